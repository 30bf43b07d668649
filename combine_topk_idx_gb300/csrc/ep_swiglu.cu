// Gated activation between the experts' two products, its 8-bit checkpoint,
// and its gradient from that checkpoint.
//
// Rows of h are gate | up, F elements each.  Forward, per element:
//   a = w * g * sigmoid(g) * u   (w: the row's weight, or 1)
// written as bf16 and/or e4m3 with one fp32 scale per 1x128 block; the
// checkpoint is h itself quantised the same way.  Backward, with g and u read
// back from the checkpoint, sg = sigmoid(g) and t = w * ga:
//   gu = t * g * sg,  gg = t * u * sg * (1 + g * (1 - sg)),
//   gw = sum over the row of ga * g * sg * u.
//
// A CTA takes tiles of whole rows; a thread takes 16 elements of the gate and
// the same of up per step, so eight neighbouring lanes hold one scale block of
// each and share its largest magnitude in three shuffles.  Alignment padding
// costs no reads: its rows are recognised by their source token and, where the
// layout zeroes padding, written as 0.
//
// 4096 tokens x 8 experts, F = 2048, FP8 out and checkpoint kept: 100 to 104 us, 4.6
// TB/s of the rows in use, between memory (71 us at a copy's rate) and the issue
// of its instructions (66 % of the cycles).  8192 rows without checkpoint: 17.3
// us, 4.9 TB/s; a call of a few rows takes 5.  36 bytes a thread are spilt at three
// CTAs to an SM.  Units dealt to the threads of the whole grid, without tiles and
// their barriers, take 112 us for the first, and with copies into shared memory
// three units ahead 133.  The gradient's figures are at its kernel.
#include <algorithm>

#include "ep_internal.cuh"
#include "ep_ptx.cuh"
#include "ep_quant.cuh"
#include "ep_rows.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kTileElems = 32768;  // of F per tile, at most
constexpr int kMaxTileRows = 64;

struct TileRow {
  int64_t row;  // -1: nothing to do
  float w;
  int pad;
};

// Row i of a tile of n rows from item i0 (threads i < n).
__device__ __forceinline__ TileRow load_row(const RowsParams &r, const float *row_w, int64_t i0,
                                            int n, int64_t items) {
  TileRow t{-1, 0.f, 0};
  if ((int)threadIdx.x < n) {
    bool pad;
    t.row = item_row(r, i0 + threadIdx.x, items, &pad);
    t.pad = pad;
    t.w = (row_w != nullptr && t.row >= 0 && !pad) ? __ldg(row_w + t.row) : 1.f;
    if (pad && !r.zero_padding) t.row = -1;
  }
  return t;
}

// A thread's walk over the units of a tile: unit (row i, column unit v), `nu`
// units per row, kThreads units a step.
struct Walk {
  int i, v, di, dv, nu;
  __device__ __forceinline__ Walk(int units) : nu(units) {
    i = threadIdx.x / nu;
    v = threadIdx.x - i * nu;
    di = kThreads / nu;
    dv = kThreads - di * nu;
  }
  __device__ __forceinline__ void step() {
    i += di;
    v += dv;
    if (v >= nu) {
      v -= nu;
      ++i;
    }
  }
};

// A unit is U vectors: 16 elements (F a multiple of 128, where 8 neighbouring
// lanes hold one scale block), or 8 (BF16 output only).  A thread loads a unit
// while it works on the one before.
template <int U>
struct Unit {
  TileRow t;
  uint4 g[U], u[U];
  __device__ __forceinline__ bool use() const { return t.row >= 0 && !t.pad; }
  __device__ __forceinline__ void load(const SwigluParams &p, const TileRow *rows, const Walk &k,
                                       bool any) {
    t = TileRow{-1, 0.f, 0};
    if (any) t = rows[k.i];
    const uint16_t *h = p.h + t.row * 2 * p.F + k.v * (8 * U);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      g[i] = use() ? ld_stream_v4(h + 8 * i) : make_uint4(0, 0, 0, 0);
      u[i] = use() ? ld_stream_v4(h + p.F + 8 * i) : make_uint4(0, 0, 0, 0);
    }
  }
};

// U vectors of zeros.
template <int U>
__device__ __forceinline__ void store_zeros(void *p) {
#pragma unroll
  for (int i = 0; i < U; ++i)
    st_stream_v4(static_cast<uint8_t *>(p) + 16 * i, make_uint4(0, 0, 0, 0));
}

template <int U>
__global__ void __launch_bounds__(kThreads, 3) swiglu_kernel(SwigluParams p, int tile_rows) {
  constexpr int N = 8 * U;
  __shared__ TileRow rows[2][kMaxTileRows];
  griddep_wait();
  const int64_t items = item_count(p.r);
  const int64_t step = (int64_t)gridDim.x * tile_rows;
  const Walk w0(p.F / N);
  const int total = tile_rows * w0.nu;  // with U = 2 blocks never split over warps
  int par = 0;
  int64_t i0 = (int64_t)blockIdx.x * tile_rows;
  TileRow next = load_row(p.r, p.row_w, i0, tile_rows, items);
  for (; i0 < items; i0 += step, par ^= 1) {
    if ((int)threadIdx.x < tile_rows) rows[par][threadIdx.x] = next;
    __syncthreads();
    next = load_row(p.r, p.row_w, i0 + step, tile_rows, items);  // used a tile later
    Walk k = w0;
    Unit<U> ahead;
    ahead.load(p, rows[par], k, (int)threadIdx.x < total);
    for (int id = threadIdx.x; id - (int)(threadIdx.x & 31) < total; id += kThreads) {
      const Unit<U> x = ahead;
      const TileRow t = x.t;
      const bool use = x.use();
      const int v = k.v, c = v * N;  // first column
      k.step();
      ahead.load(p, rows[par], k, id + kThreads < total);
      const int j = v >> 3;
      const bool first = (v & 7) == 0;
      if (!__any_sync(0xffffffffu, use)) {  // padding of the whole warp: zeros, if anything
        if (t.row >= 0) {
          if (p.act != nullptr) store_zeros<U>(p.act + t.row * p.F + c);
          if (U == 2 && p.q != nullptr) {
            store_zeros<1>(p.q + t.row * p.F + c);
            if (first) p.sf[sf_at(p.sfl, t.row, j)] = 0.f;
          }
        }
        continue;
      }
      if constexpr (U == 2) {
        if (p.ckpt != nullptr) {  // one at a time: fewer values live
          uint8_t *o = p.ckpt + t.row * 2 * p.F + c;
          float *os = p.ckpt_sf + t.row * (p.F / 64) + j;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint64_t f[N / 2];
            uint32_t b[4];
            float sc;
            bf16_to_f32<U>(half ? x.u : x.g, f);
            quantise_block16(f, b, &sc);
            if (use) {
              store_bytes16(o + half * p.F, b);
              if (first) os[half * (p.F / 128)] = sc;
            }
          }
        }
      }
      uint64_t g[N / 2], u[N / 2];
      bf16_to_f32<U>(x.g, g);
      bf16_to_f32<U>(x.u, u);
      const uint64_t w2 = f32x2_pack(t.w, t.w);
#pragma unroll
      for (int q = 0; q < N / 2; ++q)
        g[q] = f32x2_mul_rn(f32x2_mul_rn(g[q], sigmoid2(g[q])), f32x2_mul_rn(u[q], w2));
      if (p.act != nullptr && t.row >= 0) store_bf16<U>(p.act + t.row * p.F + c, g);
      if constexpr (U == 2) {
        if (p.q != nullptr) {
          float sc;
          uint32_t b[4];
          quantise_block16(g, b, &sc);
          if (t.row >= 0) {
            store_bytes16(p.q + t.row * p.F + c, b);
            if (first) p.sf[sf_at(p.sfl, t.row, j)] = sc;
          }
        }
      }
    }
  }
}

// 4096 tokens x 8 experts, F = 2048, FP8 in and out: 107 to 111 us, 3.8 TB/s of the
// rows in use; BF16 out 117 us, 4.6 TB/s.  52 bytes a thread are spilt at four CTAs
// to an SM.  Between the issue of its instructions (59 % of the cycles) and its
// loads: loading a unit ahead as above costs registers, and so resident warps
// (114 -> 122 us); whole rows to a warp, without the tile's barrier, gain nothing
// (108 us); copies into shared memory three units ahead cost more than the wait
// that they save (129 us).
__global__ void __launch_bounds__(kThreads)
    swiglu_backward_kernel(SwigluBackwardParams p, int tile_rows) {
  constexpr int U = 2, N = 8 * U;
  __shared__ TileRow rows[2][kMaxTileRows];
  // one sum per row and 1x128 block of F, two tiles
  extern __shared__ float gws[];
  griddep_wait();
  const int nb = p.F / 128;
  const int64_t items = item_count(p.r);
  const int64_t step = (int64_t)gridDim.x * tile_rows;
  const Walk w0(p.F / N);
  const int total = tile_rows * w0.nu;
  int par = 0;
  int64_t i0 = (int64_t)blockIdx.x * tile_rows;
  TileRow next = load_row(p.r, p.row_w, i0, tile_rows, items);
  for (; i0 < items; i0 += step, par ^= 1) {
    if ((int)threadIdx.x < tile_rows) rows[par][threadIdx.x] = next;
    __syncthreads();
    next = load_row(p.r, p.row_w, i0 + step, tile_rows, items);
    float *sum = gws + par * tile_rows * nb;
    Walk k = w0;
    for (int id = threadIdx.x; id - (int)(threadIdx.x & 31) < total; id += kThreads, k.step()) {
      TileRow t{-1, 0.f, 0};
      if (id < total) t = rows[par][k.i];
      const bool use = t.row >= 0 && !t.pad;
      const int c = k.v * N, j = k.v >> 3;
      const bool first = (k.v & 7) == 0;
      if (!__any_sync(0xffffffffu, use)) {  // without this 113 us, a third of the rows padding
        if (id < total && first && p.gw != nullptr) sum[k.i * nb + j] = 0.f;
        if (t.row >= 0) {
          if (p.gh != nullptr) {
            uint16_t *o = p.gh + t.row * 2 * p.F + c;
            store_zeros<U>(o);
            store_zeros<U>(o + p.F);
          }
          if (p.q != nullptr) {
            uint8_t *o = p.q + t.row * 2 * p.F + c;
            store_zeros<1>(o);
            store_zeros<1>(o + p.F);
            if (first) {
              p.sf[sf_at(p.sfl, t.row, j)] = 0.f;
              p.sf[sf_at(p.sfl, t.row, j + nb)] = 0.f;
            }
          }
        }
        continue;
      }
      const uint8_t *cp = p.ckpt + t.row * 2 * p.F + c;
      const float *cs = p.ckpt_sf + t.row * (2 * nb) + j;
      const uint16_t *ga = p.ga + t.row * p.F + c;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const uint4 gq = use ? ld_stream_v4(cp) : zero, uq = use ? ld_stream_v4(cp + p.F) : zero;
      uint4 dv[U];
#pragma unroll
      for (int i = 0; i < U; ++i) dv[i] = use ? ld_stream_v4(ga + 8 * i) : zero;
      const float gs = use ? __ldg(cs) : 0.f, us = use ? __ldg(cs + nb) : 0.f;
      uint64_t gg[N / 2], gu[N / 2];  // the checkpoint's gate and up, then their gradients
      const uint32_t gw4[4] = {gq.x, gq.y, gq.z, gq.w}, uw4[4] = {uq.x, uq.y, uq.z, uq.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        e4m3x4_to_f32(gw4[q], gg + 2 * q);
        e4m3x4_to_f32(uw4[q], gu + 2 * q);
      }
      uint64_t d[N / 2], dot2 = 0;
      bf16_to_f32<U>(dv, d);
      const uint64_t gs2 = f32x2_pack(gs, gs), us2 = f32x2_pack(us, us);
      const uint64_t w2 = f32x2_pack(t.w, t.w), one = f32x2_pack(1.f, 1.f);
      const uint64_t minus = f32x2_pack(-1.f, -1.f);
#pragma unroll
      for (int q = 0; q < N / 2; ++q) {
        const uint64_t g = f32x2_mul_rn(gg[q], gs2), u = f32x2_mul_rn(gu[q], us2);
        const uint64_t sg = sigmoid2(g), sl = f32x2_mul_rn(g, sg);
        const uint64_t du = f32x2_mul_rn(d[q], u);
        dot2 = f32x2_fma_rn(du, sl, dot2);
        gu[q] = f32x2_mul_rn(f32x2_mul_rn(d[q], w2), sl);
        gg[q] = f32x2_mul_rn(f32x2_mul_rn(du, w2),
                             f32x2_fma_rn(sl, f32x2_fma_rn(sg, minus, one), sg));
      }
      if (p.gw != nullptr) {
        float dot = f32x2_lo(dot2) + f32x2_hi(dot2);
#pragma unroll
        for (int o = 1; o < 8; o *= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (id < total && first) sum[k.i * nb + j] = dot;
      }
      if (p.gh != nullptr && t.row >= 0) {
        uint16_t *o = p.gh + t.row * 2 * p.F + c;
        store_bf16<U>(o, gg);
        store_bf16<U>(o + p.F, gu);
      }
      if (p.q != nullptr) {
        float sc, su;
        uint32_t b[4];
        uint8_t *o = p.q + t.row * 2 * p.F + c;
        quantise_block16(gg, b, &sc);
        if (t.row >= 0) store_bytes16(o, b);
        quantise_block16(gu, b, &su);
        if (t.row >= 0) {
          store_bytes16(o + p.F, b);
          if (first) {
            p.sf[sf_at(p.sfl, t.row, j)] = sc;
            p.sf[sf_at(p.sfl, t.row, j + nb)] = su;
          }
        }
      }
    }
    if (p.gw != nullptr) {
      __syncthreads();
      if ((int)threadIdx.x < tile_rows && rows[par][threadIdx.x].row >= 0) {
        float v = 0.f;
        for (int j = 0; j < nb; ++j) v += sum[threadIdx.x * nb + j];
        p.gw[rows[par][threadIdx.x].row] = v;
      }
    }
  }
}

// Rows per tile and CTAs: tiles of up to kTileElems elements (a barrier each; of
// 8192, 32,768 rows of F = 2048 take 122 us against 108 with the checkpoint),
// shorter where the rows would not give every CTA four, so that the CTAs' loads
// differ little (8192 rows: 24.7 us against 27.8 with the longest).
cudaError_t shape_for(const void *func, int64_t rows, int F, bool sums, int sm_cap, int *tile,
                      unsigned *grid, size_t *smem) {
  const int most = std::max(1, std::min(kMaxTileRows, kTileElems / F));
  *smem = sums ? 2 * sizeof(float) * (size_t)most * (F / kFp8Block) : 0;
  int dev = 0, per_sm = 0;
  const cudaError_t e = launch_geometry(func, kThreads, *smem, &dev, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)sms_to_use(dev, sm_cap) * std::max(per_sm, 1);
  *tile = (int)std::max<int64_t>(1, std::min<int64_t>(most, rows / (4 * ctas)));
  *grid = (unsigned)std::min<int64_t>((rows + *tile - 1) / *tile, ctas);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_swiglu(const SwigluParams &p, int sm_cap, cudaStream_t s) {
  auto kern = p.F % kFp8Block == 0 ? swiglu_kernel<2> : swiglu_kernel<1>;
  int tile = 0;
  unsigned grid = 0;
  size_t smem = 0;
  const cudaError_t e = shape_for(reinterpret_cast<const void *>(kern), p.r.rows, p.F, false,
                                  sm_cap, &tile, &grid, &smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, grid, kThreads, smem, s, p, tile);
}

cudaError_t launch_swiglu_backward(const SwigluBackwardParams &p, int sm_cap, cudaStream_t s) {
  int tile = 0;
  unsigned grid = 0;
  size_t smem = 0;
  const cudaError_t e = shape_for(reinterpret_cast<const void *>(swiglu_backward_kernel), p.r.rows,
                                  p.F, true, sm_cap, &tile, &grid, &smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(swiglu_backward_kernel, grid, kThreads, smem, s, p, tile);
}

}  // namespace ep
