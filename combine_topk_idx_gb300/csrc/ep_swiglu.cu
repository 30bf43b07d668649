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
// each and share its largest magnitude in three shuffles.  Alignment padding costs no reads: its rows are recognised
// by their source token and, where the layout zeroes padding, written as 0.
#include <algorithm>

#include "ep_internal.cuh"
#include "ep_ptx.cuh"
#include "ep_quant.cuh"
#include "ep_rows.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kTileVecs = 1024;  // vectors of F per tile: rows per tile = kTileVecs / (F / 8)
constexpr int kMaxTileRows = 64; // F >= 128: at most 1024 / 16 rows

// 1 / (1 + e^-g): relative error about 2^-21 plus the rounding of g's exponent
// (|g| 2^-24); 0 where e^-g overflows.
__device__ __forceinline__ float sigmoid(float g) {
  return rcp_approx(1.0f + exp2_approx(g * -1.4426950408889634f));
}

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
// lanes hold one scale block), or 8 (BF16 output only).
template <int U>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(SwigluParams p, int tile_rows) {
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
    for (int id = threadIdx.x; id - (int)(threadIdx.x & 31) < total; id += kThreads, k.step()) {
      TileRow t{-1, 0.f, 0};
      if (id < total) t = rows[par][k.i];
      const bool use = t.row >= 0 && !t.pad;
      const int c = k.v * N;  // first column
      uint4 gv[U], uv[U];
      const uint16_t *h = p.h + t.row * 2 * p.F + c;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        gv[i] = use ? ld_stream_v4(h + 8 * i) : make_uint4(0, 0, 0, 0);
        uv[i] = use ? ld_stream_v4(h + p.F + 8 * i) : make_uint4(0, 0, 0, 0);
      }
      float g[N], u[N], a[N];
      bf16_to_f32<U>(gv, g);
      bf16_to_f32<U>(uv, u);
#pragma unroll
      for (int q = 0; q < N; ++q) a[q] = g[q] * sigmoid(g[q]) * (u[q] * t.w);
      if (p.act != nullptr && t.row >= 0) store_bf16<U>(p.act + t.row * p.F + c, a);
      if constexpr (U == 2) {
        float sc;
        uint32_t b[4];
        const int j = k.v >> 3;
        const bool first = (k.v & 7) == 0;
        if (p.q != nullptr) {
          quantise_block<N>(a, b, &sc);
          if (t.row >= 0) {
            store_bytes<U>(p.q + t.row * p.F + c, b);
            if (first) p.sf[sf_at(p.sfl, t.row, j)] = sc;
          }
        }
        if (p.ckpt != nullptr) {
          uint8_t *o = p.ckpt + t.row * 2 * p.F + c;
          float *os = p.ckpt_sf + t.row * (p.F / 64) + j;
          quantise_block<N>(g, b, &sc);
          if (use) {
            store_bytes<U>(o, b);
            if (first) os[0] = sc;
          }
          quantise_block<N>(u, b, &sc);
          if (use) {
            store_bytes<U>(o + p.F, b);
            if (first) os[p.F / 128] = sc;
          }
        }
      }
    }
  }
}

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
      const uint8_t *cp = p.ckpt + t.row * 2 * p.F + c;
      const float *cs = p.ckpt_sf + t.row * (2 * nb) + j;
      const uint16_t *ga = p.ga + t.row * p.F + c;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const uint4 gq = use ? ld_stream_v4(cp) : zero, uq = use ? ld_stream_v4(cp + p.F) : zero;
      uint4 dv[U];
#pragma unroll
      for (int i = 0; i < U; ++i) dv[i] = use ? ld_stream_v4(ga + 8 * i) : zero;
      const float gs = use ? __ldg(cs) : 0.f, us = use ? __ldg(cs + nb) : 0.f;
      float gg[N], gu[N];  // the checkpoint's gate and up, then their gradients
      e4m3x8_to_f32(make_uint2(gq.x, gq.y), gg);
      e4m3x8_to_f32(make_uint2(gq.z, gq.w), gg + 8);
      e4m3x8_to_f32(make_uint2(uq.x, uq.y), gu);
      e4m3x8_to_f32(make_uint2(uq.z, uq.w), gu + 8);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float d[8];
        bf16x8_to_f32(dv[i], d);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float g = gg[8 * i + q] * gs, u = gu[8 * i + q] * us;
          const float sg = sigmoid(g), sl = g * sg;
          const float du = d[q] * u;
          dot = fmaf(du, sl, dot);
          gu[8 * i + q] = d[q] * t.w * sl;
          gg[8 * i + q] = du * t.w * fmaf(sl, 1.f - sg, sg);
        }
      }
      if (p.gw != nullptr) {
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
        quantise_block<N>(gg, b, &sc);
        if (t.row >= 0) store_bytes<U>(o, b);
        quantise_block<N>(gu, b, &su);
        if (t.row >= 0) {
          store_bytes<U>(o + p.F, b);
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

int rows_per_tile(int F) { return std::max(1, std::min(kMaxTileRows, kTileVecs / (F / 8))); }

cudaError_t grid_for(const void *func, size_t smem, int64_t rows, int tile, unsigned *grid) {
  int dev = 0, per_sm = 0;
  const cudaError_t e = launch_geometry(func, kThreads, smem, &dev, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (rows + tile - 1) / tile;
  *grid = (unsigned)std::min<int64_t>(tiles, (int64_t)device_sm_count(dev) * std::max(per_sm, 1));
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_swiglu(const SwigluParams &p, cudaStream_t s) {
  const int tile = rows_per_tile(p.F);
  auto kern = p.F % kFp8Block == 0 ? swiglu_kernel<2> : swiglu_kernel<1>;
  unsigned grid = 0;
  const cudaError_t e = grid_for(reinterpret_cast<const void *>(kern), 0, p.r.rows, tile, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, grid, kThreads, 0, s, p, tile);
}

cudaError_t launch_swiglu_backward(const SwigluBackwardParams &p, cudaStream_t s) {
  const int tile = rows_per_tile(p.F);
  const size_t smem = 2 * sizeof(float) * (size_t)tile * (p.F / 128);
  unsigned grid = 0;
  const cudaError_t e = grid_for(reinterpret_cast<const void *>(swiglu_backward_kernel), smem,
                                 p.r.rows, tile, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(swiglu_backward_kernel, grid, kThreads, smem, s, p, tile);
}

}  // namespace ep
