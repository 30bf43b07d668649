// Gradient of the weighted combine.
//
// The combine is out[t] = sum over the token's slots k of
// w[t,k] * (y[dst[t,k]] + bias[e(t,k)]) (+ per-token terms), so with g the
// gradient of out:
//   gy[row]    = (sum of w over the token's slots on that row) * g[t]
//   gw[t,k]    = <g[t], y[dst[t,k]] + bias[e(t,k)]>
//   gbias[e]   = sum over the slots (t,k) routed to e of w[t,k] * g[t]
// (the per-token terms' gradient is g itself).  In the rank layout several
// slots of a token share a row; in the expanded layout each has its own.
//
// Row kernel: one CTA per token (persistent), the token's gradient in
// registers while its rows go by: each row of y is read once and the row of
// gy written once, g once per token.  As FP8 rows, g is quantised once per
// token: the bytes are those of g (with the sign of the weight), the scale is
// the scale of g times |w|, so K rows cost one quantisation.  gy's alignment
// padding is zeroed by the same CTAs afterwards.  Memory bounds it: 4096 tokens
// x 8 experts, H = 7168, FP8 rows, 164 us for 771 MB and 117 MB of zeroed
// padding, 5.4 TB/s; each row of y waits for its token's slots and is then
// read in two pieces a thread, so the loads in flight limit it.  The registers of
// three CTAs to an SM leave 72 bytes a thread spilt (432 for H above 8192); with
// registers without limit, and nothing spilt, it takes 250.
//
// Bias gradient: a sum over tokens per expert, so the slots of each chunk of
// kChunkTokens tokens are first sorted by expert (stably, once for all columns);
// then each warp owns 256 columns, a few experts and a part of the chunks and
// walks an expert's slots with its sums in registers, which meet the sums in
// shared memory once per chunk and expert.  The parts are added afterwards in a
// fixed order.  (No atomics, and no dense product with the mostly empty
// weight matrix: there 0 * inf of one token's gradient would reach experts that
// the token never chose.)
#include <algorithm>

#include "ep_internal.cuh"
#include "ep_ptx.cuh"
#include "ep_quant.cuh"
#include "ep_rows.cuh"

namespace ep {
namespace {

constexpr int kMaxWarps = 32;

struct Slots {       // a token's slots, one per lane
  int d, e;
  float w;           // weight of the slot
  float ws;          // weight of its row (sum over the slots sharing it, in slot order)
  int64_t sf;        // where its row's first scale lies (FP8 output)
  unsigned first;    // lanes holding the first slot of their row
  int lead;          // lane of the first slot of this slot's row
};

__device__ __forceinline__ Slots load_slots(const CombineGradParams &p, int64_t t, int lane) {
  Slots s{-1, -1, 0.f, 0.f, 0, 0u, 0};
  if (lane < p.K) {
    s.d = __ldg(p.dst + t * p.K + lane);
    s.w = __ldg(p.topk_w + t * p.K + lane);
    if (p.ebias != nullptr) s.e = __ldg(p.topk32 + t * p.K + lane);
  }
  const unsigned peers = __match_any_sync(0xffffffffu, s.d);
  s.lead = __ffs(peers) - 1;
  s.first = __ballot_sync(0xffffffffu, s.d >= 0 && s.lead == lane);
  s.ws = s.w;
  if (!p.do_expand) {  // several slots may share a row
    s.ws = 0.f;
    for (int k = 0; k < p.K; ++k) {
      const float w = __shfl_sync(0xffffffffu, s.w, k);
      if ((peers >> k) & 1) s.ws += w;
    }
  }
  if (p.q != nullptr && s.d >= 0) s.sf = sf_at(p.sfl, s.d, 0);
  return s;
}

// Sums of a and of b over the warp: lanes 0..15 get a's, lanes 16..31 b's.
__device__ __forceinline__ float warp_sum2(float a, float b) {
  const bool hi = (threadIdx.x & 16) != 0;
  float v = (hi ? b : a) + __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A thread's share of a row: NV units of U vectors, blockDim.x units apart.
template <int U, int NV>
struct Share {
  uint4 v[NV][U];
  template <bool STREAM>
  __device__ __forceinline__ void load(const uint16_t *row, int H, bool any) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * 8 * U;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const uint16_t *a = row + c + 8 * k;
        v[i][k] = any && c < H ? (STREAM ? ld_stream_v4(a) : ld_cached_v4(a))
                               : make_uint4(0, 0, 0, 0);
      }
    }
  }
  // This thread's part of the inner product with another share: each product
  // of two BF16 values is exact, each sum rounded once.
  __device__ __forceinline__ float dot(const Share &o) const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < U; ++k) {
        s = fma2_bf16_f32(v[i][k].x, o.v[i][k].x, s);
        s = fma2_bf16_f32(v[i][k].y, o.v[i][k].y, s);
        s = fma2_bf16_f32(v[i][k].z, o.v[i][k].z, s);
        s = fma2_bf16_f32(v[i][k].w, o.v[i][k].w, s);
      }
    return s;
  }
};

// The token's gradient as FP8 bytes and scales, a thread's share of them.
template <int U, int NV>
struct ShareFp8 {
  uint32_t b[NV][2 * U];
  float s[NV];
};

// Writes w * g to `row` of the outputs; sf0: where the row's scales begin.
template <int U, int NV>
__device__ __forceinline__ void write_row(const CombineGradParams &p, const Share<U, NV> &g,
                                          const ShareFp8<U, NV> &q, int64_t row, float w,
                                          int64_t sf0) {
  constexpr int N = 8 * U;
  const int64_t at = row * p.H;
  if (p.gy != nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * N;
      uint64_t f[N / 2];
      bf16_to_f32<U>(g.v[i], f);
      const uint64_t w2 = f32x2_pack(w, w);
#pragma unroll
      for (int k = 0; k < N / 2; ++k) f[k] = f32x2_mul_rn(f[k], w2);
      if (c < p.H) store_bf16<U>(p.gy + at + c, f);
    }
  }
  if constexpr (U == 2) {
    if (p.q != nullptr) {
      const uint32_t flip = w < 0.f ? 0x80808080u : 0u;
      const uint32_t keep = w != 0.f ? 0xffffffffu : 0u;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * blockDim.x + threadIdx.x;
        if (v * N < p.H) {
          uint32_t b[2 * U];
#pragma unroll
          for (int k = 0; k < 2 * U; ++k) b[k] = (q.b[i][k] ^ flip) & keep;
          store_bytes16(p.q + at + v * N, b);
          if ((v & 7) == 0)  // weight 0: a scale of 0, whatever the gradient holds
            p.sf[sf0 + (v >> 3) * p.sfl.hs] = w != 0.f ? fabsf(w) * q.s[i] : 0.f;
        }
      }
    }
  }
}

// U = 2 where H is a multiple of 16: eight neighbouring lanes then hold a
// scale block.
template <int U, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 3 : 1)
    combine_grad_kernel(CombineGradParams p) {
  constexpr int N = 8 * U;
  __shared__ float red_y[2][EP_MAX_TOPK][kMaxWarps + 1];
  __shared__ float red_b[2][EP_MAX_TOPK][kMaxWarps + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int64_t H = p.H;
  griddep_wait();
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    Share<U, NV> g;
    g.template load<true>(p.g + t * H, p.H, true);
    const Slots s = load_slots(p, t, lane);
    ShareFp8<U, NV> q;
    if constexpr (U == 2) {
      if (p.q != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          uint64_t f[N / 2];
          bf16_to_f32<U>(g.v[i], f);
          quantise_block16(f, q.b[i], &q.s[i]);
        }
      }
    }
    // the token's rows, two at a time
    for (unsigned m = s.first; m;) {
      const int k0 = __ffs(m) - 1;
      m &= m - 1;
      const bool two = m != 0;
      const int k1 = two ? __ffs(m) - 1 : k0;
      m &= m - 1;
      const int64_t row0 = __shfl_sync(0xffffffffu, s.d, k0);
      const int64_t row1 = __shfl_sync(0xffffffffu, s.d, k1);
      Share<U, NV> y0, y1;
      if (p.gw != nullptr) {
        y0.template load<true>(p.y + row0 * H, p.H, true);
        y1.template load<true>(p.y + row1 * H, p.H, two);
      }
      write_row<U, NV>(p, g, q, row0, __shfl_sync(0xffffffffu, s.ws, k0),
                       __shfl_sync(0xffffffffu, s.sf, k0));
      if (two)
        write_row<U, NV>(p, g, q, row1, __shfl_sync(0xffffffffu, s.ws, k1),
                         __shfl_sync(0xffffffffu, s.sf, k1));
      if (p.gw != nullptr) {
        const float v = warp_sum2(g.dot(y0), g.dot(y1));
        if (lane == 0) red_y[par][k0][warp] = v;
        if (lane == 16 && two) red_y[par][k1][warp] = v;
      }
    }
    if (p.gw != nullptr && p.ebias != nullptr) {
      for (unsigned m = __ballot_sync(0xffffffffu, s.d >= 0); m;) {
        const int k0 = __ffs(m) - 1;
        m &= m - 1;
        const bool two = m != 0;
        const int k1 = two ? __ffs(m) - 1 : k0;
        m &= m - 1;
        Share<U, NV> b0, b1;
        b0.template load<false>(p.ebias + __shfl_sync(0xffffffffu, s.e, k0) * H, p.H, true);
        b1.template load<false>(p.ebias + __shfl_sync(0xffffffffu, s.e, k1) * H, p.H, two);
        const float v = warp_sum2(g.dot(b0), g.dot(b1));
        if (lane == 0) red_b[par][k0][warp] = v;
        if (lane == 16 && two) red_b[par][k1][warp] = v;
      }
    }
    if (p.gw != nullptr) {
      __syncthreads();
      // lane k of warp 0 holds slot k; the other warps go on to the next token
      if (warp == 0 && lane < p.K) {
        float v = 0.f;
        if (s.d >= 0) {
          for (int i = 0; i < nw; ++i) v += red_y[par][s.lead][i];
          if (p.ebias != nullptr) {
            float b = 0.f;
            for (int i = 0; i < nw; ++i) b += red_b[par][lane][i];
            v += b;
          }
        }
        p.gw[t * p.K + lane] = v;
      }
    }
  }
  if (!p.zero_padding || (p.gy == nullptr && p.q == nullptr)) return;
  const int npad = __ldg(p.psum_pad + p.E);
  for (int64_t i = blockIdx.x; i < npad; i += gridDim.x) {
    const int e = padding_expert(p.psum_pad, p.E, (int)i);
    const int64_t row =
        (int64_t)__ldg(p.psum_e + e) + __ldg(p.cnt_e + e) + (i - __ldg(p.psum_pad + e));
    if (row >= p.rows_alloc) continue;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (p.gy != nullptr)
      for (int c = threadIdx.x * 8; c < p.H; c += blockDim.x * 8)
        st_stream_v4(p.gy + row * H + c, zero);
    if (p.q != nullptr) {
      for (int c = threadIdx.x * 16; c < p.H; c += blockDim.x * 16) {
        st_stream_v4(p.q + row * H + c, zero);
        if (c % kFp8Block == 0) p.sf[sf_at(p.sfl, row, c / kFp8Block)] = 0.f;
      }
    }
  }
}

// 16,384 tokens x 6 of 64 experts, H = 4096, skewed: the whole call takes 295 us,
// 197 of them the row kernel's and 10 the sort's.  With 8 experts a warp and half
// as many parts 25 us more, with 16 experts and 128 columns 53: eight columns a
// lane halve what is spent per slot on its entry and address.  Many small parts
// even out a skewed load (40 warps' parts 14 us more, 27 warps' 35) and cost an
// even one 1 %.  Their sums take about 50 MB; the parts are rounded up, so that it
// can be just under twice that (E 772, H 16128, two parts: 99.6 MB).  Loads in
// flight bound it; the gradient rows come from L2.
constexpr int kChunkTokens = 256;
constexpr int kSortWarps = 8;
constexpr int kSortAhead = 8;      // steps of 32 slots whose loads are in flight
constexpr int kBiasCols = 256;     // columns of a warp, eight per lane
constexpr int kBiasExperts = 4;    // experts of a warp: 4 KB of sums
constexpr int kBiasWarps = 80;     // warps of an SM that the parts are made for
constexpr int kBiasAhead = 8;      // slots whose rows are in flight

// Sorts a chunk's slots by expert: entries (token, weight) in (token, slot)
// order within an expert, off[e] the first entry of expert e.  Each warp takes
// consecutive tokens, 32 slots at a step.
__device__ __forceinline__ void sort_chunk(const CombineGradParams &p, int chunk, int *cnt,
                                           int *warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nt = kSortWarps * 32;
  int *const mine = cnt + warp * p.E;
  for (int i = threadIdx.x; i < kSortWarps * p.E; i += nt) cnt[i] = 0;
  __syncthreads();
  constexpr int per = kChunkTokens / kSortWarps;
  const int64_t t0 = (int64_t)chunk * kChunkTokens + warp * per;
  const int64_t s0 = min(t0, (int64_t)p.T) * p.K, s1 = min(t0 + per, (int64_t)p.T) * p.K;
  auto expert = [&](int64_t s) {
    return s < s1 && __ldg(p.dst + s) >= 0 ? __ldg(p.topk32 + s) : -1;
  };
  // kSortAhead steps' loads at once: 16,384 tokens x 6 take 10 us, and 16 with the
  // loads one after the other
  for (int64_t s = s0 + lane; s - lane < s1; s += 32 * kSortAhead) {
    int ex[kSortAhead];
#pragma unroll
    for (int q = 0; q < kSortAhead; ++q) ex[q] = expert(s + 32 * q);
#pragma unroll
    for (int q = 0; q < kSortAhead; ++q) {
      const unsigned peers = __match_any_sync(0xffffffffu, ex[q]);
      if (ex[q] >= 0 && lane == __ffs(peers) - 1) mine[ex[q]] += __popc(peers);
      __syncwarp();
    }
  }
  __syncthreads();
  // counts -> first entry of each (expert, warp)
  int32_t *off = p.off + (int64_t)chunk * (p.E + 1);
  int base = 0;
  for (int e0 = 0; e0 < p.E; e0 += nt) {
    const int e = e0 + threadIdx.x;
    int n = 0;
    if (e < p.E)
      for (int w = 0; w < kSortWarps; ++w) n += cnt[w * p.E + e];
    int v = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    int first = base + v - n, all = base;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) first += warp_sum[w];
      all += warp_sum[w];
    }
    if (e < p.E) {
      off[e] = first;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = cnt[w * p.E + e];
        cnt[w * p.E + e] = first;
        first += c;
      }
    }
    base = all;
    __syncthreads();
  }
  if (threadIdx.x == 0) off[p.E] = base;
  int2 *ent = p.ent + (int64_t)chunk * kChunkTokens * p.K;
  for (int64_t s = s0 + lane; s - lane < s1; s += 32 * kSortAhead) {
    int ex[kSortAhead];
    float w[kSortAhead];
#pragma unroll
    for (int q = 0; q < kSortAhead; ++q) {
      ex[q] = expert(s + 32 * q);
      w[q] = s + 32 * q < s1 ? __ldg(p.topk_w + s + 32 * q) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < kSortAhead; ++q) {
      const unsigned peers = __match_any_sync(0xffffffffu, ex[q]);
      const int at = ex[q] >= 0 ? mine[ex[q]] : 0;
      __syncwarp();
      if (ex[q] >= 0) {
        ent[at + __popc(peers & lanemask_lt())] =
            make_int2((int)((s + 32 * q) / p.K), __float_as_int(w[q]));
        if (lane == __ffs(peers) - 1) mine[ex[q]] = at + __popc(peers);
      }
      __syncwarp();
    }
  }
}

// A CTA sorts one chunk, or with CAPPED the chunks in turn.
template <bool CAPPED>
__global__ void __launch_bounds__(kSortWarps * 32)
    bias_sort_kernel(CombineGradParams p, int chunks) {
  extern __shared__ int cnt[];  // [kSortWarps, E]
  __shared__ int warp_sum[kSortWarps];
  griddep_wait();
  if constexpr (!CAPPED) {
    sort_chunk(p, blockIdx.x, cnt, warp_sum);
  } else {
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
      sort_chunk(p, c, cnt, warp_sum);
      __syncthreads();  // the next chunk clears the counts
    }
  }
}

// A warp's share (x, y, z): columns x * kBiasCols .., experts y, y + ny, ... (popular
// experts, often neighbours, fall to different warps), chunks z, z + parts, ...
__device__ __forceinline__ void bias_share(const CombineGradParams &p, int x, int y, int z, int ny,
                                           float4 *sum) {
  const int lane = threadIdx.x;
  const int ne = (p.E - y + ny - 1) / ny;
  const int col = x * kBiasCols + lane * 8;
  const bool in = col < p.H;
  for (int i = 0; i < ne * 2; ++i) sum[i * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int chunks = (p.T + kChunkTokens - 1) / kChunkTokens;
  const uint16_t *g = p.g + (in ? col : 0);
  for (int c = z; c < chunks; c += p.parts) {
    const int32_t *off = p.off + (int64_t)c * (p.E + 1) + y;
    const int2 *ent = p.ent + (int64_t)c * kChunkTokens * p.K;
    for (int i = 0; i < ne; ++i, off += ny) {
      int first = __ldg(off);
      const int end = __ldg(off + 1);
      if (first == end) continue;
      const float4 a = sum[i * 64 + lane], b = sum[i * 64 + 32 + lane];
      uint64_t s[4] = {f32x2_pack(a.x, a.y), f32x2_pack(a.z, a.w), f32x2_pack(b.x, b.y),
                       f32x2_pack(b.z, b.w)};
      for (; first < end; first += kBiasAhead) {
        uint4 v[kBiasAhead];
        float w[kBiasAhead];
#pragma unroll
        for (int q = 0; q < kBiasAhead; ++q) {
          const int2 x = first + q < end ? __ldg(ent + first + q) : make_int2(-1, 0);
          w[q] = __int_as_float(x.y);
          v[q] = x.x >= 0 ? ld_cached_v4(g + (int64_t)x.x * p.H)
                          : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < kBiasAhead; ++q) {
          const uint64_t w2 = f32x2_pack(w[q], w[q]);
          uint64_t f[4];
          bf16_to_f32<1>(&v[q], f);
#pragma unroll
          for (int k = 0; k < 4; ++k) s[k] = f32x2_fma_rn(w2, f[k], s[k]);
        }
      }
      sum[i * 64 + lane] = make_float4(f32x2_lo(s[0]), f32x2_hi(s[0]), f32x2_lo(s[1]), f32x2_hi(s[1]));
      sum[i * 64 + 32 + lane] =
          make_float4(f32x2_lo(s[2]), f32x2_hi(s[2]), f32x2_lo(s[3]), f32x2_hi(s[3]));
    }
  }
  if (!in) return;
  float *o = p.part + ((int64_t)z * p.E + y) * p.H + col;
  for (int i = 0; i < ne; ++i) {
    float4 *const r = reinterpret_cast<float4 *>(o + (int64_t)i * ny * p.H);
    r[0] = sum[i * 64 + lane];
    r[1] = sum[i * 64 + 32 + lane];
  }
}

// A warp's share is its place in the grid, or with CAPPED warps take the nx * ny *
// parts shares in turn (the skewed case above takes 300 us that way).
template <bool CAPPED>
__global__ void __launch_bounds__(32) bias_grad_kernel(CombineGradParams p, int nx, int ny) {
  extern __shared__ float4 sum[];  // [experts, 2, 32]; a lane touches its own columns only
  griddep_wait();
  if constexpr (!CAPPED) {
    bias_share(p, blockIdx.x, blockIdx.y, blockIdx.z, gridDim.y, sum);
  } else {
    for (int b = blockIdx.x; b < nx * ny * p.parts; b += gridDim.x)
      bias_share(p, b % nx, b / nx % ny, b / (nx * ny), ny, sum);
  }
}

int bias_experts(int E) { return std::min(E, kBiasExperts); }
int bias_chunks(const CombineGradParams &p) { return (p.T + kChunkTokens - 1) / kChunkTokens; }

template <int U, int NV, int MAXT>
cudaError_t launch_rows(const CombineGradParams &p, int threads, int sm_cap, cudaStream_t s) {
  auto kern = combine_grad_kernel<U, NV, MAXT>;
  int dev = 0, per_sm = 0;
  const cudaError_t e =
      launch_geometry(reinterpret_cast<const void *>(kern), threads, 0, &dev, &per_sm);
  if (e != cudaSuccess) return e;
  const int use = sms_to_use(dev, sm_cap);
  const int64_t items = (int64_t)p.T + (p.zero_padding ? p.rows_alloc : 0);  // tokens, then padding
  const int64_t grid = std::min<int64_t>((int64_t)use * std::max(per_sm, 1), items);
  return launch_pdl(kern, (unsigned)grid, threads, 0, s, p);
}

}  // namespace

cudaError_t combine_grad_workspace(CombineGradParams *p, size_t *bytes, void *base) {
  // enough warps for about kBiasWarps on each SM, at least a chunk each
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int64_t experts = bias_experts(p->E), chunks = bias_chunks(*p);
  const int64_t blocks = (int64_t)((p->H + kBiasCols - 1) / kBiasCols) *
                         ((p->E + experts - 1) / experts);
  const int64_t want = (kBiasWarps * (int64_t)device_sm_count(dev) + blocks - 1) / blocks;
  p->parts = (int)std::max<int64_t>(1, std::min(want, chunks));
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 255) / 256 * 256;
    return o;
  };
  const size_t o_ent = take(sizeof(int2) * (size_t)chunks * kChunkTokens * p->K);
  const size_t o_off = take(sizeof(int32_t) * (size_t)chunks * (p->E + 1));
  const size_t o_part = take(p->parts > 1 ? sizeof(float) * (size_t)p->parts * p->E * p->H : 0);
  *bytes = std::max<size_t>(at, 256);
  if (base != nullptr) {
    uint8_t *b = static_cast<uint8_t *>(base);
    p->ent = reinterpret_cast<int2 *>(b + o_ent);
    p->off = reinterpret_cast<int32_t *>(b + o_off);
    p->part = p->parts > 1 ? reinterpret_cast<float *>(b + o_part) : p->gbias;
  }
  return cudaSuccess;
}

cudaError_t launch_combine_grad(const CombineGradParams &p, int sm_cap, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.T > 0 && (p.gy != nullptr || p.q != nullptr || p.gw != nullptr)) {
    // 32 elements per thread.  Up to 256 threads, H = 8192, with registers for
    // three CTAs to an SM: 4096 tokens x 8, H = 7168, 165 us against 180 where
    // the bound is that of longer rows, and 250 with registers without limit.
    const int threads = std::max(32, ((p.H + 31) / 32 + 31) / 32 * 32);
    if (p.H % 16 == 0)
      e = threads <= 256 ? launch_rows<2, 2, 256>(p, threads, sm_cap, s)
                         : launch_rows<2, 2, 1024>(p, threads, sm_cap, s);
    else
      e = threads <= 256 ? launch_rows<1, 4, 256>(p, threads, sm_cap, s)
                         : launch_rows<1, 4, 1024>(p, threads, sm_cap, s);
  }
  if (e != cudaSuccess || p.gbias == nullptr) return e;
  const int experts = bias_experts(p.E);
  const size_t sort_smem = sizeof(int) * kSortWarps * (size_t)p.E;
  const size_t smem = (size_t)experts * kBiasCols * sizeof(float);
  int dev = 0, sort_per_sm = 0, per_sm = 0;
  const auto sort = sm_cap > 0 ? bias_sort_kernel<true> : bias_sort_kernel<false>;
  e = launch_geometry(reinterpret_cast<const void *>(sort), kSortWarps * 32, sort_smem, &dev,
                      &sort_per_sm);
  if (e != cudaSuccess) return e;
  const auto bias = sm_cap > 0 ? bias_grad_kernel<true> : bias_grad_kernel<false>;
  e = launch_geometry(reinterpret_cast<const void *>(bias), 32, smem, &dev, &per_sm);
  if (e != cudaSuccess) return e;
  // as many CTAs as the SMs of a cap hold
  auto most = [&](int64_t items, int per) {
    return (unsigned)std::min(items, (int64_t)sms_to_use(dev, sm_cap) * std::max(per, 1));
  };
  const int chunks = bias_chunks(p);
  if (p.T > 0) {
    e = launch_pdl(sort, sm_cap > 0 ? most(chunks, sort_per_sm) : (unsigned)chunks,
                   kSortWarps * 32, sort_smem, s, p, chunks);
    if (e != cudaSuccess) return e;
  }
  const int nx = (p.H + kBiasCols - 1) / kBiasCols, ny = (p.E + experts - 1) / experts;
  const dim3 grid = sm_cap > 0 ? dim3(most((int64_t)nx * ny * p.parts, per_sm))
                               : dim3(nx, ny, p.parts);
  e = launch_pdl(bias, grid, 32, smem, s, p, nx, ny);
  if (e != cudaSuccess || p.part == p.gbias) return e;
  return launch_column_sum(p.part, p.parts, (int64_t)p.E * p.H, p.gbias, sm_cap, s);
}

}  // namespace ep
