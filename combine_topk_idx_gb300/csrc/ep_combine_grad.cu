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
// padding is zeroed by the same CTAs afterwards.
//
// Bias kernel: each warp owns 64 columns and a part of the tokens and adds
// w * g to shared-memory sums of up to kBiasExperts experts, in token order;
// the parts are added afterwards in a fixed order (no atomics).
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
      float f[N];
      bf16_to_f32<U>(g.v[i], f);
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] *= w;
      if (c < p.H) store_bf16<U>(p.gy + at + c, f);
    }
  }
  if (U == 2 && p.q != nullptr) {
    const uint32_t flip = w < 0.f ? 0x80808080u : 0u;
    const uint32_t keep = w != 0.f ? 0xffffffffu : 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v * N < p.H) {
        uint32_t b[2 * U];
#pragma unroll
        for (int k = 0; k < 2 * U; ++k) b[k] = (q.b[i][k] ^ flip) & keep;
        store_bytes<U>(p.q + at + v * N, b);
        if ((v & 7) == 0) p.sf[sf0 + (v >> 3) * p.sfl.hs] = fabsf(w) * q.s[i];
      }
    }
  }
}

// U = 2 where H is a multiple of 16: eight neighbouring lanes then hold a
// scale block.
template <int U, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) combine_grad_kernel(CombineGradParams p) {
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
    if (U == 2 && p.q != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[N];
        bf16_to_f32<U>(g.v[i], f);
        quantise_block<N>(f, q.b[i], &q.s[i]);
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

constexpr int kBiasCols = 64;      // columns of a warp, two per lane
constexpr int kBiasExperts = 256;  // experts of a warp's sums (64 KB of shared memory)

__global__ void __launch_bounds__(32) bias_grad_kernel(CombineGradParams p, int experts) {
  extern __shared__ float2 sum[];  // [experts, 32]
  const int lane = threadIdx.x;
  const int e0 = blockIdx.y * experts, ne = min(experts, p.E - e0);
  const int col = blockIdx.x * kBiasCols + lane * 2;
  const bool in = col < p.H;
  for (int e = 0; e < ne; ++e) sum[e * 32 + lane] = make_float2(0.f, 0.f);
  griddep_wait();
  const int64_t per = ((int64_t)p.T + p.parts - 1) / p.parts;
  const int64_t t0 = blockIdx.z * per, t1 = min((int64_t)p.T, t0 + per);
  for (int64_t t = t0; t < t1; ++t) {
    int e = -1;
    float w = 0.f;
    if (lane < p.K) {
      e = __ldg(p.dst + t * p.K + lane) >= 0 ? __ldg(p.topk32 + t * p.K + lane) - e0 : -1;
      w = __ldg(p.topk_w + t * p.K + lane);
    }
    unsigned m = __ballot_sync(0xffffffffu, e >= 0 && e < ne);
    if (m == 0) continue;
    const uint32_t gv = in ? __ldg(reinterpret_cast<const uint32_t *>(p.g + t * p.H + col)) : 0u;
    const float g0 = bf16_lo(gv), g1 = bf16_hi(gv);
    for (; m; m &= m - 1) {
      const int k = __ffs(m) - 1;
      const int ek = __shfl_sync(0xffffffffu, e, k);
      const float wk = __shfl_sync(0xffffffffu, w, k);
      float2 a = sum[ek * 32 + lane];
      a.x = fmaf(wk, g0, a.x);
      a.y = fmaf(wk, g1, a.y);
      sum[ek * 32 + lane] = a;
    }
  }
  if (!in) return;
  float *o = p.part + ((int64_t)blockIdx.z * p.E + e0) * p.H + col;
  for (int e = 0; e < ne; ++e)
    *reinterpret_cast<float2 *>(o + (int64_t)e * p.H) = sum[e * 32 + lane];
}

int bias_experts(int E) { return std::min(E, kBiasExperts); }

template <int U, int NV, int MAXT>
cudaError_t launch_rows(const CombineGradParams &p, int threads, int sm_cap, cudaStream_t s) {
  auto kern = combine_grad_kernel<U, NV, MAXT>;
  int dev = 0, per_sm = 0;
  const cudaError_t e =
      launch_geometry(reinterpret_cast<const void *>(kern), threads, 0, &dev, &per_sm);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count(dev);
  const int use = (sm_cap > 0 && sm_cap < sms) ? sm_cap : sms;
  const int64_t items = (int64_t)p.T + (p.zero_padding ? p.rows_alloc : 0);  // tokens, then padding
  const int64_t grid = std::min<int64_t>((int64_t)use * std::max(per_sm, 1), items);
  return launch_pdl(kern, (unsigned)grid, threads, 0, s, p);
}

}  // namespace

int combine_grad_parts(const CombineGradParams &p) {
  // enough warps to fill the GPU once, at least 64 tokens each
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const int experts = bias_experts(p.E);
  const int per_sm = std::max(1, std::min(14, (int)(220 * 1024 / (experts * 256))));
  const int64_t blocks = (int64_t)((p.H + kBiasCols - 1) / kBiasCols) *
                         ((p.E + experts - 1) / experts);
  const int64_t want = ((int64_t)device_sm_count(dev) * per_sm + blocks - 1) / blocks;
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, ((int64_t)p.T + 63) / 64));
}

cudaError_t launch_combine_grad(const CombineGradParams &p, int sm_cap, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.T > 0 && (p.gy != nullptr || p.q != nullptr || p.gw != nullptr)) {
    // 32 elements per thread
    const int threads = std::max(32, ((p.H + 31) / 32 + 31) / 32 * 32);
    if (p.H % 16 == 0)
      e = threads <= 256   ? launch_rows<2, 2, 256>(p, threads, sm_cap, s)
          : threads <= 512 ? launch_rows<2, 2, 512>(p, threads, sm_cap, s)
                           : launch_rows<2, 2, 1024>(p, threads, sm_cap, s);
    else
      e = threads <= 512 ? launch_rows<1, 4, 512>(p, threads, sm_cap, s)
                         : launch_rows<1, 4, 1024>(p, threads, sm_cap, s);
  }
  if (e != cudaSuccess || p.gbias == nullptr) return e;
  const int experts = bias_experts(p.E);
  const size_t smem = (size_t)experts * kBiasCols * sizeof(float);
  int dev = 0;
  e = launch_geometry(reinterpret_cast<const void *>(bias_grad_kernel), 32, smem, &dev, nullptr);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((p.H + kBiasCols - 1) / kBiasCols, (p.E + experts - 1) / experts, p.parts);
  lc.blockDim = dim3(32);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  e = cudaLaunchKernelEx(&lc, bias_grad_kernel, p, experts);
  if (e != cudaSuccess || p.part == p.gbias) return e;
  return launch_column_sum(p.part, p.parts, (int64_t)p.E * p.H, p.gbias, s);
}

}  // namespace ep
