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
  unsigned first;    // lanes holding the first slot of their row
  int lead;          // lane of the first slot of this slot's row
};

__device__ __forceinline__ Slots load_slots(const CombineGradParams &p, int64_t t, int lane) {
  Slots s{-1, -1, 0.f, 0.f, 0u, 0};
  if (lane < p.K) {
    s.d = __ldg(p.dst + t * p.K + lane);
    s.w = __ldg(p.topk_w + t * p.K + lane);
    if (p.ebias != nullptr) s.e = __ldg(p.topk32 + t * p.K + lane);
  }
  const unsigned peers = __match_any_sync(0xffffffffu, s.d);
  s.lead = __ffs(peers) - 1;
  s.first = __ballot_sync(0xffffffffu, s.d >= 0 && s.lead == lane);
  s.ws = 0.f;
  for (int k = 0; k < p.K; ++k) {
    const float w = __shfl_sync(0xffffffffu, s.w, k);
    if ((peers >> k) & 1) s.ws += w;
  }
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) combine_grad_kernel(CombineGradParams p) {
  __shared__ float red_y[2][EP_MAX_TOPK][kMaxWarps + 1];
  __shared__ float red_b[2][EP_MAX_TOPK][kMaxWarps + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int nvec = p.H / 8;
  const int64_t H = p.H;
  griddep_wait();
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    uint4 gv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      gv[i] = v < nvec ? ld_stream_v4(p.g + t * H + v * 8) : make_uint4(0, 0, 0, 0);
    }
    const Slots s = load_slots(p, t, lane);
    uint2 gq[NV];
    float gs[NV];
    if (p.q != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8];
        bf16x8_to_f32(gv[i], f);
        gq[i] = quantise_block(f, &gs[i]);
      }
    }
    unsigned slots = __ballot_sync(0xffffffffu, s.d >= 0);
    for (; slots; slots &= slots - 1) {
      const int k = __ffs(slots) - 1;
      const int64_t row = __shfl_sync(0xffffffffu, s.d, k);
      const float w = __shfl_sync(0xffffffffu, s.ws, k);
      if ((s.first >> k) & 1) {
        uint4 yv[NV];
        if (p.gw != nullptr) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int v = i * blockDim.x + threadIdx.x;
            yv[i] = v < nvec ? ld_stream_v4(p.y + row * H + v * 8) : make_uint4(0, 0, 0, 0);
          }
        }
        if (p.gy != nullptr) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int v = i * blockDim.x + threadIdx.x;
            float f[8];
            bf16x8_to_f32(gv[i], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] *= w;
            if (v < nvec) st_stream_v4(p.gy + row * H + v * 8, f32_to_bf16x8(f));
          }
        }
        if (p.q != nullptr) {
          const uint32_t flip = w < 0.f ? 0x80808080u : 0u;
          const uint32_t keep = w != 0.f ? 0xffffffffu : 0u;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int v = i * blockDim.x + threadIdx.x;
            if (v < nvec) {
              st_stream_v2(p.q + row * H + v * 8,
                           make_uint2((gq[i].x ^ flip) & keep, (gq[i].y ^ flip) & keep));
              if ((v & 15) == 0) p.sf[sf_at(p.sfl, row, v >> 4)] = fabsf(w) * gs[i];
            }
          }
        }
        if (p.gw != nullptr) {
          float dot = 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            float f[8], y[8];
            bf16x8_to_f32(gv[i], f);
            bf16x8_to_f32(yv[i], y);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot = fmaf(f[q], y[q], dot);
          }
          dot = warp_sum(dot);
          if (lane == 0) red_y[par][k][warp] = dot;
        }
      }
      if (p.gw != nullptr && p.ebias != nullptr) {
        const int e = __shfl_sync(0xffffffffu, s.e, k);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = i * blockDim.x + threadIdx.x;
          if (v < nvec) {
            float f[8], b[8];
            bf16x8_to_f32(gv[i], f);
            bf16x8_to_f32(ld_cached_v4(p.ebias + e * H + v * 8), b);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot = fmaf(f[q], b[q], dot);
          }
        }
        dot = warp_sum(dot);
        if (lane == 0) red_b[par][k][warp] = dot;
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
  for (int64_t q = blockIdx.x; q < npad; q += gridDim.x) {
    const int e = padding_expert(p.psum_pad, p.E, (int)q);
    const int64_t row =
        (int64_t)__ldg(p.psum_e + e) + __ldg(p.cnt_e + e) + (q - __ldg(p.psum_pad + e));
    if (row >= p.rows_alloc) continue;
    for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
      if (p.gy != nullptr) st_stream_v4(p.gy + row * H + v * 8, make_uint4(0, 0, 0, 0));
      if (p.q != nullptr) {
        st_stream_v2(p.q + row * H + v * 8, make_uint2(0, 0));
        if ((v & 15) == 0) p.sf[sf_at(p.sfl, row, v >> 4)] = 0.f;
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

template <int NV, int MAXT>
cudaError_t launch_rows(const CombineGradParams &p, int threads, int sm_cap, cudaStream_t s) {
  auto kern = combine_grad_kernel<NV, MAXT>;
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
  const int nvec = p.H / 8;
  cudaError_t e = cudaSuccess;
  if (p.T > 0 && (p.gy != nullptr || p.q != nullptr || p.gw != nullptr)) {
    const int threads = std::max(32, ((nvec + 3) / 4 + 31) / 32 * 32);
    e = threads <= 256   ? launch_rows<4, 256>(p, threads, sm_cap, s)
        : threads <= 512 ? launch_rows<4, 512>(p, threads, sm_cap, s)
                         : launch_rows<4, 1024>(p, threads, sm_cap, s);
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
