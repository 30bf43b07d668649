// Root-mean-square norm with the residual's addition, and its gradient.
//
// Forward, per row of H elements:
//   s = x + residual (fp32), r = bf16(s), k = 1 / sqrt(mean(s^2) + eps),
//   v = s * k * gamma; written as bf16(v) and/or as e4m3 bytes with one fp32
//   scale per 1x128 block (amax * (1 / 448)), the input of a pre-quantised dispatch.
// Backward, with xh = r * k:
//   m = mean(gy * gamma * xh), gx = k * (gy * gamma - xh * m) + gres,
//   ggamma = sum over rows of gy * xh.
//
// Both read each input once and write each output once: a row stays in
// registers between the sum and the result, as 16-byte vectors of eight
// elements.  What bounds them is memory.  4096 rows of 7168, residual in and
// out, FP8 out: 33.7 us for 206 MB, 6.1 TB/s, where a copy reaches 6.7.
// Gradient of 16,384 rows of 4096 with a residual's: 92 us for 537 MB, 5.8 TB/s.
// One row of 7168: 6.5 us in a CUDA graph, most of it the launch.
#include <algorithm>

#include "ep_internal.cuh"
#include "ep_ptx.cuh"
#include "ep_quant.cuh"

namespace ep {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kWideSum = 65536;  // columns
constexpr int kWarpRow = 512;  // elements of a row that a warp takes, at most

// Sum over the threads of a row: a warp, or the whole CTA (`red` then holds
// one value per warp; one barrier per call, the caller alternates buffers).
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (WARP_ROW) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void load_gamma(const void *gamma, int f32, int v, float *f) {
  if (f32) {
    const float4 a = __ldg(static_cast<const float4 *>(gamma) + 2 * v);
    const float4 b = __ldg(static_cast<const float4 *>(gamma) + 2 * v + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    bf16x8_to_f32(ld_cached_v4(static_cast<const uint4 *>(gamma) + v), f);
  }
}

// A thread holds NV units of U vectors; WARP_ROW: one warp per row, else one
// CTA per row.  U = 2 where H is a multiple of 16, as FP8 output needs: eight
// neighbouring lanes then hold one scale block.
template <int U, int NV, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 128 : kMaxThreads) norm_kernel(NormParams p) {
  constexpr int N = 8 * U;
  __shared__ float red[32];
  const int tpr = WARP_ROW ? 32 : blockDim.x;  // threads per row
  const int tid = WARP_ROW ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t t = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                             : (int64_t)blockIdx.x;
  if (WARP_ROW && t >= p.T) return;
  const float inv_h = 1.0f / (float)p.H;
  const uint64_t inv2 = f32x2_pack(inv_h, inv_h);
  griddep_wait();
  uint64_t f[NV][N / 2];  // pairs
  uint64_t ss2 = 0;
  uint4 xv[NV][U], rv[NV][U];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + tid) * N;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      xv[i][k] = rv[i][k] = make_uint4(0, 0, 0, 0);
      if (c < p.H) {
        xv[i][k] = ld_stream_v4(p.x + t * p.x_stride + c + 8 * k);
        // a plain load: the sum may be written over the residual
        if (p.residual != nullptr) rv[i][k] = ld_plain_v4(p.residual + t * p.res_stride + c + 8 * k);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + tid) * N;
    bf16_to_f32<U>(xv[i], f[i]);
    if (p.residual != nullptr) {
      uint64_t r[N / 2];
      bf16_to_f32<U>(rv[i], r);
#pragma unroll
      for (int q = 0; q < N / 2; ++q) f[i][q] = f32x2_add_rn(f[i][q], r[q]);
    }
    if (c < p.H && p.res_out != nullptr) store_bf16<U>(p.res_out + t * (int64_t)p.H + c, f[i]);
    // each term over H before the sum: the mean then fits fp32 as long as it
    // does itself, although the sum of squares may not
#pragma unroll
    for (int q = 0; q < N / 2; ++q) ss2 = f32x2_fma_rn(f32x2_mul_rn(f[i][q], inv2), f[i][q], ss2);
  }
  const float ss = row_sum<WARP_ROW>(f32x2_lo(ss2) + f32x2_hi(ss2), red);
  const float k = rsqrtf(ss + p.eps);
  if (tid == 0 && p.rstd != nullptr) p.rstd[t] = k;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * tpr + tid, c = v * N;
    if ((v - (tid & 31)) * N >= p.H) break;  // whole warps only: the scale blocks shuffle
    const bool valid = c < p.H;
    if (valid) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float g[8];
        load_gamma(p.gamma, p.gamma_f32, v * U + j, g);
        const uint64_t k2 = f32x2_pack(k, k);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          f[i][4 * j + q] = f32x2_mul_rn(f32x2_mul_rn(f[i][4 * j + q], k2),
                                         f32x2_pack(g[2 * q], g[2 * q + 1]));
      }
      if (p.y != nullptr) store_bf16<U>(p.y + t * (int64_t)p.H + c, f[i]);
    }
    if constexpr (U == 2) {
      if (p.q != nullptr) {
        float sc;
        uint32_t b[4];
        quantise_block16(f[i], b, &sc);
        if (valid) {
          store_bytes16(p.q + t * (int64_t)p.H + c, b);
          if ((v & 7) == 0) p.sf[t * p.sf_ts + (v >> 3) * p.sf_hs] = sc;
        }
      }
    }
  }
}

template <int U, int NV, bool WARP_ROW>
cudaError_t launch_forward(const NormParams &p, int threads, cudaStream_t s) {
  const int rows = WARP_ROW ? threads / 32 : 1;
  return launch_pdl(norm_kernel<U, NV, WARP_ROW>, (unsigned)((p.T + (int64_t)rows - 1) / rows),
                    threads, 0, s, p);
}

// Persistent CTAs take rows blockIdx.x, + gridDim.x, ...; every thread keeps
// its columns, so the gradient of gamma is summed in registers and leaves as
// one row of partial sums per CTA.
template <int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_backward_kernel(NormBackwardParams p) {
  __shared__ float red[2][32];
  const int nvec = p.H / 8;
  const float inv_h = 1.0f / (float)p.H;
  griddep_wait();
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[i][q] = 0.f;
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    uint4 gv[NV], rv[NV], av[NV];
    const float k = __ldg(p.rstd + t);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      gv[i] = rv[i] = av[i] = make_uint4(0, 0, 0, 0);
      if (v < nvec) {
        const int64_t at = t * p.H + v * 8;
        gv[i] = ld_stream_v4(p.gy + at);
        rv[i] = ld_stream_v4(p.r + at);
        if (p.gres != nullptr) av[i] = ld_plain_v4(p.gres + at);  // gx may be written over it
      }
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v < nvec) {
        float g[8], r[8], w[8];
        bf16x8_to_f32(gv[i], g);
        bf16x8_to_f32(rv[i], r);
        load_gamma(p.gamma, p.gamma_f32, v, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float gx = g[q] * (r[q] * k);
          acc[i][q] += gx;
          m = fmaf(gx, w[q], m);
        }
      }
    }
    m = row_sum<false>(m, red[par]) * inv_h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v < nvec) {
        float g[8], r[8], w[8], a[8], o[8];
        bf16x8_to_f32(gv[i], g);
        bf16x8_to_f32(rv[i], r);
        bf16x8_to_f32(av[i], a);
        load_gamma(p.gamma, p.gamma_f32, v, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = k * (g[q] * w[q] - r[q] * k * m) + a[q];
        st_stream_v4(p.gx + t * (int64_t)p.H + v * 8, f32_to_bf16x8(o));
      }
    }
  }
  if (p.ggamma == nullptr) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < nvec) {
      float4 *o = reinterpret_cast<float4 *>(p.part + (int64_t)blockIdx.x * p.H + v * 8);
      o[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      o[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
}

// out[c] = sum over i < parts of part[i, c], in a fixed order, for the 32 * V
// columns from c0: SPLIT threads of a column sum every SPLIT-th row, then one adds
// their sums.  A thread has V columns, V * 4 bytes of each row.
template <int V, int SPLIT>
__device__ __forceinline__ void column_block(const float *part, int parts, int64_t n, float *out,
                                             int64_t c0, float (*s)[32 * V]) {
  const int c = (threadIdx.x & 31) * V, k = threadIdx.x >> 5;
  const int64_t col = c0 + c;
  float v[V] = {};
  if (col < n) {
#pragma unroll 4
    for (int i = k; i < parts; i += SPLIT) {
      const float *a = part + (int64_t)i * n + col;
      if constexpr (V == 4) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(a));
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
      } else {
        v[0] += __ldg(a);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) s[k][c + j] = v[j];
  __syncthreads();
  const int o = threadIdx.x;
  if (o < 32 * V && c0 + o < n) {
    float t = s[0][o];
    for (int i = 1; i < SPLIT; ++i) t += s[i][o];
    out[c0 + o] = t;
  }
}

// A CTA takes one block of columns, or with CAPPED blocks in turn (the loop's
// registers cost 0.7 us of 10 where every block has its CTA).
template <int V, int SPLIT, bool CAPPED>
__global__ void __launch_bounds__(32 * SPLIT)
    column_sum_kernel(const float *part, int parts, int64_t n, float *out) {
  __shared__ float s[SPLIT][32 * V];
  griddep_wait();
  int64_t c0 = (int64_t)blockIdx.x * (32 * V);
  if constexpr (!CAPPED) {
    column_block<V, SPLIT>(part, parts, n, out, c0, s);
  } else {
    for (; c0 < n; c0 += (int64_t)gridDim.x * (32 * V)) {
      column_block<V, SPLIT>(part, parts, n, out, c0, s);
      __syncthreads();
    }
  }
}

template <int V, int SPLIT>
cudaError_t launch_columns(const float *part, int parts, int64_t n, float *out, int sm_cap,
                           cudaStream_t s) {
  const int64_t blocks = (n + 32 * V - 1) / (32 * V);
  if (sm_cap <= 0)
    return launch_pdl(column_sum_kernel<V, SPLIT, false>, (unsigned)blocks, 32 * SPLIT, 0, s, part,
                      parts, n, out);
  auto kern = column_sum_kernel<V, SPLIT, true>;
  int dev = 0, per_sm = 0;
  const cudaError_t e =
      launch_geometry(reinterpret_cast<const void *>(kern), 32 * SPLIT, 0, &dev, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)sms_to_use(dev, sm_cap) * std::max(per_sm, 1);
  return launch_pdl(kern, (unsigned)std::min(blocks, ctas), 32 * SPLIT, 0, s, part, parts, n, out);
}

// Four vectors per thread (two: 74 us against 60 for 4096 rows of 7168, for the
// barrier spans more warps), but two warps from H = 1024 on (16,384 rows 45 us
// against 49 with one; at H = 512 one is better, 78 us against 100 for 65,536).
int backward_threads(int H) {
  const int nvec = H / 8;
  return std::min(kMaxThreads, std::max(H < 1024 ? 32 : 64, ((nvec + 3) / 4 + 31) / 32 * 32));
}

// The bound gives a short row's CTAs the registers they need: with that of the
// longest, 4096 rows of 7168 take 74 us against 60.  Rows above 16384 spill 308
// bytes a thread: 1024 threads have 64 registers each.
auto backward_kernel(int threads) {
  return threads <= 256   ? norm_backward_kernel<4, 256>
         : threads <= 512 ? norm_backward_kernel<4, 512>
                          : norm_backward_kernel<4, 1024>;
}

}  // namespace

cudaError_t launch_column_sum(const float *part, int parts, int64_t n, float *out, int sm_cap,
                              cudaStream_t s) {
  // Few columns: 32 threads of each; many: 16 bytes a thread, 8 of a column.  608
  // rows of 4096 take 6.7 us one way and 10 the other, 24 of 262,144 33 and 7.8.
  return n >= kWideSum ? launch_columns<4, 8>(part, parts, n, out, sm_cap, s)
                       : launch_columns<1, 32>(part, parts, n, out, sm_cap, s);
}

cudaError_t launch_norm(const NormParams &p, cudaStream_t s) {
  // Short rows take a warp each: H = 128, 262,144 rows 99 us against 140 with a
  // CTA each, H = 256, 131,072 rows 60 against 75; at 512 both take 52.  Longer
  // ones a CTA with 32 elements per thread (16 take 52 us for 4096 rows of 7168
  // where these take 48).
  if (p.H <= kWarpRow)
    return p.H % 16 == 0 ? launch_forward<2, 1, true>(p, 128, s)
                         : launch_forward<1, 2, true>(p, 128, s);
  const int threads = ((p.H + 31) / 32 + 31) / 32 * 32;
  return p.H % 16 == 0 ? launch_forward<2, 2, false>(p, threads, s)
                       : launch_forward<1, 4, false>(p, threads, s);
}

cudaError_t norm_backward_parts(const NormBackwardParams &p, int *parts) {
  const int threads = backward_threads(p.H);
  int dev = 0, per_sm = 0;
  const cudaError_t e = launch_geometry(reinterpret_cast<const void *>(backward_kernel(threads)),
                                        threads, 0, &dev, &per_sm);
  if (e != cudaSuccess) return e;
  *parts = (int)std::min<int64_t>(p.T, (int64_t)device_sm_count(dev) * std::max(per_sm, 1));
  return cudaSuccess;
}

cudaError_t launch_norm_backward(const NormBackwardParams &p, cudaStream_t s) {
  const int threads = backward_threads(p.H);
  const cudaError_t e = launch_pdl(backward_kernel(threads), (unsigned)p.parts, threads, 0, s, p);
  if (e != cudaSuccess || p.ggamma == nullptr) return e;
  return launch_column_sum(p.part, p.parts, p.H, p.ggamma, 0, s);
}

}  // namespace ep
