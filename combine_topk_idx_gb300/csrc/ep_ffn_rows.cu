// The gated product and the product of a few rows with one matrix: a decode step.
//
// Every weight is read once, for at most 16 rows of x, so the time is that of reading the
// matrix.  A CTA takes 16 rows of the matrix (gated: 8 of the gate, the 8 of up beside them);
// its warps share the reduction in chunks of 32 elements, each lane reading 16 bytes of a row,
// several chunks ahead, straight into registers.  There 16 x 8 x 16 products of a warp take
// them as they lie: a lane's eight elements are not the ones that the fragment's layout names,
// but the same ones of the matrix and of x, and a sum has no order.  The warps' sums meet in
// shared memory, in a fixed order.
//
// No stages, no cluster, no TMEM: what the tcgen05 form does around its products is a third of
// so short a call.  Weights read from HBM, 7168 x 4096 gated (58.7 MB, 8.8 us at what a copy
// reaches): 10.5 us for 1 row, 10.9 for 8, 12.3 for 16, where that form takes 14.5; 2048 x
// 7168 as a product 6.6, 6.8 and 8.9 us for 10.4.  What a row more costs is reading x in every
// CTA.  Half or twice as many warps, CTAs per SM or loads ahead change nothing.
#include <algorithm>

#include "ep_ffn.cuh"
#include "ep_ptx.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kPerSm = 2;
constexpr int kUnit = 16;   // rows of the matrix of a CTA

// d += a b, a 16 x 16 and b 16 x 8 of BF16.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kN: groups of 8 rows of x.
template <bool kGated, int kN>
__global__ void __launch_bounds__(kThreads, kPerSm) ffn_rows_kernel(const __grid_constant__ FfnParams p) {
  constexpr int kAhead = 8 / kN;                    // chunks of a warp in flight
  __shared__ float part[kWarps][kUnit][8 * kN];
  const int T = (int)p.s.rows, K = p.K, N = p.N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  constexpr int kOut = kGated ? kUnit / 2 : kUnit;  // columns of the output of a CTA
  const int units = (N + kOut - 1) / kOut;
  griddep_wait();
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int n0 = unit * kOut;
    // this lane's rows of the matrix, in the upper and the lower half of the products' 16;
    // behind the last column any row will do
    const uint16_t *w[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int c = min(n0 + (kGated ? 0 : r * 8) + g, N - 1);
      w[r] = p.b + (int64_t)(kGated && r ? N + c : c) * K + 8 * t;
    }
    const uint16_t *x[kN];
#pragma unroll
    for (int q = 0; q < kN; ++q) x[q] = p.a + (int64_t)(8 * q + g) * p.a_stride + 8 * t;
    float d[kN][4] = {};
    for (int k0 = 32 * warp; k0 < K; k0 += 32 * kWarps * kAhead) {
      uint4 a[kAhead][2], b[kAhead][kN];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * 32 * kWarps;
        const bool in = k + 8 * t < K;
#pragma unroll
        for (int r = 0; r < 2; ++r) a[u][r] = in ? ld_stream_v4(w[r] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < kN; ++q)
          b[u][q] = in && 8 * q + g < T ? ld_cached_v4(x[q] + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int q = 0; q < kN; ++q) {
          const uint4 lo = a[u][0], hi = a[u][1], y = b[u][q];
          mma16816(d[q], lo.x, hi.x, lo.y, hi.y, y.x, y.y);
          mma16816(d[q], lo.z, hi.z, lo.w, hi.w, y.z, y.w);
        }
    }
    __syncthreads();  // the unit before is read
#pragma unroll
    for (int q = 0; q < kN; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        part[warp][8 * (i >> 1) + g][8 * q + 2 * t + (i & 1)] = d[q][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kOut * 8 * kN; i += kThreads) {
      const int c = i % kOut, row = i / kOut, col = n0 + c;
      if (row >= T || col >= N) continue;
      float s = 0.f, u = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        s += part[v][c][row];
        if constexpr (kGated) u += part[v][8 + c][row];
      }
      if constexpr (kGated) {
        const float act = s * f32x2_lo(sigmoid2(f32x2_pack(s, s))) * u;
        if (p.out != nullptr) p.out[(int64_t)row * N + col] = (uint16_t)cvt_bf16x2(act, 0.f);
        if (p.out2 != nullptr) {
          p.out2[(int64_t)row * 2 * N + col] = (uint16_t)cvt_bf16x2(s, 0.f);
          p.out2[(int64_t)row * 2 * N + N + col] = (uint16_t)cvt_bf16x2(u, 0.f);
        }
      } else {
        p.out[(int64_t)row * N + col] = (uint16_t)cvt_bf16x2(s, 0.f);
      }
    }
  }
}

template <bool kGated, int kN>
cudaError_t launch(const FfnParams &p, int sms, cudaStream_t s) {
  constexpr int kOut = kGated ? kUnit / 2 : kUnit;
  const int grid = std::min(sms * kPerSm, (p.N + kOut - 1) / kOut);
  return launch_pdl(ffn_rows_kernel<kGated, kN>, (unsigned)grid, kThreads, 0, s, p);
}

}  // namespace

bool ffn_few_rows(int mode, const FfnParams &p) {
  return p.s.cnt_e == nullptr && (mode == kFfnGated || mode == kFfnProduct) &&
         p.s.rows <= kFfnFewRows;
}

cudaError_t launch_ffn_rows(int mode, const FfnParams &p, int sms, cudaStream_t s) {
  if (p.s.rows <= 8)
    return mode == kFfnGated ? launch<true, 1>(p, sms, s) : launch<false, 1>(p, sms, s);
  return mode == kFfnGated ? launch<true, 2>(p, sms, s) : launch<false, 2>(p, sms, s);
}

}  // namespace ep
