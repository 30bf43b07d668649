// The gated product and the product of a few rows: a decode step.
//
// At most 16 rows, with one matrix or in a layout, each with its expert's.  Every weight is
// read once, so the time is that of reading the matrices.  A CTA takes 16 rows of the matrix
// (gated: 8 of the gate, the 8 of up beside them); its warps share the reduction in chunks of
// 32 elements, each lane reading 16 bytes of a row, several chunks ahead, straight into
// registers.  There 16 x 8 x 16 products of a warp take them as they lie: a lane's eight
// elements are not the ones that the fragment's layout names, but the same ones of the matrix
// and of x, and a sum has no order.  The warps' sums meet in shared memory, in a fixed order.
//
// No stages, no cluster, no TMEM: what the tcgen05 form does around its products is a third of
// so short a call.  Weights read from HBM, 4096 x 7168 gated (58.7 MB, 8.8 us at what a copy
// reaches): 10.5 us for 1 row, 10.9 for 8, 12.3 for 16, where that form takes 14.5; 7168 x
// 2048 as a product 6.6, 6.8 and 8.9 us for 10.4.  What a row more costs is reading x in every
// CTA.  Half or twice as many warps, CTAs per SM or loads ahead change nothing.  One token
// through 2 of 8 experts (4096 x 4096 gated): 14.4 us, by tcgen05 27; through 8 of 256 (4096 x
// 7168) 76 and 79.
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

// kN: groups of 8 rows of x; kLayout: the rows are a layout's.
template <bool kGated, int kN, bool kLayout>
__global__ void __launch_bounds__(kThreads, kPerSm)
    ffn_rows_kernel(const __grid_constant__ FfnParams p) {
  constexpr int kAhead = 8 / kN;                    // chunks of a warp in flight
  __shared__ float part[kWarps][kUnit][8 * kN];
  __shared__ int busy[kFfnFewRows], found[kWarps];
  const int K = p.K, N = p.N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  constexpr int kOut = kGated ? kUnit / 2 : kUnit;  // columns of the output of a CTA
  const int units = (N + kOut - 1) / kOut;          // of an expert
  griddep_wait();
  // the experts with rows, in order, at most as many as there are rows
  int count = kLayout ? 0 : 1;
  for (int e0 = 0; kLayout && e0 < p.s.E; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    const bool has = e < p.s.E && segment_rows(p.s, e).used > 0;
    const uint32_t all = __ballot_sync(0xffffffffu, has);
    if (lane == 0) found[warp] = __popc(all);
    __syncthreads();
    int at = count + __popc(all & lanemask_lt());
    for (int v = 0; v < kWarps; ++v) {
      at += v < warp ? found[v] : 0;
      count += found[v];
    }
    if (has) busy[at] = e;
    __syncthreads();
  }
  for (int item = blockIdx.x; item < count * units; item += gridDim.x) {
    const int e = kLayout ? busy[item / units] : 0, n0 = (kLayout ? item % units : item) * kOut;
    const SegmentRows rows = kLayout ? segment_rows(p.s, e) : SegmentRows{0, p.s.rows, p.s.rows};
    const int T = (int)rows.used;
    const uint16_t *matrix = p.b + (int64_t)e * (kGated ? 2 : 1) * N * K;
    // this lane's rows of the matrix, in the upper and the lower half of the products' 16;
    // behind the last column any row will do
    const uint16_t *w[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int c = min(n0 + (kGated ? 0 : r * 8) + g, N - 1);
      w[r] = matrix + (int64_t)(kGated && r ? N + c : c) * K + 8 * t;
    }
    const uint16_t *x[kN];
#pragma unroll
    for (int q = 0; q < kN; ++q)
      x[q] = p.a + (rows.first + 8 * q + g) * p.a_stride + 8 * t;
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
    // the sums, then zeros in alignment padding
    for (int i = threadIdx.x; i < kOut * (int)rows.write; i += kThreads) {
      const int c = i % kOut, r = i / kOut, col = n0 + c;
      if (col >= N) continue;
      const int64_t row = rows.first + r;
      float v = 0.f, u = 0.f;
      if (r < T) {
#pragma unroll
        for (int q = 0; q < kWarps; ++q) {
          v += part[q][c][r];
          if constexpr (kGated) u += part[q][8 + c][r];
        }
      }
      if constexpr (kGated) {
        const float act = v * f32x2_lo(sigmoid2(f32x2_pack(v, v))) * u;
        if (p.out != nullptr) p.out[row * N + col] = (uint16_t)cvt_bf16x2(act, 0.f);
        if (p.out2 != nullptr) {
          p.out2[row * 2 * N + col] = (uint16_t)cvt_bf16x2(v, 0.f);
          p.out2[row * 2 * N + N + col] = (uint16_t)cvt_bf16x2(u, 0.f);
        }
      } else {
        p.out[row * N + col] = (uint16_t)cvt_bf16x2(v, 0.f);
      }
    }
  }
}

template <bool kGated, int kN, bool kLayout>
cudaError_t launch(const FfnParams &p, int sms, cudaStream_t s) {
  constexpr int kOut = kGated ? kUnit / 2 : kUnit;
  const int64_t experts = std::min<int64_t>(p.max_segments, p.s.E);
  if (experts == 0) return cudaSuccess;  // a layout of no tokens: rows, but none in use
  const int64_t grid = std::min<int64_t>(sms * kPerSm, experts * ((p.N + kOut - 1) / kOut));
  return launch_pdl(ffn_rows_kernel<kGated, kN, kLayout>, (unsigned)grid, kThreads, 0, s, p);
}

// Rows in use, at most: of one matrix all, of a layout its slots.
int64_t most_rows(const FfnParams &p) {
  return p.s.cnt_e == nullptr ? p.s.rows : p.max_segments;
}

}  // namespace

bool ffn_few_rows(int mode, const FfnParams &p) {
  return (mode == kFfnGated || mode == kFfnProduct) && most_rows(p) <= kFfnFewRows;
}

cudaError_t launch_ffn_rows(int mode, const FfnParams &p, int sms, cudaStream_t s) {
  const bool layout = p.s.cnt_e != nullptr, gated = mode == kFfnGated;
  if (most_rows(p) <= 8) {
    if (layout)
      return gated ? launch<true, 1, true>(p, sms, s) : launch<false, 1, true>(p, sms, s);
    return gated ? launch<true, 1, false>(p, sms, s) : launch<false, 1, false>(p, sms, s);
  }
  if (layout) return gated ? launch<true, 2, true>(p, sms, s) : launch<false, 2, true>(p, sms, s);
  return gated ? launch<true, 2, false>(p, sms, s) : launch<false, 2, false>(p, sms, s);
}

}  // namespace ep
