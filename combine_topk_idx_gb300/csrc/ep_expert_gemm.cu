// The experts' FP8 product over the rows of an expanded layout:
//   out[r, n] = bf16( sum over blocks j of  sa[r, j] * sb[e, n / 128, j]
//                     * sum over k in block j of a[r, k] * w[e, n, k] )
// for the rows r of expert e; a and w are e4m3, a scaled by 1x128 blocks, w by
// 128x128 blocks.
//
// One persistent CTA per SM takes output tiles of kTileM rows x kTileN
// columns of one expert, found on the device from the layout's counts.  Warp 0
// copies the operands (tiled TMA, 128-byte swizzle) into a ring of stages of
// one 128-element block each; one thread of warp 1 issues the tcgen05 products
// of a block into one of two TMEM accumulators; the epilogue warps (4..11)
// read a finished block's accumulator and add it, times its scales, to fp32
// sums in registers (a thread holds one row and 128 columns), while the next
// block is multiplied into the other accumulator.  Each block's sum has its
// own scales, so it cannot stay in TMEM: per block the tensor cores need
// kTileN * 2 cycles (8192 multiply-adds a cycle), reading the accumulator half
// of that and its multiply-adds as much again, on other units.
//
// Every mbarrier wait is bounded: one that gives up sets EP_ERRBIT_TIMEOUT in
// the handle's error word, and the CTA waits (bounded) for what it has in
// flight, frees its TMEM and returns.
#include <algorithm>

#include "ep_internal.cuh"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"
#include "ep_tcgen05.cuh"

namespace ep {
namespace {

constexpr int kTileM = 128, kTileN = 256, kBlockK = 128;
constexpr int kStages = 4;
constexpr int kABytes = kTileM * kBlockK, kBBytes = kTileN * kBlockK;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
constexpr int kTmemColumns = 512;         // two accumulators of kTileN columns
// registers of a control and of an epilogue thread: 128 * 88 + 256 * 208 are
// the 168 * 384 of the launch
constexpr int kControlRegs = 88, kEpilogueRegs = 208;
constexpr int kWaitIters = 4000;          // x kWaitHintNs: gives up after ~2 s
constexpr uint32_t kWaitHintNs = 500000;

struct Tile {
  int e;             // expert
  int64_t row0;      // first row
  int rows, out_rows;  // rows in use from row0, and rows to write (then zeros)
  int n0;            // first column
};

// Rows of expert e: first, in use, and to write (alignment padding zeroed).
__device__ __forceinline__ void expert_rows(const ExpertGemmParams &p, int e, int64_t *first,
                                            int *used, int *write) {
  const int cnt = __ldg(p.cnt_e + e);
  if (p.fixed_cap > 0) {
    *first = (int64_t)e * p.fixed_cap;
    *used = *write = min(cnt, p.fixed_cap);
    return;
  }
  const int64_t r0 = __ldg(p.psum_e + e);
  const int64_t left = max((int64_t)0, p.rows_alloc - r0);
  *first = r0;
  *used = (int)min((int64_t)cnt, left);
  *write = p.zero_padding ? (int)min((int64_t)__ldg(p.psum_e + e + 1) - r0, left) : *used;
}

// cum[e]: row tiles of the experts before e (e <= E).  All threads.
__device__ __forceinline__ void count_tiles(const ExpertGemmParams &p, int *cum, int *warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int e0 = 0; e0 < p.E; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    int m = 0;
    if (e < p.E) {
      int64_t first;
      int used, write;
      expert_rows(p, e, &first, &used, &write);
      m = (write + kTileM - 1) / kTileM;
    }
    int v = m;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    int before = base, all = base;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    if (e < p.E) cum[e] = before + v - m;
    base = all;
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[p.E] = base;
  __syncthreads();
}

// Tile i of the experts' tiles: row tiles first, so that the CTAs at work
// share a weight tile through L2.
__device__ __forceinline__ Tile find_tile(const ExpertGemmParams &p, const int *cum, int64_t i,
                                          int tiles_n) {
  int lo = 0, hi = p.E - 1;  // the last expert with cum[e] * tiles_n <= i
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)cum[mid] * tiles_n <= i) lo = mid; else hi = mid - 1;
  }
  const int tm = cum[lo + 1] - cum[lo];
  const int k = (int)(i - (int64_t)cum[lo] * tiles_n);
  const int n = k / tm, m = k - n * tm;
  Tile t;
  int used, write;
  int64_t first;
  expert_rows(p, lo, &first, &used, &write);
  t.e = lo;
  t.row0 = first + (int64_t)m * kTileM;
  t.rows = max(0, min(kTileM, used - m * kTileM));
  t.out_rows = min(kTileM, write - m * kTileM);
  t.n0 = n * kTileN;
  return t;
}

struct __align__(8) Barriers {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain;
};

__global__ void __launch_bounds__(kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, ExpertGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int warp_sum[kThreads / 32];
  // stages on 1024-byte boundaries (the swizzle's period), then cum[E + 1]
  uint8_t *smem = smem_raw + (1024 - smem_u32(smem_raw) % 1024) % 1024;
  int *cum = reinterpret_cast<int *>(smem + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bar.acc_full[b], 1);
      mbar_init(&bar.acc_empty[b], kEpilogueWarps);
    }
    mbar_init(&bar.drain, 1);
    fence_mbar_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kTmemColumns);
    tmem_relinquish();
  }
  griddep_wait();
  count_tiles(p, cum, warp_sum);  // ends with a barrier
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int tiles_n = (p.N + kTileN - 1) / kTileN;
  const int64_t tiles = (int64_t)cum[p.E] * tiles_n;
  const int nk = p.K / kBlockK;

  if (warp < 4) {
    setmaxnreg_dec<kControlRegs>();
    if (warp == 0 && lane == 0) {
      // ---------------- copies ----------------
      int64_t it = 0;
      bool ok = true;
      for (int64_t i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
        const Tile t = find_tile(p, cum, i, tiles_n);
        if (t.rows == 0) continue;  // padding only: nothing to multiply
        const int b_row = t.e * p.N + t.n0;
        for (int k = 0; k < nk; ++k, ++it) {
          const int s = (int)(it % kStages);
          if (it >= kStages &&
              !mbar_wait_bounded(&bar.empty[s], (uint32_t)((it / kStages - 1) & 1), kWaitIters,
                                 kWaitHintNs)) {
            ok = false;
            break;
          }
          uint8_t *a = smem + s * kStageBytes;
          mbar_arrive_expect_tx(&bar.full[s], kStageBytes);
          tma_load_2d(a, &map_a, k * kBlockK, (int)t.row0, &bar.full[s]);
          tma_load_2d(a + kABytes, &map_b, k * kBlockK, b_row, &bar.full[s]);
        }
      }
      if (!ok) {
        atomicOr(p.err, EP_ERRBIT_TIMEOUT);
        for (int64_t j = it > kStages ? it - kStages : 0; j < it; ++j)  // copies in flight
          mbar_wait_bounded(&bar.full[j % kStages], (uint32_t)((j / kStages) & 1), kWaitIters,
                            kWaitHintNs);
      }
    } else if (warp == 1 && lane == 0) {
      // ---------------- products ----------------
      constexpr uint32_t idesc = idesc_e4m3(kTileM, kTileN);
      int64_t it = 0;
      bool ok = true;
      for (int64_t i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
        if (find_tile(p, cum, i, tiles_n).rows == 0) continue;
        for (int k = 0; k < nk; ++k, ++it) {
          const int s = (int)(it % kStages), b = (int)(it & 1);
          if ((it >= 2 && !mbar_wait_bounded(&bar.acc_empty[b], (uint32_t)((it / 2 - 1) & 1),
                                             kWaitIters, kWaitHintNs)) ||
              !mbar_wait_bounded(&bar.full[s], (uint32_t)((it / kStages) & 1), kWaitIters,
                                 kWaitHintNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + s * kStageBytes);
          const uint64_t da = smem_desc_k128(a), db = smem_desc_k128(a + kABytes);
#pragma unroll
          for (int q = 0; q < kBlockK / 32; ++q)
            mma_fp8(tmem + b * kTileN, da + q * 2, db + q * 2, idesc, q > 0);
          mma_commit(&bar.empty[s]);
          mma_commit(&bar.acc_full[b]);
        }
      }
      if (!ok) {
        atomicOr(p.err, EP_ERRBIT_TIMEOUT);
        mma_commit(&bar.drain);
        mbar_wait_bounded(&bar.drain, 0, kWaitIters, kWaitHintNs);
      }
    }
  } else {
    // ---------------- scaled sums and output ----------------
    setmaxnreg_inc<kEpilogueRegs>();
    const int quarter = warp & 3;           // TMEM lanes of this warp
    const int half = (warp - 4) >> 2;       // columns half * 128 ..
    const int m = quarter * 32 + lane;
    const uint32_t taddr = tmem + (uint32_t)(quarter * 32) * 65536u + half * 128;
    const int nb = (p.N + 127) / 128;
    int64_t it = 0;
    bool ok = true;
    for (int64_t i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
      const Tile t = find_tile(p, cum, i, tiles_n);
      const int64_t row = t.row0 + m;
      const int col = t.n0 + half * 128;
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.f;
      if (t.rows > 0) {
        const bool mine = m < t.rows;
        const float *sa = p.sf + (mine ? sf_at(p.sfl, row, 0) : 0);
        const float *sb =
            p.w_sf + ((int64_t)t.e * nb + min(col / 128, nb - 1)) * nk;
        float a_next = mine ? __ldg(sa) : 0.f, b_next = __ldg(sb);
        for (int k = 0; k < nk; ++k, ++it) {
          const float scale = a_next * b_next;
          if (k + 1 < nk) {
            a_next = mine ? __ldg(sa + (int64_t)(k + 1) * p.sfl.hs) : 0.f;
            b_next = __ldg(sb + k + 1);
          }
          const int b = (int)(it & 1);
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar.acc_full[b], (uint32_t)((it / 2) & 1),
                                                         kWaitIters, kWaitHintNs));
          if (!ok) break;
          tc_fence_after();
          float d[2][16];
          tmem_load16(taddr + b * kTileN, d[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tmem_load_wait16(d[c & 1]);
            if (c < 7) {
              tmem_load16(taddr + b * kTileN + (c + 1) * 16, d[(c + 1) & 1]);
            } else {  // the accumulator is read: the next block may overwrite it
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar.acc_empty[b]);
            }
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[c * 16 + q] = fmaf(d[c & 1][q], scale, acc[c * 16 + q]);
          }
        }
      }
      if (ok && m < t.out_rows) {
        const bool in = m < t.rows;
        uint16_t *o = p.out + row * p.N + col;
#pragma unroll
        for (int c = 0; c < 128; c += 16) {
          uint32_t v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            v[q] = in ? cvt_bf16x2(acc[c + 2 * q], acc[c + 2 * q + 1]) : 0u;
          const uint4 lo = make_uint4(v[0], v[1], v[2], v[3]);
          const uint4 hi = make_uint4(v[4], v[5], v[6], v[7]);
          if (p.out32 && col + c + 16 <= p.N) {
            st_stream_v8(o + c, lo, hi);
          } else {
            if (col + c + 8 <= p.N) st_stream_v4(o + c, lo);
            if (col + c + 16 <= p.N) st_stream_v4(o + c + 8, hi);
          }
        }
      }
    }
    if (!ok && lane == 0) atomicOr(p.err, EP_ERRBIT_TIMEOUT);
    tc_fence_before();
  }
  __syncthreads();
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem, kTmemColumns);
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Rows of K bytes, copied as boxes of 128 bytes x box_rows, zeros outside.
bool make_map(CUtensorMap *map, const void *base, int64_t rows, int K, int box_rows) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K};
  const cuuint32_t box[2] = {(cuuint32_t)kBlockK, (cuuint32_t)box_rows};
  const cuuint32_t step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
            step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_expert_gemm(const ExpertGemmParams &p, int sm_cap, cudaStream_t s) {
  CUtensorMap map_a, map_b;
  if (!make_map(&map_a, p.a, p.rows_alloc, p.K, kTileM) ||
      !make_map(&map_b, p.w, (int64_t)p.E * p.N, p.K, kTileN))
    return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)kStages * kStageBytes + sizeof(int) * (p.E + 1);
  const void *func = reinterpret_cast<const void *>(expert_gemm_kernel);
  int dev = 0;
  const cudaError_t e = launch_geometry(func, kThreads, smem, &dev, nullptr);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count(dev);
  const int use = (sm_cap > 0 && sm_cap < sms) ? sm_cap : sms;
  // at most this many row tiles hold rows (every expert's last one may be partial)
  const int64_t tiles_m = std::min<int64_t>(p.max_slots, p.E) + p.rows_alloc / kTileM;
  const int64_t tiles = tiles_m * ((p.N + kTileN - 1) / kTileN);
  return launch_pdl(expert_gemm_kernel, (unsigned)std::min<int64_t>(use, std::max<int64_t>(tiles, 1)),
                    kThreads, smem, s, map_a, map_b, p);
}

}  // namespace ep
