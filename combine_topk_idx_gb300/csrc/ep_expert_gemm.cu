// The experts' FP8 product over the rows of an expanded layout:
//   out[r, n] = bf16( sum over blocks j of  sa[r, j] * sb[e, n / 128, j]
//                     * sum over k in block j of a[r, k] * w[e, n, k] )
// for the rows r of expert e; a and w are e4m3, a scaled by 1x128 blocks, w by
// 128x128 blocks.
//
// One persistent CTA per SM takes tiles of up to kTileR rows and kTileC columns
// of one expert, found on the device from the layout's counts.  The rows are the
// tensor cores' M operand, the weights their N operand.
//   warp 0       copies the operands, a 128-element block per stage, into a
//                ring of stages (tiled TMA, 128-byte swizzle)
//   warp 1       issues the products of a block into one of two TMEM
//                accumulators of kTileC columns
//   warps 4..11  four for each half of the columns: read a finished accumulator
//                and add it, times the scales of its rows and of its weights,
//                to fp32 sums in registers (a thread holds one row and 128
//                columns) while the next block is multiplied
// Each block's sum has its own scales, so it cannot stay in TMEM.  With the
// rows in TMEM lanes a block's scale is one register per thread; with the
// columns there it would be one per accumulator column, and fetching those from
// shared memory takes longer than the products (2310 us against 1569 in the
// last case below).  A row leaves as 32-byte stores straight from registers:
// through shared memory, which the tensor cores keep busy, they took 3 % more.
//
// What bounds it.  Few rows, the weights' bytes: 8 rows, each its expert, N 4096,
// K 7168, 41 us for 235 MB, 5.7 TB/s of 6.7 that a copy reaches.  128 rows per
// expert, 256 experts: 1374 to 1475 us, by GPU, for 8.0 GB, 5.4 to 5.8 TB/s.
// Many rows, the scaled sums: 96,300 rows over 64 experts, N = K = 4096, 1451 to
// 1513 us, 2.1 to 2.2 PFLOP/s, tensor cores busy 53 % of the time.  The products of a
// block take 512 cycles, its operands' way into shared memory and out 768, the
// scaled sums 730 by themselves; with the barriers over two accumulators, all that
// TMEM holds, a block takes about 970.  Pairs of CTAs sharing the operands (1480
// us where one CTA a tile took 1486) did not help, nor does any layout in which an
// epilogue thread spills (20 to 60 % slower): hence 232 registers for it.
//
// Every mbarrier wait is bounded: one that gives up sets EP_ERRBIT_TIMEOUT in
// the handle's error word.  However it ends, the CTA waits (bounded) for what it
// has in flight, frees its TMEM and returns.
#include <algorithm>

#include "ep_internal.cuh"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"
#include "ep_tcgen05.cuh"
#include "ep_tma_host.cuh"

namespace ep {
namespace {

constexpr int kTileR = 128, kTileC = 256, kBlockK = 128;
constexpr int kRowStep = 16;              // a tile's rows are rounded up to this
constexpr int kRowMaps = 4;               // TMA boxes of 16, 32, 64 and 128 rows
constexpr int kStages = 4;
constexpr int kABytes = kTileR * kBlockK;
constexpr int kStageBytes = kABytes + kTileC * kBlockK;
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
constexpr int kTmemColumns = 2 * kTileC;  // two accumulators
constexpr int kWarpC = kTileC / 2;        // columns of an epilogue warp
constexpr int kChunk = 64;                // accumulator columns per TMEM load
// Row tiles that pass over the weights together.  Row tiles first, so that the
// CTAs at work share a weight tile, but no more of them than stay in L2 for the
// next column tile: 98,304 rows over 64 experts with a few large ones, K 7168,
// take 2320 us this way and 2776 with all of an expert's row tiles first.
constexpr int kRaster = 32;
// An epilogue thread loads the scales of one block, or of two together, as long
// ahead of their use.  Two are better where weights stream in for few rows (128
// rows per expert, 256 experts, N 4096, K 7168: 1358 us against 1446; 375 rows,
// K 4096: 1606 against 1626), one where the epilogue is all that counts (1500
// rows per expert, K 4096: 1362 us against 1413).  This many rows per expert, of
// those allocated, is where the choice turns.
constexpr int kGroupRows = 512;
// registers of a control and of an epilogue thread: 128 * 40 + 256 * 232 are
// the 168 * 384 of the launch
constexpr int kControlRegs = 40, kEpilogueRegs = 232;
constexpr int kWaitIters = 4000;          // x kWaitHintNs: gives up after ~2 s
constexpr uint32_t kWaitHintNs = 500000;

struct Tile {
  int e;               // expert
  int64_t row0;        // first row
  int rows, out_rows;  // rows in use from row0, and rows to write (then zeros)
  int height;          // rows multiplied: out_rows up to a multiple of kRowStep
  int c0;              // first column
};

// Height of the row tiles of an expert with n rows to write: all about the same.
__device__ __forceinline__ int tile_height(int n) {
  const int m = max(1, (n + kTileR - 1) / kTileR);
  return max(1, ((n + m - 1) / m + kRowStep - 1) / kRowStep) * kRowStep;
}

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
      const int th = tile_height(write);
      m = (write + th - 1) / th;
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

// Tile i of the experts' tiles.  Whole warps: a search by one thread would be a
// chain of shared-memory reads, each slow while the tensor cores read there.
__device__ __forceinline__ Tile find_tile(const ExpertGemmParams &p, const int *cum, int64_t i,
                                          int tiles_c) {
  const int lane = threadIdx.x & 31;
  int lo = -1;  // the last expert with cum[e] * tiles_c <= i
  for (int e = lane; e - lane < p.E; e += 32)
    lo += __popc(__ballot_sync(0xffffffffu, e < p.E && (int64_t)cum[e] * tiles_c <= i));
  const int tr = cum[lo + 1] - cum[lo];
  const int k = (int)(i - (int64_t)cum[lo] * tiles_c);
  const int g = k / (kRaster * tiles_c) * kRaster;
  const int n = min(kRaster, tr - g), u = k - g * tiles_c;
  const int c = u / n, r = g + u - c * n;
  Tile t;
  int used, write;
  int64_t first;
  expert_rows(p, lo, &first, &used, &write);
  const int th = tile_height(write);
  t.e = lo;
  t.row0 = first + (int64_t)r * th;
  t.rows = max(0, min(th, used - r * th));
  t.out_rows = min(th, write - r * th);
  t.height = (t.out_rows + kRowStep - 1) / kRowStep * kRowStep;
  t.c0 = c * kTileC;
  return t;
}

struct __align__(8) Barriers {
  uint64_t full[kStages];   // a stage's copies landed
  uint64_t empty[kStages];  // the products that read a stage are done
  uint64_t acc_full[2];     // an accumulator is complete
  uint64_t acc_empty[2];    // an accumulator is read
  uint64_t drain;
};

struct Maps {
  CUtensorMap a[kRowMaps], w;
};

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t phase) {
  return mbar_wait_bounded(bar, phase, kWaitIters, kWaitHintNs);
}

// Position in a ring of N slots: slot and the parity of the current round.  A
// consumer waits for `phase`, a producer for the round before (`phase ^ 1`,
// which a fresh barrier passes at once).
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

template <int kGroup>
__global__ void __launch_bounds__(kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ Maps maps, ExpertGemmParams p) {
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
    for (int i = 0; i < kRowMaps; ++i) tma_prefetch_map(&maps.a[i]);
    tma_prefetch_map(&maps.w);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, kTmemColumns);
  griddep_wait();
  count_tiles(p, cum, warp_sum);  // ends with a barrier
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int tiles_c = (p.N + kTileC - 1) / kTileC;
  const int64_t tiles = (int64_t)cum[p.E] * tiles_c;
  const int nk = p.K / kBlockK;

  if (warp < 4) {
    setmaxnreg_dec<kControlRegs>();
    if (warp == 0) {
      // ---------------- copies ----------------
      Ring<kStages> st;
      int issued = 0;  // stages filled, counted up to kStages
      bool ok = true;
      for (int64_t i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
        const Tile t = find_tile(p, cum, i, tiles_c);
        if (t.rows == 0) continue;  // padding only: nothing to multiply
        if (lane == 0) {
          const uint32_t bytes = (uint32_t)((t.height + kTileC) * kBlockK);
          const int w_row = t.e * p.N + t.c0;
          for (int k = 0; k < nk; ++k) {
            if (!wait(&bar.empty[st.slot], st.phase ^ 1)) {
              ok = false;
              break;
            }
            uint8_t *a = smem + st.slot * kStageBytes;
            uint64_t *const full = &bar.full[st.slot];
            mbar_arrive_expect_tx(full, bytes);
            tma_load_2d(a + kABytes, &maps.w, k * kBlockK, w_row, full);
            int r = 0;
#pragma unroll
            for (int b = kRowMaps - 1; b >= 0; --b)  // height = 16 * (sum of 2^b)
              if (t.height & (kRowStep << b)) {
                tma_load_2d(a + r * kBlockK, &maps.a[b], k * kBlockK, (int)t.row0 + r, full);
                r += kRowStep << b;
              }
            st.next();
            if (issued < kStages) ++issued;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (lane == 0) {
        // The products' last arrivals on the stages' barriers: nothing else waits
        // for them, and they must not come after the CTA's shared memory is gone.
        Ring<kStages> left = st;
        for (int s = 0; s < kStages && ok; ++s, left.next())
          ok = wait(&bar.empty[left.slot], left.phase ^ 1);
        if (!ok) {
          atomicOr(p.err, EP_ERRBIT_TIMEOUT);
          // copies in flight: slots below st.slot in this round, the others in
          // the round before
          for (int s = 0; s < kStages; ++s)
            if (s < st.slot || issued == kStages)
              wait(&bar.full[s], s < st.slot ? st.phase : st.phase ^ 1);
        }
      }
    } else if (warp == 1) {
      // ---------------- products ----------------
      // the lanes poll the two barriers of a block side by side
      constexpr uint32_t idesc = idesc_e4m3(kTileR, kTileC);
      Ring<kStages> st;
      Ring<2> acc;
      const uint32_t smem0 = smem_u32(smem);
      bool ok = true;
      for (int64_t i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
        if (find_tile(p, cum, i, tiles_c).rows == 0) continue;
        for (int k = 0; k < nk; ++k) {
          uint64_t *b = lane & 1 ? &bar.acc_empty[acc.slot] : &bar.full[st.slot];
          ok = __all_sync(0xffffffffu, wait(b, lane & 1 ? acc.phase ^ 1 : st.phase));
          if (!ok) break;
          tc_fence_after();
          const uint64_t da = smem_desc_k128(smem0 + st.slot * kStageBytes);
          const uint64_t dw = smem_desc_k128(smem0 + st.slot * kStageBytes + kABytes);
          if (elect_one()) {
#pragma unroll
            for (int q = 0; q < kBlockK / 32; ++q)
              mma_fp8(tmem + acc.slot * kTileC, da + q * 2, dw + q * 2, idesc, q > 0);
            mma_commit(&bar.acc_full[acc.slot]);
            mma_commit(&bar.empty[st.slot]);
          }
          __syncwarp();
          acc.next();
          st.next();
        }
      }
      if (!ok) {
        if (elect_one()) {
          atomicOr(p.err, EP_ERRBIT_TIMEOUT);
          mma_commit(&bar.drain);
        }
        __syncwarp();
        wait(&bar.drain, 0);
      }
    }
  } else {
    // ---------------- scaled sums and output ----------------
    setmaxnreg_inc<kEpilogueRegs>();
    const int quarter = warp & 3;           // TMEM lanes of this warp
    const int j = (warp - 4) >> 2;          // half of the columns
    const int m = quarter * 32 + lane;      // row of the tile
    const uint32_t taddr = tmem + (uint32_t)(quarter * 32) * 65536u + j * kWarpC;
    const int nc = (p.N + 127) / 128;
    Ring<2> acc;
    // After a wait that gave up, the rest of the tile is walked without waiting.
    bool ok = true;
    for (int64_t i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
      const Tile t = find_tile(p, cum, i, tiles_c);
      const bool mine = m < t.rows;
      const bool work = quarter * 32 < t.out_rows;  // any row of the warp
      const int blocks = t.rows > 0 ? nk : 0;
      const float *sa = p.sf + (mine ? sf_at(p.sfl, t.row0 + m, 0) : 0);
      const float *sw =
          p.w_sf + ((int64_t)t.e * nc + min(t.c0 / 128 + j, nc - 1)) * nk;
      uint64_t sum[kWarpC / 2];             // pairs of columns
#pragma unroll
      for (int c = 0; c < kWarpC / 2; ++c) sum[c] = 0;
      // scales of the next kGroup blocks, loaded together a group ahead
      float na[kGroup], nw[kGroup];
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        na[u] = mine && u < blocks ? __ldg(sa + u * p.sfl.hs) : 0.f;
        nw[u] = u < blocks ? __ldg(sw + u) : 0.f;
      }
      for (int k0 = 0; k0 < blocks; k0 += kGroup) {
        float s[kGroup];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) s[u] = na[u] * nw[u];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          const int k = k0 + kGroup + u;
          na[u] = mine && k < blocks ? __ldg(sa + k * p.sfl.hs) : 0.f;
          nw[u] = k < blocks ? __ldg(sw + k) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          if (k0 + u < blocks) {
            if (ok) ok = __all_sync(0xffffffffu, wait(&bar.acc_full[acc.slot], acc.phase));
            tc_fence_after();
            const uint32_t ta = taddr + acc.slot * kTileC;
            if (work) {
              const uint64_t s2 = f32x2_pack(s[u], s[u]);
#pragma unroll
              for (int c = 0; c < kWarpC / kChunk; ++c) {
                uint32_t d[kChunk];
                tmem_load64(ta + c * kChunk, d);
                tmem_load_wait(d);
                if (c + 1 == kWarpC / kChunk) {  // read: a later block may overwrite it
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&bar.acc_empty[acc.slot]);
                }
#pragma unroll
                for (int q = 0; q < kChunk / 2; ++q)
                  sum[c * kChunk / 2 + q] = f32x2_fma_rn(
                      f32x2_pack(__uint_as_float(d[2 * q]), __uint_as_float(d[2 * q + 1])), s2,
                      sum[c * kChunk / 2 + q]);
              }
            } else if (lane == 0) {
              mbar_arrive(&bar.acc_empty[acc.slot]);
            }
            acc.next();
          }
        }
      }
      if (!ok || !work) continue;
      if (m < t.out_rows) {
        const int col = t.c0 + j * kWarpC;
        uint16_t *o = p.out + (t.row0 + m) * p.N + col;
#pragma unroll
        for (int c = 0; c < kWarpC; c += 16) {
          uint32_t v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint64_t x = sum[c / 2 + q];
            v[q] = mine ? cvt_bf16x2(f32x2_lo(x), f32x2_hi(x)) : 0u;
          }
          if (p.out32 && col + c + 16 <= p.N) {
            st_stream_v8(o + c, v);
          } else {
            if (col + c + 8 <= p.N) st_stream_v4(o + c, make_uint4(v[0], v[1], v[2], v[3]));
            if (col + c + 16 <= p.N) st_stream_v4(o + c + 8, make_uint4(v[4], v[5], v[6], v[7]));
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
  Maps maps;
  bool ok = make_map(&maps.w, p.w, (int64_t)p.E * p.N, p.K, kTileC);
  for (int i = 0; i < kRowMaps; ++i)
    ok = ok && make_map(&maps.a[i], p.a, p.rows_alloc, p.K, kRowStep << i);
  if (!ok) return cudaErrorInvalidValue;
  const auto kernel = p.rows_alloc <= (int64_t)kGroupRows * p.E ? expert_gemm_kernel<2>
                                                                 : expert_gemm_kernel<1>;
  const size_t smem = 1024 + (size_t)kStages * kStageBytes + sizeof(int) * (p.E + 1);
  int dev = 0;
  const cudaError_t e = launch_geometry(reinterpret_cast<const void *>(kernel),
                                        kThreads, smem, &dev, nullptr);
  if (e != cudaSuccess) return e;
  const int use = sms_to_use(dev, sm_cap);
  // at most this many row tiles hold rows (every expert's last one may be partial)
  const int64_t tiles_r = std::min<int64_t>(p.max_slots, p.E) + 2 * (p.rows_alloc / kTileR);
  const int64_t tiles = std::max<int64_t>(1, tiles_r * ((p.N + kTileC - 1) / kTileC));
  return launch_pdl(kernel, (unsigned)std::min<int64_t>(use, tiles), kThreads, smem, s,
                    maps, p);
}

}  // namespace ep
