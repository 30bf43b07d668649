// The BF16 products of a trained feed-forward block, with what stands around
// them fused into their last step.  W [E, ...] one matrix per expert, rows r of
// a layout sorted by expert (or E = 1 and all rows):
//   gated        h = x W^T, W [2F, K] gate rows then up rows;
//                act = silu(h_gate) * h_up, and h itself for the backward pass
//   gated grad   d = g W, W [K, F] the down projection; with the forward's h:
//                dh = (d h_up silu'(h_gate), d silu(h_gate)), and act of h as kept
//   product      out = a W^T, W [N, K], or a W, W [K, N] (transposed)
//   weight grad  W'[e] = sum over e's rows of g[r]^T a[r]
// Sums in fp32 (TMEM; long ones of a weight gradient joined of parts), each output rounded
// once.
//
// A tile is 128 rows x 256 columns of a CTA's TMEM (gated: 128 gate columns and
// the 128 up columns beside them).  Warps of a CTA:
//   0       copies the operands, 64 reduction elements per stage, into a ring of
//           stages (tiled TMA, 128-byte swizzle)
//   1       issues the products into one of two accumulators
//   4..11   four for each half of the columns: read a finished accumulator, apply
//           the rest of the formula and store, while the next tile is multiplied
// An operand whose contiguous dimension is the reduction is taken row by row, one
// whose contiguous dimension is the output's as it lies in memory too (the tensor
// cores transpose): no operand is laid out again.
//
// Three forms of one kernel:
//   kPair 1   persistent, a CTA per SM
//   kPair 2   persistent, two CTAs on a 256 x 256 tile: each holds its 128 rows and
//             half of the columns' operand
//   kSplit    few tiles: 128 x 128 ones (of pairs 256 x 256), a cluster per tile, its CTAs
//             or pairs share the reduction and add up through each other's shared memory, in
//             a fixed order
// Up to 16 rows in all are ep_ffn_rows.cu's, if gated or a product on W's rows.
//
// What bounds it (times move by 8 % with the GPU and what it ran before: the power cap sets
// its clock; sizes are rows x n x k as the calls name them, n of a gated product gate and up
// together).  Large tiles, the tensor cores: a block of a 256 x 256 tile takes 521 cycles
// where its products need 512; 8192 x 8192 x 4096 takes 268 to 290 us, up to 2.05 PFLOP/s, and
// as torch.matmul, timed in turn with it, 266 to 290.  What an epilogue reads and writes competes with the operands for L2:
// the gated gradient of that size moves 670 MB more and takes 353 us.  128 rows per expert,
// the weights' bytes: 256 experts of 4096 x 7168, 2.46 ms for 15.9 GB, 6.5 TB/s.  Few rows
// through one matrix, latency: 128 x 7168 x 2048 takes 10.0 us, of them 1.2 before the first
// copy and 2 from the last product to the end.
//
// Rows that are not an expert's own never reach its results: in the row products
// they are other rows of the accumulator; in the weight gradient, where they
// would be summed, an expert's tensor map ends with its last row, and what a copy
// reads behind it is zero.
//
// Every mbarrier wait is bounded.  One that gives up sets EP_ERRBIT_TIMEOUT in
// the handle's error word (where there is one) and the tiles that are not done
// hold NaN.  However it ends, the CTA waits (bounded) for what it has in flight,
// frees its TMEM and returns.
#include <algorithm>
#include <mutex>
#include <type_traits>
#include <vector>

#include "ep_ffn.cuh"
#include "ep_ptx.cuh"
#include "ep_tcgen05.cuh"
#include "ep_tma_host.cuh"

namespace ep {
namespace {

constexpr int kTileM = 128, kBlockK = 64;
constexpr int kRowStep = 16;   // a tile's rows are copied up to a multiple of this
constexpr int kRowMaps = 4;    // boxes of 16, 32, 64 and 128 rows
constexpr int kBoxBytes = 64 * kBlockK * 2;  // 64 columns of a 64-element block
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
// Blocks that a weight gradient in 32 bits adds up in TMEM before its sums go on in
// registers, rounded to nearest: the tensor cores cut off what does not fit, which
// over 4096 rows is 4.4e-6 of the result, over 512 at a time 4.7e-7.
constexpr int kJoin = 8;
// The same of one in BF16, whose rounding is 2^-8.  The tensor cores add 16 rows at a time and
// cut off at most 2^-23 of the sum so far: at most 2^-10 of sums of one sign after this many
// blocks (131072 rows).  Without end, 2^20 positive products were off by 4e-3 beside the
// rounding and 2^22 by 2e-2.
constexpr int kLongBlocks = 2048;
constexpr int kSumsBytes = kTileM * 256 * 4;  // of a CTA between two parts
// registers of a control and of an epilogue thread where the latter need more than
// 168: 128 * 88 + 256 * 208 are the 168 * 384 of the launch.  With 72 the copies' loop
// spilt and took 690 cycles a block, whose products take 512.
constexpr int kControlRegs = 88, kEpilogueRegs = 208;
constexpr int kMaxSplit = 4;   // CTAs, or pairs, that share a tile's reduction
constexpr int kPairSplitBlocks = 24;  // of each pair; see launch_mode
constexpr int kRaster = 16;    // row tiles that pass over the columns together
constexpr int kWaitIters = 4000;          // x kWaitHintNs: gives up after ~2 s
constexpr uint32_t kWaitHintNs = 500000;

__host__ __device__ constexpr bool weight_grad16(int mode) {
  return mode == kFfnWeightGrad || mode == kFfnWeightGradLong;
}
__host__ __device__ constexpr bool weight_grad(int mode) {
  return weight_grad16(mode) || mode == kFfnWeightGrad32;
}

// A pair's weight gradients in 32 bits leave by TMA, through 8 KB of each epilogue warp: 256
// x 4096 x 7168 takes 33 us where 32-byte stores of each thread's row took 39.  What is BF16
// is stored from registers, and the memory is a sixth stage: 8192 x 8192 x 4096 took 281 us
// as a product where TMA and five stages took 287, 358 as the gated gradient where they took
// 385 (all measured on the same GPU).
template <int kMode, int kPair, bool kSplit>
struct Ring_ {
  static constexpr int kCols = kSplit && kPair == 1 ? 128 : 256;  // accumulator columns of a tile
  static constexpr int kABytes = kTileM * kBlockK * 2;
  static constexpr int kBBytes = kCols / kPair * kBlockK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr bool kTmaOut = kPair == 2 && kMode == kFfnWeightGrad32;
  static constexpr int kStages = kTmaOut ? 5 : 2 * kABytes == kStageBytes ? 6 : 4;
  static constexpr int kOutBytes = kTmaOut ? 8192 : 0;  // of an epilogue warp
  static constexpr int kSmem = kStages * kStageBytes + kEpilogueWarps * kOutBytes;
};

struct Maps {
  CUtensorMap a[kRowMaps], b, b_small;  // operands; b in boxes of a split tile's half
  CUtensorMap out;             // a pair's weight gradients in 32 bits
};

struct __align__(8) Barriers {
  uint64_t full[6];       // a stage's copies landed (the pair's first CTA)
  uint64_t empty[6];      // the products that read a stage are done
  uint64_t acc_full[2];   // an accumulator is complete
  uint64_t acc_empty[2];  // an accumulator is read (the pair's first CTA)
  uint64_t drain;
};

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t phase) {
  return mbar_wait_bounded(bar, phase, kWaitIters, kWaitHintNs);
}

// Position in a ring of N slots; see the waits: a consumer waits for `phase`, a
// producer for the round before (`phase ^ 1`, which a fresh barrier passes).
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

struct Tile {
  int e;         // expert
  int64_t row0;  // first row of the output (weight gradient: within the expert's matrix)
  int used;      // rows of the tile with a result
  int write;     // rows to write: the used ones, then zeros
  int n0;        // first column
  int cols;      // columns: of a whole tile, or of half of one
  int64_t k0;    // weight gradient: first row of the sum
  int blocks;    // blocks of the reduction
};

// Row tiles of the experts before e (row products; e <= E) in cum[e].  All threads.
__device__ __forceinline__ void count_tiles(const FfnParams &p, int rows_per_tile, int *cum,
                                            int *warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int e0 = 0; e0 < p.s.E; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    int m = 0;
    if (e < p.s.E) {
      const SegmentRows r = segment_rows(p.s, e);
      m = (int)((r.write + rows_per_tile - 1) / rows_per_tile);
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
    if (e < p.s.E) cum[e] = before + v - m;
    base = all;
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[p.s.E] = base;
  __syncthreads();
}

// a / b with b's Reciprocal: at most one short before the correction.  (Divisions by registers
// take a few hundred cycles, and a tile's place several of them, before the first copy.)
__device__ __forceinline__ uint32_t divide(uint32_t a, Reciprocal b) {
  const uint32_t q = __umulhi(a, b.magic);
  return q + (a - q * b.of >= b.of ? 1 : 0);
}

// (row, column) of tile k of tr x tc: kRaster row tiles pass over the columns together.
__device__ __forceinline__ void raster(int k, int tr, int tc, Reciprocal per, int *r, int *c) {
  const int g = (int)divide((uint32_t)k, per) * kRaster;
  const int n = min(kRaster, tr - g), u = k - g * tc;
  // u < 2^14, n <= 16: (u + 1/2) / n lies 1/32 off every whole number, fp32 2^-9 off at most
  *c = (int)(((float)u + 0.5f) * rcp_approx((float)n));
  *r = g + u - *c * n;
}

// Tile i.  Whole warps.
template <int kMode, int kCols>
__device__ __forceinline__ Tile find_tile(const FfnParams &p, const int *cum, int i,
                                          int rows_per_tile, int tiles_n) {
  Tile t;
  int r, c;
  if constexpr (weight_grad(kMode)) {
    const int tr = (p.M + rows_per_tile - 1) / rows_per_tile;
    t.e = (int)divide((uint32_t)i, p.expert_tiles);
    raster(i - t.e * (int)p.expert_tiles.of, tr, tiles_n, p.raster_tiles, &r, &c);
    const SegmentRows s = segment_rows(p.s, t.e);
    t.row0 = (int64_t)r * rows_per_tile;
    t.used = t.write = min(rows_per_tile, p.M - (int)t.row0);
    t.k0 = s.first;
    t.blocks = (int)((s.used + kBlockK - 1) / kBlockK);
  } else {
    int lo = 0;
    if (p.s.cnt_e == nullptr) {
      raster(i, (int)((p.s.rows + rows_per_tile - 1) / rows_per_tile), tiles_n, p.raster_tiles,
             &r, &c);
    } else {
      const int lane = threadIdx.x & 31;
      lo = -1;  // the last expert with cum[e] * tiles_n <= i
      for (int e = lane; e - lane < p.s.E; e += 32)
        lo += __popc(__ballot_sync(0xffffffffu, e < p.s.E && cum[e] * tiles_n <= i));
      raster(i - cum[lo] * tiles_n, cum[lo + 1] - cum[lo], tiles_n, p.raster_tiles, &r, &c);
    }
    const SegmentRows s = segment_rows(p.s, lo);
    const int64_t off = (int64_t)r * rows_per_tile;
    t.e = lo;
    t.row0 = s.first + off;
    t.used = (int)max((int64_t)0, min((int64_t)rows_per_tile, s.used - off));
    t.write = (int)min((int64_t)rows_per_tile, s.write - off);
    t.k0 = 0;
    t.blocks = t.used > 0 ? (p.K + kBlockK - 1) / kBlockK : 0;
  }
  t.n0 = c * kCols;
  t.cols = kCols;
  return t;
}

// Columns of a tile's accumulator.
template <int kMode>
__device__ __forceinline__ int acc_columns(const Tile &t) {
  return kMode == kFfnGated ? 2 * t.cols : t.cols;
}

// Rows of a tile that CTA `rank` of a pair takes: from which, and how many of n.
// Halves are multiples of kRowStep, so that few rows are shared out too.
template <int kMode, int kPair>
__device__ __forceinline__ int half_of(const Tile &t) {
  if (kPair == 1) return kTileM;
  if (weight_grad(kMode)) return kTileM;
  return ((t.write + 1) / 2 + kRowStep - 1) / kRowStep * kRowStep;
}

// ---- what is computed of 16 accumulated columns -----------------------------------------
// In pairs of columns, two to a register pair (8192 x 8192 x 4096 gated 316 us, 327 singly).

typedef uint64_t Pairs[8];

__device__ __forceinline__ uint64_t join(uint32_t lo, uint32_t hi) {
  return f32x2_pack(__uint_as_float(lo), __uint_as_float(hi));
}

__device__ __forceinline__ bool on_32(const void *p) {
  return (reinterpret_cast<uintptr_t>(p) & 31) == 0;
}

// 16 columns of a row from `o` on (16-byte aligned), of which `left` are in the row.
__device__ __forceinline__ void store16(uint16_t *o, int left, const uint32_t (&w)[8]) {
  if (left >= 16 && on_32(o)) {
    st_stream_v8(o, w);
  } else {
    if (left >= 8) st_stream_v4(o, make_uint4(w[0], w[1], w[2], w[3]));
    if (left >= 16) st_stream_v4(o + 8, make_uint4(w[4], w[5], w[6], w[7]));
  }
}

// A row's output, 16 columns after another.  Where the row starts in the middle of a sector
// (every second row of 8 more than a multiple of 16 columns), each piece's last 8 columns wait
// for the next one's first 8, so that sectors are still stored whole: the gated gradient of
// 8192 x 6776 x 2048 takes 225 us, 347 in half sectors (of the loads too, see RowIn) and 171
// at 6784 columns.
struct RowOut {
  uint16_t *o;
  int left;       // columns in the row
  bool odd, has;  // starts in the middle of a sector; 8 columns wait
  uint4 rest;
  __device__ __forceinline__ void begin(uint16_t *at, int columns) {
    o = at;
    left = columns;
    odd = !on_32(at);
    has = false;
  }
  __device__ __forceinline__ void put(const uint32_t (&w)[8]) {
    if (!odd) {
      store16(o, left, w);
    } else if (left >= 8) {
      if (has) {
        const uint32_t v[8] = {rest.x, rest.y, rest.z, rest.w, w[0], w[1], w[2], w[3]};
        st_stream_v8(o - 8, v);
      } else {
        st_stream_v4(o, make_uint4(w[0], w[1], w[2], w[3]));
      }
      has = left >= 16;
      rest = make_uint4(w[4], w[5], w[6], w[7]);
    }
    o += 16;
    left -= 16;
  }
  __device__ __forceinline__ void end() {
    if (has) st_stream_v4(o - 8, rest);
  }
};

// 16 BF16 values from `a` on, of which `left` are there; zeros behind them.  A sector at once
// where it starts there: in two halves it is fetched twice.
template <bool kReadOnly>
__device__ __forceinline__ uint4 load8(const uint16_t *a) {
  return kReadOnly ? ld_stream_v4(a) : ld_plain_v4(a);
}
template <bool kReadOnly>
__device__ __forceinline__ void load16(const uint16_t *a, int left, uint4 &lo, uint4 &hi) {
  if (left >= 16 && on_32(a)) {
    uint4 v[2];
    if (kReadOnly)
      ld_stream_v8(a, v);
    else
      ld_plain_v8(a, v);
    lo = v[0], hi = v[1];
    return;
  }
  lo = left >= 8 ? load8<kReadOnly>(a) : make_uint4(0, 0, 0, 0);
  hi = left >= 16 ? load8<kReadOnly>(a + 8) : make_uint4(0, 0, 0, 0);
}

// A row's input, 32 columns after another, each loaded while the ones before are worked on.
// In a row that starts in the middle of a sector the loads are 8 columns ahead of their use.
template <bool kShifted, bool kReadOnly>  // not shifted: no row does; not written by the kernel
struct RowIn {
  uint4 r[4], first;
  bool odd;
  __device__ __forceinline__ void begin(const uint16_t *at, int left) {
    odd = kShifted && !on_32(at);
    first = odd && left >= 8 ? load8<kReadOnly>(at) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const uint16_t *at, int left) {
    const int skip = odd ? 8 : 0;
    load16<kReadOnly>(at + skip, left - skip, r[0], r[1]);
    load16<kReadOnly>(at + skip + 16, left - skip - 16, r[2], r[3]);
  }
  // the 32 columns loaded last
  __device__ __forceinline__ void take(uint4 (&v)[4]) {
    v[0] = odd ? first : r[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) v[i] = odd ? r[i - 1] : r[i];
    first = r[3];
  }
};

// Pair i of 8 BF16 values.
__device__ __forceinline__ uint64_t pair_of(const uint4 &h, int i) {
  const uint32_t w = i == 0 ? h.x : i == 1 ? h.y : i == 2 ? h.z : h.w;
  return f32x2_pack(bf16_lo(w), bf16_hi(w));
}

// Gate and up of the forward at 16 columns of a row.
struct Kept {
  uint4 g[2], u[2];
};

// What is written of a row's 16 columns.  Gated: act, gate, up; gated gradient: of gate, of
// up, act; else one.
template <int kMode>
constexpr int kOuts = kMode == kFfnGated || kMode == kFfnGatedGrad ? 3 : 1;
template <int kMode>
struct Words {
  uint32_t w[kOuts<kMode>][8];
};

// The row's output i (of a weight gradient in BF16: within expert e's matrix), from its first
// column on; nullptr: not asked for.
template <int kMode>
__device__ __forceinline__ uint16_t *out_row(const FfnParams &p, int i, int64_t row, int e) {
  const int64_t N = p.N;
  if constexpr (kMode == kFfnGated) {
    if (i == 0) return p.out == nullptr ? nullptr : p.out + row * N;
    return p.out2 == nullptr ? nullptr : p.out2 + row * 2 * N + (i == 2 ? N : 0);
  } else if constexpr (kMode == kFfnGatedGrad) {
    if (i < 2) return p.out + row * 2 * N + (i == 1 ? N : 0);
    return p.out2 == nullptr ? nullptr : p.out2 + row * N;
  } else if constexpr (weight_grad(kMode)) {
    return p.out + ((int64_t)e * p.M + row) * N;
  } else {
    return p.out + row * N;
  }
}

// From 16 columns' accumulated v (gated: gate v, up u).
template <int kMode>
__device__ __forceinline__ void compute16(const FfnParams &p, const Pairs &v, const Pairs &u,
                                          const Kept &k, Words<kMode> &o) {
  if constexpr (kMode == kFfnGated) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t a = f32x2_mul_rn(f32x2_mul_rn(v[i], sigmoid2(v[i])), u[i]);
      o.w[0][i] = cvt_bf16x2(f32x2_lo(a), f32x2_hi(a));
    }
    if (p.out2 != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o.w[1][i] = cvt_bf16x2(f32x2_lo(v[i]), f32x2_hi(v[i]));
        o.w[2][i] = cvt_bf16x2(f32x2_lo(u[i]), f32x2_hi(u[i]));
      }
    }
  } else if constexpr (kMode == kFfnGatedGrad) {
    // one column at a time: in packed pairs 8192 x 8192 x 4096 took 376 us instead of 353
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t g2 = pair_of(k.g[i >> 2], i & 3), u2 = pair_of(k.u[i >> 2], i & 3);
      float r[2][3];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float g = q ? f32x2_hi(g2) : f32x2_lo(g2), up = q ? f32x2_hi(u2) : f32x2_lo(u2);
        const float d = q ? f32x2_hi(v[i]) : f32x2_lo(v[i]);
        const float s = rcp_approx(1.f + exp2_approx(-1.4426950408889634f * g)), silu = g * s;
        r[q][0] = d * up * (s + silu * (1.f - s));
        r[q][1] = d * silu;
        r[q][2] = silu * up;
      }
#pragma unroll
      for (int x = 0; x < 3; ++x) o.w[x][i] = cvt_bf16x2(r[0][x], r[1][x]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.w[0][i] = cvt_bf16x2(f32x2_lo(v[i]), f32x2_hi(v[i]));
  }
}

// 16 columns of a row, zeros: alignment padding, a weight's gradient without rows.
template <int kMode>
__device__ __forceinline__ void zero16(const FfnParams &p, int64_t row, int e, int col) {
  const uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const int left = p.N - col;
  if constexpr (kMode == kFfnWeightGrad32) {
    uint16_t *o = p.out + 2 * (((int64_t)e * p.M + row) * p.N + col);  // two of these a column
    store16(o, 16, w);
    if (left >= 16) store16(o + 16, 16, w);
  } else {
#pragma unroll
    for (int i = 0; i < kOuts<kMode>; ++i) {
      uint16_t *o = out_row<kMode>(p, i, row, e);
      if (o != nullptr) store16(o + col, left, w);
    }
  }
}

// Writes 16 columns of a row by themselves.
template <int kMode>
__device__ __forceinline__ void finish16(const FfnParams &p, int64_t row, int e, int col,
                                         const Pairs &v, const Pairs &u, const Kept &k,
                                         bool add) {
  const int left = p.N - col;
  if constexpr (kMode == kFfnWeightGrad32) {
    float *o = reinterpret_cast<float *>(p.out) + ((int64_t)e * p.M + row) * p.N + col;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (left < 8 * q + 8) break;
      uint32_t w[8];
#pragma unroll
      for (int x = 0; x < 8; ++x)
        w[x] = (uint32_t)(v[4 * q + x / 2] >> (x & 1 ? 32 : 0));
      if (add) {
        const uint4 b0 = ld_plain_v4(o + 8 * q), b1 = ld_plain_v4(o + 8 * q + 4);
        const uint32_t b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
        for (int x = 0; x < 8; ++x)
          w[x] = __float_as_uint(__uint_as_float(w[x]) + __uint_as_float(b[x]));
      }
      store16(reinterpret_cast<uint16_t *>(o + 8 * q), 16, w);
    }
  } else {
    Pairs s;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = v[i];
    if constexpr (weight_grad16(kMode))
      if (add) {
        const uint16_t *b = out_row<kMode>(p, 0, row, e) + col;
        const uint4 lo = ld_plain_v4(b);
        const uint4 hi = left >= 16 ? ld_plain_v4(b + 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = f32x2_add_rn(s[i], pair_of(i < 4 ? lo : hi, i & 3));
      }
    Words<kMode> words;
    compute16<kMode>(p, s, u, k, words);
#pragma unroll
    for (int i = 0; i < kOuts<kMode>; ++i) {
      uint16_t *o = out_row<kMode>(p, i, row, e);
      if (o != nullptr) store16(o + col, left, words.w[i]);
    }
  }
}

// What a warp writes by TMA: pieces of 32 rows x 32 fp32 columns through a ring in shared
// memory, in the swizzle of their rows.
struct Out {
  static constexpr int kBytes = 4096, kRing = 2;
  uint8_t *base;
  int slot = 0;

  // 16 of the piece's columns, from column 16 * part; all lanes, each its row
  __device__ __forceinline__ void put16(int part, bool zero, const float *v) {
    const int lane = threadIdx.x & 31;
    uint8_t *row = base + slot * kBytes + lane * 128;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 w = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
      *reinterpret_cast<float4 *>(row + (((part * 4 + c) ^ (lane & 7)) << 4)) = w;
    }
  }
  // before the first put16 of a piece: its slot is free
  __device__ __forceinline__ void open() {
    if (elect_one()) bulk_wait_read<kRing - 1>();
    __syncwarp();
  }
  __device__ __forceinline__ void send(const CUtensorMap *map, int x, int y, int z, bool add) {
    fence_proxy_async_smem();
    __syncwarp();
    if (elect_one()) {
      if (add)
        tma_add_3d(map, x, y, z, base + slot * kBytes);
      else
        tma_store_3d(map, x, y, z, base + slot * kBytes);
      bulk_commit();
    }
    if (++slot == kRing) slot = 0;
  }
  __device__ __forceinline__ void finish() {
    if (elect_one()) bulk_wait_all<0>();
    __syncwarp();
  }
};

// An epilogue warp has read an accumulator: what it loaded is in registers (the loads were
// waited for), so nothing needs a release, which in a pair would wait for all its stores:
// 1,600 cycles at the end of each tile.
template <int kPair>
__device__ __forceinline__ void release(uint64_t *acc_empty) {
  if ((threadIdx.x & 31) != 0) return;
  if constexpr (kPair == 2)
    mbar_arrive_cluster_relaxed(cluster_map(acc_empty, 0));
  else
    mbar_arrive(acc_empty);
}

// Adds `parts` accumulators of 2 * kHalf columns, as they become complete, up in sum: `cols`
// (64 or 128) columns from `taddr` of this warp's lanes.  Rows nobody needs (!work) are not
// read.
template <int kPair, int kHalf>
__device__ __forceinline__ void join_sums(Barriers &bar, uint32_t taddr, int cols, int parts,
                                          bool work, Ring<2> &acc, bool &ok,
                                          float (&sum)[kHalf]) {
#pragma unroll
  for (int c = 0; c < kHalf; ++c) sum[c] = 0.f;
  for (int i = 0; i < parts; ++i) {
    if (ok) ok = __all_sync(0xffffffffu, wait(&bar.acc_full[acc.slot], acc.phase));
    tc_fence_after();
    if (work) {
#pragma unroll
      for (int c = 0; c < kHalf; c += 64) {
        if (c >= cols) break;
        uint32_t d[64];
        tmem_load64(taddr + acc.slot * 2 * kHalf + c, d);
        tmem_load_wait(d);
#pragma unroll
        for (int x = 0; x < 64; ++x) sum[c + x] += __uint_as_float(d[x]);
      }
      tc_fence_before();
      __syncwarp();
    }
    release<kPair>(&bar.acc_empty[acc.slot]);
    acc.next();
  }
  if (!ok)
#pragma unroll
    for (int c = 0; c < kHalf; ++c) sum[c] = __uint_as_float(0x7fffffffu);
}

// A tile whose sum is of several accumulators, `apart` columns from one another: `cols` columns
// from `taddr`.  Between them the sums are in memory, where no other thread looks at them (one
// part is 2,048 blocks, a million cycles; held in registers they made every tile of such a call
// 8 % slower).
template <int kMode, int kPair>
__device__ __forceinline__ void sum_parts(const FfnParams &p, Barriers &bar, const Tile &t,
                                          uint32_t taddr, int apart, int cols, int col,
                                          int64_t row, bool mine, bool work, Ring<2> &acc,
                                          bool &ok) {
  constexpr int kMine = 32 * kEpilogueWarps;
  float4 *sums = p.sums + (int64_t)blockIdx.x * (kSumsBytes / 16) + (threadIdx.x - 128);
  const int parts = (t.blocks + kLongBlocks - 1) / kLongBlocks;
  for (int i = 0; i < parts; ++i) {
    if (ok) ok = __all_sync(0xffffffffu, wait(&bar.acc_full[acc.slot], acc.phase));
    tc_fence_after();
    if (work) {
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        uint32_t d[32];
        tmem_load32(taddr + acc.slot * apart + c, d);
        tmem_load_wait(d);
        float4 *at = sums + (c >> 2) * kMine;
        float4 v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          v[x] = make_float4(__uint_as_float(d[4 * x]), __uint_as_float(d[4 * x + 1]),
                             __uint_as_float(d[4 * x + 2]), __uint_as_float(d[4 * x + 3]));
          if (i > 0) {
            const float4 b = at[x * kMine];
            v[x].x += b.x, v[x].y += b.y, v[x].z += b.z, v[x].w += b.w;
          }
          if (!ok) v[x].x = v[x].y = v[x].z = v[x].w = __uint_as_float(0x7fffffffu);
          if (i + 1 < parts) at[x * kMine] = v[x];
        }
        if (i + 1 == parts && mine)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (col + c + 16 * q >= p.N) break;
            Pairs w;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              w[2 * x] = f32x2_pack(v[4 * q + x].x, v[4 * q + x].y);
              w[2 * x + 1] = f32x2_pack(v[4 * q + x].z, v[4 * q + x].w);
            }
            finish16<kMode>(p, row, t.e, col + c + 16 * q, w, w, Kept{}, p.accumulate);
          }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
    }
    release<kPair>(&bar.acc_empty[acc.slot]);
    acc.next();
  }
}

// ---- the kernel ---------------------------------------------------------------------------

// kShifted: rows of the output (or of `kept`) may start in the middle of a sector.  A variant of
// its own, as RowOut costs the others instructions: 8192 x 13568 x 256 gated takes 50 us, with
// it 61.  kAdds: a weight's gradient in BF16 is added to what is there (64 experts of 2048 x
// 4096, 512 tokens, top-8, without adding: 198 us, with the code for it 239).
template <int kMode, int kPair, bool kSplit, bool kShifted, bool kAdds>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ FfnParams p) {
  using R = Ring_<kMode, kPair, kSplit>;
  constexpr int kStages = R::kStages, kTileN = R::kCols;
  constexpr int kTmemColumns = 2 * kTileN;  // two accumulators
  constexpr bool kAMn = weight_grad(kMode);
  constexpr bool kBMn = kMode == kFfnGatedGrad || kMode == kFfnProductT || kAMn;
  constexpr bool kF32 = kMode == kFfnWeightGrad32, kLong = kMode == kFfnWeightGradLong;
  constexpr bool kJoins = kF32 || kLong;
  constexpr int kPart = kF32 ? kJoin : kLongBlocks;  // blocks of an accumulator, where joined
  constexpr bool kMoreRegs = kF32 || (kLong && kSplit) || (kMode == kFfnGatedGrad && !kSplit);
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int warp_sum[kThreads / 32];
  // stages on 1024-byte boundaries (the swizzle's period), outputs, then cum[E + 1]
  uint8_t *smem = smem_raw + (1024 - smem_u32(smem_raw) % 1024) % 1024;
  int *cum = reinterpret_cast<int *>(smem + R::kSmem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair == 2 || kSplit ? (int)cluster_rank() : 0;
  // of the CTAs of a pair, and the cluster's rank of its first; the part of a reduction
  const int half_rank = kPair == 2 ? rank & 1 : 0, leader = rank - half_rank;
  const int part_rank = kSplit ? rank >> (kPair - 1) : 0;

  if (threadIdx.x == 64) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bar.acc_full[b], 1);
      mbar_init(&bar.acc_empty[b], kEpilogueWarps * kPair);
    }
    mbar_init(&bar.drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_group<kPair>(&tmem_slot, kTmemColumns);
  griddep_wait();
  if (!kAMn && p.s.cnt_e != nullptr) count_tiles(p, kTileM * kPair, cum, warp_sum);
  constexpr int kCols = kMode == kFfnGated ? kTileN / 2 : kTileN;
  const int tiles_n = (p.N + kCols - 1) / kCols;
  int tiles;
  if constexpr (kAMn)
    tiles = p.s.E * (int)p.expert_tiles.of;
  else
    tiles = (p.s.cnt_e == nullptr ? (int)((p.s.rows + kTileM * kPair - 1) / (kTileM * kPair))
                                  : cum[p.s.E]) * tiles_n;
  // a cluster of a split tile, or a pair, or a CTA, takes every step-th tile
  const int first = (int)blockIdx.x >> (kSplit ? (p.split >> 1) + kPair - 1 : kPair - 1);
  const int step = (int)p.groups.of;
  // The tiles of the last round, where they are at most half as many as there are pairs,
  // are halved, so that the round takes half as long.
  const int last =
      kPair == 2 && !kSplit ? tiles - (int)divide((uint32_t)tiles, p.groups) * step : 0;
  const int whole_tiles = tiles - (2 * last <= step ? last : 0);
  const int items = whole_tiles + 2 * (tiles - whole_tiles);
  const auto tile_at = [&](int i) {
    const int h = i - whole_tiles;
    const bool half = kPair == 2 && h >= 0;
    Tile t = find_tile<kMode, kCols>(p, cum, half ? whole_tiles + (h >> 1) : i, kTileM * kPair,
                                     tiles_n);
    if (half) {
      t.cols = kCols / 2;
      t.n0 += (h & 1) * t.cols;
      if (t.n0 >= p.N) t.used = t.write = t.blocks = 0;
    }
    return t;
  };
  Tile tile0;  // while the barriers and TMEM are got ready
  if (first < items) tile0 = tile_at(first);
  __syncthreads();
  if constexpr (kPair == 2) {  // the other CTA's barriers are ready (it fenced them)
    cluster_arrive_relaxed();
    cluster_wait();
  }
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // this CTA's part of a tile's reduction
  const auto part = [&](int blocks, int r) {
    return kSplit ? (int)((int64_t)blocks * r >> (p.split >> 1)) : (r == 0 ? 0 : blocks);
  };
  bool ok = true;

  if (warp < 4) {
   if constexpr (kMoreRegs) setmaxnreg_dec<kControlRegs>();
   if (warp == 0) {
    // ---------------- copies ----------------
    // The warp stays whole and one lane of it issues, so that the copies' addresses
    // and coordinates are in uniform registers: from a branch of lane 0 alone a
    // stage's two copies took 540 cycles to issue, longer than its products run.
    Ring<kStages> st;
    int issued = 0;  // stages filled, counted up to kStages
    int acquired = -1;  // the expert whose maps were last made visible
    const uint32_t full0 = kPair == 2 ? cluster_map(&bar.full[0], leader) : smem_u32(&bar.full[0]);
    Tile next = tile0;
    for (int i = first; i < items && ok; i += step) {
      const Tile t = next;
      const int kb = part(t.blocks, part_rank), ke = part(t.blocks, part_rank + 1);
      if (kb == ke) {
        if (i + step < items) next = tile_at(i + step);
        continue;
      }
      const int half = half_of<kMode, kPair>(t);
      // rows copied: up to a multiple of kRowStep; of both CTAs of a pair
      const int left = kPair == 2 ? min(half, t.used) : t.used;
      const auto up = [](int n) { return max(0, (n + kRowStep - 1) / kRowStep * kRowStep); };
      const int rows0 = kAMn ? kTileM : up(left);
      const int rows1 = kPair == 1 ? 0 : kAMn ? kTileM : up(t.used - half);
      const int rows = half_rank ? rows1 : rows0;
      const int width = acc_columns<kMode>(t);
      const uint32_t bytes = (uint32_t)((rows0 + rows1 + width) * kBlockK * 2);
      const CUtensorMap *ma = &maps.a[0], *mb = width == 128 && !kBMn ? &maps.b_small : &maps.b;
      if (kAMn && p.seg_maps != nullptr) {
        ma = reinterpret_cast<const CUtensorMap *>(p.seg_maps) + 2 * t.e;
        mb = ma + 1;
        if (t.e != acquired) {
          tma_acquire_map(ma);
          tma_acquire_map(mb);
          acquired = t.e;
        }
      }
      const int a_row = (int)t.row0 + half_rank * half;
      for (int k = kb; k < ke; ++k) {
        ok = __all_sync(0xffffffffu, wait(&bar.empty[st.slot], st.phase ^ 1));
        if (!ok) break;
        uint8_t *a = smem + st.slot * R::kStageBytes, *b = a + R::kABytes;
        const uint32_t full = full0 + st.slot * 8;
        if (elect_one()) {
          if (half_rank == 0) mbar_arrive_expect_tx(&bar.full[st.slot], bytes);
          if constexpr (kAMn) {
            const int y = (int)(t.k0 + (int64_t)k * kBlockK);
#pragma unroll
            for (int j = 0; j < kTileM / 64; ++j)
              tma_load_3d<kPair>(a + j * kBoxBytes, ma, a_row + 64 * j, y, 0, full);
          } else if (rows == kTileM) {
            tma_load_3d<kPair>(a, &maps.a[kRowMaps - 1], k * kBlockK, a_row, 0, full);
          } else {
            int r = 0;
#pragma unroll
            for (int q = kRowMaps - 2; q >= 0; --q)  // rows = 16 * (sum of 2^q)
              if (rows & (kRowStep << q)) {
                tma_load_3d<kPair>(a + r * kBlockK * 2, &maps.a[q], k * kBlockK, a_row + r, 0,
                                   full);
                r += kRowStep << q;
              }
          }
          if constexpr (kBMn) {
            const int y = kAMn ? (int)(t.k0 + (int64_t)k * kBlockK) : k * kBlockK;
            const int x = t.n0 + half_rank * (width / 2);
#pragma unroll
            for (int j = 0; j < kTileN / kPair / 64; ++j)
              if (j < width / kPair / 64)
                tma_load_3d<kPair>(b + j * kBoxBytes, mb, x + 64 * j, y, kAMn ? 0 : t.e, full);
          } else {
            // half of the tile's rows of the matrix per box: gate and up, or two neighbours
            const int far = kMode == kFfnGated ? p.N : width / 2;
#pragma unroll
            for (int j = 0; j < 2 / kPair; ++j)
              tma_load_3d<kPair>(b + j * (R::kBBytes * kPair / 2), mb, k * kBlockK,
                                 t.n0 + (half_rank + j) * far, t.e, full);
          }
        }
        __syncwarp();
        st.next();
        if (issued < kStages) ++issued;
        // while the ring is full: where the next tile's copies come from
        if (k == min(kb + kStages, ke) - 1 && i + step < items) next = tile_at(i + step);
      }
    }
    if (lane == 0) {
      // The products' last arrivals on the stages' barriers: nothing else waits for
      // them, and they must not come after the CTA's shared memory is gone.
      Ring<kStages> left = st;
      for (int s = 0; s < kStages && ok; ++s, left.next())
        ok = wait(&bar.empty[left.slot], left.phase ^ 1);
      if (!ok) {
        if (p.err != nullptr) atomicOr(p.err, EP_ERRBIT_TIMEOUT);
        // copies in flight: slots below st.slot in this round, the others in the
        // round before
        if (half_rank == 0)
          for (int s = 0; s < kStages; ++s)
            if (s < st.slot || issued == kStages)
              wait(&bar.full[s], s < st.slot ? st.phase : st.phase ^ 1);
      }
    }
    __syncwarp();
   } else if (warp == 1 && half_rank == 0) {
    // ---------------- products ----------------
    constexpr int kAStep = kAMn ? 2048 >> 4 : 32 >> 4, kBStep = kBMn ? 2048 >> 4 : 32 >> 4;
    Ring<kStages> st;
    Ring<2> acc;
    const uint32_t smem0 = smem_u32(smem);
    for (int i = first; i < items && ok; i += step) {
      const Tile t = i == first ? tile0 : tile_at(i);
      const int kb = part(t.blocks, part_rank), ke = part(t.blocks, part_rank + 1);
      if (kb == ke) continue;
      const uint32_t idesc = idesc_bf16(kTileM * kPair, acc_columns<kMode>(t), kAMn, kBMn);
      for (int k = kb; k < ke && ok; ++k) {
        // an accumulator takes the whole sum, or kPart blocks of it
        const bool begins = kJoins ? (k - kb) % kPart == 0 : k == kb;
        const bool ends = k + 1 == ke || (kJoins && (k + 1 - kb) % kPart == 0);
        if (begins) ok = __all_sync(0xffffffffu, wait(&bar.acc_empty[acc.slot], acc.phase ^ 1));
        if (ok) ok = __all_sync(0xffffffffu, wait(&bar.full[st.slot], st.phase));
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = smem0 + st.slot * R::kStageBytes, b = a + R::kABytes;
        const uint64_t da = kAMn ? smem_desc_mn128(a) : smem_desc_k128(a);
        const uint64_t db = kBMn ? smem_desc_mn128(b) : smem_desc_k128(b);
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < kBlockK / 16; ++q)
            mma_bf16<kPair>(tmem + acc.slot * kTileN, da + q * kAStep, db + q * kBStep, idesc,
                            q > 0 || !begins);
          mma_commit_group<kPair>(&bar.empty[st.slot], (uint16_t)(3 << leader));
          if (ends) mma_commit_group<kPair>(&bar.acc_full[acc.slot], (uint16_t)(3 << leader));
        }
        __syncwarp();
        st.next();
        if (ends) acc.next();
      }
    }
    // The other CTA's last arrivals here: nothing else waits for them, and relaxed as they
    // are, the cluster's barrier at the end does not either.
    if constexpr (kPair == 2 && !kSplit)
      for (int b = 0; b < 2 && ok; ++b, acc.next())
        ok = __all_sync(0xffffffffu, wait(&bar.acc_empty[acc.slot], acc.phase ^ 1));
    if (!ok) {
      if (elect_one()) {
        if (p.err != nullptr) atomicOr(p.err, EP_ERRBIT_TIMEOUT);
        mma_commit_here<kPair>(&bar.drain);
      }
      __syncwarp();
      wait(&bar.drain, 0);
    }
   }
   __syncwarp();
   if constexpr (kSplit) {  // see below
     cluster_arrive_release();
     cluster_wait();
     cluster_arrive_release();
     cluster_wait();
   }
  } else if (!kSplit) {
    // ---------------- the rest of the formula, and output ----------------
    if constexpr (kMoreRegs) setmaxnreg_inc<kEpilogueRegs>();
    const int quarter = warp & 3;       // TMEM lanes of this warp
    const int j = (warp - 4) >> 2;      // half of the columns
    const int m = quarter * 32 + lane;  // row of the CTA's part of the tile
    const uint32_t taddr = tmem + (uint32_t)(quarter * 32) * 65536u;
    constexpr int kMostCols = kCols / 2;  // of a warp
    Out o{smem + kStages * R::kStageBytes + (warp - 4) * R::kOutBytes};
    Ring<2> acc;
    for (int i = first; i < items; i += step) {
      const Tile t = i == first ? tile0 : tile_at(i);
      const int half = half_of<kMode, kPair>(t);
      const int mine0 = half_rank * half;
      const int used = kPair == 2 ? max(0, min(half, t.used - mine0)) : t.used;
      const int write = kPair == 2 ? max(0, min(half, t.write - mine0)) : t.write;
      const int64_t row = t.row0 + mine0 + m;
      const bool mine = m < used;
      const bool work = quarter * 32 < write;  // any row of the warp
      const bool mma = t.blocks > 0;
      const int cols = t.cols / 2;  // of this warp
      const bool zero = !mma || !mine;
      const int row_w = (int)t.row0 + mine0 + quarter * 32;
      if constexpr (kF32) {
        if (!mma && p.accumulate) continue;
        float sum[kMostCols];
        join_sums<kPair, kMostCols>(bar, taddr + j * cols, cols, (t.blocks + kPart - 1) / kPart,
                                    work, acc, ok, sum);
        if (R::kTmaOut) {
#pragma unroll
          for (int c = 0; c < kMostCols; c += 32) {
            const int col = t.n0 + j * cols + c;
            if (c >= cols || col >= p.N || !work) break;
            o.open();
#pragma unroll
            for (int q = 0; q < 2; ++q) o.put16(q, zero, sum + c + 16 * q);
            o.send(&maps.out, col, row_w, t.e, p.accumulate);
          }
        } else if (m < write)
#pragma unroll
          for (int c = 0; c < kMostCols; c += 16) {
            const int col = t.n0 + j * cols + c;
            Pairs v;
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = f32x2_pack(sum[c + 2 * x], sum[c + 2 * x + 1]);
            if (c < cols && col < p.N) {
              if (zero && !p.accumulate)
                zero16<kMode>(p, row, t.e, col);
              else
                finish16<kMode>(p, row, t.e, col, v, v, Kept{}, p.accumulate);
            }
          }
        continue;
      }
      if constexpr (kLong)
        if (t.blocks > kPart) {
          sum_parts<kMode, kPair>(p, bar, t, taddr + j * cols, kTileN, cols, t.n0 + j * cols, row,
                                  m < write, work, acc, ok);
          continue;
        }
      // the kept values of the next 32 columns are loaded while these are worked on
      const int col_w = t.n0 + j * cols, left_w = min(cols, p.N - col_w);
      RowIn<kShifted, !weight_grad(kMode)> gates, ups;
      const uint16_t *kept = weight_grad(kMode) ? out_row<kMode>(p, 0, row, t.e) + col_w
                                                     : p.kept + row * 2 * p.N + col_w;
      const bool loads = mine && (kMode == kFfnGatedGrad || kAdds);
      // gate and up 32 columns ahead; of the values that are added to, 64: every second 32
      // each (4096 tokens of kAdds' layout 578 us, 32 ahead 655; 8192 x 8192 x 4104, shifted,
      // 405 and 376)
      constexpr bool kFar = kAdds && !kShifted;
      const auto ahead = [&](int c) {
        if (!loads || c >= left_w) return;
        if (kFar && (c & 32)) {
          ups.load(kept + c, left_w - c);
          return;
        }
        gates.load(kept + c, left_w - c);
        if constexpr (kMode == kFfnGatedGrad) ups.load(kept + p.N + c, left_w - c);
      };
      if (loads && left_w > 0) {
        gates.begin(kept, left_w);
        ups.begin(kMode == kFfnGatedGrad ? kept + p.N : kept, left_w);
      }
      ahead(0);
      if (kFar) ahead(32);
      if (mma) {
        // after a wait that gave up, the rest is walked without waiting
        if (ok) ok = __all_sync(0xffffffffu, wait(&bar.acc_full[acc.slot], acc.phase));
        tc_fence_after();
      } else if (kAdds) {
        continue;
      }
      const uint32_t ta = taddr + acc.slot * kTileN;
      if (work) {
        RowOut outs[kOuts<kMode>];
        const bool stream = kShifted && m < write && !zero && left_w > 0;
        if (kShifted)
#pragma unroll
          for (int i = 0; i < kOuts<kMode>; ++i) {
            uint16_t *at = out_row<kMode>(p, i, row, t.e);
            outs[i].begin(at == nullptr ? nullptr : at + col_w, at == nullptr ? 0 : left_w);
          }
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          uint32_t d[32], d2[32];
          const int c0 = j * cols + c, col = t.n0 + c0;
          if (mma) {
            tmem_load32(ta + c0, d);
            if constexpr (kMode == kFfnGated) tmem_load32(ta + t.cols + c0, d2);
            tmem_load_wait(d);
            if constexpr (kMode == kFfnGated) tmem_load_wait(d2);
          }
          if (mma && c + 32 == cols) {  // read: a later tile may overwrite it
            tc_fence_before();
            __syncwarp();
            release<kPair>(&bar.acc_empty[acc.slot]);
          }
          uint4 g4[4], u4[4];
          if constexpr (kMode == kFfnGatedGrad || kAdds) {
            if (kFar && (c & 32))
              ups.take(g4);
            else
              gates.take(g4);
          }
          if constexpr (kMode == kFfnGatedGrad) ups.take(u4);
          ahead(c + (kFar ? 64 : 32));
          if (!ok) {
#pragma unroll
            for (int x = 0; x < 32; ++x) d[x] = d2[x] = 0x7fffffffu;
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (m >= write || col + 16 * q >= p.N) continue;
            if (zero) {
              zero16<kMode>(p, row, t.e, col + 16 * q);
              continue;
            }
            Pairs v, u;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              v[x] = join(d[16 * q + 2 * x], d[16 * q + 2 * x + 1]);
              u[x] = kMode == kFfnGated ? join(d2[16 * q + 2 * x], d2[16 * q + 2 * x + 1]) : 0;
            }
            Kept k;
            if constexpr (kMode == kFfnGatedGrad)
              k = {{g4[2 * q], g4[2 * q + 1]}, {u4[2 * q], u4[2 * q + 1]}};
            if constexpr (kAdds)
#pragma unroll
              for (int x = 0; x < 8; ++x)
                v[x] = f32x2_add_rn(v[x], pair_of(g4[2 * q + (x >> 2)], x & 3));
            if (stream) {
              Words<kMode> words;
              compute16<kMode>(p, v, u, k, words);
#pragma unroll
              for (int i = 0; i < kOuts<kMode>; ++i)
                if (outs[i].left > 0) outs[i].put(words.w[i]);
            } else {
              finish16<kMode>(p, row, t.e, col + 16 * q, v, u, k, false);
            }
          }
        }
        if (stream)
#pragma unroll
          for (int i = 0; i < kOuts<kMode>; ++i) outs[i].end();
      } else if (mma) {
        release<kPair>(&bar.acc_empty[acc.slot]);
      }
      if (mma) acc.next();
    }
    if constexpr (R::kTmaOut) o.finish();
    if (!ok && lane == 0 && p.err != nullptr) atomicOr(p.err, EP_ERRBIT_TIMEOUT);
    tc_fence_before();
  } else {
    // ---------------- a tile shared by the cluster ----------------
    if constexpr (kMoreRegs) setmaxnreg_inc<kEpilogueRegs>();
    // Each CTA gets the sums of kTileN / split columns from all of them, in shared memory
    // over the stages: [source][4 columns][row][4], so that a warp writes 512 bytes in a row
    // (rows apart, a tile of 128 rows took 25 us to change hands).  Its own part it reads from
    // TMEM again (of joined sums, which are in registers: from there too).
    const Tile t = tile0;
    const int S = p.split, wide = kTileN / S;       // accumulator columns of a CTA
    const int kb = part(t.blocks, part_rank), ke = part(t.blocks, part_rank + 1);
    const int half = half_of<kMode, kPair>(t), mine0 = half_rank * half;
    const int used = kPair == 2 ? max(0, min(half, t.used - mine0)) : t.used;
    const int write = kPair == 2 ? max(0, min(half, t.write - mine0)) : t.write;
    const int64_t row0 = t.row0 + mine0;
    const int quarter = warp & 3, j = (warp - 4) >> 2, m = quarter * 32 + lane;
    const bool work = quarter * 32 < used;  // any row of the warp
    const uint32_t ta = tmem + (uint32_t)(quarter * 32) * 65536u + j * (kTileN / 2);
    float sum[kJoins ? kTileN / 2 : 1];
    if constexpr (kJoins) {
      Ring<2> acc;
      join_sums<1, kTileN / 2>(bar, ta, kTileN / 2, (ke - kb + kPart - 1) / kPart, work, acc, ok,
                               sum);
    } else {
      ok = __all_sync(0xffffffffu, wait(&bar.acc_full[0], 0));
      tc_fence_after();
    }
    __syncwarp();
    cluster_arrive_release();  // this CTA's products are done with its stages
    cluster_wait();
    if (work) {
      const auto send = [&](int c, const float (&v)[16]) {
        // gated: a CTA's gate columns, then as many up columns
        const int cc = kMode == kFfnGated ? c : j * (kTileN / 2) + c;
        const int per = kMode == kFfnGated ? wide / 2 : wide;
        const int to = cc / per;
        if (!kJoins && to == part_rank) return;
        const int piece = (cc - to * per + (kMode == kFfnGated ? j * per : 0)) / 4;
        const uint32_t base =
            cluster_map(smem, to * kPair + half_rank) +
            (uint32_t)(((part_rank * (wide / 4) + piece) * kTileM + m) * 16);
        if (m < used)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            st_cluster_v4(base + (uint32_t)(x * kTileM * 16), v[4 * x], v[4 * x + 1],
                          v[4 * x + 2], v[4 * x + 3]);
      };
      if constexpr (kJoins) {
#pragma unroll
        for (int c = 0; c < kTileN / 2; c += 16) {
          float v[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) v[x] = sum[c + x];
          send(c, v);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < kTileN / 2; c += 32) {
          const int cc = kMode == kFfnGated ? c : j * (kTileN / 2) + c;
          const int per = kMode == kFfnGated ? wide / 2 : wide;
          if (per >= 32 && cc / per == part_rank) continue;
          uint32_t d[32];
          tmem_load32(ta + c, d);
          tmem_load_wait(d);
#pragma unroll
          for (int q = 0; q < 32; q += 16) {
            float v[16];
#pragma unroll
            for (int x = 0; x < 16; ++x)
              v[x] = ok ? __uint_as_float(d[q + x]) : __uint_as_float(0x7fffffffu);
            send(c + q, v);
          }
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    cluster_arrive_release();
    cluster_wait();
    const int per = kMode == kFfnGated ? wide / 2 : wide, groups = per / 16;
    const float4 *in = reinterpret_cast<const float4 *>(smem);
    const uint32_t own = tmem + (uint32_t)(quarter * 32) * 65536u + part_rank * per;
    // two warps to 32 rows, each with every second 16 columns
    for (int g = j; g < groups && quarter * 32 < write; g += 2) {
      const int col = t.n0 + part_rank * per + g * 16;
      if (col >= p.N) break;
      float v[16], u[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) v[x] = u[x] = 0.f;
      if constexpr (!kJoins) {
        uint32_t d[16], d2[16];
        tmem_load16(own + g * 16, d);
        if constexpr (kMode == kFfnGated) tmem_load16(own + kTileN / 2 + g * 16, d2);
        tmem_load_wait(d);
        if constexpr (kMode == kFfnGated) tmem_load_wait(d2);
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          v[x] = ok ? __uint_as_float(d[x]) : __uint_as_float(0x7fffffffu);
          if constexpr (kMode == kFfnGated) u[x] = ok ? __uint_as_float(d2[x]) : v[x];
        }
      }
      if (m < write) {
#pragma unroll
        for (int s = 0; s < kMaxSplit; ++s) {
          if (s >= S || (!kJoins && s == part_rank)) continue;
          const float4 *from = in + (s * (wide / 4) + g * 4) * kTileM + m;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float4 a = from[x * kTileM];
            v[4 * x] += a.x, v[4 * x + 1] += a.y, v[4 * x + 2] += a.z, v[4 * x + 3] += a.w;
            if constexpr (kMode == kFfnGated) {
              const float4 b = from[(per / 4 + x) * kTileM];
              u[4 * x] += b.x, u[4 * x + 1] += b.y, u[4 * x + 2] += b.z, u[4 * x + 3] += b.w;
            }
          }
        }
        Pairs vp, up;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          vp[x] = f32x2_pack(v[2 * x], v[2 * x + 1]);
          up[x] = f32x2_pack(u[2 * x], u[2 * x + 1]);
        }
        Kept k{};
        if constexpr (kMode == kFfnGatedGrad) {
          const uint16_t *kept = p.kept + (row0 + m) * 2 * p.N + col;
          load16<true>(kept, p.N - col, k.g[0], k.g[1]);
          load16<true>(kept + p.N, p.N - col, k.u[0], k.u[1]);
        }
        finish16<kMode>(p, row0 + m, t.e, col, vp, up, k, p.accumulate);
      }
      __syncwarp();
    }
    tc_fence_before();
    if (!ok && lane == 0 && p.err != nullptr) atomicOr(p.err, EP_ERRBIT_TIMEOUT);
  }
  __syncwarp();
  __syncthreads();
  if constexpr (kPair == 2) {
    // neither CTA leaves while the other may still arrive on its barriers, read
    // its operands or write into its TMEM (relaxed: no wait for the output's stores)
    cluster_arrive_relaxed();
    cluster_wait();
  }
  if (warp == 1) tmem_dealloc_group<kPair>(tmem, kTmemColumns);
}

// Tensor maps of an expert's rows for the weight gradient: the given ones with
// their rows ending at the expert's last.  Map 2 * e + (0: a, 1: b); a warp each.
__global__ void __launch_bounds__(32) ffn_segment_maps_kernel(const __grid_constant__ Maps maps,
                                                              Segments s, CUtensorMap *out) {
  griddep_wait();
  for (int i = blockIdx.x; i < 2 * s.E; i += gridDim.x) {
    const uint4 *from = reinterpret_cast<const uint4 *>(i & 1 ? &maps.b : &maps.a[0]);
    uint4 *to = reinterpret_cast<uint4 *>(out + i);
    if (threadIdx.x < sizeof(CUtensorMap) / 16) to[threadIdx.x] = from[threadIdx.x];
    __syncwarp();
    if (threadIdx.x == 0) {
      const SegmentRows r = segment_rows(s, i >> 1);
      tma_replace_rows(out + i, (uint32_t)max((int64_t)1, r.first + r.used));
    }
  }
}

// An array [z, y, x] of BF16 (or fp32), x contiguous, copied in boxes of box_x (128 bytes)
// x box_y x 1 in 128-byte swizzle; zeros outside.  Strides in elements.
bool make_map(CUtensorMap *map, const void *base, int64_t x, int64_t y, int64_t z,
              int64_t y_stride, int64_t z_stride, int box_x, int box_y, bool f32 = false) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const int size = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
  const cuuint64_t strides[2] = {(cuuint64_t)(size * y_stride), (cuuint64_t)(size * z_stride)};
  const cuuint32_t box[3] = {(cuuint32_t)box_x, (cuuint32_t)box_y, 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void *>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `share` CTAs that are resident together, looked up once per kernel and device.
cudaError_t max_clusters(const void *func, int dev, int share, const cudaLaunchConfig_t &lc,
                         int *out) {
  struct Entry {
    const void *func;
    int device, share, clusters;
  };
  static std::mutex mu;
  static std::vector<Entry> known;
  std::lock_guard<std::mutex> g(mu);
  for (const Entry &e : known)
    if (e.func == func && e.device == dev && e.share == share) {
      *out = e.clusters;
      return cudaSuccess;
    }
  const cudaError_t e = cudaOccupancyMaxActiveClusters(out, func, &lc);
  if (e == cudaSuccess) try {
      known.push_back({func, dev, share, *out});
    } catch (...) {  // no memory: looked up again
    }
  return e;
}

template <int kMode, int kPair, bool kSplit, bool kShifted = false, bool kAdds = false>
cudaError_t launch_form(const Maps &maps, FfnParams p, int64_t tiles, int use, int share,
                        cudaStream_t s, bool *fits) {
  using R = Ring_<kMode, kPair, kSplit>;
  const auto kernel = ffn_kernel<kMode, kPair, kSplit, kShifted, kAdds>;
  const size_t cum = weight_grad(kMode) ? 0 : sizeof(int) * (p.s.E + 1);
  const size_t smem = 1024 + (size_t)R::kSmem + cum;
  int dev = 0;
  cudaError_t e = launch_geometry(reinterpret_cast<const void *>(kernel), kThreads, smem, &dev,
                                  nullptr);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)share);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)share;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = share > 1 ? 2 : 1;
  // (a pair's last tiles may be halved)
  int64_t groups = std::min<int64_t>(use / share, kPair == 2 && !kSplit ? 2 * tiles : tiles);
  if (share > 1) {
    int fit = 0;  // clusters that run at a time: no tile waits for one that does not
    e = max_clusters(reinterpret_cast<const void *>(kernel), dev, share, lc, &fit);
    if (e != cudaSuccess) return e;
    groups = std::min<int64_t>(groups, fit);
  }
  groups = std::max<int64_t>(1, groups);
  if constexpr (kSplit) {  // a cluster for every tile, or not this way
    *fits = groups == tiles;
    if (!*fits) return cudaSuccess;
  }
  lc.gridDim.x = (unsigned)(groups * share);
  constexpr int kCols = kMode == kFfnGated ? R::kCols / 2 : R::kCols;
  const int64_t tiles_n = (p.N + kCols - 1) / kCols;
  const int64_t expert = (p.M + kTileM * kPair - 1) / (kTileM * kPair) * tiles_n;
  if (2 * tiles > 0x7fffffffLL) return cudaErrorInvalidValue;  // (more than memory holds)
  p.groups = Reciprocal((uint32_t)groups);
  p.raster_tiles = Reciprocal((uint32_t)(kRaster * tiles_n));
  p.expert_tiles = Reciprocal((uint32_t)std::max<int64_t>(1, expert));
  return cudaLaunchKernelEx(&lc, kernel, maps, p);
}

// Rows per expert, on average, above which pairs of CTAs take the tiles of a layout.  With 64
// experts of 4096 x 4096, a gated product of 128 rows each takes 365 us by single CTAs and 364
// by pairs, of 160 rows 422 and 372, of 1024 1477 and 1300; the product on W as it lies of 128
// rows 342 and 350, of 160 406 and 358; a weight gradient in BF16 of 128 rows 430 and 470 us
// (all of it stores, which two CTAs wait for together), of 192 520 and 485, of 1024 1590 and
// 1400, in 32 bits of 128 820 and 785.
template <int kMode>
constexpr int64_t kPairRows = weight_grad16(kMode) ? 176 : weight_grad(kMode) ? 0 : 128;

template <int kMode>
cudaError_t launch_mode(const FfnParams &p0, int sm_cap, cudaStream_t s) {
  constexpr bool kAMn = weight_grad(kMode);
  FfnParams p = p0;
  Maps maps{};
  bool ok = true;
  const auto matrix = [&](int64_t x, int64_t y, bool rows = true) {
    return make_map(&maps.b, p.b, x, y, p.s.E, x, x * y, kBlockK, rows ? 128 : kBlockK) &&
           (!rows || make_map(&maps.b_small, p.b, x, y, p.s.E, x, x * y, kBlockK, 64));
  };
  if constexpr (kAMn) {
    ok = make_map(&maps.a[0], p.a, p.M, p.s.rows, 1, p.a_stride, p.a_stride, 64, kBlockK);
    ok = ok && make_map(&maps.b, p.b, p.N, p.s.rows, 1, p.b_stride, p.b_stride, 64, kBlockK);
  } else {
    for (int i = 0; i < kRowMaps; ++i)
      ok = ok && make_map(&maps.a[i], p.a, p.K, p.s.rows, 1, p.a_stride, p.a_stride, kBlockK,
                          kRowStep << i);
    if constexpr (kMode == kFfnGated)
      ok = ok && matrix(p.K, 2 * (int64_t)p.N);
    else if constexpr (kMode == kFfnProduct)
      ok = ok && matrix(p.K, p.N);
    else
      ok = ok && matrix(p.N, p.K, false);
  }
  if (!ok) return cudaErrorInvalidValue;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int use = sms_to_use(dev, sm_cap);
  // at most this many row tiles of `m` rows hold rows (every expert's last one may be partial)
  const auto tiles_of = [&](int m, int n) {
    if (kMode == kFfnGated) n /= 2;
    const int64_t tiles_n = (p.N + n - 1) / n;
    const int64_t r = kAMn ? (int64_t)p.s.E * ((p.M + m - 1) / m)
                           : std::min<int64_t>(p.max_segments, p.s.E) + (p.s.rows - 1) / m;
    return r * tiles_n;
  };
  if (p.s.cnt_e == nullptr) {
    // Few tiles: a cluster of 2 or 4 CTAs, or pairs of them, shares each one's reduction, as
    // long as all run at once: CTAs on smaller tiles where there are enough, else pairs.  A
    // block of either takes an SM 512 cycles, of a pair's half tile 384, but the sums that
    // change hands cost 2,000 to 6,000 once, hence kPairSplitBlocks: 384 x 4096 x 7168 gated
    // takes 24.3 us, unshared 30.7; 256 x 7168 x 2048 (32 blocks) 13.0 and 11.9.  Where CTAs
    // share as often, pairs are no faster: 256 x 4096 x 7168 gated 23.2 and, by CTAs, 22.2.
    const int64_t tiles = tiles_of(kTileM, 128), pairs = tiles_of(2 * kTileM, 256);
    const int64_t blocks = ((kAMn ? p.s.rows : p.K) + kBlockK - 1) / kBlockK;
    for (p.split = kMaxSplit; p.split > 1; p.split /= 2) {
      bool fits = false;
      if (tiles * p.split <= use && blocks >= p.split * 4) {
        e = launch_form<kMode, 1, true>(maps, p, tiles, use, p.split, s, &fits);
        if (e != cudaSuccess || fits) return e;
      }
      if constexpr (!kAMn)
        if (p.s.rows > kTileM && 2 * pairs * p.split <= use &&
            blocks >= p.split * kPairSplitBlocks) {
          e = launch_form<kMode, 2, true>(maps, p, pairs, use, 2 * p.split, s, &fits);
          if (e != cudaSuccess || fits) return e;
        }
    }
  } else if constexpr (kAMn) {
    e = launch_pdl(ffn_segment_maps_kernel, (unsigned)std::min(2 * p.s.E, 8 * use), 32, 0, s,
                   maps, p.s, static_cast<CUtensorMap *>(p.seg_maps));
    if (e != cudaSuccess) return e;
  }
  bool pair = use > 1 && (p.s.cnt_e == nullptr || p.max_segments > kPairRows<kMode> * p.s.E);
  if constexpr (!kAMn)
    if (pair && p.s.cnt_e == nullptr) {
      // By the rounds of tiles, in cycles of a block: a round of pairs' tiles 512, of their
      // halves 384, of single CTAs' 600.  The latter have fewer empty rows: 640 x 7168 x 4096
      // (84 tiles for 76 pairs, 140 for 152 CTAs) takes 28 us, by pairs 40; 1152 x 4096 x 4096
      // 24 and 37; 1024 x 7168 x 2048 (two rounds of either) 21 by pairs.
      const int64_t ones = tiles_of(kTileM, 256), twos = tiles_of(2 * kTileM, 256), at = use / 2;
      const int64_t last = twos % at;
      pair = 600 * ((ones + use - 1) / use) >=
             512 * (twos / at) + (last == 0 ? 0 : 2 * last <= at ? 384 : 512);
    }
  if constexpr (kMode == kFfnWeightGrad32)
    if (pair &&
        !make_map(&maps.out, p.out, p.N, p.M, p.s.E, p.N, (int64_t)p.N * p.M, 32, 32, true))
      return cudaErrorInvalidValue;
  const int64_t tiles = tiles_of(pair ? 2 * kTileM : kTileM, 256);
  const auto launch = [&](auto shifted, auto adds) {
    constexpr bool kShifted = decltype(shifted)::value, kAdds = decltype(adds)::value;
    return pair
               ? launch_form<kMode, 2, false, kShifted, kAdds>(maps, p, tiles, use, 2, s, nullptr)
               : launch_form<kMode, 1, false, kShifted, kAdds>(maps, p, tiles, use, 1, s, nullptr);
  };
  const std::true_type yes;
  const std::false_type no;
  if constexpr (kMode != kFfnWeightGrad32) {
    const auto on_32 = [](const void *x) { return reinterpret_cast<uintptr_t>(x) % 32 == 0; };
    const bool shifted = p.N % 16 != 0 || !on_32(p.out) || !on_32(p.out2) || !on_32(p.kept);
    if constexpr (weight_grad(kMode))
      if (p.accumulate) return shifted ? launch(yes, yes) : launch(no, yes);
    if (shifted) return launch(yes, no);
  }
  return launch(no, no);
}

// Whether an expert may have more rows than one accumulator takes.
bool long_sums(int mode, const FfnParams &p) {
  int64_t most = p.s.rows;
  if (p.s.cnt_e != nullptr)
    most = std::min(p.max_segments, p.s.fixed_cap > 0 ? (int64_t)p.s.fixed_cap : p.s.rows);
  return mode == kFfnWeightGrad && most > (int64_t)kLongBlocks * kBlockK;
}

}  // namespace

size_t ffn_workspace(int mode, FfnParams *p, void *ws) {
  if (!weight_grad(mode)) return 0;
  const size_t maps = p->s.cnt_e != nullptr ? 2 * sizeof(CUtensorMap) * p->s.E : 0;
  size_t sums = 0;
  if (long_sums(mode, *p)) {
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess) sums = (size_t)kSumsBytes * device_sm_count(dev);
  }
  if (ws != nullptr) {
    if (maps > 0) p->seg_maps = ws;
    if (sums > 0) p->sums = reinterpret_cast<float4 *>(static_cast<char *>(ws) + maps);
  }
  return maps + sums;
}

cudaError_t launch_ffn(int mode, const FfnParams &p, int sm_cap, cudaStream_t s) {
  if (ffn_few_rows(mode, p)) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : launch_ffn_rows(mode, p, sms_to_use(dev, sm_cap), s);
  }
  switch (mode) {
    case kFfnGated:
      return launch_mode<kFfnGated>(p, sm_cap, s);
    case kFfnGatedGrad:
      return launch_mode<kFfnGatedGrad>(p, sm_cap, s);
    case kFfnProduct:
      return launch_mode<kFfnProduct>(p, sm_cap, s);
    case kFfnProductT:
      return launch_mode<kFfnProductT>(p, sm_cap, s);
    case kFfnWeightGrad:
      return long_sums(mode, p) ? launch_mode<kFfnWeightGradLong>(p, sm_cap, s)
                                : launch_mode<kFfnWeightGrad>(p, sm_cap, s);
    default:
      return launch_mode<kFfnWeightGrad32>(p, sm_cap, s);
  }
}

}  // namespace ep
