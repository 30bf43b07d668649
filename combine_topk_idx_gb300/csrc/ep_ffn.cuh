// The products of the trained feed-forward block: parameters and launchers.
#pragma once

#include "ep_internal.cuh"

namespace ep {

// Weight gradients: BF16, in 32 bits, and BF16 where an expert may have so many rows that
// their sum is joined of parts (a form of the first that its launch chooses).
enum FfnMode {
  kFfnGated, kFfnGatedGrad, kFfnProduct, kFfnProductT, kFfnWeightGrad, kFfnWeightGrad32,
  kFfnWeightGradLong
};

// The rows of each expert: of an expanded layout, or (cnt_e NULL, E = 1) all rows.
struct Segments {
  const int32_t *psum_e, *cnt_e;
  int E, fixed_cap, zero_padding;
  int64_t rows;             // rows allocated
};

struct SegmentRows {
  int64_t first, used, write;  // first row, rows in use, rows to write (then zeros)
};

__device__ __forceinline__ SegmentRows segment_rows(const Segments &s, int e) {
  if (s.cnt_e == nullptr) return {0, s.rows, s.rows};
  const int64_t cnt = __ldg(s.cnt_e + e);
  if (s.fixed_cap > 0) {
    const int64_t n = cnt < s.fixed_cap ? cnt : s.fixed_cap;
    return {(int64_t)e * s.fixed_cap, n, n};
  }
  const int64_t r0 = __ldg(s.psum_e + e);
  const int64_t left = max((int64_t)0, s.rows - r0);
  const int64_t used = min(cnt, left);
  return {r0, used, s.zero_padding ? min((int64_t)__ldg(s.psum_e + e + 1) - r0, left) : used};
}

// A divisor, and 2^32 / it rounded down.
struct Reciprocal {
  uint32_t of, magic;
  Reciprocal() = default;
  explicit Reciprocal(uint32_t b) : of(b), magic((uint32_t)(0xffffffffull / b)) {}
};

struct FfnParams {
  Segments s;
  int64_t max_segments;     // experts that can have rows; of a layout, its slots
  // a: the rows [rows, K] (weight gradient: the gradient [rows, M]); b: the matrix of
  // each expert (weight gradient: the rows [rows, N]); strides of rows, in elements
  const uint16_t *a, *b;
  int64_t a_stride, b_stride;
  int M, N, K;              // N: columns of the output (gated: F); M: weight gradient only
  const uint16_t *kept;     // gated gradient: [rows, 2N] gate | up of the forward
  uint16_t *out;            // gated: act; gated gradient: of gate_up; else the output
  uint16_t *out2;           // gated: gate_up; gated gradient: act; may be nullptr
  int accumulate;           // weight gradient: out is added to
  int split;                // CTAs that share a tile's reduction
  // filled in by the launch: CTAs, pairs or clusters that take tiles; tiles of kRaster rows
  // of tiles; weight gradient: of an expert's matrix
  Reciprocal groups, raster_tiles, expert_tiles;
  void *seg_maps;           // workspace: two tensor maps per expert
  float4 *sums;             // workspace: sums between the parts of a long one
  unsigned *err;            // the handle's error word (EP_ERRBIT_TIMEOUT), or nullptr
};

// Bytes of workspace (128-byte aligned), which p is pointed into if it is given; 0: none.
size_t ffn_workspace(int mode, FfnParams *p, void *ws);
cudaError_t launch_ffn(int mode, const FfnParams &p, int sm_cap, cudaStream_t s);

// Few rows, weights streamed into registers: whether a call is one of these, and its launch.
constexpr int kFfnFewRows = 16;
bool ffn_few_rows(int mode, const FfnParams &p);
cudaError_t launch_ffn_rows(int mode, const FfnParams &p, int sms, cudaStream_t s);

}  // namespace ep
