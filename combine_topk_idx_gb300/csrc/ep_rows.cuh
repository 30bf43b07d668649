// Device-side walks over the rows of a layout (sm_103a).
#pragma once

#include "ep_internal.cuh"

namespace ep {

// Expert whose padding range holds padding row q: the last e with psum_pad[e] <= q.
__device__ __forceinline__ int padding_expert(const int32_t *psum_pad, int E, int q) {
  int lo = 0, hi = E;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(psum_pad + mid) <= q) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Items of a layout: its rows below the device total, or, in the fixed-capacity
// layout, the used rows of all experts one after another.  Row of item i (-1:
// none), and whether it is alignment padding.
__device__ __forceinline__ int64_t item_row(const RowsParams &r, int64_t i, int64_t items,
                                            bool *pad) {
  *pad = false;
  if (i >= items) return -1;
  if (r.num_rows == nullptr) return i;
  if (r.fixed_cap > 0) {
    int lo = 0, hi = r.E - 1;  // the last expert with psum_e[e] <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(r.psum_e + mid) <= i) lo = mid; else hi = mid - 1;
    }
    const int64_t k = i - __ldg(r.psum_e + lo);
    return k < r.fixed_cap ? (int64_t)lo * r.fixed_cap + k : -1;
  }
  *pad = __ldg(r.meta + 2 * i) < 0;
  return i;
}

__device__ __forceinline__ int64_t sf_at(const SfLayout &l, int64_t row, int j) {
  if (l.es > 0) {
    const int64_t e = row / l.cap;
    return e * l.es + (row - e * l.cap) * l.ts + j * l.hs;
  }
  return row * l.ts + j * l.hs;
}

__device__ __forceinline__ int64_t item_count(const RowsParams &r) {
  return r.num_rows == nullptr ? r.rows
         : r.fixed_cap > 0     ? (int64_t)__ldg(r.num_rows)
                               : min((int64_t)__ldg(r.num_rows), r.rows);
}

}  // namespace ep
