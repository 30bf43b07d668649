// The global norm of many gradients, and their clipping to it:
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// Two passes over the gradients with the norm between them: the first leaves a sum
// per CTA, the second starts by adding all of these up, in the same fixed order in
// every CTA, so neither a counter nor a third launch stands between them.  The
// tensors' addresses travel as launch parameters (up to kMost per launch): nothing
// is copied to the device first.  Both passes are bound by memory.  The second
// goes through each CTA's part backwards: what the first read last is still in L2.
//
// Sums.  A thread adds up the squares of at most kChunk / kThreads elements in fp32,
// then goes on in fp64, so the error does not grow with the number of elements.
// Squares that leave the range of fp32 are taken again of scaled values (2^90 or
// 2^-80, exact): any finite gradients have their norm, as far as fp32 holds it.
#include <algorithm>
#include <cmath>

#include "ep_clip.cuh"
#include "ep_ptx.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;           // elements that a CTA takes at a time
constexpr int kFew = 64, kMost = 1024; // tensors of a launch
constexpr int kPerSm = 4;              // CTAs

template <int N>
struct Table {
  const void *g[N];
  void *o[N];
  int64_t n[N];          // elements; negative: -n of BF16
  int32_t first[N + 1];  // chunks of the tensors before
  int count;
};

// Elements [i0, i1) of tensor t that chunk c holds.
struct Piece {
  int t;
  int64_t i0;
  int len;
  bool bf16;
};
template <int N>
__device__ __forceinline__ int find_tensor(const Table<N> &tab, int c) {
  int lo = 0, hi = tab.count - 1;  // the last tensor with first[t] <= c
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}
template <int N>
__device__ __forceinline__ Piece piece(const Table<N> &tab, int t, int c) {
  Piece p;
  p.t = t;
  const int64_t n = tab.n[t];
  p.bf16 = n < 0;
  p.i0 = (int64_t)(c - tab.first[t]) * kChunk;
  p.len = (int)min((int64_t)kChunk, (n < 0 ? -n : n) - p.i0);
  return p;
}

// Elements before the first 16-byte boundary of p, of at most len of `size` bytes.
__device__ __forceinline__ int head_of(const void *p, int size, int len) {
  return min(len, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / size);
}

__device__ __forceinline__ void add_squares(uint4 v, bool bf16, float scale, float &s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      const float a = bf16_lo(w[i]) * scale, b = bf16_hi(w[i]) * scale;
      s = fmaf(a, a, s);
      s = fmaf(b, b, s);
    } else {
      const float a = __uint_as_float(w[i]) * scale;
      s = fmaf(a, a, s);
    }
  }
}

// This thread's share of the squares of a piece, each value times `scale`.
template <bool kBf16>
__device__ __forceinline__ float squares(const void *base, int len, float scale) {
  constexpr int kSize = kBf16 ? 2 : 4, kVec = 16 / kSize, kLoads = kChunk / kVec / kThreads;
  const char *p = static_cast<const char *>(base);
  const int head = head_of(p, kSize, len), vecs = (len - head) / kVec;
  const char *body = p + head * kSize;
  float s = 0.f;
  uint4 v[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = threadIdx.x + u * kThreads;
    v[u] = i < vecs ? ld_plain_v4(body + 16 * (int64_t)i) : make_uint4(0, 0, 0, 0);
  }
  const int tail = head + vecs * kVec, rest = head + len - tail;
  float e = 0.f;
  if ((int)threadIdx.x < rest) {  // fewer than 2 * kVec elements about the vectors
    const int i = (int)threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
    if constexpr (kBf16)
      e = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << 16) * scale;
    else
      e = reinterpret_cast<const float *>(p)[i] * scale;
  }
#pragma unroll
  for (int u = 0; u < kLoads; ++u) add_squares(v[u], kBf16, scale, s);
  return fmaf(e, e, s);
}

// Sum of one value per thread, in a fixed order; in thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double all = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kThreads / 32; ++w) all += part[w];
  return all;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kPerSm)
    grad_squares_kernel(const __grid_constant__ Table<N> tab, double *part) {
  const int chunks = tab.first[tab.count];
  const int c0 = (int)((int64_t)chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((int64_t)chunks * (blockIdx.x + 1) / gridDim.x);
  griddep_wait();
  double sum = 0.0;
  int t = find_tensor(tab, c0);
  for (int c = c0; c < c1; ++c) {
    while (c >= tab.first[t + 1]) ++t;
    const Piece q = piece(tab, t, c);
    const char *g = static_cast<const char *>(tab.g[t]) + q.i0 * (q.bf16 ? 2 : 4);
    float s = q.bf16 ? squares<true>(g, q.len, 1.f) : squares<false>(g, q.len, 1.f);
    double w = 1.0;
    if (!(s > 1e-30f && s < INFINITY)) {
      const bool big = !(s <= 1e-30f);
      const float scale = big ? 0x1p-80f : 0x1p90f;
      s = q.bf16 ? squares<true>(g, q.len, scale) : squares<false>(g, q.len, scale);
      w = big ? 0x1p160 : 0x1p-180;
    }
    sum = fma((double)s, w, sum);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <bool kBf16>
__device__ __forceinline__ void scale_piece(const void *from, void *to, int len, float by) {
  constexpr int kSize = kBf16 ? 2 : 4, kVec = 16 / kSize, kLoads = kChunk / kVec / kThreads;
  const char *p = static_cast<const char *>(from);
  char *o = static_cast<char *>(to);
  const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
  const int head = same ? head_of(p, kSize, len) : 0;
  const int vecs = same ? (len - head) / kVec : 0;
  const char *body = p + head * kSize;
  char *obody = o + head * kSize;
  uint4 v[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = threadIdx.x + u * kThreads;
    if (i < vecs) v[u] = ld_plain_v4(body + 16 * (int64_t)i);
  }
  // about the vectors; all of a piece whose two addresses differ modulo 16 bytes
  const int tail = head + vecs * kVec, rest = head + len - tail;
  for (int j = threadIdx.x; j < rest; j += kThreads) {
    const int i = j < head ? j : tail + j - head;
    if constexpr (kBf16)
      reinterpret_cast<uint16_t *>(o)[i] = (uint16_t)cvt_bf16x2(
          __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << 16) * by, 0.f);
    else
      reinterpret_cast<float *>(o)[i] = reinterpret_cast<const float *>(p)[i] * by;
  }
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = threadIdx.x + u * kThreads;
    if (i < vecs) {
      uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int x = 0; x < 4; ++x)
        w[x] = kBf16 ? cvt_bf16x2(bf16_lo(w[x]) * by, bf16_hi(w[x]) * by)
                     : __float_as_uint(__uint_as_float(w[x]) * by);
      st_stream_v4(obody + 16 * (int64_t)i, make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

// Adds up the parts; norm (if not NULL) is written by the first CTA.
template <int N>
__global__ void __launch_bounds__(kThreads, kPerSm)
    grad_clip_kernel(const __grid_constant__ Table<N> tab, const double *part, int parts,
                     float max_norm, float *norm) {
  __shared__ float by_all;
  griddep_wait();
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) sum += __ldg(part + i);
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    const double n = sqrt(sum);
    // NaN, and not 1, for a norm that is NaN
    by_all = n + 1e-6 <= (double)max_norm ? 1.f : (float)((double)max_norm / (n + 1e-6));
    if (norm != nullptr && blockIdx.x == 0) *norm = (float)n;
  }
  __syncthreads();
  const float by = by_all;
  if (tab.count == 0) return;
  const int chunks = tab.first[tab.count];
  const int c0 = (int)((int64_t)chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((int64_t)chunks * (blockIdx.x + 1) / gridDim.x);
  int t = find_tensor(tab, max(0, c1 - 1));
  for (int c = c1 - 1; c >= c0; --c) {
    while (c < tab.first[t]) --t;
    if (by == 1.f && tab.o[t] == tab.g[t]) continue;  // in place: as it is
    const Piece q = piece(tab, t, c);
    const int64_t at = q.i0 * (q.bf16 ? 2 : 4);
    const char *g = static_cast<const char *>(tab.g[t]) + at;
    char *o = static_cast<char *>(tab.o[t]) + at;
    if (q.bf16)
      scale_piece<true>(g, o, q.len, by);
    else
      scale_piece<false>(g, o, q.len, by);
  }
}

// The next tensors of the list (from *at on) that fit a table; empty ones are left out.
template <int N>
void fill(const GradList &l, int *at, Table<N> *t) {
  t->count = 0;
  int64_t chunks = 0;
  for (; *at < l.count && t->count < N; ++*at) {
    const int i = *at;
    if (l.numels[i] == 0) continue;
    const int64_t c = (l.numels[i] + kChunk - 1) / kChunk;
    if (chunks + c > 0x7fffffffLL) break;
    t->g[t->count] = l.grads[i];
    t->o[t->count] = l.outs != nullptr ? l.outs[i] : nullptr;
    t->n[t->count] = l.is_f32[i] ? l.numels[i] : -l.numels[i];
    t->first[t->count++] = (int32_t)chunks;
    chunks += c;
  }
  t->first[t->count] = (int32_t)chunks;
}

template <int N>
cudaError_t launch(const GradList &l, float max_norm, float *norm, double *part, int sms,
                   cudaStream_t s) {
  Table<N> t;
  int parts = 0;
  cudaError_t e = cudaSuccess;
  for (int at = 0; e == cudaSuccess;) {
    fill(l, &at, &t);
    if (t.count == 0) break;
    const int grid = std::min(sms * kPerSm, (int)t.first[t.count]);
    e = launch_pdl(grad_squares_kernel<N>, (unsigned)grid, kThreads, 0, s, t, part + parts);
    parts += grid;
  }
  bool first = true;
  for (int at = 0; e == cudaSuccess; first = false) {
    if (l.outs != nullptr) fill(l, &at, &t);
    else t.count = 0, t.first[0] = 0;
    if (t.count == 0 && !(first && norm != nullptr)) break;
    const int grid = std::max(1, std::min(sms * kPerSm, (int)t.first[t.count]));
    e = launch_pdl(grad_clip_kernel<N>, (unsigned)grid, kThreads, 0, s, t,
                   const_cast<const double *>(part), parts, max_norm, first ? norm : nullptr);
    if (t.count == 0) break;
  }
  return e;
}

int in_use(const GradList &l) {
  int n = 0;
  for (int i = 0; i < l.count; ++i) n += l.numels[i] != 0;
  return n;
}

}  // namespace

size_t clip_workspace(const GradList &l, int sms) {
  // a sum per CTA of every launch; a launch ends with its table or its chunk numbers
  int64_t launches = 1 + in_use(l) / kMost, chunks = 0;
  for (int i = 0; i < l.count; ++i) chunks += (l.numels[i] + kChunk - 1) / kChunk;
  launches += 2 * (chunks / 0x7fffffffLL);
  return sizeof(double) * (size_t)(launches * sms * kPerSm);
}

cudaError_t launch_clip(const GradList &l, float max_norm, float *norm, void *workspace, int sms,
                        cudaStream_t s) {
  double *part = static_cast<double *>(workspace);
  return in_use(l) <= kFew ? launch<kFew>(l, max_norm, norm, part, sms, s)
                           : launch<kMost>(l, max_norm, norm, part, sms, s);
}

}  // namespace ep
