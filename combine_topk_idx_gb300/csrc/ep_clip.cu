// The global norm of many gradients, and their clipping to it:
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// Two passes over the gradients with the norm between them: the first leaves a sum
// per CTA, the second starts by adding all of these up, in the same fixed order in
// every CTA, so neither a counter nor a third launch stands between them.  Few and
// small tensors are one launch of a cluster, where the GPU holds it, whose CTAs read
// each other's sums.  The tensors' addresses travel as launch parameters (up to kMost
// per launch): nothing is copied to the device first.  Both passes are bound by memory.
// The second goes through each CTA's part backwards: what the first read last is still
// in L2.
//
// Sums.  A thread adds up the squares of at most 64 elements in fp32, then goes on in
// fp64, so the error does not grow with the number of elements.  Squares that leave
// the range of fp32 are taken again of scaled values (2^90 or 2^-80, exact): any
// finite gradients have their norm, as far as fp32 holds it.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <vector>

#include "ep_clip.cuh"
#include "ep_ptx.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256, kPerSm = 4;  // of a CTA; CTAs
// 16-byte loads a thread has in flight: a CTA takes 32 KB at a time
constexpr int kLoads = 8;
constexpr int kFew = 64, kMost = 1024;     // tensors of a launch
// One cluster, whose warps take a piece each: up to kFew tensors and this many pieces (4 MB).
// 24 tensors of 1.2 MB take 8.8 us and 11 us of a CPU, in two launches 7.0 us and 16.
constexpr int kClusterCtas = 16, kClusterThreads = 1024, kClusterPieces = 1024;

// Elements that kT threads take at a time.
template <int kT>
__host__ __device__ constexpr int chunk(bool bf16) {
  return kT * kLoads * (bf16 ? 8 : 4);
}

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
template <int kT, int N>
__device__ __forceinline__ Piece piece(const Table<N> &tab, int t, int c) {
  Piece p;
  p.t = t;
  const int64_t n = tab.n[t];
  p.bf16 = n < 0;
  const int per = chunk<kT>(p.bf16);
  p.i0 = (int64_t)(c - tab.first[t]) * per;
  p.len = (int)min((int64_t)per, (n < 0 ? -n : n) - p.i0);
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
template <bool kBf16, int kT>
__device__ __forceinline__ float squares(const void *base, int len, float scale, int tid) {
  constexpr int kSize = kBf16 ? 2 : 4, kVec = 16 / kSize;
  const char *p = static_cast<const char *>(base);
  const int head = head_of(p, kSize, len), vecs = (len - head) / kVec;
  const char *body = p + head * kSize;
  uint4 v[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = tid + u * kT;
    v[u] = i < vecs ? ld_plain_v4(body + 16 * (int64_t)i) : make_uint4(0, 0, 0, 0);
  }
  const int tail = head + vecs * kVec, rest = head + len - tail;
  float e = 0.f;
  if (tid < rest) {  // fewer than 2 * kVec elements about the vectors
    const int i = tid < head ? tid : tail + tid - head;
    if constexpr (kBf16)
      e = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << 16) * scale;
    else
      e = reinterpret_cast<const float *>(p)[i] * scale;
  }
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) add_squares(v[u], kBf16, scale, s);
  return fmaf(e, e, s);
}

template <int kT>
__device__ __forceinline__ double piece_squares(const char *g, const Piece &q, int tid) {
  const auto sum = [&](float scale) {
    return q.bf16 ? squares<true, kT>(g, q.len, scale, tid)
                  : squares<false, kT>(g, q.len, scale, tid);
  };
  float s = sum(1.f);
  double w = 1.0;
  if (!(s > 1e-30f && s < INFINITY)) {
    const bool big = !(s <= 1e-30f);
    s = sum(big ? 0x1p-80f : 0x1p90f);
    w = big ? 0x1p160 : 0x1p-180;
  }
  return (double)s * w;
}

// Sum of one value per thread, in a fixed order; in thread 0.
template <int kT>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kT / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = threadIdx.x < kT / 32 ? part[threadIdx.x] : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float factor(double norm, float max_norm) {
  // NaN, and not 1, for a norm that is NaN
  return norm + 1e-6 <= (double)max_norm ? 1.f : (float)((double)max_norm / (norm + 1e-6));
}

template <bool kBf16>
__device__ __forceinline__ uint4 scaled(const uint32_t (&w)[4], float by) {
  uint32_t r[4];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    r[x] = kBf16 ? cvt_bf16x2(bf16_lo(w[x]) * by, bf16_hi(w[x]) * by)
                 : __float_as_uint(__uint_as_float(w[x]) * by);
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// to[0, len) = from[0, len) * by.  Stores are of 16 bytes, on the boundaries of `to`; where
// `from` lies otherwise, a vector is put together of two of its own, this lane's and the
// next one's (1e9 elements: 1.77 ms where single elements took 3.98).
template <bool kBf16, int kT>
__device__ __forceinline__ void scale_piece(const void *from, void *to, int len, float by,
                                            int tid) {
  constexpr int kSize = kBf16 ? 2 : 4, kVec = 16 / kSize;
  const char *p = static_cast<const char *>(from);
  char *o = static_cast<char *>(to);
  int head = head_of(o, kSize, len), vecs = (len - head) / kVec;
  const int m = (int)(reinterpret_cast<uintptr_t>(p + head * kSize) & 15);
  if (m != 0) {  // the first and the last vector singly: no read before or behind the piece
    head = min(len, head + kVec);
    vecs = max(0, vecs - 2);
  }
  const int reads = vecs == 0 ? 0 : vecs + (m != 0);  // vectors of `from`
  const char *body = p + head * kSize - m;
  char *obody = o + head * kSize;
  const int lane = tid & 31;
  // about the vectors
  const int tail = head + vecs * kVec, rest = head + len - tail;
  for (int j = tid; j < rest; j += kT) {
    const int i = j < head ? j : tail + j - head;
    if constexpr (kBf16)
      reinterpret_cast<uint16_t *>(o)[i] = (uint16_t)cvt_bf16x2(
          __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << 16) * by, 0.f);
    else
      reinterpret_cast<float *>(o)[i] = reinterpret_cast<const float *>(p)[i] * by;
  }
  // in flight; with the 64 registers of four CTAs to an SM 52 bytes spill
  constexpr int kBatch = 4;
#pragma unroll 1
  for (int u0 = 0; u0 < kLoads; u0 += kBatch) {
    // kBatch * 32 vectors of a warp in a row
    const int i0 = u0 * kT + (tid >> 5) * (kBatch * 32) + lane;
    if (i0 - lane >= vecs) break;
    uint4 v[kBatch], behind = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (i0 + u * 32 < reads) v[u] = ld_plain_v4(body + 16 * (int64_t)(i0 + u * 32));
    if (m == 0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * 32;
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        if (i < vecs) st_stream_v4(obody + 16 * (int64_t)i, scaled<kBf16>(w, by));
      }
      continue;
    }
    if (lane == 31 && i0 + (kBatch - 1) * 32 < vecs)
      behind = ld_plain_v4(body + 16 * (int64_t)(i0 + (kBatch - 1) * 32 + 1));
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * 32;
      // lane 31's neighbour is lane 0 of the next 32
      const uint4 after = u + 1 < kBatch ? v[u + 1 < kBatch ? u + 1 : u] : behind;
      const uint32_t mine[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      const uint32_t next[4] = {after.x, after.y, after.z, after.w};
      uint32_t c[8];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        // lane 0 offers the next 32's first word to lane 31, which keeps `behind` itself
        const uint32_t offer = lane == 0 && u + 1 < kBatch ? next[x] : mine[x];
        const uint32_t n = __shfl_sync(0xffffffffu, offer, (lane + 1) & 31);
        c[x] = mine[x];
        c[4 + x] = lane == 31 && u + 1 == kBatch ? next[x] : n;
      }
#pragma unroll
      for (int x = 0; x < 7; ++x) c[x] = m & 4 ? c[x + 1] : c[x];
#pragma unroll
      for (int x = 0; x < 5; ++x) c[x] = m & 8 ? c[x + 2] : c[x];
      uint32_t w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) w[x] = __funnelshift_r(c[x], c[x + 1], (m & 3) * 8);
      if (i < vecs) st_stream_v4(obody + 16 * (int64_t)i, scaled<kBf16>(w, by));
    }
  }
}

template <int kT, int N>
__device__ __forceinline__ void clip_piece(const Table<N> &tab, int t, int c, float by, int tid) {
  if (by == 1.f && tab.o[t] == tab.g[t]) return;  // in place: as it is
  const Piece q = piece<kT>(tab, t, c);
  const int64_t at = q.i0 * (q.bf16 ? 2 : 4);
  const char *g = static_cast<const char *>(tab.g[t]) + at;
  char *o = static_cast<char *>(tab.o[t]) + at;
  if (q.bf16)
    scale_piece<true, kT>(g, o, q.len, by, tid);
  else
    scale_piece<false, kT>(g, o, q.len, by, tid);
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
    const Piece q = piece<kThreads>(tab, t, c);
    sum += piece_squares<kThreads>(
        static_cast<const char *>(tab.g[t]) + q.i0 * (q.bf16 ? 2 : 4), q, threadIdx.x);
  }
  sum = block_sum<kThreads>(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
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
  sum = block_sum<kThreads>(sum);
  if (threadIdx.x == 0) {
    const double n = sqrt(sum);
    by_all = factor(n, max_norm);
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
    clip_piece<kThreads>(tab, t, c, by, threadIdx.x);
  }
}

// Both passes in one cluster.  write: the clipped gradients too.
__global__ void __launch_bounds__(kClusterThreads, 1)
    grad_cluster_kernel(const __grid_constant__ Table<kFew> tab, bool write, float max_norm,
                        float *norm) {
  __shared__ double mine;
  __shared__ float by_all;
  const int chunks = tab.first[tab.count];
  griddep_wait();
  double sum = 0.0;
  const int lane = threadIdx.x & 31, warp = blockIdx.x + kClusterCtas * (threadIdx.x >> 5);
  constexpr int kWarps = kClusterCtas * kClusterThreads / 32;
  for (int c = warp; c < chunks; c += kWarps) {
    const int t = find_tensor(tab, c);
    const Piece q = piece<32>(tab, t, c);
    sum += piece_squares<32>(static_cast<const char *>(tab.g[t]) + q.i0 * (q.bf16 ? 2 : 4), q,
                             lane);
  }
  sum = block_sum<kClusterThreads>(sum);
  if (threadIdx.x == 0) mine = sum;
  cluster_arrive_release();
  cluster_wait();
  if (threadIdx.x < 32) {
    sum = lane < kClusterCtas ? ld_cluster_f64(smem_u32(&mine), lane) : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_down_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      const double n = sqrt(sum);
      by_all = factor(n, max_norm);
      if (norm != nullptr && blockIdx.x == 0) *norm = (float)n;
    }
  }
  cluster_arrive_release();  // no CTA leaves while its sum may be read
  cluster_wait();
  if (write)
    for (int c = warp; c < chunks; c += kWarps)
      clip_piece<32>(tab, find_tensor(tab, c), c, by_all, lane);
}

template <int kT>
int64_t chunks_of(const GradList &l, int i) {
  const int per = chunk<kT>(!l.is_f32[i]);
  return (l.numels[i] + per - 1) / per;
}

// The next tensors of the list (from *at on) that fit a table; empty ones are left out.
template <int kT, int N>
void fill(const GradList &l, int *at, Table<N> *t) {
  t->count = 0;
  int64_t chunks = 0;
  for (; *at < l.count && t->count < N; ++*at) {
    const int i = *at;
    if (l.numels[i] == 0) continue;
    const int64_t c = chunks_of<kT>(l, i);
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
    fill<kThreads>(l, &at, &t);
    if (t.count == 0) break;
    const int grid = std::min(sms * kPerSm, (int)t.first[t.count]);
    e = launch_pdl(grad_squares_kernel<N>, (unsigned)grid, kThreads, 0, s, t, part + parts);
    parts += grid;
  }
  bool first = true;
  for (int at = 0; e == cudaSuccess; first = false) {
    if (l.outs != nullptr) fill<kThreads>(l, &at, &t);
    else t.count = 0, t.first[0] = 0;
    if (t.count == 0 && !(first && norm != nullptr)) break;
    const int grid = std::max(1, std::min(sms * kPerSm, (int)t.first[t.count]));
    e = launch_pdl(grad_clip_kernel<N>, (unsigned)grid, kThreads, 0, s, t,
                   const_cast<const double *>(part), parts, max_norm, first ? norm : nullptr);
    if (t.count == 0) break;
  }
  return e;
}

struct Extent {
  int tensors;     // that are not empty
  int64_t chunks, pieces;  // of a CTA, of a warp
};
Extent extent(const GradList &l) {
  Extent x{0, 0, 0};
  for (int i = 0; i < l.count; ++i) {
    x.tensors += l.numels[i] != 0;
    x.chunks += chunks_of<kThreads>(l, i);
    x.pieces += chunks_of<32>(l, i);
  }
  return x;
}

cudaLaunchConfig_t cluster_config(cudaLaunchAttribute (&attr)[2], cudaStream_t s) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(kClusterCtas);
  lc.blockDim = dim3(kClusterThreads);
  lc.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kClusterCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return lc;
}

// Whether the current device takes the cluster (of more than 8 CTAs: opted in to; part of a
// GPU may not hold it).  Looked up once per device.
bool cluster_fits() {
  struct Entry {
    int device;
    bool fits;
  };
  static std::mutex mu;
  static std::vector<Entry> known;
  int dev = 0, clusters = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> g(mu);
  for (const Entry &e : known)
    if (e.device == dev) return e.fits;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t lc = cluster_config(attr, nullptr);
  const bool fits =
      cudaFuncSetAttribute(grad_cluster_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                           1) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&clusters, grad_cluster_kernel, &lc) == cudaSuccess &&
      clusters > 0;
  try {
    known.push_back({dev, fits});
  } catch (...) {  // no memory: looked up again
  }
  return fits;
}
bool one_cluster(const Extent &x) {
  return x.tensors <= kFew && x.pieces <= kClusterPieces && cluster_fits();
}

cudaError_t launch_cluster(const Table<kFew> &t, bool write, float max_norm, float *norm,
                           cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t lc = cluster_config(attr, s);
  return cudaLaunchKernelEx(&lc, grad_cluster_kernel, t, write, max_norm, norm);
}

}  // namespace

size_t clip_workspace(const GradList &l, int sms) {
  const Extent x = extent(l);
  if (one_cluster(x)) return 0;
  // a sum per CTA of every launch; a launch ends with its table or its chunk numbers
  const int64_t launches = 1 + x.tensors / kMost + 2 * (x.chunks / 0x7fffffffLL);
  return sizeof(double) * (size_t)(launches * sms * kPerSm);
}

cudaError_t launch_clip(const GradList &l, float max_norm, float *norm, void *workspace, int sms,
                        cudaStream_t s) {
  const Extent x = extent(l);
  if (workspace == nullptr) {
    Table<kFew> t;
    int at = 0;
    fill<32>(l, &at, &t);
    return launch_cluster(t, l.outs != nullptr, max_norm, norm, s);
  }
  double *part = static_cast<double *>(workspace);
  return x.tensors <= kFew ? launch<kFew>(l, max_norm, norm, part, sms, s)
                           : launch<kMost>(l, max_norm, norm, part, sms, s);
}

}  // namespace ep
