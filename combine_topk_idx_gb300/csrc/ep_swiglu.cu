// Gated activation between the experts' two products, its 8-bit checkpoint,
// and its gradient from that checkpoint.
//
// Rows of h are gate | up, F elements each.  Forward, per element:
//   a = w * g * sigmoid(g) * u   (w: the row's weight, or 1)
// written as bf16 and/or e4m3 with one fp32 scale per 1x128 block; the
// checkpoint is h itself quantised the same way.  Backward, with g and u read
// back from the checkpoint, sg = sigmoid(g) and t = w * ga:
//   gu = t * g * sg,  gg = t * u * sg * (1 + g * (1 - sg)),
//   gw = sum over the row of ga * g * sg * u.
//
// A CTA takes tiles of whole rows; a thread takes one 16-byte vector of the
// gate and the same of up per step, so 16 neighbouring lanes hold one scale
// block of each.  Alignment padding costs no reads: its rows are recognised
// by their source token and, where the layout zeroes padding, written as 0.
#include <algorithm>

#include "ep_internal.cuh"
#include "ep_ptx.cuh"
#include "ep_quant.cuh"
#include "ep_rows.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kTileVecs = 1024;  // vectors of F per tile: rows per tile = kTileVecs / (F / 8)
constexpr int kMaxTileRows = 64; // F >= 128: at most 1024 / 16 rows

__device__ __forceinline__ float sigmoid(float g) {
  return __fdividef(1.0f, 1.0f + __expf(-g));
}

struct TileRow {
  int64_t row;  // -1: nothing to do
  float w;
  int pad;
};

__device__ __forceinline__ void load_tile(const RowsParams &r, const float *row_w, int64_t i0,
                                          int n, int64_t items, TileRow *rows) {
  if ((int)threadIdx.x < n) {
    bool pad;
    TileRow t;
    t.row = item_row(r, i0 + threadIdx.x, items, &pad);
    t.pad = pad;
    t.w = (row_w != nullptr && t.row >= 0 && !pad) ? __ldg(row_w + t.row) : 1.f;
    if (pad && !r.zero_padding) t.row = -1;
    rows[threadIdx.x] = t;
  }
}

__global__ void __launch_bounds__(kThreads) swiglu_kernel(SwigluParams p, int tile_rows) {
  __shared__ TileRow rows[2][kMaxTileRows];
  griddep_wait();
  const int nv = p.F / 8;
  const int64_t items = item_count(p.r);
  int par = 0;
  for (int64_t i0 = (int64_t)blockIdx.x * tile_rows; i0 < items;
       i0 += (int64_t)gridDim.x * tile_rows, par ^= 1) {
    load_tile(p.r, p.row_w, i0, tile_rows, items, rows[par]);
    __syncthreads();
    const int total = tile_rows * nv;  // a multiple of 16: blocks never split over warps
    for (int id0 = 0; id0 < total; id0 += kThreads) {
      const int id = id0 + threadIdx.x;
      if (id0 + (int)(threadIdx.x & ~31u) >= total) break;
      const int i = id / nv, v = id - i * nv;
      TileRow t{-1, 0.f, 0};
      if (id < total) t = rows[par][i];
      float g[8], u[8], a[8];
      uint4 gv = make_uint4(0, 0, 0, 0), uv = gv;
      if (t.row >= 0 && !t.pad) {
        const uint16_t *h = p.h + t.row * 2 * p.F + v * 8;
        gv = ld_stream_v4(h);
        uv = ld_stream_v4(h + p.F);
      }
      bf16x8_to_f32(gv, g);
      bf16x8_to_f32(uv, u);
#pragma unroll
      for (int q = 0; q < 8; ++q) a[q] = g[q] * sigmoid(g[q]) * u[q] * t.w;
      if (p.act != nullptr && t.row >= 0)
        st_stream_v4(p.act + t.row * p.F + v * 8, f32_to_bf16x8(a));
      float sc;
      if (p.q != nullptr) {
        const uint2 b = quantise_block(a, &sc);
        if (t.row >= 0) {
          st_stream_v2(p.q + t.row * p.F + v * 8, b);
          if ((v & 15) == 0) p.sf[sf_at(p.sfl, t.row, v >> 4)] = sc;
        }
      }
      if (p.ckpt != nullptr) {
        uint8_t *c = p.ckpt + t.row * 2 * p.F + v * 8;
        float *cs = p.ckpt_sf + t.row * (p.F / 64) + (v >> 4);
        const bool keep = t.row >= 0 && !t.pad;
        uint2 b = quantise_block(g, &sc);
        if (keep) {
          st_stream_v2(c, b);
          if ((v & 15) == 0) cs[0] = sc;
        }
        b = quantise_block(u, &sc);
        if (keep) {
          st_stream_v2(c + p.F, b);
          if ((v & 15) == 0) cs[p.F / 128] = sc;
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    swiglu_backward_kernel(SwigluBackwardParams p, int tile_rows) {
  __shared__ TileRow rows[2][kMaxTileRows];
  // one sum per row and 1x128 block of F: tile_rows * F / 128 <= kTileVecs / 16
  // values, or F / 128 of one row
  extern __shared__ float gws[];
  griddep_wait();
  const int nv = p.F / 8, nb = p.F / 128;
  const int64_t items = item_count(p.r);
  int par = 0;
  for (int64_t i0 = (int64_t)blockIdx.x * tile_rows; i0 < items;
       i0 += (int64_t)gridDim.x * tile_rows, par ^= 1) {
    load_tile(p.r, p.row_w, i0, tile_rows, items, rows[par]);
    __syncthreads();
    const int total = tile_rows * nv;
    for (int id0 = 0; id0 < total; id0 += kThreads) {
      const int id = id0 + threadIdx.x;
      if (id0 + (int)(threadIdx.x & ~31u) >= total) break;
      const int i = id / nv, v = id - i * nv;
      TileRow t{-1, 0.f, 0};
      if (id < total) t = rows[par][i];
      uint2 gq = make_uint2(0, 0), uq = gq;
      uint4 dv = make_uint4(0, 0, 0, 0);
      float gs = 0.f, us = 0.f;
      if (t.row >= 0 && !t.pad) {
        const uint8_t *c = p.ckpt + t.row * 2 * p.F + v * 8;
        const float *cs = p.ckpt_sf + t.row * (2 * nb) + (v >> 4);
        gq = ld_stream_v2(c);
        uq = ld_stream_v2(c + p.F);
        dv = ld_stream_v4(p.ga + t.row * p.F + v * 8);
        gs = __ldg(cs);
        us = __ldg(cs + nb);
      }
      float g[8], u[8], d[8], gg[8], gu[8];
      e4m3x8_to_f32(gq, g);
      e4m3x8_to_f32(uq, u);
      bf16x8_to_f32(dv, d);
      float dot = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float gf = g[q] * gs, uf = u[q] * us;
        const float sg = sigmoid(gf), sl = gf * sg;
        dot = fmaf(d[q] * sl, uf, dot);
        const float w = d[q] * t.w;
        gu[q] = w * sl;
        gg[q] = w * uf * (sg * (1.f + gf * (1.f - sg)));
      }
      if (p.gw != nullptr) {
#pragma unroll
        for (int o = 1; o < 16; o *= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (id < total && (v & 15) == 0) gws[i * nb + (v >> 4)] = dot;
      }
      if (p.gh != nullptr && t.row >= 0) {
        uint16_t *o = p.gh + t.row * 2 * p.F + v * 8;
        st_stream_v4(o, f32_to_bf16x8(gg));
        st_stream_v4(o + p.F, f32_to_bf16x8(gu));
      }
      if (p.q != nullptr) {
        float sc, su;
        const uint2 b = quantise_block(gg, &sc), c = quantise_block(gu, &su);
        if (t.row >= 0) {
          uint8_t *o = p.q + t.row * 2 * p.F + v * 8;
          st_stream_v2(o, b);
          st_stream_v2(o + p.F, c);
          if ((v & 15) == 0) {
            p.sf[sf_at(p.sfl, t.row, v >> 4)] = sc;
            p.sf[sf_at(p.sfl, t.row, (v >> 4) + nb)] = su;
          }
        }
      }
    }
    if (p.gw != nullptr) {
      __syncthreads();
      if ((int)threadIdx.x < tile_rows && rows[par][threadIdx.x].row >= 0) {
        float v = 0.f;
        for (int j = 0; j < nb; ++j) v += gws[threadIdx.x * nb + j];
        p.gw[rows[par][threadIdx.x].row] = v;
      }
      __syncthreads();
    }
  }
}

int rows_per_tile(int F) { return std::max(1, std::min(kMaxTileRows, kTileVecs / (F / 8))); }

cudaError_t grid_for(const void *func, size_t smem, int64_t rows, int tile, unsigned *grid) {
  int dev = 0, per_sm = 0;
  const cudaError_t e = launch_geometry(func, kThreads, smem, &dev, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (rows + tile - 1) / tile;
  *grid = (unsigned)std::min<int64_t>(tiles, (int64_t)device_sm_count(dev) * std::max(per_sm, 1));
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_swiglu(const SwigluParams &p, cudaStream_t s) {
  const int tile = rows_per_tile(p.F);
  unsigned grid = 0;
  const cudaError_t e =
      grid_for(reinterpret_cast<const void *>(swiglu_kernel), 0, p.r.rows, tile, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(swiglu_kernel, grid, kThreads, 0, s, p, tile);
}

cudaError_t launch_swiglu_backward(const SwigluBackwardParams &p, cudaStream_t s) {
  const int tile = rows_per_tile(p.F);
  const size_t smem = sizeof(float) * (size_t)tile * (p.F / 128);
  unsigned grid = 0;
  const cudaError_t e = grid_for(reinterpret_cast<const void *>(swiglu_backward_kernel), smem,
                                 p.r.rows, tile, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(swiglu_backward_kernel, grid, kThreads, smem, s, p, tile);
}

}  // namespace ep
