// FP8 (e4m3) quantisation by 1x128 blocks and BF16 vectors, shared by the
// kernels that write quantised rows (sm_103a).
#pragma once

#include "ep_ptx.cuh"

namespace ep {

// e4m3 bytes of x / sc for eight elements (f: x as fp32), equal to the
// round-to-nearest-even, saturating conversion of the IEEE fp32 quotients.
// With r the reciprocal of sc within 2 ulp (relative error 2^-22), the
// products x * r * (1 -+ 2^-17), each rounded, bracket the rounded quotient
// strictly (every rounding error is below 2^-21 of the 2^-17 margin).  The
// conversion is monotonic in the magnitude, so where both ends of the
// bracket convert to the same byte, the quotient does too; where they differ
// -- a rounding boundary of the e4m3 grid inside the bracket, about 1 element
// in 200 of BF16 data, mostly exact ties -- that pair of quotients is taken
// by IEEE division (per pair, so a warp runs the divisions only for pairs
// where some lane needs them).  Outside sc in [2^-120, 2^120) the reciprocal
// loses its accuracy and every quotient is a division.
__device__ __forceinline__ uint2 e4m3_block8(const float *f, float sc) {
  const uint32_t sb = __float_as_uint(sc);
  uint32_t c[4];
  if (sb >= 0x03800000u && sb < 0x7B800000u) {
    const float r = __fdividef(1.0f, sc);
    const float rl = r * 0.99999237060546875f, rh = r * 1.00000762939453125f;  // 1 -+ 2^-17
    const uint64_t rl2 = f32x2_pack(rl, rl), rh2 = f32x2_pack(rh, rh);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t x2 = f32x2_pack(f[2 * q], f[2 * q + 1]);
      const uint64_t lo = f32x2_mul_rn(x2, rl2), hi = f32x2_mul_rn(x2, rh2);
      c[q] = cvt_e4m3x2(f32x2_lo(lo), f32x2_hi(lo));
      if (c[q] != cvt_e4m3x2(f32x2_lo(hi), f32x2_hi(hi)))
        c[q] = cvt_e4m3x2(__fdiv_rn(f[2 * q], sc), __fdiv_rn(f[2 * q + 1], sc));
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      c[q] = cvt_e4m3x2(__fdiv_rn(f[2 * q], sc), __fdiv_rn(f[2 * q + 1], sc));
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The eight BF16 values of a 16-byte vector as fp32, and back (round to
// nearest even).
__device__ __forceinline__ void bf16x8_to_f32(const uint4 &v, float *f) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
  f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
  f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float *f) {
  return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                    cvt_bf16x2(f[6], f[7]));
}

// Four e4m3 values as two pairs of fp32 (exact; through f16, which holds every
// e4m3 value).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t v, uint64_t *f) {
  float a, b, c, d;
  asm("{\n\t.reg .b16 l, h, e0, e1, e2, e3;\n\t.reg .b32 p, q;\n\t"
      "mov.b32 {l, h}, %4;\n\t"
      "cvt.rn.f16x2.e4m3x2 p, l;\n\tcvt.rn.f16x2.e4m3x2 q, h;\n\t"
      "mov.b32 {e0, e1}, p;\n\tmov.b32 {e2, e3}, q;\n\t"
      "cvt.f32.f16 %0, e0;\n\tcvt.f32.f16 %1, e1;\n\t"
      "cvt.f32.f16 %2, e2;\n\tcvt.f32.f16 %3, e3;\n\t}"
      : "=f"(a), "=f"(b), "=f"(c), "=f"(d)
      : "r"(v));
  f[0] = f32x2_pack(a, b);
  f[1] = f32x2_pack(c, d);
}

// Largest magnitude of 16 values held in pairs; NaN if any is one.
__device__ __forceinline__ float amax_of16(const uint64_t *f) {
  float m = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(f32x2_lo(f[q])), "f"(f32x2_hi(f[q])));
  return m;
}

// Quantises a 1x128 block held by 8 consecutive lanes, 16 fp32 values each:
// scale = amax * (1 / 448), bytes = e4m3(value * r) in fp32, r the scale's
// reciprocal to 1 ulp, to nearest even, saturating.  The dispatch divides both
// times.  Where the values are fp32 results (norm, activation, its gradient) they
// carry errors larger than that.  The checkpoint and the combine gradient have
// BF16 values, which meet exact ties as the dispatch's do: there 1 byte in 1000
// is the other neighbour of the dispatch's, equally near, and more than half of
// the scales are one unit in the last place off its.  The reason for the product
// is its cost: with the dispatch's divisions the norm of 4096 rows of 7168 takes
// 37.4 us against 33.7, the activation of 4096 x 8 rows, F = 2048, with its
// checkpoint 204 against 103, its gradient 146 against 108, the combine gradient
// in FP8 174 against 165.  Every lane of the warp calls it.  An all-zero block,
// or one whose scale rounds to 0, has scale 0 and zero bytes; a block holding a
// NaN a NaN scale and the NaN code in every byte; one holding an infinity scale
// +inf, zeros for its finite values and the NaN code for the infinite ones.
__device__ __forceinline__ void quantise_block16(const uint64_t *f, uint32_t *bytes, float *scale) {
  float amax = amax_of16(f);
#pragma unroll
  for (int o = 1; o < 8; o *= 2)
    amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float sc = amax * (1.0f / 448.0f);
  *scale = sc;
  if (amax < 0x1p-100f) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = f32x2_lo(f[4 * i + q]);
        v[2 * q + 1] = f32x2_hi(f[4 * i + q]);
      }
      const uint2 b = sc != 0.f ? e4m3_block8(v, sc) : make_uint2(0, 0);
      bytes[2 * i] = b.x;
      bytes[2 * i + 1] = b.y;
    }
    return;
  }
  const float r = rcp_approx(sc);  // sc in [2^-109, 2^120), infinite or NaN
  const uint64_t r2 = f32x2_pack(r, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t v = f32x2_mul_rn(f[2 * i], r2), w = f32x2_mul_rn(f[2 * i + 1], r2);
    bytes[i] = cvt_e4m3x4(f32x2_lo(v), f32x2_hi(v), f32x2_lo(w), f32x2_hi(w));
  }
}

// A thread's U vectors of eight BF16 values as pairs of fp32, and 16 e4m3 bytes.
template <int U>
__device__ __forceinline__ void bf16_to_f32(const uint4 *v, uint64_t *f) {
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) f[4 * i + q] = f32x2_pack(bf16_lo(w[q]), bf16_hi(w[q]));
  }
}
template <int U>
__device__ __forceinline__ void store_bf16(void *p, const uint64_t *f) {
#pragma unroll
  for (int i = 0; i < U; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = cvt_bf16x2(f32x2_lo(f[4 * i + q]), f32x2_hi(f[4 * i + q]));
    st_stream_v4(static_cast<uint8_t *>(p) + 16 * i, make_uint4(w[0], w[1], w[2], w[3]));
  }
}
__device__ __forceinline__ void store_bytes16(void *p, const uint32_t *b) {
  st_stream_v4(p, make_uint4(b[0], b[1], b[2], b[3]));
}

}  // namespace ep
