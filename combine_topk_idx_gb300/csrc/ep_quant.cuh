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

// The eight e4m3 values of an 8-byte vector as fp32 (exact; through f16,
// which holds every e4m3 value).
__device__ __forceinline__ void e4m3x8_to_f32(const uint2 &v, float *f) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    asm("{\n\t.reg .b16 l, h, e0, e1, e2, e3;\n\t.reg .b32 p, q;\n\t"
        "mov.b32 {l, h}, %4;\n\t"
        "cvt.rn.f16x2.e4m3x2 p, l;\n\tcvt.rn.f16x2.e4m3x2 q, h;\n\t"
        "mov.b32 {e0, e1}, p;\n\tmov.b32 {e2, e3}, q;\n\t"
        "cvt.f32.f16 %0, e0;\n\tcvt.f32.f16 %1, e1;\n\t"
        "cvt.f32.f16 %2, e2;\n\tcvt.f32.f16 %3, e3;\n\t}"
        : "=f"(f[4 * i]), "=f"(f[4 * i + 1]), "=f"(f[4 * i + 2]), "=f"(f[4 * i + 3])
        : "r"(w[i]));
  }
}

// Quantises a 1x128 block held by 16 consecutive lanes, eight fp32 values
// each: scale = amax / 448 (fp32 division), bytes = e4m3(value / scale).
// Every lane of the warp calls it.  An all-zero block has scale 0 and zero
// bytes; a block holding a NaN a NaN scale and the NaN code in every byte.
__device__ __forceinline__ uint2 quantise_block(const float *f, float *scale) {
  float amax = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) amax = fmax_nan(amax, fabsf(f[q]));
#pragma unroll
  for (int o = 1; o < 16; o *= 2) amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float sc = __fdiv_rn(amax, 448.0f);
  *scale = sc;
  if (amax != amax) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  // a block so small that its scale rounds to 0 counts as zero
  return sc != 0.f ? e4m3_block8(f, sc) : make_uint2(0, 0);
}

}  // namespace ep
