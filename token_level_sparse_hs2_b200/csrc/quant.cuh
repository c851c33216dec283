// quant.cuh -- the FP8 (e4m3) cache row quantiser shared by every kernel that writes cache rows.
// Per row and matrix, from the format's definition value = scale * code: scale = max|x| / 448 in
// float32 (1 for an all-zero row); code of x = round-to-nearest-even e4m3 of the float32
// quotient x / scale (IEEE division, correctly rounded), saturated at the largest finite e4m3
// value (448).
//
// The quotient is formed with Markstein's correction of the reciprocal product (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev.
// 34(1), 1990): r = RN(1 / scale) once per row, then per value q0 = RN(x r), e = RN(x - scale q0)
// (exact, one fused multiply-add) and q = RN(q0 + e r). Three rounded operations instead of a
// full division per value. For scales in [2^-100, 2^100] it equals the IEEE quotient for every
// bf16 x with |x| <= 448 scale whenever |x / scale| >= 2^-11, and gives a value of the same sign
// below 2^-11 in magnitude, where every such value has the code +-0 (an exhaustive check over
// all bf16 pairs is part of the tests); other scales divide directly.
#pragma once

#include <cuda_fp8.h>

namespace hs2 {

__device__ __forceinline__ float fp8_row_scale(float amax) {
  return amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
}

// The same value in three instructions: the corrected reciprocal product again, whose divisor is a
// constant here (equal to the division for every float32 significand, exponents 2^-100 ... 2^100: a
// test goes through them). Of a block so small that the quotient rounds to zero the scale is 1, as of zeros.
__device__ __forceinline__ float fp8_block_scale(float amax) {
  if (!(amax >= 0x1p-100f && amax <= 0x1p100f)) {
    const float s = fp8_row_scale(amax);
    return s == 0.f ? 1.f : s;
  }
  constexpr float r = 1.f / 448.f;
  const float q0 = __fmul_rn(amax, r);
  return __fmaf_rn(__fmaf_rn(-448.f, q0, amax), r, q0);
}

// The per-row constant of fp8_quotient: RN(1 / scale), or 0 to divide directly.
__device__ __forceinline__ float fp8_row_recip(float sc) {
  return (sc >= 0x1p-100f && sc <= 0x1p100f) ? __frcp_rn(sc) : 0.f;
}

// RN(x / sc), given rc = fp8_row_recip(sc)
__device__ __forceinline__ float fp8_quotient(float x, float sc, float rc) {
  if (rc == 0.f) return __fdiv_rn(x, sc);
  const float q0 = __fmul_rn(x, rc);
  const float e = __fmaf_rn(-sc, q0, x);
  return __fmaf_rn(e, rc, q0);
}

// two codes (low byte = a) of a row whose scale is sc (rc = fp8_row_recip(sc))
__device__ __forceinline__ uint32_t fp8_pair(float a, float b, float sc, float rc) {
  return __nv_cvt_float2_to_fp8x2(make_float2(fp8_quotient(a, sc, rc), fp8_quotient(b, sc, rc)),
                                  __NV_SATFINITE, __NV_E4M3);
}

// eight codes of a block whose scale is sc (rc = fp8_row_recip(sc)); the quotients as in fp8_quotient, two per
// instruction
__device__ __forceinline__ uint2 fp8_codes8(const float2 (&v)[4], float sc, float rc) {
  uint32_t p[4];
  if (rc != 0.f) {
    const float2 r2 = make_float2(rc, rc), n2 = make_float2(-sc, -sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q0 = fmul2(v[i], r2), e = ffma2(n2, q0, v[i]), q = ffma2(e, r2, q0);
      p[i] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[i].x, sc), __fdiv_rn(v[i].y, sc)), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}

}  // namespace hs2
