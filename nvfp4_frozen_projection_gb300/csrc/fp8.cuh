// Device helpers of the FP8 kernels: E4M3 values with one FP32 scale per block of
// 128 (activations: 128 consecutive values of a row; weights: a 128 x 128 tile).
//
// A block with largest magnitude amax is held with
//   t = max(amax, 448 * 2^-126),  s = RN(t / 448),  r = RN(448 / t),
//   q = e4m3_rne_satfinite(RN(x r)),   value = q s.
// The floor on t keeps s and r normal FP32 numbers, so a zero block needs no case of
// its own (its values are zeros).  The product with r instead of a division by s is
// part of the definition: one instruction per value, and the two differ only where a
// quotient lies within 2^-22 of a rounding border of E4M3, whose steps are 2^-4.  Of BF16
// values those are exact ties, either side of which is a nearest code: on normal data 3 codes
// in 10,000 are the other side from e4m3(448 x / t) (of a division by s: 6 in a million), so
// a tensor that another program made by division does not match code for code.
// A NaN or an infinity is taken as it is (its code is a NaN), so the FP8 kernels have none
// of the debug build's checks for NaN.
#pragma once

#include "common.cuh"

namespace pact {

constexpr float kE4m3Max = 448.0f;
constexpr float kFp8TMin = 0x1.cp-118f;  // 448 * 2^-126

struct Fp8Scale {
  float s;  // decode scale
  float r;  // encode factor
};
__device__ __forceinline__ Fp8Scale fp8_scale(float amax) {
  const float t = fmaxf(amax, kFp8TMin);
  Fp8Scale f;
  f.s = __fdiv_rn(t, kE4m3Max);
  f.r = __fdiv_rn(kE4m3Max, t);
  return f;
}

// Two FP32 values -> E4M3 bytes (RN, satfinite), lo in bits 0..7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// e4m3(RN(x r)) of eight values, element 0 in the low byte of .x.
__device__ __forceinline__ uint2 e4m3x8(const float* x, float r) {
  float p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = __fmul_rn(x[i], r);
  return make_uint2(e4m3x2(p[0], p[1]) | (e4m3x2(p[2], p[3]) << 16),
                    e4m3x2(p[4], p[5]) | (e4m3x2(p[6], p[7]) << 16));
}

// max |.| over the 16 lanes of a half warp, which hold one block of 128 values.
__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

}  // namespace pact
