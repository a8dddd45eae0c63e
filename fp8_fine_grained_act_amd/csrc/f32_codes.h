// Device helpers of the kernels that code FP32 values into E4M3 groups themselves (gated.hip, adamw.hip, the gated
// tiles of gemm.hip).
#pragma once

#include "common.h"

namespace fp8bs {

// the larger magnitude of the two, a NaN if either is one (v_maximum3_f32; fmaxf would drop it)
__device__ __forceinline__ float top_of(float a, float b) {
  return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}

// max of non-negative floats (they order as their bits, a NaN above all others) over aligned groups of 16
// lanes, and with the lane 16 or 32 away (a swap of the operand with itself leaves
// both lanes' values in each)
__device__ __forceinline__ float max16_f32(float v) {
  const uint32_t m = max8_u32(__float_as_uint(v));
  return __uint_as_float(max(m, dpp_shuffle<0x140>(m)));
}
__device__ __forceinline__ float max_xor16_f32(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(max(s[0], s[1]));
}
__device__ __forceinline__ float max_xor32_f32(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(max(s[0], s[1]));
}

// two such values at once: a's maximum with the lane 16 (32) away in the even groups (the
// lower half), b's in the odd ones (the upper half)
__device__ __forceinline__ float max_swap16_f32(float a, float b) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(max(s[0], s[1]));
}
__device__ __forceinline__ float max_swap32_f32(float a, float b) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(max(s[0], s[1]));
}

// Groups of FP32 values that never were bf16 (a gated product, a gradient, an
// optimizer state): s = amax / 448 and E4M3 codes, to nearest even, of x / s.
//   s is correctly rounded: with 1 / 448 correctly rounded, one fma gives the
//   remainder of the first quotient and one more the correction (below 2^-100, where
//   the remainder could be subnormal, the division itself).
//   For amax below 2^-64 both sides of x / s are scaled by 2^64 (s may be subnormal);
//   such an s carries fewer bits, so the quotient is clipped to 448 there (elsewhere it
//   stays below 448 (1 + 2^-21), which codes as 448).  Where s underflows to zero
//   (amax < 2^-141) the codes are signed zeros.
//   An amax that is NaN (top_of) or infinite gives s = NaN and NaN codes: such a group is NaN as a whole.
// F32Scale holds 1 / s as r + rl, to about 2^-46: x / s by f32_quotient, two operations
// that round once more: the binary32 quotient, but where the exact one lies within 2^-46 of a
// boundary between two of them.  (x * r alone is within two units in the last place; a few codes in 10^5 are
// then not the nearest.)
struct F32Scale {
  float s, r, rl, up;
};
__device__ __forceinline__ float over_448_normal(float amax) {   // amax >= 2^-100
  constexpr float kInv = 1.0f / kE4M3Max;
  const float q = amax * kInv;
  return __builtin_fmaf(__builtin_fmaf(-kE4M3Max, q, amax), kInv, q);
}
__device__ __forceinline__ float over_448(float amax) {
  return amax < 0x1p-100f ? amax / kE4M3Max : over_448_normal(amax);
}
constexpr float kTinyGroup = 0x1p-64f;         // below: the slow forms
__device__ __forceinline__ F32Scale f32_scale_as(float s, float amax) {   // s near amax / 448
  F32Scale g;
  g.s = s;
  g.up = amax < kTinyGroup ? kTinyScale : 1.0f;
  const float d = g.s * g.up;
  g.r = d == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(d);
  g.rl = __builtin_fmaf(-d, g.r, 1.0f) * g.r;
  return g;
}
__device__ __forceinline__ F32Scale f32_scale(float amax) { return f32_scale_as(over_448(amax), amax); }
__device__ __forceinline__ F32Scale f32_scale_ordinary(float amax) {     // not below kTinyGroup
  const float s = over_448_normal(amax), r = __builtin_amdgcn_rcpf(s);
  return F32Scale{s, r, __builtin_fmaf(-s, r, 1.0f) * r, 1.0f};
}
// SLOW: some group of the wave may be that small.  Only such groups are clipped, which hold no NaN (v_med3_f32
// would make it a number).
__device__ __forceinline__ float clip_tiny(float q, float up) {
  return up != 1.0f ? __builtin_amdgcn_fmed3f(q, -kE4M3Max, kE4M3Max) : q;
}
template <bool SLOW>
__device__ __forceinline__ float f32_quotient(float x, const F32Scale& g) {
  if (!SLOW) return __builtin_fmaf(x, g.r, x * g.rl);
  const float v = x * g.up;
  return clip_tiny(__builtin_fmaf(v, g.r, v * g.rl), g.up);
}
// The second conversion overwrites the first one's upper half, for which a stands (no register to clear).
__device__ __forceinline__ uint32_t code4_f32(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, __float_as_int(a), false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// act(z) and act'(z) from one sigma.
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& a, float& slope) {
  if (ACT == FP8BS_ACT_RELU) {
    a = z < 0.0f ? 0.0f : z;
    slope = z > 0.0f ? 1.0f : 0.0f;
  } else if (ACT == FP8BS_ACT_GELU_TANH) {
    const float c = z == z ? gelu_clip(z) : z, cc = c * c;
    const float p = sigmoid_of(c * __builtin_fmaf(kGeluC1, cc, kGeluC0));
    a = z * p;
    slope = __builtin_fmaf(c * p * (1.0f - p), __builtin_fmaf(3.0f * kGeluC1, cc, kGeluC0), p);
  } else if (ACT == FP8BS_ACT_SILU) {
    const float p = sigmoid_of(z);
    a = z * p;
    slope = __builtin_fmaf(a, 1.0f - p, p);
  } else {
    a = z;
    slope = 1.0f;
  }
}

}  // namespace fp8bs
