// E4M3 (OCP FN) quantisation with one FP32 scale per 128 values, shared by the standalone
// quantiser and the FP8 GEMMs' SwiGLU epilogue:
//   scale = max(amax / 448, 2^-126),   code = e4m3_rne(value / scale),   in FP32.
// Both quotients round as IEEE divisions do, so a group's codes depend on its values alone (not
// on which kernel wrote them). The floor keeps the scale a normal FP32 number: a group of zeros gets
// scale 2^-126 and codes 0. |value| / scale rounds to at most 448 (amax / 448 is off by half
// an ulp at most), so no code saturates. A NaN in a group makes its scale and codes NaN; an
// infinity makes the scale infinite, its own code NaN and the finite values' codes 0.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "fp8_plan.h"  // kFp8Block

namespace moe {

constexpr float kE4m3Max = 448.0f;

// The scale of a group whose largest magnitude has the FP32 bits `amax_bits` (the maximum
// of sign-less bit patterns: NaN orders above infinity, so it is not lost).
__device__ __forceinline__ float fp8_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) / kE4m3Max;
  return s < 0x1p-126f ? 0x1p-126f : s;  // a select: NaN stays NaN
}

// Scales whose quotients need no division: nothing that matters to a code over- or underflows.
__device__ __forceinline__ bool fp8_ordinary(float s) { return s >= 0x1p-64f && s <= 0x1p100f; }

// v / s as IEEE rounds it, inv = 1 / s rounded, s ordinary: the first correction leaves the
// product within an ulp, the second (its residual is exact) then rounds as the division does
// (Markstein's theorem). A zero keeps v's sign. 6 operations, a division takes 11.
__device__ __forceinline__ float fp8_quotient(float v, float s, float inv) {
  float y = v * inv;
  y = fmaf(fmaf(-y, s, v), inv, y);
  y = fmaf(fmaf(-y, s, v), inv, y);
  return __builtin_copysignf(y, v);
}

// silu(min(g, L)) * clamp(u, -L, L) in FP32 with moe::swiglu_clamp1's properties (selects keep a
// NaN; e = e^-|g|, so nothing overflows; full range) in 20 operations instead of 50, for
// outputs quantised to 4 significant bits. The hardware exponential ends at the normal numbers:
// below g = -87 it takes e 2^64. Its argument's rounding moves e by |g| 2^-24, as the rounding
// of the sum g itself does; the reciprocal is off by an ulp.
__device__ __forceinline__ float fp8_swiglu(float g, float u, float limit) {
  const float gc = g > limit ? limit : g;
  const float uc = u > limit ? limit : (u < -limit ? -limit : u);
  const float t = -1.44269504f * fabsf(gc);  // log2(e)
  const bool tiny = t < -125.0f;
  float e = __builtin_amdgcn_exp2f(tiny ? t + 64.0f : t);
  e = tiny ? e * 0x1p-64f : e;
  const float num = gc >= 0.0f ? gc : gc * e;
  return num * __builtin_amdgcn_rcpf(1.0f + e) * uc;
}

// The codes of four quotients as four bytes, the first lowest.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

}  // namespace moe
