// E4M3 (OCP FN) quantisation with one FP32 scale per 128 values, shared by the standalone
// quantiser and the FP8 GEMMs' SwiGLU epilogue:
//   scale = max(amax / 448, 2^-126),   code = e4m3_rne(value / scale),   in FP32.
// Both divisions are IEEE, so a group's codes depend on its values alone (not on which
// kernel wrote them). The floor keeps the scale a normal FP32 number: a group of zeros gets
// scale 2^-126 and codes 0. |value| / scale rounds to at most 448 (amax / 448 is off by half
// an ulp at most), so no code saturates. A NaN in a group makes its scale and codes NaN; an
// infinity makes the scale infinite, its own code NaN and the finite values' codes 0.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

constexpr int kFp8Block = 128;  // values per scale
constexpr float kE4m3Max = 448.0f;

// The scale of a group whose largest magnitude has the FP32 bits `amax_bits` (the maximum
// of sign-less bit patterns: NaN orders above infinity, so it is not lost).
__device__ __forceinline__ float fp8_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) / kE4m3Max;
  return s < 0x1p-126f ? 0x1p-126f : s;  // a select: NaN stays NaN
}

// The codes of four quotients as four bytes, the first lowest.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

}  // namespace moe
