// INT8 quantisation with one FP32 scale per row, shared by the row quantiser and the norm:
//   scale = max(amax / 127, 2^-126),   code = rint(value / scale) in [-127, 127],   in FP32.
// Both quotients round as IEEE divisions do, the codes to nearest, ties to even. The floor keeps
// the scale a normal FP32 number: a row of zeros gets scale 2^-126 and codes 0. |value| / scale
// rounds to at most 127 (1 + 2^-24), so no code saturates. A row with a NaN or an infinity gets
// a NaN or infinite scale and codes 0: every product with it is NaN.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "fp8.h"  // fp8_quotient: a quotient as IEEE rounds it, without a division per value

namespace moe {

constexpr float kInt8Max = 127.0f;

// moe_quant_int8 of contiguous FP32 rows (16-byte aligned), reporting errors as `name`.
int quant_int8_f32(const char *name, const float *x, int8_t *q, float *scale, int32_t rows,
                   int32_t cols, void *stream);

// The scale of a row whose largest magnitude has the FP32 bits `amax_bits` (the maximum of
// sign-less bit patterns: NaN orders above infinity, so it is not lost).
__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) / kInt8Max;
  return s < 0x1p-126f ? 0x1p-126f : s;  // a select: NaN stays NaN
}

// Codes of 8 values (bytes, the first lowest), inv = 1 / s. Adding 1.5 2^23 rounds a quotient of
// at most 127 to an integer, ties to even, whose two's complement byte is the sum's lowest one.
__device__ __forceinline__ uint2 int8_codes8(const float (&v)[8], float s, float inv) {
  uint32_t b[8];
  if (fp8_ordinary(s)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      b[i] = __float_as_uint(fp8_quotient(v[i], s, inv) + 0x1.8p23f);
  } else if (s < 0x1p-64f || (s > 0x1p100f && s < INFINITY)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(v[i] / s + 0x1.8p23f);
  } else {  // NaN or infinite: a whole row at a time
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0;
  }
  const auto pack4 = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x0C0C0400u);
    return lo | hi << 16;
  };
  return make_uint2(pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]));
}

}  // namespace moe
