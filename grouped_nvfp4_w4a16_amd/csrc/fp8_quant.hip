// moe_quant_fp8: BF16 rows to E4M3 codes with one FP32 scale per (row, 128 columns), the
// form the FP8 GEMMs take their rows in.
//
// Bound by memory: 2 bytes read and 1.03 written per value: 4096 x 6144 in 13.0 us, 32768 rows
// in 104 us (5.9 TB/s; a plain copy reaches 4.8, a plain read 6.3). 8 lanes share a group of 128
// values, 16 values (two 16-byte loads, one 16-byte store) per lane, so a wave reads 2 KB and
// writes 1 KB of consecutive columns. The magnitudes' maximum is taken on pairs of BF16
// patterns at once (16-bit integer maxima). The quotients are the IEEE ones without a division
// per value: with inv = 1 / s rounded, q = x inv is corrected once by its exact residual,
// q + (x - q s) inv, which rounds as the division does (checked over every pair of BF16
// mantissas) as long as nothing underflows; other scales take the division itself.
#include "common.h"
#include "fp8.h"

namespace {

constexpr int kThreads = 256;
constexpr int kLaneVals = 16;
constexpr int kGroupLanes = moe::kFp8Block / kLaneVals;  // 8
constexpr int kGroupsPerBlock = kThreads / kGroupLanes;  // 32

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// The larger of two pairs of 16-bit patterns.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                          __builtin_bit_cast(u16x2_t, b)));
}

__global__ __launch_bounds__(kThreads) void quant_kernel(
    const uint16_t *__restrict__ x, int64_t ld_x, uint8_t *__restrict__ q, int64_t ld_q,
    float *__restrict__ scale, int64_t ld_s, int64_t groups, int32_t groups_per_row,
    int32_t cols) {
  const int64_t grp = static_cast<int64_t>(blockIdx.x) * kGroupsPerBlock +
                      (threadIdx.x / kGroupLanes);
  if (grp >= groups) return;  // whole 8-lane groups leave together
  const int64_t row = grp / groups_per_row;
  const int g = static_cast<int>(grp - row * groups_per_row);
  const int sub = threadIdx.x % kGroupLanes;
  const int col = g * moe::kFp8Block + sub * kLaneVals;
  const bool live = col < cols;  // the width is a multiple of 16
  uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
  if (live) {
    const uint4 *src = reinterpret_cast<const uint4 *>(x + row * ld_x + col);
    v0 = src[0];
    v1 = src[1];
  }
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  // |BF16| bit patterns order as the magnitudes do, NaN above infinity.
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m2 = max_u16x2(m2, w[i] & 0x7FFF7FFFu);
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
  for (int d = 1; d < kGroupLanes; d <<= 1)
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, kGroupLanes)));
  const float s = moe::fp8_scale(m << 16);
  if (sub == 0) scale[row * ld_s + g] = s;
  if (!live) return;
  float f[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  if (moe::fp8_ordinary(s)) {
    const float inv = 1.0f / s;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = f[i] * inv;
      f[i] = fmaf(fmaf(-y, s, f[i]), inv, y);
    }
  } else {  // NaN, infinite or tiny: a whole group at a time
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = f[i] / s;
  }
  uint4 o;
  uint32_t *op = &o.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // A zero's sign is lost in the correction: every code takes its value's.
    const uint32_t sign = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x07050301u) & 0x80808080u;
    op[i] = moe::e4m3x4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]) | sign;
  }
  *reinterpret_cast<uint4 *>(q + row * ld_q + col) = o;
}

}  // namespace

extern "C" int moe_quant_fp8(const uint16_t *x, int64_t ld_x, uint8_t *q, int64_t ld_q,
                             float *scale, int64_t ld_scale, int32_t rows, int32_t cols,
                             void *stream) {
  moe::clear_error();
  MOE_REQUIRE(rows >= 0 && cols >= 0 && cols % 16 == 0,
              "quant_fp8: need rows >= 0 and cols >= 0 a multiple of 16 (rows=%d cols=%d)", rows,
              cols);
  const int32_t per_row = (cols + moe::kFp8Block - 1) / moe::kFp8Block;
  MOE_REQUIRE(ld_x >= cols && ld_x % 8 == 0, "quant_fp8: ld_x must be >= cols and a multiple of 8");
  MOE_REQUIRE(ld_q >= cols && ld_q % 16 == 0,
              "quant_fp8: ld_q must be >= cols and a multiple of 16");
  MOE_REQUIRE(ld_scale >= per_row, "quant_fp8: ld_scale must be >= ceil(cols / 128)");
  if (rows == 0 || cols == 0) return MOE_OK;
  MOE_REQUIRE(x && q && scale, "quant_fp8: a required pointer is NULL");
  MOE_REQUIRE(moe::aligned16(x) && moe::aligned16(q) &&
                  (reinterpret_cast<uintptr_t>(scale) & 3u) == 0,
              "quant_fp8: x and q must be 16-byte aligned, scale 4-byte aligned");
  const int64_t groups = static_cast<int64_t>(rows) * per_row;
  const int64_t blocks = (groups + kGroupsPerBlock - 1) / kGroupsPerBlock;
  // A launch holds fewer than 2^32 threads.
  MOE_REQUIRE(blocks < (1ll << 32) / kThreads, "quant_fp8: matrix too large");
  return moe::launch("moe_quant_fp8", quant_kernel, dim3(static_cast<unsigned>(blocks)),
                     dim3(kThreads), 0, stream, x, ld_x, q, ld_q, scale, ld_scale, groups,
                     per_row, cols);
}
