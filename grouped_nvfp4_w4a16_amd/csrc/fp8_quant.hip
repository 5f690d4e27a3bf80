// moe_quant_fp8: BF16 rows to E4M3 codes with one FP32 scale per (row, 128 columns), the
// form the FP8 GEMMs take their rows in.
//
// Bound by memory: 2 bytes read and 1.03 written per value. 16 lanes share a group of 128
// values, 8 values (one 16-byte load, one 8-byte store) per lane, so a wave moves 1 KB of
// consecutive columns; the group's maximum is taken over the 16 lanes.
#include "common.h"
#include "fp8.h"

namespace {

constexpr int kThreads = 256;
constexpr int kLaneVals = 8;
constexpr int kGroupLanes = moe::kFp8Block / kLaneVals;  // 16
constexpr int kGroupsPerBlock = kThreads / kGroupLanes;  // 16

__global__ __launch_bounds__(kThreads) void quant_kernel(
    const uint16_t *__restrict__ x, int64_t ld_x, uint8_t *__restrict__ q, int64_t ld_q,
    float *__restrict__ scale, int64_t ld_s, int64_t groups, int32_t groups_per_row,
    int32_t cols) {
  const int64_t grp = static_cast<int64_t>(blockIdx.x) * kGroupsPerBlock +
                      (threadIdx.x / kGroupLanes);
  if (grp >= groups) return;  // whole 16-lane groups leave together
  const int64_t row = grp / groups_per_row;
  const int g = static_cast<int>(grp - row * groups_per_row);
  const int sub = threadIdx.x % kGroupLanes;
  const int col = g * moe::kFp8Block + sub * kLaneVals;
  const bool live = col < cols;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (live) v = *reinterpret_cast<const uint4 *>(x + row * ld_x + col);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // |BF16| bit patterns order as the magnitudes do.
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = max(m, w[i] & 0x7FFF0000u);
    m = max(m, (w[i] << 16) & 0x7FFF0000u);
  }
#pragma unroll
  for (int d = 1; d < kGroupLanes; d <<= 1)
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, kGroupLanes)));
  const float s = moe::fp8_scale(m);
  if (sub == 0) scale[row * ld_s + g] = s;
  if (!live) return;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16) / s;
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) / s;
  }
  uint2 o;
  o.x = moe::e4m3x4(f[0], f[1], f[2], f[3]);
  o.y = moe::e4m3x4(f[4], f[5], f[6], f[7]);
  *reinterpret_cast<uint2 *>(q + row * ld_q + col) = o;
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
