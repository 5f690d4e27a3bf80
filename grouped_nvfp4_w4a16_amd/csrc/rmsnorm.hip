// moe_rmsnorm_bf16, moe_rmsnorm_fp8, moe_rmsnorm_int8 and moe_quant_int8: the rows a
// feed-forward layer starts from. One pass per row:
//
//   h = bf16(x + residual)                      (the residual stream, stored where asked for)
//   y = h * g * rstd,   rstd = 1 / sqrt(mean(h^2) + eps)                             (FP32)
//   BF16 output: bf16(y)
//   E4M3 output: s = max(amax(y) / 448, 2^-126) per 128 columns, code = e4m3(y / s)
//   INT8 output: s = max(amax(y) / 127, 2^-126) per row, code = rint(y / s)
//
// The norm is taken of the stored sum h, so a row's output is a function of the residual stream
// that the next layer reads. Nothing else is rounded before the codes: y stays FP32.
// Because a rounded product by rstd is monotonic, amax(y) = amax(h g) rstd exactly: the row's
// maxima are found in the pass that sums the squares, before rstd is known, and one barrier per
// row serves both.
//
// Bound by memory: 4 bytes read, up to 5 written per value: 4096 x 6144 with every output in 43 us,
// 5.3 TB/s (a copy reaches 4.9); 8 rows in 3.7 to 4.0 us, the chain of a launch, the loads of x and
// the residual, the row's sum, the weight's load behind it (the INT8 form's stands before) and the
// stores. moe_quant_int8 of 4096 x 6144 takes 18 us (4.2 TB/s). A lane holds 8 consecutive columns
// per iteration (16-byte loads and stores, 16 lanes to a group of 128), the row stays in registers
// between the passes.
#include "common.h"
#include "fp8.h"
#include "int8.h"
#include "nvfp4_decode.h"  // moe::pack_bf16x2

namespace {

constexpr int kLaneVals = 8;
constexpr int kGroupLanes = moe::kFp8Block / kLaneVals;  // 16
constexpr int kMaxThreads = 1024;

enum class Out { kBf16, kFp8, kInt8 };

struct NormArgs {
  const void *x;        // BF16, or FP32 (the quantiser of the shared expert's activations)
  const uint16_t *res;  // or NULL
  const uint16_t *g;
  uint16_t *h, *y;      // or NULL
  uint8_t *q;
  float *scale;
  int64_t ld_x, ld_res, ld_h, ld_y, ld_q, ld_s;
  int32_t cols;
  float eps;
};

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// The largest of the sign-less bit patterns (NaN orders above infinity) of `lanes` lanes.
__device__ __forceinline__ uint32_t lanes_max(uint32_t m, int lanes) {
  for (int d = 1; d < lanes; d <<= 1)
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, 64)));
  return m;
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(moe::pack_bf16x2(f[0], f[1]), moe::pack_bf16x2(f[2], f[3]),
                    moe::pack_bf16x2(f[4], f[5]), moe::pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
  f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
  f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

// 8 values of a row as they are held: BF16 patterns, or FP32.
struct Bf16x8 {
  uint4 v;
};
struct F32x8 {
  float4 a, b;
};

__device__ __forceinline__ void unpack8(const Bf16x8 &v, float (&f)[8]) { unpack8(v.v, f); }
__device__ __forceinline__ void unpack8(const F32x8 &v, float (&f)[8]) {
  f[0] = v.a.x; f[1] = v.a.y; f[2] = v.a.z; f[3] = v.a.w;
  f[4] = v.b.x; f[5] = v.b.y; f[6] = v.b.z; f[7] = v.b.w;
}

__device__ __forceinline__ void fetch8(const NormArgs &p, int64_t row, int col, F32x8 &o) {
  const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) +
                                                       row * p.ld_x + col);
  o = {src[0], src[1]};
}

// The 8 columns' sum h of a row. Not __restrict__: h may be x or the residual (each element is
// read by the thread that then writes it).
__device__ __forceinline__ void fetch8(const NormArgs &p, int64_t row, int col, Bf16x8 &o) {
  uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + row * p.ld_x +
                                             col);
  if (p.res != nullptr) {
    const uint4 r = *reinterpret_cast<const uint4 *>(p.res + row * p.ld_res + col);
    float a[8], b[8];
    unpack8(v, a);
    unpack8(r, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] += b[i];
    v = pack8(a);
  }
  o.v = v;
}

// Codes of 8 values with an E4M3 scale, or an INT8 one.
__device__ __forceinline__ uint2 fp8_codes8(const float (&y)[8], float s) {
  float q[8];
  if (moe::fp8_ordinary(s)) {
    const float inv = 1.0f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = moe::fp8_quotient(y[i], s, inv);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = y[i] / s;
  }
  return make_uint2(moe::e4m3x4(q[0], q[1], q[2], q[3]), moe::e4m3x4(q[4], q[5], q[6], q[7]));
}

// One row per block. kIter > 0: the row fits kIter iterations of the block and stays in
// registers; 0: any width, h is formed again for the output.
template <Out kOut, bool kNorm, class Held, int kIter>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(NormArgs p) {
  constexpr int kHeld = kIter > 0 ? kIter : 1;
  __shared__ float s_sum[kMaxThreads / 64];
  __shared__ uint32_t s_max[kMaxThreads / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n_waves = static_cast<int>(blockDim.x >> 6);
  const int step = static_cast<int>(blockDim.x) * kLaneVals;

  // 1. The row's sums of squares, and the largest |h g| (INT8: of the row, E4M3: of the lane's
  //    group of 128, found in step 2).
  Held held[kHeld];
  float sum = 0.0f;
  uint32_t top = 0;
  const auto scan = [&](const Held &v, int col) {
    float f[8];
    unpack8(v, f);
    if (kNorm) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
    }
    if (kOut == Out::kInt8) {
      float g[8];
      if (kNorm) unpack8(*reinterpret_cast<const uint4 *>(p.g + col), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, magnitude(kNorm ? f[i] * g[i] : f[i]));
    }
  };
  if (kIter > 0) {
#pragma unroll
    for (int it = 0; it < kHeld; ++it) {
      const int col = tid * kLaneVals + it * step;
      held[it] = {};
      if (col < p.cols) fetch8(p, row, col, held[it]);
    }
#pragma unroll
    for (int it = 0; it < kHeld; ++it) {
      const int col = tid * kLaneVals + it * step;
      if (col < p.cols) scan(held[it], col);
    }
  } else {
    for (int64_t col = tid * kLaneVals; col < p.cols; col += step) {
      fetch8(p, row, static_cast<int>(col), held[0]);
      scan(held[0], static_cast<int>(col));
    }
  }
  float rstd = 1.0f;
  if (kNorm || kOut == Out::kInt8) {
    sum = wave_sum(sum);
    if (kOut == Out::kInt8) top = lanes_max(top, 64);
    if (lane == 0) {
      s_sum[wave] = sum;
      s_max[wave] = top;
    }
    __syncthreads();
    sum = 0.0f;
    for (int w = 0; w < n_waves; ++w) {
      sum += s_sum[w];
      top = max(top, s_max[w]);
    }
    if (kNorm) rstd = 1.0f / sqrtf(sum / static_cast<float>(p.cols) + p.eps);
  }
  float row_scale = 0.0f, row_inv = 0.0f;
  if (kOut == Out::kInt8) {
    row_scale = moe::int8_scale(magnitude(__uint_as_float(top) * rstd));
    row_inv = 1.0f / row_scale;
    if (tid == 0) p.scale[row] = row_scale;
  }

  // 2. The outputs. Every lane of a wave takes part while one has columns (the groups' maxima).
  const auto put = [&](const Held &v, int64_t col) {
    const bool live = col < p.cols;
    float f[8];
    unpack8(v, f);
    if (kNorm && live) {
      float g[8];
      unpack8(*reinterpret_cast<const uint4 *>(p.g + col), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * g[i] * rstd;
    }
    if constexpr (kNorm)
      if (live && p.h != nullptr) *reinterpret_cast<uint4 *>(p.h + row * p.ld_h + col) = v.v;
    if (kNorm && live && p.y != nullptr)
      *reinterpret_cast<uint4 *>(p.y + row * p.ld_y + col) = pack8(f);
    if (kOut == Out::kFp8) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, live ? magnitude(f[i]) : 0u);
      const float s = moe::fp8_scale(lanes_max(m, kGroupLanes));
      if (live) {
        if (lane % kGroupLanes == 0) p.scale[row * p.ld_s + col / moe::kFp8Block] = s;
        *reinterpret_cast<uint2 *>(p.q + row * p.ld_q + col) = fp8_codes8(f, s);
      }
    }
    if (kOut == Out::kInt8 && live)
      *reinterpret_cast<uint2 *>(p.q + row * p.ld_q + col) =
          moe::int8_codes8(f, row_scale, row_inv);
  };
  if (kIter > 0) {
#pragma unroll
    for (int it = 0; it < kHeld; ++it) {
      const int base = wave * 64 * kLaneVals + it * step;  // wave-uniform
      if (base < p.cols) put(held[it], tid * kLaneVals + it * step);
    }
  } else {
    for (int64_t base = wave * 64 * kLaneVals; base < p.cols; base += step) {
      const int64_t col = base + lane * kLaneVals;
      held[0] = {};
      if (col < p.cols) fetch8(p, row, static_cast<int>(col), held[0]);
      put(held[0], col);
    }
  }
}

int check_norm(const char *name, const NormArgs &p, bool norm, int32_t rows) {
  const auto rows_ok = [&](const void *ptr, int64_t ld) {
    return ptr == nullptr || (ld >= p.cols && ld % 8 == 0);
  };
  MOE_REQUIRE(rows >= 0 && p.cols >= 0 && p.cols % 8 == 0,
              "%s: need rows >= 0 and cols >= 0 a multiple of 8 (rows=%d cols=%d)", name, rows,
              p.cols);
  MOE_REQUIRE(p.eps >= 0.0f && p.eps < INFINITY, "%s: eps must be finite and >= 0", name);
  MOE_REQUIRE(p.ld_x >= p.cols && p.ld_x % 8 == 0 && rows_ok(p.res, p.ld_res) &&
                  rows_ok(p.h, p.ld_h) && rows_ok(p.y, p.ld_y) && rows_ok(p.q, p.ld_q),
              "%s: leading dimensions must be >= cols and multiples of 8", name);
  if (rows == 0 || p.cols == 0) return MOE_OK;
  MOE_REQUIRE(p.x && (!norm || p.g), "%s: a required pointer is NULL", name);
  MOE_REQUIRE(moe::aligned16(p.x) && moe::aligned16(p.res) && moe::aligned16(p.g) &&
                  moe::aligned16(p.h) && moe::aligned16(p.y),
              "%s: x, residual, weight, h and y must be 16-byte aligned", name);
  MOE_REQUIRE((reinterpret_cast<uintptr_t>(p.q) & 7u) == 0 &&
                  (reinterpret_cast<uintptr_t>(p.scale) & 3u) == 0,
              "%s: q must be 8-byte aligned, scale 4-byte aligned", name);
  MOE_REQUIRE(p.h == nullptr || p.h != p.y, "%s: h and y must not be the same buffer", name);
  // In place: a row's output over that row's input, not over another row's.
  const auto place_ok = [&](const void *out, int64_t ld, const void *in, int64_t ld_in) {
    return rows == 1 || out == nullptr || out != in || ld == ld_in;
  };
  MOE_REQUIRE(place_ok(p.h, p.ld_h, p.x, p.ld_x) && place_ok(p.h, p.ld_h, p.res, p.ld_res) &&
                  place_ok(p.y, p.ld_y, p.x, p.ld_x),
              "%s: an output in place of an input needs its leading dimension", name);
  // A launch holds fewer than 2^32 threads.
  MOE_REQUIRE(rows < (1ll << 32) / kMaxThreads, "%s: at most 2^22 - 1 rows (got %d)", name, rows);
  return MOE_OK;
}

// The block: as many threads as a row has lanes' worth of columns, up to 1024. Fewer threads with
// several iterations each, which hold more loads in flight per wave, took longer at every number of
// rows: 6144 columns on 256 threads (3 iterations) against 768, us: 8 rows 5.1 / 3.7, 512 8.8 / 7.9,
// 4096 49.0 / 42.8.
template <Out kOut, bool kNorm, class Held = Bf16x8>
int launch_norm(const char *name, const NormArgs &p, int32_t rows, void *stream) {
  const int64_t lanes = (static_cast<int64_t>(p.cols) + kLaneVals - 1) / kLaneVals;
  const int64_t waves = (lanes + 63) / 64;
  const int64_t iter = (waves + 15) / 16;
  const int64_t per = std::min<int64_t>((waves + iter - 1) / iter, 16);
  const dim3 grid(static_cast<unsigned>(rows)), block(static_cast<unsigned>(64 * per));
  const auto go = [&](auto kern) { return moe::launch(name, kern, grid, block, 0, stream, p); };
  // Rows of up to 32768 columns stay in registers.
  if (iter == 1) return go(norm_kernel<kOut, kNorm, Held, 1>);
  if (iter == 2) return go(norm_kernel<kOut, kNorm, Held, 2>);
  if (iter == 3) return go(norm_kernel<kOut, kNorm, Held, 3>);
  if (iter == 4) return go(norm_kernel<kOut, kNorm, Held, 4>);
  return go(norm_kernel<kOut, kNorm, Held, 0>);
}

}  // namespace

extern "C" int moe_rmsnorm_bf16(const uint16_t *x, int64_t ld_x, const uint16_t *residual,
                                int64_t ld_res, const uint16_t *weight, float eps, uint16_t *h,
                                int64_t ld_h, uint16_t *y, int64_t ld_y, int32_t rows,
                                int32_t cols, void *stream) {
  moe::clear_error();
  const NormArgs p = {x, residual, weight, h, y, nullptr, nullptr, ld_x, ld_res, ld_h, ld_y, 0, 0,
                      cols, eps};
  const int rc = check_norm("rmsnorm_bf16", p, true, rows);
  if (rc != MOE_OK || rows == 0 || cols == 0) return rc;
  MOE_REQUIRE(y, "rmsnorm_bf16: a required pointer is NULL");
  return launch_norm<Out::kBf16, true>("moe_rmsnorm_bf16", p, rows, stream);
}

extern "C" int moe_rmsnorm_fp8(const uint16_t *x, int64_t ld_x, const uint16_t *residual,
                               int64_t ld_res, const uint16_t *weight, float eps, uint16_t *h,
                               int64_t ld_h, uint16_t *y, int64_t ld_y, uint8_t *q, int64_t ld_q,
                               float *scale, int64_t ld_scale, int32_t rows, int32_t cols,
                               void *stream) {
  moe::clear_error();
  const NormArgs p = {x, residual, weight, h, y, q, scale, ld_x, ld_res, ld_h, ld_y, ld_q,
                      ld_scale, cols, eps};
  const int rc = check_norm("rmsnorm_fp8", p, true, rows);
  if (rc != MOE_OK) return rc;
  MOE_REQUIRE(ld_q >= cols && ld_q % 8 == 0,
              "rmsnorm_fp8: ld_q must be >= cols and a multiple of 8");
  MOE_REQUIRE(ld_scale >= (static_cast<int64_t>(cols) + moe::kFp8Block - 1) / moe::kFp8Block,
              "rmsnorm_fp8: ld_scale must be >= ceil(cols / 128)");
  if (rows == 0 || cols == 0) return MOE_OK;
  MOE_REQUIRE(q && scale, "rmsnorm_fp8: a required pointer is NULL");
  return launch_norm<Out::kFp8, true>("moe_rmsnorm_fp8", p, rows, stream);
}

extern "C" int moe_rmsnorm_int8(const uint16_t *x, int64_t ld_x, const uint16_t *residual,
                                int64_t ld_res, const uint16_t *weight, float eps, uint16_t *h,
                                int64_t ld_h, uint16_t *y, int64_t ld_y, int8_t *q, int64_t ld_q,
                                float *scale, int32_t rows, int32_t cols, void *stream) {
  moe::clear_error();
  const NormArgs p = {x, residual, weight, h, y, reinterpret_cast<uint8_t *>(q), scale, ld_x,
                      ld_res, ld_h, ld_y, ld_q, 0, cols, eps};
  const int rc = check_norm("rmsnorm_int8", p, true, rows);
  if (rc != MOE_OK) return rc;
  MOE_REQUIRE(ld_q >= cols && ld_q % 8 == 0,
              "rmsnorm_int8: ld_q must be >= cols and a multiple of 8");
  if (rows == 0 || cols == 0) return MOE_OK;
  MOE_REQUIRE(q && scale, "rmsnorm_int8: a required pointer is NULL");
  return launch_norm<Out::kInt8, true>("moe_rmsnorm_int8", p, rows, stream);
}

extern "C" int moe_quant_int8(const uint16_t *x, int64_t ld_x, int8_t *q, int64_t ld_q,
                              float *scale, int32_t rows, int32_t cols, void *stream) {
  moe::clear_error();
  const NormArgs p = {x, nullptr, nullptr, nullptr, nullptr, reinterpret_cast<uint8_t *>(q), scale,
                      ld_x, 0, 0, 0, ld_q, 0, cols, 0.0f};
  const int rc = check_norm("quant_int8", p, false, rows);
  if (rc != MOE_OK) return rc;
  MOE_REQUIRE(ld_q >= cols && ld_q % 8 == 0,
              "quant_int8: ld_q must be >= cols and a multiple of 8");
  if (rows == 0 || cols == 0) return MOE_OK;
  MOE_REQUIRE(q && scale, "quant_int8: a required pointer is NULL");
  return launch_norm<Out::kInt8, false>("moe_quant_int8", p, rows, stream);
}

namespace moe {

int quant_int8_f32(const char *name, const float *x, int8_t *q, float *scale, int32_t rows,
                   int32_t cols, void *stream) {
  const NormArgs p = {x, nullptr, nullptr, nullptr, nullptr, reinterpret_cast<uint8_t *>(q), scale,
                      cols, 0, 0, 0, cols, 0, cols, 0.0f};
  const int rc = check_norm(name, p, false, rows);
  if (rc != MOE_OK || rows == 0 || cols == 0) return rc;
  return launch_norm<Out::kInt8, false, F32x8>(name, p, rows, stream);
}

}  // namespace moe
