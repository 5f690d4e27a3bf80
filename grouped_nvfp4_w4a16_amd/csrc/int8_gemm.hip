// moe_dense_gemm_int8 and moe_dense_gate_up_swiglu_int8: INT8 rows with one FP32 scale per row
// (token), times INT8 weights with one FP32 scale per output channel.
//
//   S[m, n] = sum_k a[m, k] * w[n, k]               exact in int32 (K <= MOE_INT8_MAX_K)
//   y[m, n] = (float(S) * sa[m]) * sw[n]            FP32, in this order
//   c[m, n] = bf16(y), or bf16(silu(min(G, L)) * clamp(U, -L, L)) of the gate's and up's y
//
// Because the sums are exact, every tile, split and order of K gives the same bits.
//
// Two kernels:
//   - few rows (m <= 64): the weights stream from memory straight into the registers of the
//     matrix instruction, K split over the waves of a block;
//   - tiles: stages of 128 k (KS of them side by side) loaded straight into LDS, ST - 1 ahead.
// The product is v_mfma_i32_16x16x64_i8 with weights as operand A and rows as B: a lane holds 4
// consecutive outputs of one row.
#include "buffer_io.h"
#include "common.h"
#include "fp8.h"  // fp8_swiglu
#include "int8.h"
#include "lds_limit.h"
#include "nvfp4_decode.h"  // moe::pack_bf16x2

namespace {

using moe::kNoLoad;
using moe::make_rsrc;
using moe::u32x4_t;

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kRowBytes = 128;  // one LDS row: 128 k
constexpr int kMaxK = MOE_INT8_MAX_K;
constexpr int kGroupM = 4;  // row tiles that run next to each other

struct GemmArgs {
  const int8_t *a;       // [m, lda]
  const float *a_scale;  // [m]
  const int8_t *w0, *w1; // the weight, or gate and up
  const float *s0, *s1;  // their scales per output channel
  uint16_t *c;           // BF16 output [m, ldc] ...
  float *c32;            // ... or, where not NULL, FP32 output [m, ldc] (SwiGLU form)
  int64_t lda, ldw, ldc;
  int32_t m, n, k;
  float limit;
};

__device__ __forceinline__ i32x4_t mma(u32x4_t w, u32x4_t x, i32x4_t d) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, w),
                                               __builtin_bit_cast(i32x4_t, x), d, 0, 0, 0);
}

// Four consecutive outputs of a row.
template <bool kSwiglu>
__device__ __forceinline__ void store4(const GemmArgs &p, int64_t row, int col,
                                       const float (&y)[4]) {
  if (kSwiglu && p.c32 != nullptr) {  // uniform
    *reinterpret_cast<float4 *>(p.c32 + row * p.ldc + col) = make_float4(y[0], y[1], y[2], y[3]);
    return;
  }
  const uint2 o = make_uint2(moe::pack_bf16x2(y[0], y[1]), moe::pack_bf16x2(y[2], y[3]));
  *reinterpret_cast<uint2 *>(p.c + row * p.ldc + col) = o;
}

__device__ __forceinline__ float scaled(int sum, float sa, float sw) {
  return (static_cast<float>(sum) * sa) * sw;
}

// ------------------------------------------------------------------------------ few rows

// A block owns 16 weight rows (8 gate and the same 8 up rows in the SwiGLU form) and all m <=
// 16 TT rows; wave w takes the chunks of 128 k w, w + kWaves, ... Both operands come straight
// into registers: lane (r16, g4) loads 16 bytes of row r16 at k 16 g4 and 64 + 16 g4 of a
// chunk, whole 128-byte lines per row.
template <int TT, int kWaves, bool kSwiglu>
__global__ __launch_bounds__(64 * kWaves) void few_kernel(GemmArgs p) {
  constexpr int kAhead = TT >= 4 ? 2 : 4;  // chunks in flight per wave
  constexpr int kOut = kSwiglu ? 8 : 16;   // output columns
  __shared__ __attribute__((aligned(16))) i32x4_t red[kWaves][TT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const int n0 = blockIdx.x * kOut;
  const uint32_t ldw = static_cast<uint32_t>(p.ldw), lda = static_cast<uint32_t>(p.lda);
  // n is a multiple of 16: the tile's columns all exist.
  const int wr = kSwiglu ? r16 & 7 : r16;
  const int8_t *w_base = p.w0 + static_cast<int64_t>(n0) * p.ldw;
  const int8_t *u_base = (kSwiglu ? p.w1 : p.w0) + static_cast<int64_t>(n0) * p.ldw;
  const int8_t *w_row = (kSwiglu && r16 >= 8 ? u_base : w_base) + static_cast<int64_t>(wr) * ldw;
  const __amdgpu_buffer_rsrc_t x_rsrc = make_rsrc(p.a, static_cast<uint32_t>(p.m) * lda);

  i32x4_t acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = i32x4_t{0, 0, 0, 0};
  const int chunks = (p.k + 127) / 128;
  for (int c0 = wave; c0 < chunks; c0 += kWaves * kAhead) {
    u32x4_t w[kAhead][2], x[kAhead][2][TT];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (c0 + u * kWaves) * 128 + 64 * h + 16 * g4;  // past K: zeros
        w[u][h] = u32x4_t{0u, 0u, 0u, 0u};
        if (k < p.k) w[u][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(w_row + k));
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint32_t off = static_cast<uint32_t>(16 * t + r16) * lda + static_cast<uint32_t>(k);
          x[u][h][t] = moe::load16(x_rsrc, k < p.k ? off : kNoLoad, 0);
        }
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = mma(w[u][h], x[u][h][t], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) red[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < TT; t += kWaves) {  // wave-uniform
    i32x4_t sum = red[0][t][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += red[w][t][lane];
    const int row = 16 * t + r16;
    const bool live = row < p.m;
    const float sa = live ? p.a_scale[row] : 0.0f;
    float y[4];
    if (kSwiglu) {
      const int col = n0 + 4 * (g4 & 1);
      float up[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float *s = g4 < 2 ? p.s0 : p.s1;
        y[x] = scaled(sum[x], sa, s[col + x]);
        up[x] = __shfl_xor(y[x], 32, 64);
        y[x] = moe::fp8_swiglu(y[x], up[x], p.limit);
      }
      if (live && g4 < 2) store4<true>(p, row, col, y);
    } else {
      const int col = n0 + 4 * g4;
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] = scaled(sum[x], sa, p.s0[col + x]);
      if (live) store4<false>(p, row, col, y);
    }
  }
}

// --------------------------------------------------------------------------------- tiles

// NT 16-row weight tiles and TT 16-row row tiles per wave, WN x WT waves over the tile, KS
// groups of waves that split the slices of a stage, ST stages.
template <int NT_, int TT_, int WN_, int WT_, int KS_, int ST_>
struct Cfg {
  static constexpr int NT = NT_, TT = TT_, WN = WN_, WT = WT_, KS = KS_, ST = ST_;
  static constexpr int BN = 16 * NT * WN, BT = 16 * TT * WT;
  static constexpr int kSliceWaves = WN * WT;
  static constexpr int kWaves = kSliceWaves * KS, kThreads = 64 * kWaves;
  static constexpr int kWBytes = BN * kRowBytes, kSlice = (BN + BT) * kRowBytes;
  static constexpr int kStage = KS * kSlice;
  static constexpr int kRedRow = BN + 4;  // words of a row of sums in the epilogue
  static constexpr int kRed = KS * BT * kRedRow * 4;
  static constexpr int kLds = ST * kStage > kRed ? ST * kStage : kRed;
  // 1 KB wave instructions (8 LDS rows) per wave and stage
  static constexpr int kWLoads = BN / 8 / kSliceWaves, kXLoads = BT / 8 / kSliceWaves;
  static constexpr int kLoads = kWLoads + kXLoads;
  static_assert(BN / 8 % kSliceWaves == 0 && BT / 8 % kSliceWaves == 0, "whole instructions");
  static_assert(kSliceWaves % 2 == 0, "a wave's weights lie in one half of a SwiGLU tile");
  static_assert(kLds <= 160 * 1024, "LDS");
  static constexpr int kMinWaves = kLds <= 80 * 1024 ? kWaves / 2 : (kWaves + 3) / 4;
};

// The tile of this block: XCD x takes a contiguous eighth of the tiles (workgroups go to the 8
// XCDs round-robin), kGroupM row tiles at a time with the row tile fastest, so that the tiles an
// XCD runs at once share weights and rows in its L2.
struct Tile {
  int m0, n0;
};

__device__ __forceinline__ Tile tile_of(uint32_t b, uint32_t m_tiles, uint32_t n_tiles, int bt,
                                        int bn) {
  const uint32_t total = m_tiles * n_tiles, xcd = b & 7;
  const uint32_t item = xcd * (total >> 3) + min(xcd, total & 7) + (b >> 3);
  const uint32_t g0 = item / (kGroupM * n_tiles) * kGroupM;
  const uint32_t g_rows = min(static_cast<uint32_t>(kGroupM), m_tiles - g0);
  const uint32_t in_grp = item - g0 * n_tiles;
  const uint32_t col = in_grp / g_rows;
  return {static_cast<int>(g0 + in_grp - col * g_rows) * bt, static_cast<int>(col) * bn};
}

// A wave-uniform pointer in scalar registers.
template <class T>
__device__ __forceinline__ const T *uniform(const T *ptr) {
  const uint64_t u = reinterpret_cast<uint64_t>(ptr);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
  return reinterpret_cast<const T *>(static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint8_t *dst, uint32_t voff,
                                           int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16,
                                           static_cast<int>(voff), soff, 0, 0);
}

template <class C, bool kSwiglu>
__global__ __launch_bounds__(C::kThreads, C::kMinWaves) void tile_kernel(GemmArgs p) {
  constexpr int NT = C::NT, TT = C::TT, WN = C::WN, KS = C::KS, ST = C::ST;
  constexpr int BN = C::BN, BT = C::BT;
  constexpr int kBnOut = kSwiglu ? BN / 2 : BN;  // output columns per tile
  static_assert(!kSwiglu || NT % 2 == 0, "gate and up tiles in pairs");
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slice = wave / C::kSliceWaves, sw = wave % C::kSliceWaves;
  const int wn = sw % WN, wt = sw / WN;
  const int r16 = lane & 15, g4 = lane >> 4;
  const Tile tile = tile_of(blockIdx.x, (p.m + BT - 1) / BT, (p.n + kBnOut - 1) / kBnOut, BT,
                            kBnOut);
  const int m0 = tile.m0, n0 = tile.n0;
  const int cnt = min(BT, p.m - m0), n_valid = min(kBnOut, p.n - n0);

  const int8_t *w_src = kSwiglu && 8 * sw * C::kWLoads >= kBnOut ? p.w1 : p.w0;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(uniform(w_src + static_cast<int64_t>(n0) * p.ldw),
                                              static_cast<uint32_t>(n_valid * p.ldw));
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(uniform(p.a + static_cast<int64_t>(m0) * p.lda),
                                              static_cast<uint32_t>(cnt * p.lda));
  // Instruction i fills 8 LDS rows, lane l the physical piece l % 8 of row l / 8, which holds the
  // logical piece (l % 8) ^ (l / 8): the operand reads below then hit every bank once. Rows past
  // the tile's valid ones lie past the buffer's end and read zeros.
  const int piece = (lane & 7) ^ (lane >> 3);
  uint32_t w_voff[C::kWLoads], x_voff[C::kXLoads];
#pragma unroll
  for (int i = 0; i < C::kWLoads; ++i) {
    const int r = 8 * (sw * C::kWLoads + i) + (lane >> 3);
    w_voff[i] = static_cast<uint32_t>(kSwiglu ? r % kBnOut : r) * static_cast<uint32_t>(p.ldw) +
                16u * piece;
  }
#pragma unroll
  for (int i = 0; i < C::kXLoads; ++i) {
    const int r = 8 * (sw * C::kXLoads + i) + (lane >> 3);
    x_voff[i] = static_cast<uint32_t>(r) * static_cast<uint32_t>(p.lda) + 16u * piece;
  }
  const auto load_stage = [&](int j, int stage_off) {
    uint8_t *st = lds + stage_off + slice * C::kSlice;
    const int k0 = (j * KS + slice) * kRowBytes;
    const int left = p.k - k0;
    const uint32_t dead = 16 * piece < left ? 0u : kNoLoad;  // past K: zeros
    const int soff = left > 0 ? k0 : 0;
#pragma unroll
    for (int i = 0; i < C::kWLoads; ++i)
      load_lds16(wr, st + 1024 * (sw * C::kWLoads + i), w_voff[i] | dead, soff);
#pragma unroll
    for (int i = 0; i < C::kXLoads; ++i)
      load_lds16(xr, st + C::kWBytes + 1024 * (sw * C::kXLoads + i), x_voff[i] | dead, soff);
  };
  const int steps = (p.k + KS * kRowBytes - 1) / (KS * kRowBytes);
#pragma unroll
  for (int j = 0; j < ST - 1; ++j) load_stage(j, j * C::kStage);

  // acc[i][t][x]: tile column w_row(i) + 4 g4 + x of tile row 16 (t WT + wt) + r16. A wave of
  // the SwiGLU form owns gate rows and the same up rows.
  i32x4_t acc[NT][TT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = i32x4_t{0, 0, 0, 0};
  const auto w_row = [&](int i) {
    if (kSwiglu) return (i < NT / 2 ? 0 : kBnOut) + (wn * (NT / 2) + i % (NT / 2)) * 16;
    return (wn * NT + i) * 16;
  };
  constexpr int kWaitN = C::kLoads * (ST - 2);
  static_assert(ST >= 2 && kWaitN < 64, "vmcnt holds 6 bits");
  constexpr int kWaitImm = (kWaitN & 15) | ((kWaitN >> 4) << 14) | (7 << 4) | (15 << 8);
  const int frag = r16 * kRowBytes + 16 * (g4 ^ (r16 & 7));
  int cur = 0, fill = (ST - 1) * C::kStage;
  for (int s = 0; s < steps; ++s) {
    __builtin_amdgcn_s_waitcnt(kWaitImm);  // this wave's loads of stage s are in LDS
    __builtin_amdgcn_s_barrier();           // every wave's; and stage s - 1 is read
    asm volatile("" ::: "memory");          // no read of the stage moves up
    load_stage(s + ST - 1, fill);           // into stage s - 1's buffer
    const uint8_t *st = lds + cur + slice * C::kSlice;
    const uint8_t *xs = st + C::kWBytes + wt * 16 * kRowBytes;
    cur = cur == (ST - 1) * C::kStage ? 0 : cur + C::kStage;
    fill = fill == (ST - 1) * C::kStage ? 0 : fill + C::kStage;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4_t w[NT], x[TT];
#pragma unroll
      for (int i = 0; i < NT; ++i)
        w[i] = *reinterpret_cast<const u32x4_t *>(st + w_row(i) * kRowBytes + (frag ^ (64 * h)));
#pragma unroll
      for (int t = 0; t < TT; ++t)
        x[t] = *reinterpret_cast<const u32x4_t *>(xs + t * C::WT * 16 * kRowBytes +
                                                  (frag ^ (64 * h)));
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i][t] = mma(w[i], x[t], acc[i][t]);
    }
  }
  // The past-the-end stages' loads write LDS (zeros) too: they finish first.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();  // every wave's operand reads are done: the stages are free

  // ---- epilogue: the slice groups' sums through LDS, then 4 columns per thread
  constexpr int kRow = C::kRedRow;
  int *red = reinterpret_cast<int *>(lds);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t)
      *reinterpret_cast<i32x4_t *>(red + (slice * BT + 16 * (t * C::WT + wt) + r16) * kRow +
                                   w_row(i) + 4 * g4) = acc[i][t];
  __syncthreads();
  for (int u = tid; u < BT * (kBnOut / 4); u += C::kThreads) {
    const int r = u / (kBnOut / 4), q = 4 * (u % (kBnOut / 4));
    if (r >= cnt || q >= n_valid) continue;
    const auto sums = [&](int col) {
      i32x4_t v = *reinterpret_cast<const i32x4_t *>(red + r * kRow + col);
#pragma unroll
      for (int z = 1; z < KS; ++z)
        v += *reinterpret_cast<const i32x4_t *>(red + (z * BT + r) * kRow + col);
      return v;
    };
    const float sa = p.a_scale[m0 + r];
    const i32x4_t v = sums(q);
    float y[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) y[x] = scaled(v[x], sa, p.s0[n0 + q + x]);
    if (kSwiglu) {
      const i32x4_t up = sums(kBnOut + q);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        y[x] = moe::fp8_swiglu(y[x], scaled(up[x], sa, p.s1[n0 + q + x]), p.limit);
    }
    store4<kSwiglu>(p, m0 + r, n0 + q, y);
  }
}

template <class C, bool kSwiglu>
int launch_tile(const char *name, const GemmArgs &p, void *stream) {
  constexpr int kBnOut = kSwiglu ? C::BN / 2 : C::BN;
  const int64_t tiles = static_cast<int64_t>((p.m + C::BT - 1) / C::BT) *
                        ((p.n + kBnOut - 1) / kBnOut);
  MOE_REQUIRE(tiles < (1ll << 32) / C::kThreads, "%s: matrix too large", name);
  constexpr auto kern = tile_kernel<C, kSwiglu>;
  if (C::kLds > 64 * 1024)
    MOE_REQUIRE_CODE(moe::allow_lds<kern>(C::kLds), MOE_ELAUNCH, "%s: %d bytes of LDS were refused", name,
                   C::kLds);
  return moe::launch(name, kern, dim3(static_cast<unsigned>(tiles)), dim3(C::kThreads), C::kLds,
                     stream, p);
}

template <int TT, int kWaves, bool kSwiglu>
int launch_few(const char *name, const GemmArgs &p, void *stream) {
  const unsigned blocks = static_cast<unsigned>(p.n / (kSwiglu ? 8 : 16));
  return moe::launch(name, few_kernel<TT, kWaves, kSwiglu>, dim3(blocks), dim3(64 * kWaves), 0,
                     stream, p);
}

template <bool kSwiglu>
int launch_gemm(const char *name, const GemmArgs &p, void *stream) {
  if (p.m <= 16) return launch_few<1, 8, kSwiglu>(name, p, stream);
  if (p.m <= 32) return launch_few<2, 8, kSwiglu>(name, p, stream);
  if (p.m <= 64) return launch_few<4, 8, kSwiglu>(name, p, stream);
  if (p.m <= 512) return launch_tile<Cfg<2, 2, 2, 2, 2, 3>, kSwiglu>(name, p, stream);
  return launch_tile<Cfg<4, 4, 2, 2, 1, 2>, kSwiglu>(name, p, stream);
}

int check_gemm(const char *name, const GemmArgs &p, bool swiglu) {
  MOE_REQUIRE(p.m >= 0 && p.n > 0 && p.n % 16 == 0 && p.k > 0 && p.k % 16 == 0 && p.k <= kMaxK,
              "%s: need m >= 0, n > 0 and k > 0 multiples of 16, k <= %d (m=%d n=%d k=%d)", name,
              kMaxK, p.m, p.n, p.k);
  MOE_REQUIRE(p.lda >= p.k && p.lda % 16 == 0 && p.ldw >= p.k && p.ldw % 16 == 0 &&
                  p.lda < (1 << 22) && p.ldw < (1 << 22),
              "%s: leading dimensions must be >= k, multiples of 16 and below 2^22", name);
  MOE_REQUIRE(p.ldc >= p.n && p.ldc % 4 == 0, "%s: ldc must be >= n and a multiple of 4", name);
  if (p.m == 0) return MOE_OK;
  MOE_REQUIRE(p.a && p.a_scale && p.w0 && p.s0 && p.c && (!swiglu || (p.w1 && p.s1)),
              "%s: a required pointer is NULL", name);
  MOE_REQUIRE(moe::aligned16(p.a) && moe::aligned16(p.w0) && moe::aligned16(p.w1),
              "%s: rows and weights must be 16-byte aligned", name);
  MOE_REQUIRE((reinterpret_cast<uintptr_t>(p.c) & 7u) == 0, "%s: the output must be 8-byte aligned",
              name);
  MOE_REQUIRE(((reinterpret_cast<uintptr_t>(p.a_scale) | reinterpret_cast<uintptr_t>(p.s0) |
                reinterpret_cast<uintptr_t>(p.s1)) & 3u) == 0,
              "%s: scales must be 4-byte aligned", name);
  return MOE_OK;
}

}  // namespace

extern "C" int moe_dense_gemm_int8(const int8_t *a, int64_t lda, const float *a_scale,
                                   const int8_t *b, int64_t ldb, const float *b_scale,
                                   uint16_t *c, int64_t ldc, int32_t m, int32_t n, int32_t k,
                                   void *stream) {
  moe::clear_error();
  const GemmArgs p = {a, a_scale, b, nullptr, b_scale, nullptr, c, nullptr, lda, ldb, ldc, m, n, k, 0.0f};
  const int rc = check_gemm("dense_gemm_int8", p, false);
  if (rc != MOE_OK || m == 0) return rc;
  return launch_gemm<false>("moe_dense_gemm_int8", p, stream);
}

extern "C" int moe_dense_gate_up_swiglu_int8(const int8_t *a, int64_t lda, const float *a_scale,
                                             const int8_t *gate_w, const float *gate_scale,
                                             const int8_t *up_w, const float *up_scale,
                                             int64_t ldw, uint16_t *act, int64_t ld_act, int32_t m,
                                             int32_t inter, int32_t k, float limit, void *stream) {
  moe::clear_error();
  const GemmArgs p = {a,       a_scale, gate_w, up_w,   gate_scale, up_scale, act, nullptr,
                      lda,     ldw,     ld_act, m,      inter,      k,        limit};
  MOE_REQUIRE(limit > 0.0f, "dense_gate_up_swiglu_int8: limit must be > 0");
  const int rc = check_gemm("dense_gate_up_swiglu_int8", p, true);
  if (rc != MOE_OK || m == 0) return rc;
  return launch_gemm<true>("moe_dense_gate_up_swiglu_int8", p, stream);
}

namespace {

// The shared expert's workspace: FP32 activations, their codes, their scales.
struct Layout {
  int64_t codes, scales, bytes;
};

Layout layout_of(int64_t m, int64_t inter) {
  const auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  Layout l;
  l.codes = up(m * inter * 4);
  l.scales = l.codes + up(m * inter);
  l.bytes = l.scales + up(m * 4);
  return l;
}

}  // namespace

extern "C" int64_t moe_shared_expert_int8_workspace_bytes(int32_t m, int32_t inter) {
  return m <= 0 || inter <= 0 ? 0 : layout_of(m, inter).bytes;
}

extern "C" int moe_shared_expert_int8(const int8_t *a, int64_t lda, const float *a_scale,
                                      const int8_t *gate_w, const float *gate_scale,
                                      const int8_t *up_w, const float *up_scale, int64_t ldw,
                                      const int8_t *down_w, int64_t ld_down,
                                      const float *down_scale, uint16_t *out, int64_t ld_out,
                                      int32_t m, int32_t inter, int32_t hidden, float limit,
                                      void *workspace, int64_t workspace_bytes, void *stream) {
  moe::clear_error();
  constexpr const char *name = "shared_expert_int8";
  MOE_REQUIRE(limit > 0.0f, "%s: limit must be > 0", name);
  MOE_REQUIRE(m < (1 << 22), "%s: at most 2^22 - 1 rows (got %d)", name, m);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const Layout l = layout_of(m < 0 ? 0 : m, inter < 0 ? 0 : inter);
  int8_t *codes = reinterpret_cast<int8_t *>(ws + l.codes);
  float *act = reinterpret_cast<float *>(ws), *scales = reinterpret_cast<float *>(ws + l.scales);
  // `out` stands for the FP32 activations' place in the checks.
  const GemmArgs gu = {a, a_scale, gate_w, up_w, gate_scale, up_scale, out, act, lda, ldw, inter, m,
                       inter, hidden, limit};
  const GemmArgs dn = {codes, scales, down_w, nullptr, down_scale, nullptr, out, nullptr, inter,
                       ld_down, ld_out, m, hidden, inter, 0.0f};
  int rc = check_gemm(name, gu, true);
  if (rc == MOE_OK) rc = check_gemm(name, dn, false);
  if (rc != MOE_OK || m == 0) return rc;
  MOE_REQUIRE(workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0,
              "%s: the workspace must be non-NULL and 256-byte aligned", name);
  MOE_REQUIRE_CODE(workspace_bytes >= l.bytes, MOE_ECAPACITY,
                   "%s: the workspace has %lld bytes, %lld are needed", name,
                   static_cast<long long>(workspace_bytes), static_cast<long long>(l.bytes));
  rc = launch_gemm<true>("moe_shared_expert_int8", gu, stream);
  if (rc == MOE_OK) rc = moe::quant_int8_f32(name, act, codes, scales, m, inter, stream);
  if (rc == MOE_OK) rc = launch_gemm<false>("moe_shared_expert_int8", dn, stream);
  return rc;
}
