// moe_dense_gemm_int8 and moe_dense_gate_up_swiglu_int8: INT8 rows with one FP32 scale per row
// (token), times INT8 weights with one FP32 scale per output channel.
//
//   S[m, n] = sum_k a[m, k] * w[n, k]               exact in int32 (K <= MOE_INT8_MAX_K)
//   y[m, n] = (float(S) * sa[m]) * sw[n]            FP32, in this order
//   c[m, n] = bf16(y), or bf16(silu(min(G, L)) * clamp(U, -L, L)) of the gate's and up's y
//
// Because the sums are exact, every tile, split and order of K gives the same bits.
//
// Two kernels (which one and which tile: int8_plan.h):
//   - tile_kernel, up to 128 x 128: stages of 128 k (KS of them side by side, multiplied by as
//     many groups of waves) loaded straight into LDS, ST - 1 ahead;
//   - wide_kernel, 256 rows: persistent blocks in which half of the waves reads while the other
//     half multiplies.
// Weights are the matrix instruction's operand A and rows its operand B: a lane holds 4
// consecutive outputs of one row.
//
// What bounds it (256 CUs):
//   - One row to some dozens: the weights from memory, the start of a block and of a launch: 6144 x
//     2048 in 3.4 us of kernel (1 to 16 rows, weights in the last-level cache; 5.0 from memory).
//   - Hundreds: what a CU takes in from its L2 (36 bytes a clock), each block all of K: 256 rows in
//     8.1 to 9.0 us. (K in parts on several blocks is not built.)
//   - Thousands: power. At 4096 x 6144 x 2048 the chip runs at 1.45 to 1.7 GHz of its 2.4; a step of
//     the 192 x 256 tile takes 1980 clocks of which 1536 are products. 52 to 63 us by the codes
//     (small ones toggle fewer bits) and by what the chip ran before, 1640 to 1980 TOPS; 8192^3 in
//     419 to 441 us, 2490 to 2630.
#include <algorithm>

#include "buffer_io.h"
#include "common.h"
#include "int8.h"
#include "int8_plan.h"
#include "lds_limit.h"
#include "nvfp4_decode.h"  // moe::pack_bf16x2

namespace {

using moe::kNoLoad;
using moe::make_rsrc;
using moe::u32x4_t;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kRowBytes = 128;  // one LDS row: 128 k
constexpr int kMaxK = MOE_INT8_MAX_K;
// Rows and output columns: rounded up to whole tiles (256 at most) they stay within 32 bits.
constexpr int kMaxOut = 0x7FFFFFFF - 255;
constexpr int kGroupM = 4;  // row tiles that run next to each other
constexpr int kCus = 256;

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

// silu(min(g, L)) * clamp(u, -L, L), NaN kept by the IEEE minimum and maximum, in 15 operations (the
// large tiles' epilogues are bound by them: 28 took 91 us where these take 87 at 4096 rows, width
// 2048, K 6144). The rounding of the exponential's argument moves the result by |g| 2^-24 of
// itself; below g = -126 ln 2 = -87.34 the reciprocal leaves the normal numbers and the result is 0
// (|silu| is below 1.03e-36 there).
__device__ __forceinline__ float swiglu(float g, float u, float limit) {
  const float gc = __builtin_elementwise_minimum(g, limit);
  const float uc = __builtin_elementwise_maximum(__builtin_elementwise_minimum(u, limit), -limit);
  const float e = __builtin_amdgcn_exp2f(gc * -1.44269504f);  // log2(e)
  return gc * __builtin_amdgcn_rcpf(1.0f + e) * uc;
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
        y[x] = swiglu(y[x], scaled(up[x], sa, p.s1[n0 + q + x]), p.limit);
    }
    store4<kSwiglu>(p, m0 + r, n0 + q, y);
  }
}

// ---------------------------------------------------------------------------- large tiles

typedef int i32x16_t __attribute__((ext_vector_type(16)));

// NT 32-row weight tiles and TT 32-row row tiles per wave, WN x WT = 8 waves, two stages of 128 k.
template <int NT_, int TT_, int WN_, int WT_>
struct WideCfg {
  static constexpr int NT = NT_, TT = TT_, WN = WN_, WT = WT_;
  static constexpr int BN = 32 * NT * WN, BT = 32 * TT * WT;
  static constexpr int kWaves = WN * WT, kThreads = 64 * kWaves;
  static constexpr int kWBytes = BN * kRowBytes, kStage = (BN + BT) * kRowBytes;
  static constexpr int kOutBytes = 32 * 64 * NT;  // a wave's 32 rows of 32 NT BF16 outputs
  static constexpr int kLds = 2 * kStage + kWaves * kOutBytes;
  static constexpr int kWLoads = BN / 8 / kWaves, kXLoads = BT / 8 / kWaves;
  static constexpr int kLoads = kWLoads + kXLoads;
  static_assert(kWaves == 8, "two waves per SIMD, one of each group");
  static_assert(BN / 8 % kWaves == 0 && BT / 8 % kWaves == 0, "whole instructions");
  static_assert(kLds <= 160 * 1024, "LDS");
};

__device__ __forceinline__ i32x16_t mma_wide(u32x4_t w, u32x4_t x, i32x16_t d) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, w),
                                               __builtin_bit_cast(i32x4_t, x), d, 0, 0, 0);
}

// Persistent blocks, one per CU. Two phases per step of 128 k and wave: read the step's operands
// from LDS, then multiply. Waves 0-3 and 4-7 (one of each on every SIMD) run them in opposite
// order, the second group one barrier behind, so that a SIMD's matrix core is fed by one wave
// while the other reads. In slots between barriers, step s is read in slot 2 s by the first group
// and in 2 s + 1 by the second, and multiplied in the slot after. The buffer of stage s - 1 is
// free from slot 2 s on: there both groups issue their loads of stage s + 1 (the first beside its
// reads, the second between its products), and both have waited for them when slot 2 s + 1
// ends. Steps are counted through all of a block's tiles, so a tile's first stages are loaded
// during the last steps of the one before; a finished tile's outputs take one more slot of each
// group, and their stores are waited for behind the next tile's first loads.
template <class C, bool kSwiglu>
__global__ __launch_bounds__(C::kThreads, 2) void wide_kernel(GemmArgs p) {
  constexpr int NT = C::NT, TT = C::TT, WN = C::WN, WT = C::WT, BN = C::BN, BT = C::BT;
  constexpr int kBnOut = kSwiglu ? BN / 2 : BN;
  static_assert(!kSwiglu || NT == 2, "a gate tile and its up tile per wave");
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wt = wave / WN, group = wave / 4;
  const int rl = lane & 31, gl = lane >> 5;
  const uint32_t m_tiles = (p.m + BT - 1) / BT, n_tiles = (p.n + kBnOut - 1) / kBnOut;
  const uint32_t total = m_tiles * n_tiles;
  const int steps = (p.k + kRowBytes - 1) / kRowBytes;
  const int8_t *w_src = kSwiglu && 8 * wave * C::kWLoads >= kBnOut ? p.w1 : p.w0;

  // Instruction i fills the 8 LDS rows from 8 i on; row r holds its logical piece c at c ^ (r / 2 %
  // 8): the 32-row operand reads below then hit every bank once. So lane l loads piece (l % 8) ^
  // (l / 16) of row l / 8, or that ^ 4 where i is odd.
  const uint32_t w_lane = static_cast<uint32_t>(lane >> 3) * static_cast<uint32_t>(p.ldw);
  const uint32_t x_lane = static_cast<uint32_t>(lane >> 3) * static_cast<uint32_t>(p.lda);
  const uint32_t piece16 = 16u * ((lane & 7) ^ (lane >> 4));
  // What is loaded next: a step of a tile, and the stage buffer it goes to. Past the last tile
  // the buffers have no bytes.
  struct Next {
    uint32_t item;
    int step, buf;
    __amdgpu_buffer_rsrc_t w, x;
  };
  Next next;
  const auto aim = [&]() __attribute__((always_inline)) {
    const bool in = next.item < total;
    const Tile t = tile_of(in ? next.item : 0, m_tiles, n_tiles, BT, kBnOut);
    const int cnt = min(BT, p.m - t.m0), n_valid = min(kBnOut, p.n - t.n0);
    next.w = make_rsrc(uniform(w_src + static_cast<int64_t>(t.n0) * p.ldw),
                       in ? static_cast<uint32_t>(n_valid * p.ldw) : 0u);
    next.x = make_rsrc(uniform(p.a + static_cast<int64_t>(t.m0) * p.lda),
                       in ? static_cast<uint32_t>(cnt * p.lda) : 0u);
  };
  const auto load = [&](int n) __attribute__((always_inline)) {
    uint8_t *st = lds + next.buf;
    const int k0 = next.step * kRowBytes;
    const bool is_w = n < C::kWLoads;
    const int inst = is_w ? wave * C::kWLoads + n : wave * C::kXLoads + n - C::kWLoads;
    const uint32_t at = piece16 ^ (64u * (inst & 1));
    const uint32_t dead = static_cast<int>(at) < p.k - k0 ? 0u : kNoLoad;  // past K: zeros
    if (is_w) {
      const int row = kSwiglu ? 8 * inst % kBnOut : 8 * inst;
      load_lds16(next.w, st + 1024 * inst,
                 (w_lane + static_cast<uint32_t>(row) * static_cast<uint32_t>(p.ldw) + at) | dead, k0);
    } else {
      load_lds16(next.x, st + C::kWBytes + 1024 * inst,
                 (x_lane + static_cast<uint32_t>(8 * inst) * static_cast<uint32_t>(p.lda) + at) | dead,
                 k0);
    }
  };
  const auto advance = [&]() __attribute__((always_inline)) {
    next.buf ^= C::kStage;
    if (++next.step == steps) {  // uniform
      next.step = 0;
      next.item += gridDim.x;
      aim();
    }
  };
  next.item = blockIdx.x;
  next.step = next.buf = 0;
  aim();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int n = 0; n < C::kLoads; ++n) load(n);
    advance();
  }

  // acc[i][t][4 g + x]: tile column w_row(i) + 8 g + 4 gl + x of tile row 32 (t WT + wt) + rl.
  const auto w_row = [&](int i) {
    return kSwiglu ? i * kBnOut + wn * 32 : (wn * NT + i) * 32;
  };
  int frag[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) frag[j] = rl * kRowBytes + 16 * ((2 * j + gl) ^ ((rl >> 1) & 7));
  constexpr int kStageWait = (C::kLoads & 15) | ((C::kLoads >> 4) << 14) | (7 << 4) | (15 << 8);
  constexpr int kLoadsDone = (7 << 4) | (15 << 8);        // vmcnt(0)
  constexpr int kReadsDone = 15 | (3 << 14) | (7 << 4);    // lgkmcnt(0)
  __builtin_amdgcn_s_waitcnt(kStageWait);  // stage 0
  __builtin_amdgcn_s_barrier();
  if (group == 1) __builtin_amdgcn_s_barrier();
  int buf = 0;
  bool started = false;  // the first two stages are loaded above
  for (uint32_t item = blockIdx.x; item < total; item += gridDim.x) {
    i32x16_t acc[NT][TT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[i][t] = i32x16_t{};
    for (int s = 0; s < steps; ++s) {
      // Read (slot 2 s + group).
      if (group == 0 && started) {
#pragma unroll
        for (int n = 0; n < C::kLoads; ++n) load(n);
        advance();
      }
      started = true;
      const uint8_t *ws = lds + buf;
      const uint8_t *xs = ws + C::kWBytes + wt * 32 * kRowBytes;
      buf ^= C::kStage;
      u32x4_t w[NT][4], x[TT][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
          w[i][j] = *reinterpret_cast<const u32x4_t *>(ws + w_row(i) * kRowBytes + frag[j]);
#pragma unroll
        for (int t = 0; t < TT; ++t)
          x[t][j] = *reinterpret_cast<const u32x4_t *>(xs + t * WT * 32 * kRowBytes + frag[j]);
      }
      __builtin_amdgcn_s_waitcnt(kReadsDone);
      if (group == 1) __builtin_amdgcn_s_waitcnt(kLoadsDone);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      // Multiply (slot 2 s + 1 + group).
      __builtin_amdgcn_s_setprio(1);  // before the reading wave of the SIMD: 1 to 2 %
      constexpr int kProducts = 4 * NT * TT;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            acc[i][t] = mma_wide(w[i][j], x[t][j], acc[i][t]);
            if (group == 1) {  // a load behind every few products
              const int q = (j * TT + t) * NT + i;
              if ((q + 1) * C::kLoads / kProducts > q * C::kLoads / kProducts)
                load(q * C::kLoads / kProducts);
            }
          }
      __builtin_amdgcn_s_setprio(0);
      if (group == 1) advance();
      if (group == 0) __builtin_amdgcn_s_waitcnt(kLoadsDone);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }

    // The tile's outputs, 32 rows at a time through the wave's own piece of LDS, so that rows
    // leave in whole 64- to 192-byte pieces. Its 16-byte pieces are permuted within a row so that
    // neither side meets a bank more often than it must. FP32 outputs (the shared expert's
    // activations) go straight from the lanes, 16 bytes each: 109 us where BF16 ones take 105 in the
    // same trace at 4096 rows, width 2048, K 6144.
    constexpr int kCols = kSwiglu ? 32 : 32 * NT;  // the wave's output columns
    constexpr int kOutRow = 2 * kCols, kLanes = kCols / 8;
    const auto place = [](int r, int piece) {
      return r * kOutRow + 16 * (piece ^ (kLanes == 8 ? r & 7 : (r >> 1) & 3));
    };
    const Tile tile = tile_of(item, m_tiles, n_tiles, BT, kBnOut);
    const int cnt = min(BT, p.m - tile.m0);
    uint8_t *mine = lds + 2 * C::kStage + wave * C::kOutBytes;
    const int col0 = tile.n0 + wn * kCols;
    // Every scale at once: a load per value would be waited for one after the other.
    f32x4_t sw[NT][4];
    float sa[TT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float *src = kSwiglu && i == 1 ? p.s1 : p.s0;
        const int c = col0 + (kSwiglu ? 0 : 32 * i) + 8 * g + 4 * gl;
        __builtin_memcpy(&sw[i][g], src + min(c, p.n - 4), 16);  // 4-byte aligned
      }
#pragma unroll
    for (int t = 0; t < TT; ++t)
      sa[t] = p.a_scale[tile.m0 + min(32 * (t * WT + wt) + rl, cnt - 1)];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int r0 = 32 * (t * WT + wt);
#pragma unroll
      for (int i = 0; i < (kSwiglu ? 1 : NT); ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = 32 * i + 8 * g + 4 * gl;  // of the wave's columns
          float y[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            y[q] = scaled(acc[i][t][4 * g + q], sa[t], sw[i][g][q]);
            if constexpr (kSwiglu)
              y[q] = swiglu(y[q], scaled(acc[1][t][4 * g + q], sa[t], sw[1][g][q]),
                                     p.limit);
          }
          if (kSwiglu && p.c32 != nullptr) {
            if (col0 + c < p.n && r0 + rl < cnt)
              store4<true>(p, tile.m0 + r0 + rl, col0 + c, y);
          } else {
            *reinterpret_cast<uint2 *>(mine + place(rl, 4 * i + g) + 8 * gl) =
                make_uint2(moe::pack_bf16x2(y[0], y[1]), moe::pack_bf16x2(y[2], y[3]));
          }
        }
      if (kSwiglu && p.c32 != nullptr) continue;
#pragma unroll
      for (int u = 0; u < 32 * kLanes; u += 64) {
        const int r = (u + lane) / kLanes, piece = (u + lane) % kLanes, c = 8 * piece;
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>(mine + place(r, piece));
        if (r0 + r < cnt && col0 + c < p.n) {  // n is a multiple of 16
          uint16_t *dst = p.c + static_cast<int64_t>(tile.m0 + r0 + r) * p.ldc + col0 + c;
          // ldc may be any multiple of 4 (one 16-byte store where it can be was no faster)
          reinterpret_cast<uint2 *>(dst)[0] = make_uint2(v[0], v[1]);
          reinterpret_cast<uint2 *>(dst)[1] = make_uint2(v[2], v[3]);
        }
      }
    }
    __builtin_amdgcn_s_barrier();  // the slot of the outputs
    asm volatile("" ::: "memory");
  }
  if (group == 0) __builtin_amdgcn_s_barrier();
  // The past-the-end stages' loads write LDS (zeros) too: they finish first.
  __builtin_amdgcn_s_waitcnt(0);
}

template <class C, bool kSwiglu>
int launch_tile(const char *name, const GemmArgs &p, void *stream) {
  constexpr int kBnOut = kSwiglu ? C::BN / 2 : C::BN;
  const int64_t tiles = static_cast<int64_t>((p.m + C::BT - 1) / C::BT) *
                        ((p.n + kBnOut - 1) / kBnOut);
  MOE_REQUIRE(tiles < (1ll << 32) / C::kThreads, "%s: matrix too large", name);
  constexpr auto kern = tile_kernel<C, kSwiglu>;
  if (C::kLds > 64 * 1024)
    MOE_REQUIRE_CODE(moe::allow_lds<kern>(C::kLds), MOE_ELAUNCH,
                     "%s: %d bytes of LDS were refused", name,
                   C::kLds);
  return moe::launch(name, kern, dim3(static_cast<unsigned>(tiles)), dim3(C::kThreads), C::kLds,
                     stream, p);
}

template <class C, bool kSwiglu>
int launch_wide(const char *name, const GemmArgs &p, void *stream) {
  constexpr int kBnOut = kSwiglu ? C::BN / 2 : C::BN;
  const int64_t tiles = static_cast<int64_t>((p.m + C::BT - 1) / C::BT) *
                        ((p.n + kBnOut - 1) / kBnOut);
  MOE_REQUIRE(tiles < (1ll << 31), "%s: matrix too large", name);
  constexpr auto kern = wide_kernel<C, kSwiglu>;
  MOE_REQUIRE_CODE(moe::allow_lds<kern>(C::kLds), MOE_ELAUNCH, "%s: %d bytes of LDS were refused",
                   name, C::kLds);
  return moe::launch(name, kern, dim3(static_cast<unsigned>(std::min<int64_t>(tiles, kCus))),
                     dim3(C::kThreads), C::kLds, stream, p);
}

template <bool kSwiglu>
int launch_gemm(const char *name, const GemmArgs &p, void *stream) {
  const moe::Int8Tile tile = moe::int8_tile(kSwiglu, p.m, p.n, p.k);
  if constexpr (kSwiglu) {
    if (tile == moe::kInt8Tile128x128Pair)
      return launch_tile<Cfg<4, 4, 2, 2, 1, 2>, true>(name, p, stream);
  } else {
    if (tile == moe::kInt8Tile32x16)
      return launch_tile<Cfg<1, 1, 2, 1, 4, 3>, false>(name, p, stream);
    if (tile == moe::kInt8Tile128x256)
      return launch_wide<WideCfg<2, 2, 2, 4>, false>(name, p, stream);
    if (tile == moe::kInt8Tile192x256)
      return launch_wide<WideCfg<3, 2, 2, 4>, false>(name, p, stream);
  }
  switch (tile) {
    case moe::kInt8Tile32x32: return launch_tile<Cfg<2, 1, 1, 2, 4, 3>, kSwiglu>(name, p, stream);
    case moe::kInt8Tile64x32: return launch_tile<Cfg<2, 1, 2, 2, 2, 4>, kSwiglu>(name, p, stream);
    case moe::kInt8Tile64x64: return launch_tile<Cfg<2, 2, 2, 2, 2, 3>, kSwiglu>(name, p, stream);
    case moe::kInt8Tile128x64: return launch_tile<Cfg<4, 2, 2, 2, 2, 3>, kSwiglu>(name, p, stream);
    case moe::kInt8Tile128x128:
      return launch_tile<Cfg<4, 4, 2, 2, 2, 2>, kSwiglu>(name, p, stream);
    default: return launch_wide<WideCfg<2, 4, 4, 2>, kSwiglu>(name, p, stream);
  }
}

int check_gemm(const char *name, const GemmArgs &p, bool swiglu) {
  MOE_REQUIRE(p.m >= 0 && p.n > 0 && p.n % 16 == 0 && p.k > 0 && p.k % 16 == 0 && p.k <= kMaxK,
              "%s: need m >= 0, n > 0 and k > 0 multiples of 16, k <= %d (m=%d n=%d k=%d)", name,
              kMaxK, p.m, p.n, p.k);
  MOE_REQUIRE(p.m <= kMaxOut && p.n <= kMaxOut, "%s: at most %d rows and columns (m=%d n=%d)", name,
              kMaxOut, p.m, p.n);
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
  const GemmArgs p = {a,   a_scale, b,   nullptr, b_scale, nullptr, c,   nullptr,
                      lda, ldb,     ldc, m,       n,       k,       0.0f};
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
