// The FP8 (W8A8) GEMMs: E4M3 rows with one FP32 scale per 128 k, times E4M3 weights with one
// FP32 scale per 128 x 128 block.
//
//   y[s, n] = sum_b sa[s, b] * sw[n / 128, b] * (sum_{k in block b} a[s, k] * w[n, k])
//
//   moe_dense_gemm_fp8, moe_dense_gate_up_swiglu_fp8    the shared expert's products
//   moe_w8a8_grouped_gemm, moe_w8a8_grouped_gemm_swiglu one launch over all experts
//
// One kernel template computes all four. The mathematics fixes its inner step: a block of
// 128 k is exactly one v_mfma_f32_16x16x128_f8f6f4 (or four BF16 ones, below), whose FP32
// result is multiplied by the block's two scales and added to the FP32 accumulator (4 FMAs
// per lane and block product, issued under the next one). Weights are the MFMA's A operand and rows its B operand: a lane then
// holds 4 consecutive outputs of ONE row, so its scale product is one number per 16-row tile
// and weight block.
//
// Structure:
//   - A block owns BN weight rows x BT rows over the whole K, in stages of KS slices of 128 k
//     loaded straight into LDS (buffer_load ... lds), kStages - 1 stages ahead. LDS rows are
//     128 bytes, 16-byte piece c of row r at c ^ (r & 7): the operand reads are conflict-free.
//   - Waves: WN x WT over the tile, and KS groups that split the slices of a stage (the small
//     tiles, whose sums are then joined in slice order).
//   - Rows past the tile's valid ones, gather indices out of range and k past the end read
//     zeros through their offset (past the buffer's end), without memory traffic.
//   - Grouped form: blocks are persistent. Each counts the experts' row tiles from the
//     offsets once (a prefix sum kept in LDS) and takes every gridDim-th (tile, weight tile)
//     item: only experts with rows cost anything, however the rows are routed.
//   - SwiGLU form: the tile's weight rows are 128 gate rows and the same 128 up rows, a wave
//     holding both sums of an output; one block so owns whole 128-column groups of the
//     output and quantises them in its epilogue. Nothing is rounded between the FP32 sums and
//     the codes.
#include <mutex>
#include <type_traits>

#include "buffer_io.h"
#include "common.h"
#include "fp8.h"
#include "nvfp4_decode.h"  // moe::pack_bf16x2
#include "swiglu.h"

namespace {

using moe::kFp8Block;
using moe::kNoLoad;
using moe::make_rsrc;
using moe::u32x4_t;

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kRowBytes = kFp8Block;  // one LDS row: 128 k
constexpr int kMaxK = MOE_FP8_MAX_K;  // the weight scales of a tile's K sit in LDS
constexpr int kMaxExperts = MOE_ALIGN_MAX_EXPERTS;

struct GemmArgs {
  const uint8_t *a;         // [a_rows, lda] codes
  int64_t lda;
  const float *a_scale;     // [a_rows, ld_as]
  int64_t ld_as;
  const int32_t *gather;    // row of each sorted slot, or NULL
  int32_t a_rows;
  const uint8_t *w0, *w1;   // dense: the weight, or gate and up
  int64_t ldw;
  const float *ws0, *ws1;   // dense: their block scales
  const uint64_t *w_ptrs, *s_ptrs;  // grouped: per-expert weights and scales
  const int32_t *offsets;
  int32_t num_experts;
  uint16_t *c;              // plain output
  uint8_t *q;               // SwiGLU output codes ...
  float *q_scale;           // ... and scales
  int64_t ldc, ld_qs;
  int32_t rows;             // dense: m; grouped: max_rows
  int32_t n;                // output columns
  int32_t k;
  float limit;
};

// Compile-time shape of a kernel: NT 16-row weight tiles and TT 16-row row tiles per wave,
// WN x WT waves over the tile, KS slice groups, ST stages.
template <int NT_, int TT_, int WN_, int WT_, int KS_, int ST_>
struct Cfg {
  static constexpr int NT = NT_, TT = TT_, WN = WN_, WT = WT_, KS = KS_, ST = ST_;
  static constexpr int BN = 16 * NT * WN, BT = 16 * TT * WT;
  static constexpr int kSliceWaves = WN * WT;
  static constexpr int kWaves = kSliceWaves * KS, kThreads = 64 * kWaves;
  static constexpr int kScaleFloats = BT > 64 ? BT : 64;
  static constexpr int kWBytes = BN * kRowBytes, kXBytes = BT * kRowBytes;
  static constexpr int kSlice = kWBytes + kXBytes + 4 * kScaleFloats;
  static constexpr int kStage = KS * kSlice;
  // 1 KB wave instructions per wave and stage
  static constexpr int kWLoads = BN / 8 / kSliceWaves;
  static constexpr int kXInstr = BT / 8;
  static constexpr int kXLoads = kXInstr > kSliceWaves ? kXInstr / kSliceWaves : 1;
  static constexpr int kLoads = kWLoads + kXLoads + 1;
  static constexpr int kNBlocks = BN > kFp8Block ? BN / kFp8Block : 1;  // weight scale rows
  static_assert(BN / 8 % kSliceWaves == 0, "whole weight instructions per wave");
  static_assert(kXInstr % kSliceWaves == 0 || kXInstr < kSliceWaves, "row instructions");
  static_assert(kSliceWaves * 64 >= BT, "one scale instruction per wave covers the tile");
  static_assert(BN % kFp8Block == 0 || kFp8Block % BN == 0, "scale blocks");
  // LDS: stages, a dump for loads that must not land anywhere, weight scales, tile prefix
  static constexpr int kDumpOff = ST * kStage;
  static constexpr int kSbOff = kDumpOff + 1024;
};

// One lane's 32 codes of an operand tile (128 k of a row, 4 lanes per row).
struct Codes {
  u32x4_t lo, hi;
};

__device__ __forceinline__ Codes read_codes(const uint8_t *tile, int frag) {
  return {*reinterpret_cast<const u32x4_t *>(tile + frag),
          *reinterpret_cast<const u32x4_t *>(tile + (frag ^ 64))};
}

// The operand of a 16 x 16 x 128 block product. Both operands hold k in the same order, so
// which k a lane's codes are does not matter.
//
// Fp8Mma multiplies the codes as they are. The FP8 matrix cores align the products of 8
// neighbouring k (8 bytes of a lane) to the largest and cut each below 2^-13 of it before
// adding them: measured error of a block 1.5e-5 of its size (N(0, 1) operands), 1/130 of the
// rounding of a BF16 output and so invisible in it.
struct Fp8Mma {
  typedef i32x8_t Operand;
  static __device__ __forceinline__ Operand operand(const Codes &c) {
    return __builtin_bit_cast(
        i32x8_t, __builtin_shufflevector(c.lo, c.hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  static __device__ __forceinline__ f32x4_t product(const Operand &w, const Operand &x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0,
                                                            0, 0, 0, 0, 0);
  }
};

// Bf16Mma converts them to BF16 first (exact) and takes the BF16 matrix cores, which add in
// FP32 without that loss, at half the rate: for outputs that are FP32 themselves (the SwiGLU
// form's scales).
struct Bf16Mma {
  struct Operand {
    bf16x8_t part[4];
  };
  static __device__ __forceinline__ bf16x8_t eight(uint32_t a, uint32_t b) {
    const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return bf16x8_t{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  }
  static __device__ __forceinline__ Operand operand(const Codes &c) {
    return {{eight(c.lo[0], c.lo[1]), eight(c.lo[2], c.lo[3]), eight(c.hi[0], c.hi[1]),
             eight(c.hi[2], c.hi[3])}};
  }
  static __device__ __forceinline__ f32x4_t product(const Operand &w, const Operand &x) {
    f32x4_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.part[j], x.part[j], d, 0, 0, 0);
    return d;
  }
};

template <class C, bool kGrouped>
int lds_bytes(const GemmArgs &p) {
  const int kb = (p.k + kFp8Block - 1) / kFp8Block;
  const int kb_pad = (kb + C::KS - 1) / C::KS * C::KS;
  return C::kSbOff + 4 * C::kNBlocks * kb_pad + (kGrouped ? 4 * (p.num_experts + 1) : 0);
}

template <class C, bool kSwiglu, bool kGrouped>
__global__ __launch_bounds__(C::kThreads) void fp8_gemm_kernel(const GemmArgs p) {
  static_assert(!kSwiglu || (C::BN == 2 * kFp8Block && C::KS == 1 && C::NT % 2 == 0),
                "the SwiGLU form owns whole output groups");
  constexpr int NT = C::NT, TT = C::TT, WN = C::WN, KS = C::KS, ST = C::ST;
  constexpr int BN = C::BN, BT = C::BT;
  constexpr int kBnOut = kSwiglu ? BN / 2 : BN;  // output columns per tile
  using Mma = std::conditional_t<kSwiglu, Bf16Mma, Fp8Mma>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slice = wave / C::kSliceWaves, sw = wave % C::kSliceWaves;
  const int wn = sw % WN, wt = sw / WN;
  const int r16 = lane & 15, g4 = lane >> 4;

  const int kb_n = (p.k + kFp8Block - 1) / kFp8Block;
  const int steps = (kb_n + KS - 1) / KS;
  float *sb = reinterpret_cast<float *>(lds + C::kSbOff);  // [kNBlocks][steps * KS]
  int *prefix = reinterpret_cast<int *>(sb + C::kNBlocks * steps * KS);
  const int n_tiles = (p.n + kBnOut - 1) / kBnOut;

  int64_t items;
  if constexpr (kGrouped) {
    // Row tiles per expert (none where it is absent), summed over the experts: wave 0.
    if (wave == 0) {
      int carry = 0;
      for (int base = 0; base < p.num_experts; base += 64) {
        const int e = base + lane;
        int t = 0;
        if (e < p.num_experts && p.w_ptrs[e] != 0) {
          const int cnt = min(p.offsets[e + 1], p.rows) - max(p.offsets[e], 0);
          t = cnt > 0 ? (cnt + BT - 1) / BT : 0;
        }
        int incl = t;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int u = __shfl_up(incl, d, 64);
          if (lane >= d) incl += u;
        }
        if (e < p.num_experts) prefix[e] = carry + incl - t;
        carry += __shfl(incl, 63, 64);
      }
      if (lane == 0) prefix[p.num_experts] = carry;
    }
    __syncthreads();
    items = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(prefix[p.num_experts])) * n_tiles;
  } else {
    items = static_cast<int64_t>((p.rows + BT - 1) / BT) * n_tiles;
  }

  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    // ---- the item: rows [m0, m0 + cnt) and output columns [n0, n0 + n_valid)
    const int ty = static_cast<int>(item / n_tiles);
    const int n0 = static_cast<int>(item - static_cast<int64_t>(ty) * n_tiles) * kBnOut;
    const uint8_t *w0, *w1;
    const float *s0, *s1;
    int m0, cnt;
    if constexpr (kGrouped) {
      // The last expert whose prefix is at most ty (prefixes do not decrease).
      int below = 0;
      for (int base = 0; base < p.num_experts; base += 64) {
        const int e = base + lane;
        below += __popcll(__ballot(e < p.num_experts && prefix[e] <= ty));
      }
      const int e = max(below - 1, 0);
      const int lo = max(p.offsets[e], 0), hi = min(p.offsets[e + 1], p.rows);
      const int tile = ty - __builtin_amdgcn_readfirstlane(prefix[e]);
      const int64_t first = lo + static_cast<int64_t>(tile) * BT;
      // Never true for offsets that are a prefix sum; keeps every access in range if not.
      if (first < lo || first >= hi) continue;
      m0 = static_cast<int>(first);
      cnt = min(BT, hi - m0);
      w0 = reinterpret_cast<const uint8_t *>(p.w_ptrs[e]);
      s0 = reinterpret_cast<const float *>(p.s_ptrs[e]);
      if (w0 == nullptr) continue;
      w1 = w0 + static_cast<int64_t>(p.n) * p.ldw;
      s1 = s0 + static_cast<int64_t>((p.n + kFp8Block - 1) / kFp8Block) * kb_n;
    } else {
      m0 = ty * BT;
      cnt = min(BT, p.rows - m0);
      w0 = p.w0;
      w1 = p.w1;
      s0 = p.ws0;
      s1 = p.ws1;
    }
    const int n_valid = min(kBnOut, p.n - n0);
    const uint32_t w_bytes = static_cast<uint32_t>(n_valid) * static_cast<uint32_t>(p.ldw);
    const __amdgpu_buffer_rsrc_t wr0 = make_rsrc(w0 + static_cast<int64_t>(n0) * p.ldw, w_bytes);
    const __amdgpu_buffer_rsrc_t wr1 =
        kSwiglu ? make_rsrc(w1 + static_cast<int64_t>(n0) * p.ldw, w_bytes) : wr0;
    // Rows: from the tile's first row, or (gathered) from row 0.
    const bool gathered = kGrouped && p.gather != nullptr;
    const int64_t a_base = gathered ? 0 : m0;
    const int a_count = gathered ? p.a_rows : cnt;
    const __amdgpu_buffer_rsrc_t ar =
        make_rsrc(p.a + a_base * p.lda, static_cast<uint32_t>(a_count * p.lda));
    const __amdgpu_buffer_rsrc_t sr =
        make_rsrc(p.a_scale + a_base * p.ld_as, static_cast<uint32_t>(a_count * p.ld_as * 4));
    // The source row of tile row r relative to the resources, -1 past the valid ones.
    const auto src_row = [&](int r) {
      if (r >= cnt) return -1;
      if (!gathered) return r;
      const int t = p.gather[m0 + r];
      return t >= 0 && t < p.a_rows ? t : -1;
    };

    // ---- this lane's load offsets: instruction i fills 8 LDS rows, lane l the physical
    // piece l % 8 of row l / 8, so it loads logical piece (l % 8) ^ (l / 8)
    const int piece = (lane & 7) ^ (lane >> 3);
    uint32_t w_voff[C::kWLoads], x_voff[C::kXLoads], s_voff;
#pragma unroll
    for (int i = 0; i < C::kWLoads; ++i) {
      const int r = 8 * (sw * C::kWLoads + i) + (lane >> 3);
      w_voff[i] = static_cast<uint32_t>(r & (kBnOut - 1)) * static_cast<uint32_t>(p.ldw) +
                  16u * piece;
    }
#pragma unroll
    for (int i = 0; i < C::kXLoads; ++i) {
      const int inst = sw * C::kXLoads + i;
      const int r = inst < C::kXInstr ? src_row(8 * inst + (lane >> 3)) : -1;
      x_voff[i] = r < 0 ? kNoLoad : static_cast<uint32_t>(r) * static_cast<uint32_t>(p.lda) +
                                        16u * piece;
    }
    {
      const int t = 64 * (sw % (C::kScaleFloats / 64)) + lane;
      const int r = t < BT ? src_row(t) : -1;
      s_voff = r < 0 ? kNoLoad : static_cast<uint32_t>(r) * static_cast<uint32_t>(p.ld_as) * 4u;
    }
    const auto dma_stage = [&](int j) {
      const int kb = j * KS + slice;  // this wave's slice of the stage
      // Bytes of this slice inside K; a piece past them is not loaded (zeros).
      const int left = p.k - kb * kFp8Block;
      const uint32_t dead = 16 * piece < left ? 0u : kNoLoad;
      const int soff = left > 0 ? kb * kFp8Block : 0;
      uint8_t *st = lds + (j % ST) * C::kStage + slice * C::kSlice;
#pragma unroll
      for (int i = 0; i < C::kWLoads; ++i) {
        const int row = 8 * (sw * C::kWLoads + i);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            kSwiglu && row >= kBnOut ? wr1 : wr0,
            (__attribute__((address_space(3))) void *)(st + row * kRowBytes), 16,
            static_cast<int>(w_voff[i] | dead), soff, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < C::kXLoads; ++i) {
        const int inst = sw * C::kXLoads + i;
        uint8_t *dst = inst < C::kXInstr ? st + C::kWBytes + inst * 1024 : lds + C::kDumpOff;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            ar, (__attribute__((address_space(3))) void *)dst, 16,
            static_cast<int>(x_voff[i] | dead), soff, 0, 0);
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          sr,
          (__attribute__((address_space(3))) void *)(st + C::kWBytes + C::kXBytes +
                                                     256 * (sw % (C::kScaleFloats / 64))),
          4, static_cast<int>(s_voff | (left > 0 ? 0u : kNoLoad)), left > 0 ? 4 * kb : 0, 0, 0);
    };

#pragma unroll
    for (int j = 0; j < ST - 1; ++j) dma_stage(j);

    // ---- the tile's weight scales for all of K
    {
      const int nb = (p.n + kFp8Block - 1) / kFp8Block;
      for (int i = tid; i < C::kNBlocks * steps * KS; i += C::kThreads) {
        const int blk = i / (steps * KS), kb = i - blk * (steps * KS);
        float v = 0.0f;
        if (kb < kb_n) {
          if (kSwiglu)
            v = (blk == 0 ? s0 : s1)[static_cast<int64_t>(n0 / kFp8Block) * kb_n + kb];
          else if (n0 / kFp8Block + blk < nb)
            v = s0[static_cast<int64_t>(n0 / kFp8Block + blk) * kb_n + kb];
        }
        sb[i] = v;
      }
      __syncthreads();
    }

    f32x4_t acc[NT][TT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // Weight tile i of this wave: its first LDS row and its scale row.
    const auto w_row = [&](int i) {
      if (kSwiglu) return i < NT / 2 ? (wn * (NT / 2) + i) * 16 : kBnOut + (wn * (NT / 2) + i - NT / 2) * 16;
      return (wn * NT + i) * 16;
    };
    const int frag = r16 * kRowBytes + 16 * (g4 ^ (r16 & 7));

    constexpr int kWaitN = C::kLoads * (ST - 2);
    static_assert(ST >= 2 && kWaitN < 64, "vmcnt holds 6 bits");
    constexpr int kWaitImm = (kWaitN & 15) | ((kWaitN >> 4) << 14) | (7 << 4) | (15 << 8);
    for (int s = 0; s < steps; ++s) {
      __builtin_amdgcn_s_waitcnt(kWaitImm);  // this wave's loads of stage s are in LDS
      __builtin_amdgcn_s_barrier();           // every wave's; and stage s - 1 is read
      dma_stage(s + ST - 1);                  // into stage s - 1's buffer
      const uint8_t *st = lds + (s % ST) * C::kStage + slice * C::kSlice;
      const uint8_t *xs = st + C::kWBytes + wt * TT * 16 * kRowBytes;
      const float *sa =
          reinterpret_cast<const float *>(st + C::kWBytes + C::kXBytes) + wt * TT * 16 + r16;
      float sbv[C::kNBlocks];
#pragma unroll
      for (int b = 0; b < C::kNBlocks; ++b) sbv[b] = sb[b * steps * KS + s * KS + slice];
      typename Mma::Operand wf[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i)
        wf[i] = Mma::operand(read_codes(st + w_row(i) * kRowBytes, frag));
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const typename Mma::Operand xf =
            Mma::operand(read_codes(xs + t * 16 * kRowBytes, frag));
        const float sat = sa[16 * t];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const f32x4_t part = Mma::product(wf[i], xf);
          const int blk = kSwiglu ? (i < NT / 2 ? 0 : 1) : 0;
          float sbt;
          if constexpr (!kSwiglu && C::kNBlocks > 1)
            sbt = w_row(i) < kFp8Block ? sbv[0] : sbv[1];  // wave-uniform
          else
            sbt = sbv[blk];
          const float sc = sat * sbt;
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[i][t][x] = fmaf(part[x], sc, acc[i][t][x]);
        }
      }
    }
    // The past-the-end stages' loads write LDS (zeros) too: they finish first.
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();  // every wave's operand reads are done: the stages are free

    // ---- epilogue: acc[i][t][x] is output column w_row(i) + 4 g4 + x of tile row
    // (wt TT + t) 16 + r16
    if constexpr (kSwiglu) {
      constexpr int kH = NT / 2;
      constexpr int kRow = kFp8Block + 16;  // staged code row, padded
      float *red = reinterpret_cast<float *>(lds + BT * kRow);  // [WN][BT] magnitudes
      static_assert(BT * kRow + WN * BT * 4 + BT * 4 <= C::kDumpOff, "epilogue fits the stages");
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kH; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const bool in = w_row(i) + 4 * g4 + x < n_valid;
            const float v = moe::swiglu_clamp1(acc[i][t][x], acc[i + kH][t][x], p.limit);
            acc[i][t][x] = v;
            if (in) m = max(m, __float_as_uint(v) & 0x7FFFFFFFu);
          }
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16, 64)));
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32, 64)));
        if (g4 == 0) red[wn * BT + (wt * TT + t) * 16 + r16] = __uint_as_float(m);
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int r = (wt * TT + t) * 16 + r16;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < WN; ++w) m = max(m, __float_as_uint(red[w * BT + r]));
        const float s = moe::fp8_scale(m);
        if (wn == 0 && g4 == 0 && r < cnt)
          p.q_scale[static_cast<int64_t>(m0 + r) * p.ld_qs + n0 / kFp8Block] = s;
#pragma unroll
        for (int i = 0; i < kH; ++i)
          *reinterpret_cast<uint32_t *>(lds + r * kRow + w_row(i) + 4 * g4) =
              moe::e4m3x4(acc[i][t][0] / s, acc[i][t][1] / s, acc[i][t][2] / s, acc[i][t][3] / s);
      }
      __syncthreads();
      for (int u = tid; u < BT * (kFp8Block / 16); u += C::kThreads) {
        const int r = u / (kFp8Block / 16), ch = u % (kFp8Block / 16);
        if (r >= cnt || ch * 16 >= n_valid) continue;
        *reinterpret_cast<u32x4_t *>(p.q + static_cast<int64_t>(m0 + r) * p.ldc + n0 + ch * 16) =
            *reinterpret_cast<const u32x4_t *>(lds + r * kRow + ch * 16);
      }
    } else if constexpr (KS > 1) {
      // The slice groups' sums, joined in slice order.
      constexpr int kRow = BN + 4;  // floats
      static_assert(KS * BT * kRow * 4 <= C::kDumpOff, "epilogue fits the stages");
      float *red = reinterpret_cast<float *>(lds);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          *reinterpret_cast<f32x4_t *>(red + (slice * BT + (wt * TT + t) * 16 + r16) * kRow +
                                       w_row(i) + 4 * g4) = acc[i][t];
      __syncthreads();
      for (int u = tid; u < BT * (BN / 4); u += C::kThreads) {
        const int r = u / (BN / 4), q = u % (BN / 4);
        if (r >= cnt || 4 * q >= n_valid) continue;
        f32x4_t v = *reinterpret_cast<const f32x4_t *>(red + r * kRow + 4 * q);
#pragma unroll
        for (int z = 1; z < KS; ++z)
          v += *reinterpret_cast<const f32x4_t *>(red + (z * BT + r) * kRow + 4 * q);
        uint2 o;
        o.x = moe::pack_bf16x2(v[0], v[1]);
        o.y = moe::pack_bf16x2(v[2], v[3]);
        *reinterpret_cast<uint2 *>(p.c + static_cast<int64_t>(m0 + r) * p.ldc + n0 + 4 * q) = o;
      }
    } else {
      constexpr int kRow = 2 * BN + 16;  // bytes
      static_assert(BT * kRow <= C::kDumpOff, "epilogue fits the stages");
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          uint2 o;
          o.x = moe::pack_bf16x2(acc[i][t][0], acc[i][t][1]);
          o.y = moe::pack_bf16x2(acc[i][t][2], acc[i][t][3]);
          *reinterpret_cast<uint2 *>(lds + ((wt * TT + t) * 16 + r16) * kRow +
                                     2 * (w_row(i) + 4 * g4)) = o;
        }
      __syncthreads();
      for (int u = tid; u < BT * (BN / 8); u += C::kThreads) {
        const int r = u / (BN / 8), ch = u % (BN / 8);
        if (r >= cnt || ch * 8 >= n_valid) continue;
        *reinterpret_cast<u32x4_t *>(p.c + static_cast<int64_t>(m0 + r) * p.ldc + n0 + ch * 8) =
            *reinterpret_cast<const u32x4_t *>(lds + r * kRow + ch * 16);
      }
    }
    __syncthreads();  // the next item's loads overwrite the staged output
  }
}

// ------------------------------------------------------------------------------- host

constexpr int kMaxDevices = 64;

// Compute units of the current device (the persistent grid's size), looked up once each.
int compute_units(int device) {
  static std::mutex mu;
  static int cus[kMaxDevices] = {};
  if (device < 0 || device >= kMaxDevices) return 256;
  std::lock_guard<std::mutex> lock(mu);
  if (cus[device] == 0) {
    int v = 0;
    cus[device] = hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, device) ==
                              hipSuccess && v > 0
                      ? v
                      : 256;
  }
  return cus[device];
}

// Raises the kernel's dynamic LDS limit once per device.
template <class Kern>
bool allow_lds(Kern kern, int device) {
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (device >= 0 && device < kMaxDevices && done[device]) return true;
  if (hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                          hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024) != hipSuccess)
    return false;
  if (device >= 0 && device < kMaxDevices) done[device] = true;
  return true;
}

template <class C, bool kSwiglu, bool kGrouped>
int run(const char *name, const GemmArgs &p, void *stream) {
  int device = 0;
  if (hipGetDevice(&device) != hipSuccess) device = -1;
  const auto kern = fp8_gemm_kernel<C, kSwiglu, kGrouped>;
  const int bytes = lds_bytes<C, kGrouped>(p);
  if (!allow_lds(kern, device)) {
    moe::set_error("%s: the device refuses %d bytes of LDS", name, bytes);
    return MOE_ELAUNCH;
  }
  const int bn_out = kSwiglu ? C::BN / 2 : C::BN;
  const int64_t n_tiles = (p.n + bn_out - 1) / bn_out;
  // Most row tiles there can be: every expert's last tile may be partial.
  const int64_t row_tiles =
      kGrouped ? static_cast<int64_t>(p.rows) / C::BT +
                     (p.num_experts < p.rows ? p.num_experts : p.rows)
               : (static_cast<int64_t>(p.rows) + C::BT - 1) / C::BT;
  const int64_t per_cu = 160 * 1024 / bytes;
  const int64_t resident = (per_cu < 1 ? 1 : per_cu) * compute_units(device);
  const int64_t grid = row_tiles * n_tiles < resident ? row_tiles * n_tiles : resident;
  return moe::launch(name, kern, dim3(static_cast<unsigned>(grid)), dim3(C::kThreads), bytes,
                     stream, p);
}

// Tiles: rows per item from the (average) rows there are.
template <bool kSwiglu, bool kGrouped>
int dispatch(const char *name, const GemmArgs &p, void *stream) {
  int64_t avg = p.rows;
  if (kGrouped) avg = p.rows / (p.num_experts < p.rows ? p.num_experts : p.rows);
  if constexpr (kSwiglu) {
    if (avg <= 12) return run<Cfg<2, 2, 8, 1, 1, 2>, kSwiglu, kGrouped>(name, p, stream);
    if (avg <= 40) return run<Cfg<2, 4, 8, 1, 1, 3>, kSwiglu, kGrouped>(name, p, stream);
    return run<Cfg<2, 8, 8, 1, 1, 3>, kSwiglu, kGrouped>(name, p, stream);
  } else {
    if (avg <= 12) return run<Cfg<2, 2, 4, 1, 1, 3>, kSwiglu, kGrouped>(name, p, stream);
    if (avg <= 40) return run<Cfg<2, 4, 4, 1, 1, 3>, kSwiglu, kGrouped>(name, p, stream);
    return run<Cfg<2, 8, 8, 1, 1, 3>, kSwiglu, kGrouped>(name, p, stream);
  }
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The checks every call shares (n = output columns). Rows are checked where they are known.
int check_common(const char *name, const GemmArgs &p) {
  MOE_REQUIRE(p.n > 0 && p.n % 16 == 0, "%s: the output width must be a positive multiple of 16 "
              "(got %d)", name, p.n);
  MOE_REQUIRE(p.k > 0 && p.k % 16 == 0 && p.k <= kMaxK,
              "%s: k must be a multiple of 16 in [16, %d] (got %d)", name, kMaxK, p.k);
  MOE_REQUIRE(p.n <= (1 << 29), "%s: the output width is too large (got %d)", name, p.n);
  MOE_REQUIRE(p.lda >= p.k && p.lda % 16 == 0 && p.lda < (1 << 22),
              "%s: lda must be >= k, a multiple of 16 and below 2^22", name);
  MOE_REQUIRE(p.ldw >= p.k && p.ldw % 16 == 0 && p.ldw < (1 << 22),
              "%s: the weight's leading dimension must be >= k, a multiple of 16 and below 2^22",
              name);
  MOE_REQUIRE(p.ld_as >= (p.k + kFp8Block - 1) / kFp8Block && p.ld_as < (1 << 20),
              "%s: ld_a_scale must be >= ceil(k / 128) and below 2^20", name);
  MOE_REQUIRE(p.rows >= 0, "%s: the row count must be >= 0", name);
  return MOE_OK;
}

int check_out_plain(const char *name, const GemmArgs &p) {
  MOE_REQUIRE(p.ldc >= p.n && p.ldc % 8 == 0, "%s: ldc must be >= %d and a multiple of 8", name,
              p.n);
  MOE_REQUIRE(p.rows == 0 || (p.c && moe::aligned16(p.c)),
              "%s: c must be non-NULL and 16-byte aligned", name);
  return MOE_OK;
}

int check_out_swiglu(const char *name, const GemmArgs &p) {
  MOE_REQUIRE(p.limit > 0.0f, "%s: limit must be > 0", name);
  MOE_REQUIRE(p.ldc >= p.n && p.ldc % 16 == 0, "%s: ld_act must be >= %d and a multiple of 16",
              name, p.n);
  MOE_REQUIRE(p.ld_qs >= (p.n + kFp8Block - 1) / kFp8Block,
              "%s: ld_act_scale must be >= ceil(width / 128)", name);
  MOE_REQUIRE(p.rows == 0 || (p.q && p.q_scale && moe::aligned16(p.q) && aligned4(p.q_scale)),
              "%s: act must be non-NULL and 16-byte aligned, act_scale non-NULL", name);
  return MOE_OK;
}

int check_rows_in(const char *name, const GemmArgs &p) {
  MOE_REQUIRE(p.a && p.a_scale && moe::aligned16(p.a) && aligned4(p.a_scale),
              "%s: a must be non-NULL and 16-byte aligned, a_scale non-NULL", name);
  return MOE_OK;
}

int check_dense(const char *name, const GemmArgs &p, bool swiglu) {
  int rc = check_common(name, p);
  if (rc == MOE_OK) rc = swiglu ? check_out_swiglu(name, p) : check_out_plain(name, p);
  if (rc != MOE_OK || p.rows == 0) return rc;
  rc = check_rows_in(name, p);
  if (rc != MOE_OK) return rc;
  MOE_REQUIRE(p.w0 && p.ws0 && p.w1 && p.ws1, "%s: a required pointer is NULL", name);
  MOE_REQUIRE(moe::aligned16(p.w0) && moe::aligned16(p.w1) && aligned4(p.ws0) && aligned4(p.ws1),
              "%s: weights must be 16-byte aligned, scales 4-byte aligned", name);
  return MOE_OK;
}

int check_grouped(const char *name, const GemmArgs &p, bool swiglu) {
  int rc = check_common(name, p);
  if (rc == MOE_OK) rc = swiglu ? check_out_swiglu(name, p) : check_out_plain(name, p);
  if (rc != MOE_OK) return rc;
  MOE_REQUIRE(p.num_experts >= 1 && p.num_experts <= kMaxExperts,
              "%s: num_experts must be in [1, %d] (got %d)", name, kMaxExperts, p.num_experts);
  MOE_REQUIRE(p.a_rows >= 0, "%s: a_rows must be >= 0", name);
  if (p.rows == 0) return MOE_OK;
  rc = check_rows_in(name, p);
  if (rc != MOE_OK) return rc;
  MOE_REQUIRE(p.w_ptrs && p.s_ptrs && p.offsets, "%s: a required pointer is NULL", name);
  MOE_REQUIRE(p.a_rows >= 1, "%s: a_rows must be >= 1 when max_rows > 0", name);
  MOE_REQUIRE(p.gather != nullptr || p.a_rows >= p.rows,
              "%s: without a gather, a needs max_rows rows", name);
  // Gathered rows are addressed by 32-bit offsets from row 0.
  MOE_REQUIRE(p.gather == nullptr ||
                  (p.a_rows * p.lda < (1ll << 31) && p.a_rows * p.ld_as * 4 < (1ll << 31)),
              "%s: a gathered row buffer must be smaller than 2 GiB", name);
  return MOE_OK;
}

}  // namespace

extern "C" int moe_dense_gemm_fp8(const uint8_t *a, int64_t lda, const float *a_scale,
                                  int64_t ld_a_scale, const uint8_t *b, int64_t ldb,
                                  const float *b_scale, uint16_t *c, int64_t ldc, int32_t m,
                                  int32_t n, int32_t k, void *stream) {
  moe::clear_error();
  GemmArgs p = {};
  p.a = a, p.lda = lda, p.a_scale = a_scale, p.ld_as = ld_a_scale, p.a_rows = m;
  p.w0 = p.w1 = b, p.ldw = ldb, p.ws0 = p.ws1 = b_scale;
  p.c = c, p.ldc = ldc, p.rows = m, p.n = n, p.k = k;
  const int rc = check_dense("dense_gemm_fp8", p, false);
  if (rc != MOE_OK || m == 0) return rc;
  return dispatch<false, false>("moe_dense_gemm_fp8", p, stream);
}

extern "C" int moe_dense_gate_up_swiglu_fp8(const uint8_t *a, int64_t lda, const float *a_scale,
                                            int64_t ld_a_scale, const uint8_t *gate_w,
                                            const float *gate_scale, const uint8_t *up_w,
                                            const float *up_scale, int64_t ldw, uint8_t *act,
                                            int64_t ld_act, float *act_scale,
                                            int64_t ld_act_scale, int32_t m, int32_t inter,
                                            int32_t k, float limit, void *stream) {
  moe::clear_error();
  GemmArgs p = {};
  p.a = a, p.lda = lda, p.a_scale = a_scale, p.ld_as = ld_a_scale, p.a_rows = m;
  p.w0 = gate_w, p.w1 = up_w, p.ldw = ldw, p.ws0 = gate_scale, p.ws1 = up_scale;
  p.q = act, p.ldc = ld_act, p.q_scale = act_scale, p.ld_qs = ld_act_scale;
  p.rows = m, p.n = inter, p.k = k, p.limit = limit;
  const int rc = check_dense("dense_gate_up_swiglu_fp8", p, true);
  if (rc != MOE_OK || m == 0) return rc;
  return dispatch<true, false>("moe_dense_gate_up_swiglu_fp8", p, stream);
}

extern "C" int moe_w8a8_grouped_gemm(const uint8_t *a, int64_t lda, const float *a_scale,
                                     int64_t ld_a_scale, int32_t a_rows,
                                     const int32_t *a_gather, const uint64_t *weight_ptrs,
                                     const uint64_t *scale_ptrs, const int32_t *expert_offsets,
                                     int32_t num_experts, uint16_t *c, int64_t ldc,
                                     int32_t max_rows, int32_t n, int32_t k, void *stream) {
  moe::clear_error();
  GemmArgs p = {};
  p.a = a, p.lda = lda, p.a_scale = a_scale, p.ld_as = ld_a_scale, p.a_rows = a_rows;
  p.gather = a_gather, p.w_ptrs = weight_ptrs, p.s_ptrs = scale_ptrs, p.ldw = k;
  p.offsets = expert_offsets, p.num_experts = num_experts;
  p.c = c, p.ldc = ldc, p.rows = max_rows, p.n = n, p.k = k;
  const int rc = check_grouped("w8a8_grouped_gemm", p, false);
  if (rc != MOE_OK || max_rows == 0) return rc;
  return dispatch<false, true>("moe_w8a8_grouped_gemm", p, stream);
}

extern "C" int moe_w8a8_grouped_gemm_swiglu(
    const uint8_t *a, int64_t lda, const float *a_scale, int64_t ld_a_scale, int32_t a_rows,
    const int32_t *a_gather, const uint64_t *weight_ptrs, const uint64_t *scale_ptrs,
    const int32_t *expert_offsets, int32_t num_experts, uint8_t *act, int64_t ld_act,
    float *act_scale, int64_t ld_act_scale, int32_t max_rows, int32_t mi, int32_t k, float limit,
    void *stream) {
  moe::clear_error();
  GemmArgs p = {};
  p.a = a, p.lda = lda, p.a_scale = a_scale, p.ld_as = ld_a_scale, p.a_rows = a_rows;
  p.gather = a_gather, p.w_ptrs = weight_ptrs, p.s_ptrs = scale_ptrs, p.ldw = k;
  p.offsets = expert_offsets, p.num_experts = num_experts;
  p.q = act, p.ldc = ld_act, p.q_scale = act_scale, p.ld_qs = ld_act_scale;
  p.rows = max_rows, p.n = mi, p.k = k, p.limit = limit;
  const int rc = check_grouped("w8a8_grouped_gemm_swiglu", p, true);
  if (rc != MOE_OK || max_rows == 0) return rc;
  return dispatch<true, true>("moe_w8a8_grouped_gemm_swiglu", p, stream);
}
