// moe_w4a16_layer_few: a whole routed NVFP4 layer for at most 16 tokens in two kernels.
//
//   kernel 1   router (logits -> top-k), the rows' experts, gate_up + SwiGLU:
//              act[slot] = fp16 or bf16( swiglu( s2_e sum_k x[r, k] w_e[:, k] ) )
//   kernel 2   down, the weighted sum over a row's slots and the shared term:
//              out[r] = bf16( sum_slot (p_slot s2_e) sum_k act[slot, k] w_e[:, k] + shared[r] )
//
// Why two: the down products need every gate_up column of their slot, and a wait for all blocks
// inside one kernel could deadlock two such kernels on one GPU. Everything else (routing, union
// of the experts, combine) is done by each block for itself: 16 rows' worth of it costs about
// as much as one more kernel's start, and no table goes through memory.
//
// Bound by HBM: the weights of the live experts, read once. What a byte of them costs in the
// vector unit decides how near the kernel comes:
//   - A weight is e2m1 x e4m3 (the block's scale) x scale2. The first product has at most 6
//     significant bits and lies in [2^-10, 2688]: exact in FP16. One conversion and one packed
//     FP16 product decode two weights, with no table (the BF16 form, which rounds scale2 into
//     the weight, takes 14 operations per 8 weights and a table lookup in LDS per 16). scale2 is
//     applied to the FP32 sums. The matrix instruction is v_mfma_f32_16x16x32_f16.
//   - So activations are FP16 too. BF16 values times a power of two per row (that brings the
//     row's largest magnitude to [2^14, 2^15)) are exact in FP16 down to 2^-31 of the largest;
//     below, they are cut to multiples of 2^-24 there and off by less than 2^-38 of it. Beside the
//     largest value's own product that is far below what FP32 sums keep; where that one's weight
//     is zero it is what is left of the sum (moe_layer and moe_layer_decode keep BF16 rows).
//   - Kernel 1 holds its K share of all rows' activations in registers for its whole life: a wave
//     takes the same 256-k steps of every item, so nothing but weights is loaded in its loop.
//     Two items are in flight per wave (110 KB per CU at K 6144).
//   - Kernel 2's activations differ by expert: they are staged through LDS per wave, at most
//     kCap rows of an expert at a time (an expert with more is swept again).
// Measured at 6144 x 2048, 8 of 256 experts a row: 43 us for 1 row (27 for its bytes at the rate of a
// plain read), 76 for 2, 132 for 4, 214 to 233 for 8 (194), 398 for 16. The rest is:
//   - the starts of two kernels and the routing in each: the first weights are asked for 7 us into
//     kernel 1 with 1 row and 12 with 8 (table entries and logits 2 to 5, grouping 1 to 3, the tokens'
//     way through LDS 2), and 4 to 5 us into kernel 2;
//   - kernel 2's issue: with 12 weight rows to a block a quarter of every matrix instruction and of
//     every decoded register is empty. At 8 rows its waves wait 44 % of their time for an issue
//     slot and 30 % for data. The older of a CU's two blocks ends after 60 of 89 us; levelled by
//     wave priorities the two end together, no sooner.
// Sums run in a fixed order: two calls on the same inputs give the same bits. Their order
// depends on the experts of the other rows, so a row's last bits may differ in another batch.
#include <algorithm>
#include <cmath>

#include "buffer_io.h"
#include "common.h"
#include "fp8.h"  // fp8_swiglu
#include "lds_limit.h"
#include "nvfp4_decode.h"  // moe::pack_bf16x2

namespace {

using moe::kNoLoad;
using moe::load16;
using moe::make_rsrc;
using moe::u32x4_t;

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __fp16 fp16x2_t __attribute__((ext_vector_type(2)));

constexpr int kMaxRows = MOE_FEW_MAX_ROWS;  // one matrix tile of rows
constexpr int kMaxIds = MOE_FEW_MAX_IDS;    // rows * top_k
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kStepK = 256;                 // k per step: 64 per lane, 4 lanes per row
constexpr int kTable = kThreads;            // experts whose table entries a block keeps in LDS
constexpr int kCus = 256;
static_assert(kMaxIds <= kThreads, "one thread per slot");

struct Tables {
  const uint64_t *packed, *scales;
  const float *scale2;
  const uint64_t *other_packed, *other_scales;  // the other projection's: an expert needs both
};

struct FewArgs {
  const uint16_t *x;
  const float *logits, *bias;        // or NULL
  const int32_t *ids;                // [rows * top_k], read where there are no logits
  const float *wts;
  int32_t *ids_out;                  // the routing, written where there are logits
  float *wts_out;
  Tables gate_up, down;
  const uint16_t *shared;            // or NULL
  uint16_t *out;
  uint16_t *act;                     // [rows * top_k][mi]
  uint8_t *act_exp;                  // BF16: [rows * top_k][mi / 8] largest exponent of 8 columns
  int64_t ld_x, ld_logits, ld_shared, ld_out;
  int32_t rows, top_k, num_experts, hidden, mi, renormalize;
  int32_t act_half, act_shift;       // FP16 activations times 2^act_shift, or BF16 ones
  int32_t tile_rows;                 // weight rows of a block of kernel 2
  float routed_scale, limit;
};

// ------------------------------------------------------------------------------ decoding

// Eight weights (one dword of codes, k ascending) times their block's scale, exact in FP16.
__device__ __forceinline__ f16x8_t decode8(uint32_t codes, f16x2_t d) {
  const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * d;
  const f16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * d;
  const f16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * d;
  const f16x2_t e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * d;
  return f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// One step of one tile: 64 weights per lane (w[0], w[1]: 16 bytes each) with the scales of their
// four blocks, times the lane's 64 activations, into two sums (a matrix instruction that waits
// for the one before it would take twice as long).
__device__ __forceinline__ void step_product(const u32x4_t (&w)[2], uint32_t scales,
                                             const f16x8_t (&x)[8], f32x4_t (&acc)[2]) {
  const f16x2_t d01 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales, 1.0f, false);
  const f16x2_t d23 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales, 1.0f, true);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const f16x2_t pair = j < 4 ? d01 : d23;
    const _Float16 d = pair[(j >> 1) & 1];
    acc[j & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(decode8(w[j >> 2][j & 3], f16x2_t{d, d}),
                                                        x[j], acc[j & 1], 0, 0, 0);
  }
}

// A lane of the four that share a weight row holds 16 scales of it, those of one step (kb: the
// step); returns in d[i] its own four scales of step i: a 4 x 4 transposition over the lanes kb.
__device__ __forceinline__ void spread_scales(u32x4_t v, uint32_t (&d)[4]) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  const auto swap32 = [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(a, b, false, false));
  };
  const auto swap16 = [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(a, b, false, false));
  };
  const u32x2_t a = swap32(v[0], v[2]), b = swap32(v[1], v[3]);
  const u32x2_t c = swap16(a[0], b[0]), e = swap16(a[1], b[1]);
  d[0] = c[0];
  d[1] = c[1];
  d[2] = e[0];
  d[3] = e[1];
}

// The 16 scales at `off` of a row. kTail: the row may end among them (its K is no multiple of
// 256); `left` are the k from the first one's on, and scales past them are not loaded.
template <bool kTail>
__device__ __forceinline__ u32x4_t load_scales(__amdgpu_buffer_rsrc_t r, uint32_t off,
                                               uint32_t soff, int left) {
  if (!kTail) return load16(r, off, soff);
  u32x4_t v;
#pragma unroll
  for (int d = 0; d < 4; ++d)
    v[d] = static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b32(
        r, static_cast<int>(64 * d < left ? off + 4 * d : kNoLoad), static_cast<int>(soff), 0));
  return v;
}

// The power of two that brings a magnitude with this FP32 exponent field to [2^14, 2^15); none
// for infinities and NaN (which stay what they are).
__device__ __forceinline__ int shift_of(int exponent) {
  return exponent == 255 ? 0 : 141 - (exponent > 0 ? exponent : 1);
}

// Two BF16 values of a dword times 2^shift as FP16.
__device__ __forceinline__ uint32_t half2_of(uint32_t v, int shift) {
  const float lo = __builtin_amdgcn_ldexpf(__uint_as_float(v << 16), shift);
  const float hi = __builtin_amdgcn_ldexpf(__uint_as_float(v & 0xFFFF0000u), shift);
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(lo, hi));
}

__device__ __forceinline__ f16x8_t half8_of(u32x4_t v, int shift) {
  const u32x4_t o = {half2_of(v[0], shift), half2_of(v[1], shift), half2_of(v[2], shift),
                     half2_of(v[3], shift)};
  return __builtin_bit_cast(f16x8_t, o);
}

__device__ __forceinline__ uint32_t rfl(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
}

__device__ __forceinline__ const void *rfl_ptr(uint64_t v) {
  const uint64_t hi = rfl(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const void *>(hi << 32 | rfl(static_cast<uint32_t>(v)));
}

// -------------------------------------------------------------------------------- router

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// The largest of a wave's unsigned values, by lane moves within the vector unit.
template <int kCtrl>
__device__ __forceinline__ uint32_t max_moved(uint32_t v) {
  const int o = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xF, 0xF, false);
  return max(v, static_cast<uint32_t>(o));
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = max_moved<0x111>(v);  // row_shr 1, 2, 4, 8: lane 15 of each row of 16 has its maximum
  v = max_moved<0x112>(v);
  v = max_moved<0x114>(v);
  v = max_moved<0x118>(v);
  v = max_moved<0x142>(v);  // row_bcast 15, 31: lane 63 has all four rows'
  v = max_moved<0x143>(v);
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// A key's bits in an order that unsigned comparison keeps; above 0 for every number.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 -> +0
  return u >> 31 ? ~u : u | 0x80000000u;
}

// One row's top-k by one wave, as moe_router_topk computes it (same selection, same arithmetic):
// keys are the logits, or softmax + bias; the largest first, equal keys to the lower id. Lane
// j holds the id of pick j on return (-1 past the experts) and, with `weights`, its weight.
// l: the row's logits lane, lane + 64, ..., -infinity past the experts.
template <int kPerLane>
__device__ __forceinline__ void route_row(const FewArgs &p, int row, const float (&l)[kPerLane],
                                          int lane, bool weights, int &id, float &wt) {
  float m = -INFINITY, sum = 0.0f;
  if (weights || p.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (lane + 64 * i < p.num_experts) sum += __expf(l[i] - m);
    sum = wave_sum(sum);
  }
  uint32_t key[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 64 * i;
    key[i] = 0;
    if (e < p.num_experts)
      key[i] = ordered(p.bias != nullptr ? __expf(l[i] - m) / sum + p.bias[e] : l[i]);
  }
  id = -1;
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) {
      at = key[i] > best ? i : at;
      best = max(best, key[i]);
    }
    const uint32_t top = wave_umax(best);
    if (top == 0) break;  // fewer experts than top_k
    const uint64_t has = __ballot(best == top);
    int win = 64 * at + lane;
    if ((has & (has - 1)) == 0)  // one lane has it
      win = __builtin_amdgcn_readlane(win, __ffsll(static_cast<long long>(has)) - 1);
    else  // the lowest of the ids
      win = static_cast<int>(~wave_umax(best == top ? ~static_cast<uint32_t>(win) : 0u));
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) key[i] = lane + 64 * i == win ? 0u : key[i];
    id = lane == j ? win : id;
  }
  if (weights) {
    const float e =
        id >= 0 ? __expf(p.logits[static_cast<int64_t>(row) * p.ld_logits + id] - m) : 0.0f;
    const float denom = p.renormalize ? wave_sum(e) : sum;
    wt = id >= 0 ? e / denom * p.routed_scale : 0.0f;
  }
}

// ----------------------------------------------------------------------- the rows' experts

// What a block knows of the routing, in LDS. Covered slots (id in range, expert present, no
// earlier slot of the row with the same id) are grouped by expert, at most `cap` slots to an
// entry, in the order of the slots. Entries stand in the order of their first slots (up to 64 ids,
// or more than kTable experts) or of their experts.
struct Entry {
  uint64_t packed, scales;
  float scale2;
  int32_t pad;
};

__device__ __forceinline__ Entry entry_of(const Tables &t, int e) {
  const uint64_t packed = t.packed[e], scales = t.scales[e];
  const uint64_t other_packed = t.other_packed[e], other_scales = t.other_scales[e];
  const float scale2 = t.scale2[e];  // all five on their way before one is looked at
  const bool whole = (packed != 0) & (scales != 0) & (other_packed != 0) & (other_scales != 0);
  return {whole ? packed : 0, scales, scale2, 0};
}

struct Routing {
  Entry *table;      // [min(num_experts, kTable)], filled where num_experts <= kTable
  Entry *entry;      // [n_ids]
  int32_t *id;       // [kThreads]
  int32_t *num;      // [kWaves + 1], the last the number of entries
  int16_t *slot_of;  // [n_ids][16]: slot of row r in an entry, or -1
  int16_t *pos_of;   // [kThreads]: a covered slot's place in its entry
  uint32_t *mask;    // [kTable]: the rows of an expert, over 64 ids and up to kTable experts
  int16_t *base;     // [kTable]: its first entry
  int16_t *list;     // [n_ids][cap]: the entry's slots in order, -1 past them (cap < 16 only)

  static constexpr int kFixed = kThreads * 6 + 64 + kTable * 6;
  static constexpr __host__ __device__ int bytes(int n_ids, int num_experts, int cap) {
    const int table = num_experts < kTable ? num_experts : kTable;
    return kFixed + static_cast<int>(sizeof(Entry)) * (n_ids + table) +
           2 * n_ids * (16 + (cap < kMaxRows ? cap : 0));
  }

  __device__ __forceinline__ Routing(uint8_t *lds, int n_ids, int num_experts) {
    id = reinterpret_cast<int32_t *>(lds);
    num = id + kThreads;
    mask = reinterpret_cast<uint32_t *>(num + 16);
    entry = reinterpret_cast<Entry *>(mask + kTable);
    table = entry + n_ids;
    pos_of = reinterpret_cast<int16_t *>(table + min(num_experts, kTable));
    base = pos_of + kThreads;
    slot_of = base + kTable;
    list = slot_of + n_ids * 16;
  }

  // This thread's expert, for begin().
  static __device__ __forceinline__ Entry fetch(const FewArgs &p, const Tables &t, int tid) {
    if (p.num_experts <= kTable && tid < p.num_experts) return entry_of(t, tid);
    return {0, 0, 0.0f, 0};
  }

  // Before the barrier that publishes the ids: the experts' table entries and empty lists.
  template <int kCap>
  __device__ __forceinline__ void begin(const FewArgs &p, const Entry &mine, int tid) {
    const int n_ids = p.rows * p.top_k;
    if (p.num_experts <= kTable && tid < p.num_experts) table[tid] = mine;
    mask[tid] = 0;
    for (int q = tid; q < n_ids * 8; q += kThreads) reinterpret_cast<int32_t *>(slot_of)[q] = -1;
    if (kCap < kMaxRows)
      for (int q = tid; q < n_ids * kCap / 2; q += kThreads)
        reinterpret_cast<int32_t *>(list)[q] = -1;
  }

  // Slot t (row, covered, `before` slots with its id before it, `opener` the one that opened
  // its entry, whose number is `e`) goes to its places.
  template <int kCap>
  __device__ __forceinline__ void put(int t, int row, int before, int e) {
    slot_of[e * 16 + row] = static_cast<int16_t>(t);
    pos_of[t] = static_cast<int16_t>(before % kCap);
    if (kCap < kMaxRows) list[e * kCap + before % kCap] = static_cast<int16_t>(t);
  }

  // Every thread calls it, behind the barrier that publishes ids and begin()'s stores; the
  // results stand behind the caller's next barrier.
  template <int kCap>
  __device__ __forceinline__ void group(const FewArgs &p, const Tables &t, int tid) {
    const int n_ids = p.rows * p.top_k;
    const int lane = tid & 63, wave = tid >> 6;
    // Up to 64 ids: the last wave, without barriers.
    if (n_ids <= 64 && wave != kWaves - 1) return;
    const int slot = n_ids <= 64 ? lane : tid;
    const int row = slot / p.top_k, j = slot - row * p.top_k;
    int v = slot < n_ids ? id[slot] : -1;
    Entry en = {0, 0, 0.0f, 0};
    if (v >= 0 && v < p.num_experts)
      en = p.num_experts <= kTable ? table[v] : entry_of(t, v);
    if (en.packed == 0) v = -1;
    const uint64_t below = (1ull << lane) - 1ull;
    if (n_ids <= 64) {
      // The lanes with this lane's id, by one ballot per bit of the ids.
      const int bits = 32 - __clz(p.num_experts);
      uint64_t same = __ballot(v >= 0);
      for (int b = 0; b < bits; ++b) {
        const bool bit = (v >> b) & 1;
        const uint64_t ones = __ballot(bit);
        same &= bit ? ones : ~ones;
      }
      const uint64_t row_below = below & ~((1ull << ((lane - j) & 63)) - 1ull);
      const bool covered = v >= 0 && (same & row_below) == 0;  // else a repeat in the row
      same &= __ballot(covered);
      const int before = __popcll(same & below);
      const uint64_t openers = __ballot(covered && before % kCap == 0);
      // The entry's opener is the last one at or before this lane among its equals.
      const uint64_t opened = same & openers & (below | (1ull << lane));
      if (covered) {
        const int opener = 63 - __clzll(static_cast<long long>(opened));
        const int e = __popcll(openers & ((1ull << opener) - 1ull));
        if (opener == lane) entry[e] = en;
        put<kCap>(lane, row, before, e);
      }
      if (lane == 0) num[kWaves] = __popcll(openers);
      return;
    }
    for (int jj = 0; jj < j && v >= 0; ++jj)
      if (id[row * p.top_k + jj] == v) v = -1;  // a repeat in the row
    if (p.num_experts <= kTable) {
      // Entries in the order of their experts: every expert's rows as a mask, its entries counted.
      if (v >= 0) atomicOr(&mask[v], 1u << row);  // no order
      __syncthreads();
      const uint32_t rows = mask[tid];
      const int mine = (__popc(rows) + kCap - 1) / kCap;
      int upto = mine;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d, 64);
        if (lane >= d) upto += o;
      }
      if (lane == 63) num[wave] = upto;
      __syncthreads();
      int first = upto - mine, n = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        first += w < wave ? num[w] : 0;
        n += num[w];
      }
      base[tid] = static_cast<int16_t>(first);
      for (int q = 0; q < mine; ++q) entry[first + q] = table[tid];
      if (tid == 0) num[kWaves] = n;
      __syncthreads();
      if (v >= 0) {
        const int before = __popc(mask[v] & ((1u << row) - 1u));
        put<kCap>(tid, row, before, base[v] + before / kCap);
      }
      return;
    }
    __syncthreads();
    id[tid] = v;
    __syncthreads();
    int before = 0, opener = tid;
    if (wave * 64 < n_ids) {  // the slots before this one with its id
      for (int q = 0; q < min(tid, n_ids); q += 4) {
        const int4 w = *reinterpret_cast<const int4 *>(id + q);
        const int e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bool hit = v >= 0 && q + u < tid && e[u] == v;
          opener = hit && before % kCap == 0 ? q + u : opener;
          before += hit ? 1 : 0;
        }
      }
    }
    const bool opens = v >= 0 && before % kCap == 0;
    if (opens) opener = tid;
    const uint64_t ballot = __ballot(opens);
    if (lane == 0) num[wave] = __popcll(ballot);
    __syncthreads();
    int first = 0, n = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      first += w < wave ? num[w] : 0;
      n += num[w];
    }
    if (opens) {
      const int e = first + __popcll(ballot & below);
      pos_of[tid] = static_cast<int16_t>(e);  // for now: the entry that the slot opened
      entry[e] = en;
    }
    __syncthreads();
    const int mine = v >= 0 ? pos_of[opener] : -1;
    __syncthreads();
    if (mine >= 0) put<kCap>(tid, row, before, mine);
    if (tid == 0) num[kWaves] = n;
  }

  __device__ __forceinline__ int live() const {
    return static_cast<int>(rfl(static_cast<uint32_t>(num[kWaves])));
  }
};

// ------------------------------------------------------------------- kernel 1: gate and up

constexpr int kMaxPerWave = 4;  // steps of K a wave holds
// Items between two barriers. Past-the-end ones cost about 0.5 us each: with 16 of them one token's
// layer took 4 us more.
constexpr int kBatch = 8;
constexpr int kRedBytes = kBatch * kWaves * 64 * 16;
constexpr int kArrangeBytes = kWaves * 16 * 32 * 16;  // a step of every wave's share of 16 rows
static_assert(kArrangeBytes <= kRedBytes, "the rows are arranged where the partial sums go later");

// An item is 8 gate rows and the same 8 up rows of one entry. Items are dealt round-robin to the
// blocks' groups of `ways` waves, each with kSteps consecutive steps of K. Their scales come in
// one load of 16 bytes per row and step (a load per step would have every wave fetch the
// 128-byte line that holds a row's scales of 2048 k, as many bytes into the CU as the weights). The
// partial sums of 8 items per group go to LDS before the waves meet at a barrier, then each
// wave finishes its items of them (finishing every item behind a barrier of its own left 7
// waves waiting for the eighth: 3.0 us an item at K 6144).
// kRoute: logits per lane of the router, 0 where the routing is given.
// kTail: hidden is no multiple of 256.
template <int kSteps, int kRoute, bool kTail>
__global__ __launch_bounds__(kThreads, 2) void few_gate_up_kernel(FewArgs p, int ways) {
  static_assert(kRedBytes + Routing::bytes(kMaxIds, kTable, kMaxRows) + 512 <= 160 * 1024, "LDS");
  constexpr int kDepth = kSteps <= 2 ? 4 : 2;  // items in flight
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ uint32_t s_top[kWaves][16];  // largest magnitude of a wave's share of a row
  f32x4_t *red = reinterpret_cast<f32x4_t *>(dyn);  // [kBatch][kWaves][64]
  const int n_ids = p.rows * p.top_k;
  Routing rt(dyn + kRedBytes, n_ids, p.num_experts);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, kb = lane >> 4;
  const int kw = wave % ways, group = wave / ways, groups = kWaves / ways;

  // 1. Everything that needs no routing is on its way first, in the order it is waited for: the
  //    logits of this wave's rows, the experts' table entries, this wave's share of every row.
  constexpr int kLogits = kRoute > 0 ? kRoute : 1, kRouted = kMaxRows / kWaves;
  float logit[kRouted][kLogits];
  if (kRoute > 0) {
#pragma unroll
    for (int r = 0; r < kRouted; ++r)
#pragma unroll
      for (int i = 0; i < kLogits; ++i) {
        const int row = wave + r * kWaves, e = lane + 64 * i;
        logit[r][i] = -INFINITY;
        if (row < p.rows && e < p.num_experts)
          logit[r][i] = p.logits[static_cast<int64_t>(row) * p.ld_logits + e];
      }
  }
  int given = -1;
  if (kRoute == 0 && tid < n_ids) given = p.ids[tid];
  const Entry fetched = Routing::fetch(p, p.gate_up, tid);
  __builtin_amdgcn_sched_barrier(0);
  const __amdgpu_buffer_rsrc_t x_rsrc =
      make_rsrc(p.x, static_cast<uint32_t>((p.rows - 1) * p.ld_x + p.hidden) * 2u);
  u32x4_t xr[kSteps][8];  // 16 bytes of row 2 q + lane / 32 per load: whole lines
  uint32_t w_voff[kSteps];
  const uint32_t row_bytes = static_cast<uint32_t>(p.hidden) / 2;
  const uint32_t srow_bytes = static_cast<uint32_t>(p.hidden) / 16;
  const uint32_t w_row = static_cast<uint32_t>((r16 & 7) + (r16 >= 8 ? p.mi : 0));
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int k0 = (kw * kSteps + i) * kStepK, k = k0 + 64 * kb, xk = k0 + 8 * (lane & 31);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = 2 * q + (lane >> 5);
      xr[i][q] = u32x4_t{0u, 0u, 0u, 0u};
      if (2 * q < p.rows)  // wave-uniform
        xr[i][q] = load16(x_rsrc, row < p.rows && xk < p.hidden
                                      ? static_cast<uint32_t>(row * p.ld_x + xk) * 2u
                                      : kNoLoad, 0);
    }
    w_voff[i] = k < p.hidden ? w_row * row_bytes + static_cast<uint32_t>(k) / 2 : kNoLoad;
  }
  // Lane kb loads the scales of step kb.
  const int s_k = (kw * kSteps + kb) * kStepK;
  const uint32_t s_voff = kb < kSteps && s_k < p.hidden
                              ? w_row * srow_bytes + static_cast<uint32_t>(s_k) / 16
                              : kNoLoad;

  // 2. The routing, and each row's largest magnitude.
  if (kRoute > 0) {
#pragma unroll
    for (int r = 0; r < kRouted; ++r) {
      const int row = wave + r * kWaves;
      if (row >= p.rows) continue;  // wave-uniform
      int id;
      float wt = 0.0f;
      route_row(p, row, logit[r], lane, blockIdx.x == 0, id, wt);
      if (lane < p.top_k) {
        rt.id[row * p.top_k + lane] = id;
        if (blockIdx.x == 0) {
          p.ids_out[row * p.top_k + lane] = id;
          p.wts_out[row * p.top_k + lane] = wt;
        }
      }
    }
  } else if (tid < n_ids) {
    rt.id[tid] = given;
  }
  rt.begin<kMaxRows>(p, fetched, tid);
  // This wave's share of the rows goes through its piece of LDS (the place of the partial sums)
  // into the order of the matrix instruction: x[i][j] is k 64 kb + 8 j of step i of row r16. Piece
  // c of a row lies at c ^ (row % 8). With it, the rows' largest magnitudes.
  const auto arrange = [&]() __attribute__((always_inline)) {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    u32x4_t *mine = reinterpret_cast<u32x4_t *>(dyn) + wave * (16 * 32);  // kArrangeBytes in all
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int row = 2 * q + (lane >> 5);
        if (2 * q < p.rows) mine[row * 32 + ((lane & 31) ^ (row & 7))] = xr[i][q];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u32x4_t v = {0u, 0u, 0u, 0u};
        if (r16 < p.rows) v = mine[r16 * 32 + ((8 * kb + j) ^ (r16 & 7))];
        xr[i][j] = v;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, v[u] & 0x7FFF7FFFu));
      }
    }
    uint32_t top = max(m[0], m[1]);
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16, 64)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32, 64)));
    if (kb == 0) s_top[wave][r16] = top;
  };
  // The first wave, which routes when there is one row, arranges while the last one groups.
  if (wave != 0) arrange();
  __syncthreads();
  rt.group<kMaxRows>(p, p.gate_up, tid);
  if (wave == 0) arrange();
  __syncthreads();

  // 3. Items and the first loads.
  const int tiles = p.mi / 8;
  const int n_items = rt.live() * tiles;
  const int stride = static_cast<int>(gridDim.x) * groups;
  const int first = static_cast<int>(blockIdx.x) * groups;
  if (first >= n_items) return;  // uniform: the whole block
  struct Loads {
    u32x4_t w[kSteps][2];
    u32x4_t s;
  };
  const uint32_t w_total = 2u * static_cast<uint32_t>(p.mi) * row_bytes;
  const uint32_t s_total = 2u * static_cast<uint32_t>(p.mi) * srow_bytes;
  // The item whose loads come next: its number, entry and tile.
  int next = first + group, next_e = next / tiles, next_t = next - next_e * tiles;
  const auto load_w = [&](Loads &l, const Entry &en, bool in, int i)
      __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(rfl_ptr(en.packed), in ? w_total : 0u);
    const uint32_t row = static_cast<uint32_t>(next_t) * 8u;
    l.w[i][0] = load16(wr, w_voff[i], row * row_bytes);
    l.w[i][1] = load16(wr, w_voff[i] + 16, row * row_bytes);
  };
  const auto load_s = [&](Loads &l, const Entry &en, bool in) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(rfl_ptr(en.scales), in ? s_total : 0u);
    l.s = load_scales<kTail>(sr, s_voff, static_cast<uint32_t>(next_t) * 8u * srow_bytes,
                             p.hidden - s_k);
  };
  const auto advance = [&]() __attribute__((always_inline)) {
    next += stride;
    next_t += stride;
    while (next_t >= tiles) {
      next_t -= tiles;
      ++next_e;
    }
  };
  Loads l[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d) {
    const bool in = next < n_items;  // past the end: buffers of no bytes
    const Entry en = rt.entry[in ? next_e : 0];
    load_s(l[d], en, in);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) load_w(l[d], en, in, i);
    advance();
  }

  // 4. The rows as FP16, each brought to its largest magnitude's power of two.
  uint32_t top = 0;
  for (int w = 0; w < ways; ++w) top = max(top, s_top[group * ways + w][r16]);
  const int shift = shift_of(static_cast<int>(top >> 7));
  f16x8_t x[kSteps][8];
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) x[i][j] = half8_of(xr[i][j], shift);

  // 5. Items, kDepth in flight: an item's step is refilled as soon as it has been multiplied.
  const auto finish = [&](int b, int item) __attribute__((always_inline)) {
    const f32x4_t *part = red + (b * kWaves + group * ways) * 64 + lane;
    f32x4_t sum = part[0];
    for (int w = 1; w < ways; ++w) sum += part[w * 64];
    const int e = item / tiles, tile = item - e * tiles;
    const float s2 = rt.entry[e].scale2;
    float o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      // gate or up, tile row 4 kb + u
      const float v = __builtin_amdgcn_ldexpf(sum[u], -shift) * s2;
      o[u] = moe::fp8_swiglu(v, __shfl_xor(v, 32, 64), p.limit);
    }
    const int slot = rt.slot_of[e * 16 + r16];
    uint32_t lo, hi;
    if (p.act_half) {
      _Float16 h[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        h[u] = static_cast<_Float16>(__builtin_amdgcn_ldexpf(o[u], p.act_shift));
      lo = __builtin_bit_cast(uint32_t, f16x2_t{h[0], h[1]});
      hi = __builtin_bit_cast(uint32_t, f16x2_t{h[2], h[3]});
    } else {
      lo = moe::pack_bf16x2(o[0], o[1]);
      hi = moe::pack_bf16x2(o[2], o[3]);
      uint32_t m = max(max(lo & 0x7FFFu, (lo >> 16) & 0x7FFFu),
                       max(hi & 0x7FFFu, (hi >> 16) & 0x7FFFu));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16, 64)));
      if (kb == 0 && slot >= 0)
        p.act_exp[static_cast<int64_t>(slot) * tiles + tile] = static_cast<uint8_t>(m >> 7);
    }
    if (kb < 2 && slot >= 0)
      *reinterpret_cast<uint2 *>(p.act + static_cast<int64_t>(slot) * p.mi + 8 * tile + 4 * kb) =
          make_uint2(lo, hi);
  };
  for (int item0 = first + group; item0 - group < n_items; item0 += kBatch * stride) {
#pragma unroll 1
    for (int b0 = 0; b0 < kBatch; b0 += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int b = b0 + d;
        const bool mine = item0 + b * stride < n_items;  // wave-uniform
        const bool in = next < n_items;
        const Entry en = rt.entry[in ? next_e : 0];
        f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        uint32_t scales[4];
        spread_scales(l[d].s, scales);
        load_s(l[d], en, in);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          if (mine) step_product(l[d].w[i], scales[i], x[i], acc);
          load_w(l[d], en, in, i);
        }
        advance();
        if (mine) red[(b * kWaves + wave) * 64 + lane] = acc[0] + acc[1];
      }
    }
    __syncthreads();
    for (int b = kw; b < kBatch; b += ways)
      if (item0 + b * stride < n_items) finish(b, item0 + b * stride);
    __syncthreads();
  }
}

// ------------------------------------------------------------- kernel 2: down and combine

constexpr int kPiece = 64 * 2 + 16;      // a staged row's 64 k, padded
constexpr int kStaged = 4 * kPiece;      // its 256 k

// Row r16 in an entry: its coefficient p_slot scale2 / 2^shift, and its staged row (-1: none).
struct Column {
  float coef;
  int32_t pos;
};

constexpr int kUnit = 4;  // steps of a unit: their scales are 64 bytes of a row, one load

// A block owns tile_rows output columns and sweeps every entry's weight rows for them. Units of
// up to 4 steps of K of an entry are dealt round-robin to its waves, each step refilled with the
// next unit's as soon as it has been multiplied; column r16 of a product is row r16, its
// activation the row's slot in the entry.
template <int kCap, bool kHalf, bool kTail>
__global__ __launch_bounds__(kThreads, kCap <= 2 ? 4 : 2) void few_down_kernel(FewArgs p) {
  static_assert(kCap % 2 == 0, "a load stages two rows");
  constexpr int kX = kCap / 2;  // loads of a pair's activations
  constexpr int kStageBytes = kCap * kStaged > 1024 ? kCap * kStaged : 1024;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves][kStageBytes];
  __shared__ uint32_t s_exp[kHalf ? 1 : kMaxIds];
  const int n_ids = p.rows * p.top_k;
  Column *column = reinterpret_cast<Column *>(dyn);  // [n_ids][16]
  Routing rt(dyn + n_ids * 16 * sizeof(Column), n_ids, p.num_experts);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, kb = lane >> 4;
  const int n0 = blockIdx.x * p.tile_rows;

  // 1. The routing; BF16 activations: each slot's largest exponent.
  if (tid < n_ids) {
    rt.id[tid] = p.ids[tid];
    if (!kHalf) s_exp[tid] = 0;
  }
  rt.begin<kCap>(p, Routing::fetch(p, p.down, tid), tid);
  __syncthreads();
  if (!kHalf) {
    const int per = p.mi / 64;  // 8-byte pieces of a slot's exponents
    const uint2 *exps = reinterpret_cast<const uint2 *>(p.act_exp);
    for (int q = tid; q < n_ids * per; q += kThreads) {
      const uint2 v = exps[q];
      const auto top = [](uint32_t u) {
        return max(max(u & 255u, (u >> 8) & 255u), max((u >> 16) & 255u, u >> 24));
      };
      atomicMax(&s_exp[q / per], max(top(v.x), top(v.y)));
    }
  }
  rt.group<kCap>(p, p.down, tid);
  __syncthreads();
  const int n_live = rt.live();
  for (int q = tid; q < n_live * 16; q += kThreads) {
    const int slot = rt.slot_of[q];
    Column c = {0.0f, -1};
    if (slot >= 0) {
      const int shift = kHalf ? p.act_shift : shift_of(static_cast<int>(s_exp[slot]));
      c.coef = __builtin_amdgcn_ldexpf(p.wts[slot] * rt.entry[q >> 4].scale2, -shift);
      c.pos = rt.pos_of[slot];
    }
    column[q] = c;
  }

  // 2. Units, one in flight beside the one that is multiplied.
  const int steps = (p.mi + kStepK - 1) / kStepK, per_entry = (steps + kUnit - 1) / kUnit;
  const int n_units = n_live * per_entry;
  const uint32_t row_bytes = static_cast<uint32_t>(p.mi) / 2;
  const uint32_t srow_bytes = static_cast<uint32_t>(p.mi) / 16;
  const uint32_t w_row = static_cast<uint32_t>(n0 + r16);
  const bool row_in = r16 < p.tile_rows && n0 + r16 < p.hidden;
  const uint32_t w_total = static_cast<uint32_t>(p.hidden) * row_bytes;
  const uint32_t s_total = static_cast<uint32_t>(p.hidden) * srow_bytes;
  const uint32_t w_lane = w_row * row_bytes + 32u * kb;
  const uint32_t s_lane = w_row * srow_bytes + 16u * kb;  // lane kb: the scales of step kb
  const __amdgpu_buffer_rsrc_t a_rsrc =
      make_rsrc(p.act, static_cast<uint32_t>(n_ids) * static_cast<uint32_t>(p.mi) * 2u);
  struct Loads {
    u32x4_t w[kUnit][2], x[kUnit][kX];
    u32x4_t s;
  };
  // The unit whose loads come next, and the one that is multiplied: entry and first k.
  struct At {
    int unit, e, k0;
  };
  const auto advance = [&](At &a) __attribute__((always_inline)) {
    a.unit += kWaves;
    a.k0 += kWaves * kUnit * kStepK;
    while (a.k0 >= per_entry * kUnit * kStepK) {
      a.k0 -= per_entry * kUnit * kStepK;
      ++a.e;
    }
  };
  At now = {wave, wave / per_entry, wave % per_entry * kUnit * kStepK}, next = now;
  struct Want {  // what a unit's loads need from LDS
    Entry en;
    int slot[kX];
  };
  const auto want = [&]() __attribute__((always_inline)) {
    const int e = next.unit < n_units ? next.e : 0;
    Want w;
    w.en = rt.entry[e];
#pragma unroll
    for (int q = 0; q < kX; ++q) w.slot[q] = rt.list[e * kCap + 2 * q + (lane >> 5)];
    return w;
  };
  const auto load_s = [&](Loads &l, const Want &w) __attribute__((always_inline)) {
    const bool in = next.unit < n_units;  // past the end: buffers of no bytes
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(rfl_ptr(w.en.scales), in ? s_total : 0u);
    const int left = p.mi - next.k0 - kb * kStepK;
    l.s = load_scales<kTail>(sr, row_in && left > 0 ? s_lane : kNoLoad,
                             static_cast<uint32_t>(next.k0) / 16, row_in ? left : 0);
  };
  const auto load = [&](Loads &l, const Want &w, int i) __attribute__((always_inline)) {
    const bool in = next.unit < n_units;
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(rfl_ptr(w.en.packed), in ? w_total : 0u);
    const int k0 = next.k0 + i * kStepK;
    const uint32_t wv = row_in && k0 + 64 * kb < p.mi ? w_lane : kNoLoad;  // mi: a multiple of 64
    l.w[i][0] = load16(wr, wv, static_cast<uint32_t>(k0) / 2);
    l.w[i][1] = load16(wr, wv + 16, static_cast<uint32_t>(k0) / 2);
    const bool x_in = in && k0 + 8 * (lane & 31) < p.mi;
#pragma unroll
    for (int q = 0; q < kX; ++q) {
      const uint32_t off = static_cast<uint32_t>(w.slot[q] * p.mi + 8 * (lane & 31)) * 2u;
      l.x[i][q] = load16(a_rsrc, x_in && w.slot[q] >= 0 ? off : kNoLoad,
                         static_cast<uint32_t>(k0) * 2u);
    }
  };
  Loads l;
  {
    const Want w = want();
    load_s(l, w);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) load(l, w, i);
    advance(next);
  }
  __syncthreads();  // the columns

  uint8_t *mine = stage[wave];
  f32x4_t total = {0.f, 0.f, 0.f, 0.f};
  while (now.unit < n_units) {
    const Want w = want();
    const Column c = column[now.e * 16 + r16];
    uint32_t scales[4];
    spread_scales(l.s, scales);
    load_s(l, w);
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      // The staged rows: lane l's 8 values are k 8 (l % 32) of row 2 q + l / 32.
#pragma unroll
      for (int q = 0; q < kX; ++q) {
        f16x8_t v;
        if (kHalf) {
          v = __builtin_bit_cast(f16x8_t, l.x[i][q]);
        } else {
          const int slot = rt.list[now.e * kCap + 2 * q + (lane >> 5)];
          v = half8_of(l.x[i][q], slot >= 0 ? shift_of(static_cast<int>(s_exp[slot])) : 0);
        }
        *reinterpret_cast<f16x8_t *>(mine + (2 * q + (lane >> 5)) * kStaged +
                                     ((lane & 31) >> 3) * kPiece + 16 * (lane & 7)) = v;
      }
      const uint8_t *src = mine + max(c.pos, 0) * kStaged + kb * kPiece;
      f16x8_t x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = *reinterpret_cast<const f16x8_t *>(src + 16 * j);
      if (now.k0 + i * kStepK < p.mi) step_product(l.w[i], scales[i], x, acc);  // wave-uniform
      load(l, w, i);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float sum = fmaf(c.coef, acc[0][u] + acc[1][u], total[u]);
      total[u] = c.pos >= 0 ? sum : total[u];  // a select: another row's NaN stays out
    }
    advance(now);
    advance(next);
  }

  // 3. The waves' sums in order, the shared term, the output.
  f32x4_t *red = reinterpret_cast<f32x4_t *>(stage[wave]);
  red[lane] = total;
  __syncthreads();
  if (wave == 0 && r16 < p.rows && 4 * kb < p.tile_rows) {
    f32x4_t sum = total;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += reinterpret_cast<const f32x4_t *>(stage[w])[lane];
    const int col = n0 + 4 * kb;
    if (col < p.hidden) {
      if (p.shared != nullptr) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p.shared + r16 * p.ld_shared + col);
        sum[0] += __uint_as_float(v.x << 16);
        sum[1] += __uint_as_float(v.x & 0xFFFF0000u);
        sum[2] += __uint_as_float(v.y << 16);
        sum[3] += __uint_as_float(v.y & 0xFFFF0000u);
      }
      *reinterpret_cast<uint2 *>(p.out + r16 * p.ld_out + col) =
          make_uint2(moe::pack_bf16x2(sum[0], sum[1]), moe::pack_bf16x2(sum[2], sum[3]));
    }
  }
}

// ---------------------------------------------------------------------------------- host

constexpr float kHalfLimit = 128.0f;
constexpr int kRouterExperts = 512;  // 8 logits per lane

template <auto kKern>
struct Kern {
  static constexpr auto value = kKern;
};

// Workspace: activations, their exponents, ids, weights, each 16-byte aligned.
struct Layout {
  int64_t act_exp, ids, wts, bytes;
};

Layout layout_of(int64_t ids, int64_t mi) {
  const auto up = [](int64_t v) { return (v + 15) / 16 * 16; };
  Layout l;
  l.act_exp = up(ids * mi * 2);
  l.ids = l.act_exp + up(ids * (mi / 8));
  l.wts = l.ids + up(ids * 4);
  l.bytes = l.wts + up(ids * 4);
  return l;
}

// The steps of K a wave holds and the waves that share an item's K.
struct Split {
  int per_wave, ways;
};

// Steps per wave and waves per item: the fewest empty steps; among equals, the most waves.
Split split_of(int32_t hidden) {
  const int steps = (hidden + kStepK - 1) / kStepK;
  Split best = {kMaxPerWave, kWaves};
  for (int ways = kWaves; ways >= 1; ways /= 2) {
    const int per = (steps + ways - 1) / ways;
    if (per <= kMaxPerWave && per * ways < best.per_wave * best.ways) best = {per, ways};
  }
  return best;
}

template <int kRoute, bool kTail>
int launch_gate_up(const FewArgs &p, void *stream) {
  const Split s = split_of(p.hidden);
  const int64_t groups = kWaves / s.ways;
  const int64_t items = static_cast<int64_t>(p.rows) * p.top_k * (p.mi / 8);
  const int64_t blocks = std::min<int64_t>((items + groups - 1) / groups, kCus);
  const int lds = kRedBytes + Routing::bytes(p.rows * p.top_k, p.num_experts, kMaxRows);
  const auto go = [&](auto kern) -> int {
    constexpr auto k = decltype(kern)::value;
    MOE_REQUIRE_CODE(moe::allow_lds<k>(kRedBytes + Routing::bytes(kMaxIds, kTable, kMaxRows)),
                     MOE_ELAUNCH, "layer_few: LDS was refused");
    return moe::launch("moe_w4a16_layer_few", k, dim3(static_cast<unsigned>(blocks)),
                       dim3(kThreads), static_cast<size_t>(lds), stream, p, s.ways);
  };
  if (s.per_wave == 1) return go(Kern<few_gate_up_kernel<1, kRoute, kTail>>{});
  if (s.per_wave == 2) return go(Kern<few_gate_up_kernel<2, kRoute, kTail>>{});
  if (s.per_wave == 3) return go(Kern<few_gate_up_kernel<3, kRoute, kTail>>{});
  return go(Kern<few_gate_up_kernel<4, kRoute, kTail>>{});
}

// Weight rows per block: those that give the busiest CU the fewest (6144 columns: 512 blocks of
// 12, two per CU; with 384 blocks of 16, half of the CUs took twice as long: 71 and 134 us at
// 8 rows); among equals the most.
int tile_rows_of(int32_t hidden) {
  int best = 16;
  int64_t least = INT64_MAX;
  for (int rows = 16; rows >= 4; rows -= 4) {
    const int64_t blocks = (hidden + rows - 1) / rows;
    const int64_t busiest = (blocks + kCus - 1) / kCus * rows;
    if (busiest < least) {
      least = busiest;
      best = rows;
    }
  }
  return best;
}

constexpr int down_lds(int ids, int num_experts, int cap) {
  return ids * 16 * static_cast<int>(sizeof(Column)) + Routing::bytes(ids, num_experts, cap);
}

template <bool kHalf, bool kTail>
int launch_down(const FewArgs &p, void *stream) {
  const dim3 grid(static_cast<unsigned>((p.hidden + p.tile_rows - 1) / p.tile_rows));
  const int ids = p.rows * p.top_k;
  const auto go = [&](auto kern, int cap) -> int {
    constexpr auto k = decltype(kern)::value;
    const int lds = down_lds(ids, p.num_experts, cap);
    MOE_REQUIRE_CODE(moe::allow_lds<k>(down_lds(kMaxIds, kTable, 8)), MOE_ELAUNCH,
                     "layer_few: LDS was refused");
    return moe::launch("moe_w4a16_layer_few", k, grid, dim3(kThreads), static_cast<size_t>(lds),
                       stream, p);
  };
  // Rows staged at a time, by how many an expert has on average over all experts: an expert with
  // more is swept again, empty rows cost registers (fewer blocks per CU) and loads. us of the whole
  // layer for 2 / 4 / 8 rows: 8 rows of 8 among 256 experts 233.6 / 236.1 / 258.1, 16 rows of 8
  // among 64 54.8 / 51.4 / 54.5, 16 rows of 2 among 8 53.2 / 47.6 / 49.6, 16 rows of 8 among 8
  // (4 / 8 rows) 78.6 / 69.0.
  if (2 * ids <= p.num_experts || p.rows <= 2)
    return go(Kern<few_down_kernel<2, kHalf, kTail>>{}, 2);
  if (ids <= 4 * p.num_experts || p.rows <= 4)
    return go(Kern<few_down_kernel<4, kHalf, kTail>>{}, 4);
  return go(Kern<few_down_kernel<8, kHalf, kTail>>{}, 8);
}

}  // namespace

extern "C" int64_t moe_few_workspace_bytes(int32_t rows, int32_t top_k, int32_t mi) {
  if (rows <= 0 || top_k <= 0 || rows > kMaxRows ||
      static_cast<int64_t>(rows) * top_k > kMaxIds || mi <= 0 || mi % 64 != 0 ||
      mi > MOE_FEW_MAX_MI)
    return 0;
  return layout_of(static_cast<int64_t>(rows) * top_k, mi).bytes;
}

extern "C" int moe_w4a16_layer_few(
    const uint16_t *x, int64_t ld_x, const float *logits, int64_t ld_logits, const float *bias,
    float routed_scale, int32_t renormalize, int32_t *topk_ids, float *topk_weights,
    const uint64_t *gate_up_packed, const uint64_t *gate_up_scales, const float *gate_up_scale2,
    const uint64_t *down_packed, const uint64_t *down_scales, const float *down_scale2,
    int32_t num_experts, const uint16_t *shared, int64_t ld_shared, uint16_t *out, int64_t ld_out,
    int32_t rows, int32_t top_k, int32_t hidden, int32_t mi, float limit, void *workspace,
    int64_t workspace_bytes, void *stream) {
  moe::clear_error();
  constexpr const char *name = "layer_few";
  MOE_REQUIRE(rows >= 0 && rows <= kMaxRows, "%s: rows must be in [0, %d] (got %d)", name, kMaxRows,
              rows);
  MOE_REQUIRE(top_k >= 1 && static_cast<int64_t>(rows) * top_k <= kMaxIds,
              "%s: need top_k >= 1 and rows * top_k <= %d", name, kMaxIds);
  MOE_REQUIRE(num_experts >= 1, "%s: num_experts must be >= 1", name);
  MOE_REQUIRE(hidden > 0 && hidden % 64 == 0 && hidden <= MOE_FEW_MAX_HIDDEN,
              "%s: hidden must be a positive multiple of 64, at most %d (got %d)", name,
              MOE_FEW_MAX_HIDDEN, hidden);
  MOE_REQUIRE(mi > 0 && mi % 64 == 0 && mi <= MOE_FEW_MAX_MI,
              "%s: mi must be a positive multiple of 64, at most %d (got %d)", name, MOE_FEW_MAX_MI,
              mi);
  MOE_REQUIRE(limit > 0.0f, "%s: limit must be > 0", name);
  MOE_REQUIRE(ld_x >= hidden && ld_x % 8 == 0 && ld_x < (1 << 24),
              "%s: ld_x must be >= hidden, a multiple of 8 and below 2^24", name);
  MOE_REQUIRE(ld_out >= hidden && ld_out % 4 == 0 &&
                  (shared == nullptr || (ld_shared >= hidden && ld_shared % 4 == 0)),
              "%s: ld_out and ld_shared must be >= hidden and multiples of 4", name);
  if (logits != nullptr) {
    MOE_REQUIRE(num_experts <= MOE_ROUTER_MAX_EXPERTS && top_k <= MOE_ROUTER_MAX_TOPK,
                "%s: the router takes at most %d experts and top_k %d", name,
                MOE_ROUTER_MAX_EXPERTS, MOE_ROUTER_MAX_TOPK);
    MOE_REQUIRE(ld_logits >= num_experts, "%s: ld_logits must be >= num_experts", name);
    MOE_REQUIRE(routed_scale > -INFINITY && routed_scale < INFINITY,
                "%s: routed_scale must be finite", name);
  }
  if (rows == 0) return MOE_OK;
  MOE_REQUIRE(x && out && gate_up_packed && gate_up_scales && gate_up_scale2 && down_packed &&
                  down_scales && down_scale2 && workspace &&
                  (logits || (topk_ids && topk_weights)),
              "%s: a required pointer is NULL", name);
  MOE_REQUIRE(moe::aligned16(x) && moe::aligned16(workspace),
              "%s: x and the workspace must be 16-byte aligned", name);
  MOE_REQUIRE(((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(shared)) & 7u) == 0,
              "%s: out and shared must be 8-byte aligned", name);
  const Layout l = layout_of(static_cast<int64_t>(rows) * top_k, mi);
  MOE_REQUIRE_CODE(workspace_bytes >= l.bytes, MOE_ECAPACITY,
                   "%s: the workspace has %lld bytes, %lld are needed", name,
                   static_cast<long long>(workspace_bytes), static_cast<long long>(l.bytes));
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  FewArgs p = {};
  p.x = x;
  p.bias = bias;
  p.ids_out = topk_ids ? topk_ids : reinterpret_cast<int32_t *>(ws + l.ids);
  p.wts_out = topk_weights ? topk_weights : reinterpret_cast<float *>(ws + l.wts);
  p.ids = p.ids_out;
  p.wts = p.wts_out;
  p.gate_up = {gate_up_packed, gate_up_scales, gate_up_scale2, down_packed, down_scales};
  p.down = {down_packed, down_scales, down_scale2, gate_up_packed, gate_up_scales};
  p.shared = shared;
  p.out = out;
  p.act = reinterpret_cast<uint16_t *>(ws);
  p.act_exp = ws + l.act_exp;
  p.ld_x = ld_x;
  p.ld_logits = ld_logits;
  p.ld_shared = ld_shared;
  p.ld_out = ld_out;
  p.rows = rows;
  p.top_k = top_k;
  p.num_experts = num_experts;
  p.hidden = hidden;
  p.mi = mi;
  p.renormalize = renormalize;
  p.routed_scale = routed_scale;
  p.limit = limit;
  p.tile_rows = tile_rows_of(hidden);
  // |act| <= limit max(limit, 0.2785): the gate is clamped from above only, and silu's least value
  // is -0.27846. The power of two that brings this bound to [2^14, 2^15) leaves FP16 its 11 bits
  // down to 2^-28 of it. A wider limit leaves activations in BF16, with a power of two per slot.
  p.act_half = limit <= kHalfLimit;
  if (p.act_half) {
    const double l = limit;
    int exponent;
    std::frexp(l * std::max(l, 0.2785), &exponent);  // the bound is below 2^exponent
    p.act_shift = std::min(15 - exponent, 120);
  }
  const bool in_kernel = logits != nullptr && num_experts <= kRouterExperts;
  if (in_kernel) {
    p.logits = logits;
  } else if (logits != nullptr) {
    const int rc = moe_router_topk(logits, ld_logits, rows, num_experts, bias, top_k, routed_scale,
                                   renormalize, p.ids_out, p.wts_out, stream);
    if (rc != MOE_OK) return rc;
  }
  const bool few = num_experts <= 256;
  int rc;
  if (hidden % kStepK != 0)
    rc = in_kernel ? launch_gate_up<8, true>(p, stream) : launch_gate_up<0, true>(p, stream);
  else if (in_kernel)
    rc = few ? launch_gate_up<4, false>(p, stream) : launch_gate_up<8, false>(p, stream);
  else
    rc = launch_gate_up<0, false>(p, stream);
  if (rc != MOE_OK) return rc;
  if (mi % kStepK != 0)
    return p.act_half ? launch_down<true, true>(p, stream) : launch_down<false, true>(p, stream);
  return p.act_half ? launch_down<true, false>(p, stream) : launch_down<false, false>(p, stream);
}
