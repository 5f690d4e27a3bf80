// Which tile an FP8 product runs on, and in how many splits of K: host arithmetic only (no HIP),
// so that a host compiler builds it on its own.
#pragma once

#include <cstdint>

namespace moe {

constexpr int kFp8Block = 128;  // values per scale

// The tiles a launch can take: rows x weight rows (SwiGLU: gate and up rows together).
struct Fp8Tile {
  int rows, width;
};
constexpr int kFp8Tiles = 4;

template <bool kSwiglu>
constexpr Fp8Tile fp8_tile(int t) {
  constexpr Fp8Tile kPlain[kFp8Tiles] = {{32, 128}, {64, 128}, {128, 256}, {16, 32}};
  constexpr Fp8Tile kGateUp[kFp8Tiles] = {{32, 256}, {64, 256}, {128, 256}, {192, 256}};
  return kSwiglu ? kGateUp[t] : kPlain[t];
}

struct Fp8Plan {
  int tile, ways;
};

// Which tile, and how many splits of K (SwiGLU with a workspace only): the least of an
// estimate in microseconds, from two measured rates. A CU takes in about 41 KB/us
// (0.0031 us per LDS row of 128 bytes; 64 KB in flight and any tile shape end there), so a
// step costs 0.0031 us x (weight rows + rows); the SwiGLU form's conversions and BF16 products
// cost 0.0205 us per row and step (0.0165 in the two larger tiles; the two-phase loop's rows
// come in 64s), the FP8 products stay below the loads. An item costs 2 us more (its first
// loads; 2.5 in the plain 256 x 128 tile), 0.7 where two blocks fit a CU and one loads while the
// other starts, 1 where they also join slice sums (whose steps of four slices take 0.9). The
// two-stage SwiGLU tile takes 1.1 times its step and 1.5 us an item (70 slots over 107 experts,
// width 160 x K 3728: 35.6 us, 26.3 with three stages of 64 rows). A
// split adds a launch (6 with its wait) and writes and reads its sums, at 2.5 and 4 TB/s. HBM
// bounds all of it (the experts' weights at 6 TB/s); a tenth of the estimate stands for what
// does not run beside that. Over the 400 random sizes it was fitted to, the choice is 1.2 to 2.4 %
// slower than the best (geometric mean); over 400 fresh ones 1.4 % (dense), 2.3 (dense SwiGLU),
// 2.4 (grouped) and 4.1 (grouped SwiGLU), 1.32 times at worst (grouped, 148 slots over 88
// experts, 288 x 1616: 14.2 us on 32 x 16, 10.7 on 128 x 32).
//
// Both sides, measured in us (ranges: two machines), the one taken marked (where it is not the
// least, it loses up to 7 %; one matrix of few rows is bound by the host in these calls):
//   plain, N 6144 x K 2048            32 x 16   128 x 32   128 x 64   256 x 128
//     1 row                         9.3-11.1*  10.3-10.7   9.9-10.4  14.4-14.8
//     64 rows                        9.1-10.4  9.7-10.7*  12.7-13.2  15.0-15.4
//     256 rows                           26.2  13.1-13.7  13.5-13.7*      20.3
//     1024 rows                          91.4       35.5  26.6-28.3  23.1-23.4*
//     4096 rows                           352        130  89.8-95.3  68.7-72.0*
//     256 experts, 8 rows each            691   549-557*   552-562    560-561
//     256 experts, 32 rows each          1321   648-704    605-638    607-620*
//     256 experts, 128 rows each         4260       1518       1227   896-904*
//   SwiGLU, width 2048 x K 6144       256 x 32   256 x 64   256 x 128   256 x 192
//     256 experts, 8 rows each     1064-1105  1040-1080*       1126        1114
//     256 experts, 32 rows each    1365-1433  1183-1198*       1210        1232
//     256 experts, 128 rows each        3494   2712-2858  2362-2490  2026-2069*
//     4096 rows                          311    279-284    194-197*    275-278
//   (most of those experts of 128 rows pass 128 by a few: they would take two 128-row tiles)
//   split of K, the same width            1          2          4           8
//     8 rows, 256 x 32                  38.9       23.8       16.5   14.0-14.5*
//     256 rows, 256 x 64                66.5       41.7  29.8-30.6*       36.7
template <bool kSwiglu>
Fp8Plan fp8_plan(int64_t rows, int64_t experts, int64_t n, int64_t k, bool split, int cus) {
  const double used = experts > 0 ? static_cast<double>(experts < rows ? experts : rows) : 1.0;
  const double avg = static_cast<double>(rows) / used;
  const int64_t kb = (k + kFp8Block - 1) / kFp8Block;
  const double weights = used * static_cast<double>(n) * static_cast<double>(k) * (kSwiglu ? 2 : 1);
  Fp8Plan best = {0, 1};
  double best_us = 1e30;
  for (int t = 0; t < kFp8Tiles; ++t) {
    const int bt = fp8_tile<kSwiglu>(t).rows, width = fp8_tile<kSwiglu>(t).width;
    const int bn_out = kSwiglu ? width / 2 : width;
    // Row tiles per expert: exact for one matrix; for experts of `avg` rows on average, one
    // where they seldom pass the tile, else half a tile more than the rows need.
    double tiles = experts > 0 ? (avg <= 0.75 * bt ? 1.0 : avg / bt + 0.5)
                               : static_cast<double>((rows + bt - 1) / bt);
    if (tiles > avg) tiles = avg;
    const double live = experts > 0 ? avg / tiles : (avg < bt ? avg : bt);
    double step = 0.0031 * (width + live);
    if (!kSwiglu && t == 3) step *= 0.9;
    if (kSwiglu) {
      const double rows_done = t != 2 ? live : live > 64 ? 128 : 64;
      const double compute = (t < 2 ? 0.0205 : 0.0165) * rows_done;
      if (compute > step) step = compute;
      if (t == 0) step *= 1.1;
    }
    const double items = used * tiles * static_cast<double>((n + bn_out - 1) / bn_out);
    for (int ways = 1; ways <= (kSwiglu && split ? 8 : 1); ways *= 2) {
      if (ways > 1 && (items * ways > 1.5 * cus || kb < 3 * ways)) break;
      double rounds = static_cast<double>(static_cast<int64_t>((items * ways + cus - 1) / cus));
      if (rounds < 1.0) rounds = 1.0;
      const double start = kSwiglu ? (t == 0 ? 1.5 : 2.0) : t < 2 ? 0.7 : t == 2 ? 2.5 : 1.0;
      double us = rounds * (static_cast<double>((kb + ways - 1) / ways) * step + start);
      us = 0.1 * us + (us < weights / 6e6 ? weights / 6e6 : us);
      if (ways > 1)
        us += 6.0 + static_cast<double>(ways) * rows * n * 8.0 * (1.0 / 2.5e6 + 1.0 / 4e6);
      if (us < best_us) {
        best_us = us;
        best = {t, ways};
      }
    }
  }
  return best;
}

inline int64_t fp8_partial_bytes(const Fp8Plan &plan, int64_t rows, int64_t n) {
  return plan.ways > 1 ? plan.ways * rows * n * 8 : 0;
}

}  // namespace moe
