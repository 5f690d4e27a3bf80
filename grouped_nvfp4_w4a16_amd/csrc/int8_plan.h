// Which tile an INT8 product runs on: host arithmetic only (no HIP), so that a host compiler
// builds it on its own.
#pragma once

#include <cstdint>

namespace moe {

// Weight rows x rows of a tile (SwiGLU: gate and up rows together).
enum Int8Tile {
  kInt8Tile32x16,
  kInt8Tile32x32,
  kInt8Tile64x32,
  kInt8Tile64x64,
  kInt8Tile128x64,
  kInt8Tile128x128,
  kInt8Tile128x128Pair,  // two blocks per CU
  kInt8Tile128x256,
  kInt8Tile192x256,
  kInt8Tile256x256,
  kInt8Tiles
};

// A tile's shape and its estimate in microseconds: start + for every round of tiles over the
// CUs, round + step x its steps of `slices` x 128 k (pair: of a round in which both blocks of a CU
// have a tile). Fitted to the times of every tile at 260 random sizes (1 to 6000 rows, width and K
// 128 to 8192). The tile with the least estimate is 1.2 % (plain) and 0.6 % (SwiGLU) slower than the
// best of those built, in the geometric mean, 1.13 and 1.25 times at worst; at 300 fresh sizes 0.8
// and 1.1 %, 1.12 and 1.30 times (SwiGLU of two tiles a CU: 128 x 128 taken where pairs are faster).
// Without any one of the tiles the best of the others would be 0.1 to 7 % slower, up to 1.5 times at
// some size. (128 x 128 in pairs gains the plain form 0.03 %, 256 x 128 the SwiGLU form nothing:
// they are not built.)
struct Int8Shape {
  int width, rows, slices;
  float start, round, step, pair;  // step 0: not built
};

constexpr Int8Shape int8_shape(bool swiglu, int tile) {
  constexpr Int8Shape kPlain[kInt8Tiles] = {
      {32, 16, 4, 1.53f, 1.26f, 0.189f, 0.517f}, {32, 32, 4, 1.32f, 1.33f, 0.327f, 0.0f},
      {64, 32, 2, 1.16f, 1.55f, 0.273f, 0.0f},   {64, 64, 2, 0.81f, 2.09f, 0.343f, 0.0f},
      {128, 64, 2, 0.0f, 3.57f, 0.534f, 0.0f},   {128, 128, 2, 0.0f, 4.22f, 0.864f, 0.0f},
      {128, 128, 1, 0.0f, 0.0f, 0.0f, 0.0f},     {128, 256, 1, 0.0f, 5.30f, 0.730f, 0.0f},
      {192, 256, 1, 0.0f, 6.37f, 0.929f, 0.0f},  {256, 256, 1, 0.0f, 7.45f, 1.115f, 0.0f}};
  constexpr Int8Shape kSwiglu[kInt8Tiles] = {
      {32, 16, 4, 0.0f, 0.0f, 0.0f, 0.0f},       {32, 32, 4, 1.34f, 1.57f, 0.320f, 0.0f},
      {64, 32, 2, 1.26f, 1.67f, 0.271f, 0.0f},   {64, 64, 2, 1.00f, 2.06f, 0.338f, 0.0f},
      {128, 64, 2, 0.54f, 3.18f, 0.510f, 0.0f},  {128, 128, 2, 0.0f, 4.56f, 0.808f, 0.0f},
      {128, 128, 1, 0.07f, 4.67f, 0.517f, 1.37f}, {128, 256, 1, 0.0f, 0.0f, 0.0f, 0.0f},
      {192, 256, 1, 0.0f, 0.0f, 0.0f, 0.0f},     {256, 256, 1, 0.0f, 13.2f, 1.088f, 0.0f}};
  return swiglu ? kSwiglu[tile] : kPlain[tile];
}

inline double int8_estimate(bool swiglu, int tile, int64_t m, int64_t n, int64_t k) {
  constexpr int64_t kCus = 256;
  const Int8Shape s = int8_shape(swiglu, tile);
  const int64_t out = swiglu ? s.width / 2 : s.width;
  const int64_t tiles = ((m + s.rows - 1) / s.rows) * ((n + out - 1) / out);
  const int64_t busiest = (tiles + kCus - 1) / kCus;  // tiles of the CU that has the most
  const int64_t span = 128 * s.slices;
  const double steps = static_cast<double>((k + span - 1) / span);
  if (s.pair == 0.0f) return s.start + busiest * (s.round + s.step * steps);
  const double single = busiest % 2 != 0 ? s.round + s.step * steps : 0.0;
  return s.start + (busiest / 2) * (s.round + s.pair * steps) + single;
}

inline Int8Tile int8_tile(bool swiglu, int64_t m, int64_t n, int64_t k) {
  int best = kInt8Tile32x32;
  for (int t = 0; t < kInt8Tiles; ++t) {
    if (int8_shape(swiglu, t).step == 0.0f) continue;
    if (int8_estimate(swiglu, t, m, n, k) < int8_estimate(swiglu, best, m, n, k)) best = t;
  }
  return static_cast<Int8Tile>(best);
}

}  // namespace moe
