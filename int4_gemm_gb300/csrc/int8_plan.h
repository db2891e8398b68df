// How the INT8 product is cut into tiles and K parts: plain C++, so that it can be
// asked without a GPU.
#pragma once

#include <stdint.h>

#ifndef Q4_HOST_DEVICE
#ifdef __CUDACC__
#define Q4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define Q4_HOST_DEVICE inline
#endif
#endif

namespace q4 {
namespace {

constexpr int kRows = 128;        // weight rows of a CTA
constexpr int kStageK = 128;      // columns per TMA stage
constexpr int kPanel = 64;        // columns of a row of 128 bytes of f16

// How a product is cut: the kernel's form, tiles and K parts.
struct Plan {
  bool pair;
  int width, num_m, num_n, splits;  // width: tokens of a tile
};
// The cut with the least estimated time.  A form costs a fixed time and so much per
// 64 columns of a tile (measured, ns: 16 x 8192 x 8192 24.3 us with 16-token tiles,
// 28.9 with 64, 39.7 with 128, 48.3 as pairs; 512 x 512 x 512 5.6, 6.9, 7.9 and 10.5;
// 8192 x 28672 x 8192, 47 tiles per pair, 2020 us), and joining the parts of a split K
// takes a time of its own (the same 16 x 8192 x 8192 with two parts: 17.7 us; eight
// parts were never the best).
inline Plan plan_of(int64_t M, int64_t N, int64_t K, int64_t sms) {
  auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int64_t chunks = ceil_div(K, kPanel);
  Plan best = {true, 256, (int)ceil_div(M, 256), (int)ceil_div(N, 256), 1};
  int64_t least = 8000 + ceil_div((int64_t)best.num_m * best.num_n, sms / 2) * chunks * 318;
  const struct { int width, fixed, chunk, join; } forms[] = {
      {16, 4400, 155, 3000}, {32, 4400, 162, 3000}, {64, 5000, 195, 4000}, {128, 5800, 268, 5500}};
  for (const auto& f : forms) {
    const int64_t tiles = ceil_div(M, f.width) * ceil_div(N, kRows);
    for (int splits = 1; splits <= 4 && splits * kStageK < K + kStageK && (splits == 1 || splits * tiles <= sms); splits *= 2) {
      const int64_t cost = f.fixed + (splits > 1 ? f.join : 0) + ceil_div(tiles * splits, sms) * ceil_div(chunks, splits) * f.chunk;
      if (cost < least) {
        least = cost;
        best = {false, f.width, (int)ceil_div(M, f.width), (int)ceil_div(N, kRows), splits};
      }
    }
  }
  return best;
}

// The t-th tile: bands of 4096 tokens, whose codes stay in L2; within a band tokens
// first.
struct Tile {
  int m, n;  // of the tiles of tokens and of weight rows
};
Q4_HOST_DEVICE Tile tile_at(int t, int width, int num_m, int num_n) {
  const int band_m = num_m < 4096 / width ? num_m : 4096 / width;  // (a band has no more tiles than there are)
  const int band_tiles = band_m * num_n;
  const int band = t / band_tiles, r = t - band * band_tiles;
  const int left = num_m - band * band_m, rows = left < band_m ? left : band_m;
  return {band * band_m + r % rows, r / rows};
}

}  // namespace
}  // namespace q4
