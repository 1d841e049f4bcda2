// Which kernel a block-scaled FP8 product runs, with how many K splits, on how many
// columns: host arithmetic on the shape alone, free of HIP so that it compiles anywhere.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <utility>

namespace gwb {

constexpr int kCus = 256;             // compute units of an MI355X
constexpr int kTail = kCus * 3 / 8;   // 256 x 256 tiles of a last round that smaller tiles do sooner

// The kernel of a shape, its K splits, the columns of its first launch (kTile256: the rest
// go to 128 x 128 tiles; N otherwise) and its threads in all (exact: float32 outputs).
struct GemmPlan {
  int kernel, splits;
  int64_t threads, wide;
};
enum { kRows8, kRows8Deep, kRows8Narrow, kRows16, kRows16Deep, kRows16Narrow, kRows32, kRows32Deep, kRows32Narrow,
       kTile64, kTile64x128, kTile64x192, kTile128, kTile128Deep, kTile128x192, kTile256x192, kTile256 };

// One 256 x 256 tile per compute unit at a time: columns that would leave the last round
// mostly empty go to 128 x 128 tiles (512 rows of 34816: 156 -> 147 us). Whole tile columns
// go, so these can hold more tiles than the last round (2087 x 24576: 99 and not 96), or all
// of them (more tile rows than units). Returns the columns that stay, N where a split gains
// nothing, and the time of both launches in us for 40 stages (see fp8_gemm_plan).
inline std::pair<int64_t, int64_t> fp8_gemm_split256(int64_t M, int64_t N) {
  const int64_t gx = (M + 255) / 256, gy = (N + 255) / 256, all = gx * gy, full = all / kCus * kCus;
  const int64_t keep = full / gx, left = (gy - keep) * gx;
  const std::pair<int64_t, int64_t> whole{N, (all + kCus - 1) / kCus * 75};
  if (keep == 0 || left == 0 || all - full > kTail) return whole;
  const int64_t tail = left <= kTail ? 35 : (4 * left + 2 * kCus - 1) / (2 * kCus) * 53;
  const int64_t us = (keep * gx + kCus - 1) / kCus * 75 + tail;
  return us < whole.second ? std::pair<int64_t, int64_t>{keep * 256, us} : whole;
}

// By the rows of x and the tiles they make; each line's alternative measured beside it, in
// us: bf16 out, float32 scales, three weights in turn (so weights up to some 80 MB come from
// the 256 MB cache before memory: 128 x 5120 x 5120 takes 15 so and 19 from memory). The
// round times are those of 40 stages, taken in proportion to K; E8M0 scales (up to 10 %
// faster on large tiles) and float32 outputs (slower: the widening) have none of their own.
inline GemmPlan fp8_gemm_plan(int64_t M, int64_t N, int64_t K, bool exact) {
  const int64_t KB = (K + 127) / 128;
  const auto tiles = [&](int64_t b) { return ((M + b - 1) / b) * ((N + b - 1) / b); };
  const auto over = [](int64_t t) { return (t + kCus - 1) / kCus; };
  // the columns of up to 64 rows in one tile, a round of 40 stages in us: 28 with 64 x 128 tiles,
  // 36 with 64 x 192, 34 with 512 of 64 x 64, 19 with up to 256 of them (64 x 34816 x 5120, 272,
  // 182 and 544 tiles: 54, 38 and 50; 64 x 24576 x 5120, 192, 128 and 384: 29, 36 and 35)
  const auto rounds64 = [](int64_t t) {
    const int64_t rem = t % (2 * kCus);
    return t / (2 * kCus) * 34 + (rem == 0 ? 0 : rem <= kCus ? 19 : 34);
  };
  const int64_t wide128 = (N + 127) / 128, wide192 = (N + 191) / 192;
  const int64_t by64w = std::min(over(wide128) * 28, over(wide192) * 36);
  // few tiles: K splits of at least 8 stages, if the rounds they save are more than the second
  // launch and its bytes, all in us (64 x 5120 x 17408, 80 tiles: 26 with 3 splits, 32 with 4, 52
  // with none; 128 x 5120 x 5120, 160 tiles: 16 with 3, 17 with 2; 131 x 4100 x 2064, 195 tiles: 10
  // with none, 13 with 2)
  const auto split = [&](int64_t t, int64_t most, const auto& rounds) {
    std::pair<int, double> best{1, (double)rounds(t) * (double)KB / 40};
    for (int64_t s = 2; s <= KB / 8 && t * s <= most; ++s) {
      const double us = (double)rounds(t * s) * (double)((KB + s - 1) / s) / 40 + 2.5 +
                        (double)s * (double)M * (double)N * 8 / 5e6;
      if (us < best.second) best = {(int)s, us};
    }
    return best;
  };
  const auto tile64 = [&] {
    const int s = split(tiles(64), 2 * kCus, rounds64).first;
    return GemmPlan{kTile64, s, tiles(64) * s * 256, N};
  };
  const auto wide64 = [&] {
    return over(wide128) * 28 == by64w ? GemmPlan{kTile64x128, 1, wide128 * 256, N} : GemmPlan{kTile64x192, 1, wide192 * 256, N};
  };
  if (M <= 32) {
    // blocks of 32 columns; fewer than compute units: 8 wavefronts on K instead of 4 (1 x
    // 5120 x 17408: 19 and 22; 8 x 34816 x 5120, 1088 blocks: 36 and 31); where 16 columns make
    // at most a block per unit, those (1 x 4096 x 14336: 11.3 and 14.3; 16 x 2048 x 2048: 3.9
    // and 4.7; but 1 x 5120 x 17408, 320 blocks of 16: 20.8 and 18.6)
    const int64_t blocks = (N + 31) / 32;
    const bool deep = blocks < kCus && KB >= 16, narrow = deep && (N + 15) / 16 <= kCus;
    // 17 to 32 rows on a long K (32 x 5120 x 17408: tiles 22, rows 27; 20 x 4096 x 4096: 10 and 8)
    if (M > 16 && deep && !narrow && KB >= 64) return tile64();
    // or wide weights: 9 us for every 256 blocks of 40 stages (32 x 34816 x 5120, 1088 blocks: 42,
    // with 64 x 192 tiles 35; 32 x 17408 x 5120, 544 blocks: 26, 64 x 128 tiles 24)
    if (M > 16 && !exact && by64w < over(blocks) * 9) return wide64();
    const int kernel = (M <= 8 ? kRows8 : M <= 16 ? kRows16 : kRows32) + (narrow ? 2 : deep ? 1 : 0);
    return GemmPlan{kernel, 1, narrow ? (N + 15) / 16 * 512 : blocks * (deep ? 512 : 256), N};
  }
  // 128 rows are half empty below 65 (64 x 34816 x 5120: 50 us with 64 x 64 tiles, 56 with 128 x
  // 128; float32 out 60 and 117)
  if (M <= 64) return !exact && by64w < rounds64(tiles(64)) ? wide64() : tile64();
  // Big tiles hold a compute unit each, two 128 x 128 ones share it. By the rounds each shape
  // takes: one round of 40 stages is 75 us with 256 x 256 tiles, 64 with 256 x 192, 39 with
  // 128 x 192, 53 with 512 of 128 x 128, 29 with up to 256 of them. (256 x 34816 x 5120, 136
  // tiles of the first, 182 of the second and 544 of 128 x 128: 82, 69 and 105; 2048 x 5120 x
  // 5120, 160, 216 and 640: 63, 59 and 77; 2048 x 4096 x 4096, 128, 176 and 512: 55, 47 and 43;
  // 384 x 34816 x 5120, 272, 364 and 816: 122, 124 and 113; 3000 x 5120 x 5120, 240, 324 and
  // 960: 76, 114 and 100; 1024 x 5120 x 5120, 216 of 128 x 192 and 320 of 128 x 128: 40 and 44; 128 x
  // 34816 x 5120, 182 and 272: 47 and 65)
  if (!exact) {
    const int64_t t128 = tiles(128) % (2 * kCus), n192 = (N + 191) / 192;
    const int64_t by128 = tiles(128) / (2 * kCus) * 53 + (t128 == 0 ? 0 : t128 <= kCus ? 29 : 53);
    const auto [n256, by256] = fp8_gemm_split256(M, N);
    const int64_t wide = (M + 255) / 256 * n192, flat = (M + 127) / 128 * n192;
    const int64_t least = std::min({by128, by256, over(wide) * 64, over(flat) * 39});
    if (by256 == least && by256 < by128) return GemmPlan{kTile256, 1, tiles(256) * 512, n256};
    if (over(wide) * 64 == least && least < by128) return GemmPlan{kTile256x192, 1, wide * 512, N};
    if (over(flat) * 39 == least && least < by128) return GemmPlan{kTile128x192, 1, flat * 512, N};
  }
  // 128 x 128: four stages in LDS while one block fits a unit, else two blocks of two stages
  // (700 x 4096 x 4096, 192 tiles: 24 and 29; 2048 x 4096 x 4096, 512 tiles: 48 and 43)
  if (tiles(128) > kCus) return GemmPlan{kTile128, 1, tiles(128) * 512, N};
  if (tiles(128) >= 160) return GemmPlan{kTile128Deep, 1, tiles(128) * 512, N};
  // a long K splits well with these too (256 x 5120 x 17408, 80 tiles: 40 with 3 splits, 64 x 64
  // tiles 53)
  if (M > 64 && KB >= 64) {
    const auto deep = split(tiles(128), kCus, [&](int64_t t) { return over(t) * 29; });
    if (deep.second < split(tiles(64), 2 * kCus, rounds64).second)
      return GemmPlan{kTile128Deep, deep.first, tiles(128) * deep.first * 512, N};
  }
  return tile64();
}

// The splits' float32 partial sums, for any output type.
inline size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const int s = std::max(fp8_gemm_plan(M, N, K, false).splits, fp8_gemm_plan(M, N, K, true).splits);
  return s > 1 ? (size_t)s * (size_t)M * (size_t)N * sizeof(float) : 0;
}

}  // namespace gwb
