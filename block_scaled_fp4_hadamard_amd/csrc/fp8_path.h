// How an 8-bit product runs: which kernel, in how many parts, over which tiles.
// Host-only logic, no HIP types, so that it can be compiled and checked on a
// machine without a GPU.
#pragma once
#include <stdint.h>
#include <initializer_list>

namespace mx {

constexpr int kKB = 128;            // bytes (values) of a row per K step
constexpr int kXcds = 8;
constexpr int kFewWaves = 8;        // waves of a workgroup of the kernel for few rows
constexpr int kMT = 128;            // tile of the kernel for mid-sized products
constexpr int kBT = 256;            // tile of the kernel for large ones
constexpr int kGroup = 32;          // tiles of a group: one for each CU of an XCD

// Tiles are dealt in groups of 4 (M) x 8 (N) to the 8 XCDs, a group to the 32 CUs of one, so that the tiles
// an XCD computes at once share 4 A strips and 8 B strips in its L2; 2 x 16 or 1 x 32 where there are fewer than
// four rows of tiles.
struct BigMap {
  int tiles_m, tiles_n, group_m, groups_m, groups, rounds;
};

enum class Fp8Path { kFew, kMid, kBig };

struct Fp8Plan {
  Fp8Path path;
  int splits;
  BigMap big;
};

inline BigMap fp8_big_map(int64_t M, int64_t N) {
  BigMap map;
  map.tiles_m = (int)((M + kBT - 1) / kBT);
  map.tiles_n = (int)((N + kBT - 1) / kBT);
  map.group_m = map.tiles_m >= 3 ? 4 : map.tiles_m;
  map.groups_m = (map.tiles_m + map.group_m - 1) / map.group_m;
  const int group_n = kGroup / map.group_m;
  map.groups = map.groups_m * ((map.tiles_n + group_n - 1) / group_n);
  map.rounds = (map.groups + kXcds - 1) / kXcds;
  return map;
}

// Into how many parts the K blocks of at most 256 small tiles are split: the least time by what was measured (us).  A
// K block takes 0.55 to 0.68 (fp32 output: 1.0) while every CU has one workgroup at most, 0.8 to 0.9 (1.6) with two;
// the parts' float32 sums cost 0.45 a megabyte, written and read back, and the second launch 4.5.  1000 x 2000 x 2048:
// 14 us whole, 20 in two parts; 400 x 2000 x 8192: 44 whole, 23 in four; 333 x 4096 x 14336: 70 whole, 37 in five.
inline int fp8_splits(int64_t tiles, int64_t nk, double outputs, bool exact) {
  int best = 1;
  double least = 0.0;
  for (const int splits : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64}) {
    const int64_t all = tiles * splits;
    if (splits > 1 && (all > 512 || splits * 2 > nk)) break;
    const double block = exact ? (all <= 256 ? 1.0 : 1.6)
                               : (all <= 256 ? 0.55 + 0.13 * (double)all / 256 : 0.7 + 0.1 * (double)all / 256);
    const double us = block * (double)((nk + splits - 1) / splits) +
                      (splits > 1 ? 4.5 + 0.45e-6 * 4.0 * outputs * splits : 0.0);
    if (splits == 1 || us < least) {
      best = splits;
      least = us;
    }
  }
  return best;
}

// The copies of the two tiled kernels address a tile's rows by 32-bit offsets whose row pitch is a 24-bit factor
// (255 * 2^24 + 128 is below 2^32), and the large kernel a tile's second row of TILE scales by 4 * tile_scales, their
// pitch in floats (0 for line scales, whose pitch is added in 64 bits).  Operands beyond that run on the kernel for few
// rows, 32 rows of A at a time.
//
// By measurement (bf16 output, tile scales, operands in the last-level cache): up to 32 rows of A, reading B once wins
// (16 x 6144 x 4096: 8.4 us against 16; 64 rows, as four row fragments, took 22 against 16).  Above, a K block of a
// full round of the chip costs about 1.67 us in 256 x 256 tiles (one a CU) and 1.15 us in 128 x 128 tiles (two a CU,
// half the work; about 0.7 us with one a CU), and the fewest such times win.  fp32 output (exact) always takes the
// small tiles, whose wave leaves room for the widened operands.
inline Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t tile_scales, bool exact) {
  Fp8Plan plan{Fp8Path::kFew, 1, {}};
  const int64_t lim = int64_t(1) << 24;
  if (M <= 32 || lda >= lim || ldb >= lim || tile_scales >= (int64_t(1) << 30)) return plan;
  const int64_t nk = (K + kKB - 1) / kKB;
  const int64_t tiles = ((M + kMT - 1) / kMT) * ((N + kMT - 1) / kMT);
  plan.path = Fp8Path::kMid;
  if (tiles <= 256) {
    plan.splits = fp8_splits(tiles, nk, (double)M * (double)N, exact);
    return plan;
  }
  if (!exact) {
    plan.big = fp8_big_map(M, N);
    const double rest = (double)(tiles % 512);
    const double mid = 1.15 * (double)(tiles / 512) + (rest == 0 ? 0.0 : rest <= 256 ? 0.7 : 1.15);
    if (1.67 * plan.big.rounds < mid) plan.path = Fp8Path::kBig;
  }
  return plan;
}

// Column fragments of a workgroup in the kernel for few rows.  Every 256 workgroups are a round of the chip, and a
// round's time goes by the operand rows that its workgroups read, B's and A's: with K 14336 (bf16 output) 10, 17, 23
// and 29 us for 1 to 4 fragments and one row of A, 21, 29, 38 and 44 with 32 rows.  No choice reads B faster than HBM
// gives it.  fp32 output takes longer with 3 and 4 fragments, whose widened codes leave room for half the waves.  In
// units of 7 us there, the same weights again and again: 32 x 6144 x 14336 took 41 us in two rounds of one
// fragment and 29 in one of two, 16 x 28672 x 14336 104, 90, 90 and 80 with 1 to 4 fragments, 98, 92, 118 and 107 to
// fp32.  A grid holds fewer than 2^32 threads, which one fragment would pass at N = 2^27 - 1; the ABI refuses N >=
// 2^27.
inline int fp8_few_columns(int64_t M, int64_t N, bool exact) {
  const double slower[2][4] = {{1.0, 1.0, 1.3, 1.4}, {1.0, 1.0, 0.93, 1.07}};      // fp32: up to 16 rows, and above
  int best = 0;
  double least = 0.0;
  for (int j = 1; j <= 4; ++j) {
    const int64_t groups = (N + 16 * j - 1) / (16 * j), rounds = (groups + 255) / 256;
    if (groups * 64 * kFewWaves >= (int64_t(1) << 32)) continue;
    const double round = (j + 0.5 + 0.05 * (double)(M - 1)) * (exact ? slower[M > 16][j - 1] : 1.0);
    const double cost = (double)rounds * round, read = 1.4 * (double)N / 4096;
    const double units = cost > read ? cost : read;
    if (best == 0 || units < least) {
      best = j;
      least = units;
    }
  }
  return best;
}

}  // namespace mx
