// How a list of matrices is orthogonalized: the sizes of what is held of each,
// the bounds of the iteration, and the tiles of its products.  Host-only logic,
// no HIP types, so that it can be compiled and checked on a machine without a
// GPU.
#pragma once
#include <math.h>
#include <stdint.h>

namespace mx {

constexpr int kOrthoGroup = 32;                    // matrices in one launch's arguments
constexpr int kOrthoPad = 64;                      // one K step of the products: sizes are padded to it with zeros
constexpr int kOrthoRest = 192;                    // room for the rest of the last tile of 256, which holds anything
constexpr int64_t kOrthoSide = int64_t(1) << 20;   // rows and columns stay below
constexpr int64_t kOrthoMinor = int64_t(1) << 16;  // the shorter side too
constexpr int64_t kOrthoPitch = int64_t(1) << 26;  // elements between an output's rows stay below
constexpr int kOrthoParts = 256;                   // sums of squares of a matrix at most
constexpr int64_t kOrthoRun = 8192;                // elements for each of them at least

inline int64_t ortho_pad(int64_t n) { return (n + kOrthoPad - 1) / kOrthoPad * kOrthoPad; }

// A matrix's place in the workspace, in bytes: the sums of squares (float64), then X, the next X and X's low part
// [m][n], and three squares [m][m] in float16; m the shorter side, n the longer, each with room for a tile's rest.  (The rest also
// keeps the rows of a matrix whose sides are powers of two out of step with the memory's channels.)
struct OrthoSize {
  int64_t m, n;                                    // in whole K steps
  int64_t parts;                                   // sums of squares
  int64_t bytes;
};

inline OrthoSize ortho_size(int64_t rows, int64_t cols) {
  OrthoSize s;
  s.m = ortho_pad(rows < cols ? rows : cols);
  s.n = ortho_pad(rows < cols ? cols : rows);
  s.parts = (rows * cols + kOrthoRun - 1) / kOrthoRun;
  if (s.parts > kOrthoParts) s.parts = kOrthoParts;
  const int64_t lm = s.m + kOrthoRest, ln = s.n + kOrthoRest;
  s.bytes = 8 * kOrthoParts + 2 * (3 * lm * ln + 3 * lm * lm);
  return s;
}

// Matrices that are worked on together: as many of the list's next ones as one launch's arguments hold and as stay
// within this many bytes of workspace (one matrix at least).  2 GiB hold the linears of a large block, whose products
// fill the chip many times over.
constexpr int64_t kOrthoBytes = int64_t(2) << 30;

// visit(indexes, their number, bytes) for each group of a list whose entries have rows and cols, until it returns
// false; empty entries are in none.
template <typename T, typename Visit>
inline void each_ortho_group(const T* list, int32_t count, const Visit& visit) {
  int32_t at[kOrthoGroup];
  int n = 0;
  int64_t bytes = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (list[i].rows == 0 || list[i].cols == 0) continue;
    const int64_t next = ortho_size(list[i].rows, list[i].cols).bytes;
    if (n > 0 && (n == kOrthoGroup || bytes + next > kOrthoBytes)) {
      if (!visit(at, n, bytes)) return;
      n = 0;
      bytes = 0;
    }
    at[n++] = i;
    bytes += next;
  }
  if (n > 0) visit(at, n, bytes);
}

// How a product's result is cut into tiles, one for a workgroup: 64 to 256 a side; of 128 either one workgroup a CU with
// three LDS stages or two with two.
enum class OrthoTile { k64, k128, k128Two, k192, k256 };

// What a tile costs (us): `sym` or `full` for its first copies and its epilogue (of a square, of X), and a step of 64 k,
// `alone` where few CUs work and `shared` for a CU's part of a full chip, which power slows.  Fitted to 64 x 64 .. 4096 x
// 14336.  For example 4096 x 4096 (A / X): tiles of 64 163 / 223 us, of 128 105 / 158 and (two) 100 / 146, of 192 71 / 146,
// of 256 90 / 125; 1024 x 1024: 7.5 / 8.7, 11 / 13, 13 / 15, 17 / 22, 26 / 34.
struct OrthoCost {
  OrthoTile tile;
  int f, per;                                      // the tile's side in 64s, workgroups of a CU
  double sym, full, alone, shared;
};
constexpr OrthoCost kOrthoCosts[] = {{OrthoTile::k64, 1, 2, 3.0, 4.0, 0.17, 0.22},
                                     {OrthoTile::k128, 2, 1, 6.0, 8.5, 0.30, 0.58},
                                     {OrthoTile::k128Two, 2, 2, 6.0, 8.5, 0.36, 0.56},
                                     {OrthoTile::k192, 3, 1, 8.0, 14.0, 0.52, 0.95},
                                     {OrthoTile::k256, 4, 1, 12.0, 24.0, 0.87, 1.55}};
constexpr int kXcds = 8;
constexpr int kCus = 256;

// tiles of 64 f a side of a product's result: m x m of which those on and below the diagonal (sym), or m x n
inline int64_t ortho_tiles(const OrthoSize& z, bool sym, int f) {
  const int64_t tm = (z.m + 64 * f - 1) / (64 * f), tn = (z.n + 64 * f - 1) / (64 * f);
  return sym ? tm * (tm + 1) / 2 : tm * tn;
}

// The time of one product of each of these matrices, longest K first, by the costs above: whole rounds of the chip, and
// the rest, the shortest ones, in a last one.
inline double ortho_time(const OrthoSize* sizes, int count, bool sym, bool gram, const OrthoCost& c) {
  double tiles = 0.0, steps = 0.0;
  for (int i = 0; i < count; ++i) {
    const double n = (double)ortho_tiles(sizes[i], sym, c.f);
    tiles += n;
    steps += n * (double)((gram ? sizes[i].n : sizes[i].m) / 64);
  }
  const double longest = (double)((gram ? sizes[0].n : sizes[0].m) / 64);
  const double shortest = (double)((gram ? sizes[count - 1].n : sizes[count - 1].m) / 64);
  const double slots = (double)(kCus * c.per), rounds = floor(tiles / slots), rest = tiles - rounds * slots;
  const double start = sym ? c.sym : c.full;
  double us = rounds * start;
  if (rounds > 0.0) us += (steps - rest * shortest) / kCus * c.shared;
  if (rest > 0.0) {
    const double k = rounds > 0.0 ? shortest : steps / tiles;
    us += start + k * (c.alone + (c.per * c.shared - c.alone) * rest / slots);
  }
  const double least = start + longest * c.alone;
  return us > least ? us : least;
}

inline OrthoTile ortho_choose(const OrthoSize* sizes, int count, bool sym, bool gram) {
  OrthoTile best = OrthoTile::k64;
  double least = 0.0;
  for (const OrthoCost& c : kOrthoCosts) {
    const double us = ortho_time(sizes, count, sym, gram, c);
    if (&c == kOrthoCosts || us < least) {
      best = c.tile;
      least = us;
    }
  }
  return best;
}

// Bytes between the rows of a matrix of n columns (a multiple of 64) in LDS: 80 more than a multiple of 256, so that
// sixteen rows' 16-byte pieces, and four rows' 64-byte ones (almost), lie in different banks.
inline __attribute__((always_inline)) constexpr int ortho_pitch(int n) { return 2 * n + (2 * n % 256 == 0 ? 80 : 208); }

// Matrices that one workgroup takes whole: X, A and B in LDS (128 x 256: 43 us instead of 66).
inline int64_t ortho_small_bytes(const OrthoSize& z) {
  const int64_t products = z.m * ortho_pitch((int)z.n) + 2 * z.m * ortho_pitch((int)z.m), whole = 4 * z.m * (z.n + 4);
  return products > whole ? products : whole;
}
inline bool ortho_small_fits(const OrthoSize& z) { return z.m <= 128 && z.m * z.n <= 32768; }

// Whether the first two steps of these matrices run as one: it replaces 3 m^2 n multiplications by 3 m^3 (symmetric
// products counted half) and saves a pass of X, for one launch more, which large products do not notice.  Joined / apart,
// us, about the two borders: 1536 x 2048 (1.33 times as wide) 231 / 223, 2048 x 2560 (1.25) 382 / 380, 4096 x 4096 1345 /
// 1325, 4096 x 5120 1702 / 1765, 2048 x 4096 457 / 471; 1024 x 2048 (2.1e9) 152 / 152, 1024 x 4096 (4.3e9) 201 / 209, 512 x
// 8192 (2.1e9, left apart) 209 / 232; 4096 x 14336 3385 / 3848.
template <typename T>
inline bool ortho_joins(const T* list, int count) {
  double wide = 0.0, square = 0.0;
  for (int i = 0; i < count; ++i) {
    const OrthoSize z = ortho_size(list[i].rows, list[i].cols);
    wide += (double)z.m * z.m * z.n;
    square += (double)z.m * z.m * z.m;
  }
  return wide >= 1.25 * square && wide >= 4e9;
}

// The largest |p(s)|, p(s) = a s + b s^3 + c s^5, for 0 <= s <= top, and the largest |b t + c t^2| and |a + b t + c t^2|
// for 0 <= t <= top^2: what bounds X, and the factors that multiply it, in the next step.
struct OrthoReach {
  double x, factor;
};

inline OrthoReach ortho_reach(double a, double b, double c, double top) {
  OrthoReach r = {0.0, 0.0};
  const double end = top * top;
  auto at = [&](double t) {                        // t = s^2
    if (!(t >= 0.0 && t <= end)) return;
    const double x = fabs(sqrt(t) * (a + t * (b + t * c))), f = fabs(t * (b + t * c)), q = fabs(a + t * (b + t * c));
    r.x = fmax(r.x, x);
    r.factor = fmax(r.factor, fmax(f, q));
  };
  at(0.0);
  at(end);
  if (c != 0.0) at(-b / (2.0 * c));
  // p'(s) = a + 3 b t + 5 c t^2
  if (c != 0.0) {
    const double d = 9.0 * b * b - 20.0 * a * c;
    if (d >= 0.0) {
      at((-3.0 * b + sqrt(d)) / (10.0 * c));
      at((-3.0 * b - sqrt(d)) / (10.0 * c));
    }
  } else if (b != 0.0) {
    at(-a / (3.0 * b));
  }
  return r;
}

// Whether X (held times 2^12) and its factors (times 2^11) stay within float16 through all steps, with half of its
// range to spare: singular values start at 1 or below.
constexpr double kOrthoMostX = 4.0, kOrthoMostFactor = 15.0;

inline bool ortho_fits(double a, double b, double c, int steps) {
  if (!isfinite(a) || !isfinite(b) || !isfinite(c)) return false;
  double top = 1.0;
  for (int i = 0; i < steps; ++i) {
    const OrthoReach r = ortho_reach(a, b, c, top);
    if (!(r.x <= kOrthoMostX && r.factor <= kOrthoMostFactor)) return false;
    if (top * top > kOrthoMostFactor) return false;            // A itself
    if (i > 0 && r.x <= top) break;                            // from here on the bound does not grow
    top = r.x > top ? r.x : top;
  }
  return true;
}

}  // namespace mx
