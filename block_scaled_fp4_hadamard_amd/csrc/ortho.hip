// Orthogonalizing matrices by Newton-Schulz steps, alone or as the update of a
// Muon step.  From X = U / (|U| + eps), |.| the Frobenius norm, each step takes
//
//   A = X X^T,   B = b A + c A A,   X <- a X + B X
//
// which sends every singular value s of X to a s + b s^3 + c s^5: small ones
// grow by a factor a, and all end near 1.  X is held with its shorter side as
// rows (U or its transpose), so that A and B are small.  In the last step B
// takes a on its diagonal and X <- B X is all.
//
// Number formats.  The products are float16 with float32 sums: 11 bits at the
// rate of bf16's 8, and the range suffices because everything is bounded (no
// entry of X above |X|_2, about 1.2 for the usual coefficients).  X is held
// times 2^12 and A times 2^11, so that the small entries of large matrices
// (1 / sqrt(m n) in X, 1 / m in A) stay normal numbers; B adds to a I, beside
// which its subnormal entries, off by 2^-25, are nothing.  Rounding X costs most:
// what it adds in weak directions grows by a in every step, to a share of the
// result where U has few strong directions.  So X is held in two parts, high and
// low, 22 bits together (to 2^-25 in the low part's own scale); the products read
// the high part, and the sum a X takes both.  Against float64 the result is off by 0.3e-3 to 2.6e-3 of
// its norm where the entries' roundings are independent, as rounding it to bf16
// costs 1.7e-3; with the high part alone a matrix of rank 1 was 15% off.  The
// worst is a matrix of equal entries: all entries of a square round alike, which
// is an error of up to 2^-11 of B, and B at s = 1 is four times as large as the
// factor a + b s^2 + c s^4 that it is a part of: up to 1.5e-2 after five steps.
//
// A list's matrices go through each product together, up to 32 in one launch:
// the sums of squares, X, then three products a step; small ones through a single
// kernel.  Bound by the matrix cores, whose power sets the clock, and by waits:
// 1024 SIMDs on random float16 data and nothing else reach 1720 TFLOP/s (1.64 GHz), a
// large library product 1525 (8192 cubed) to 1230 (4096 x 28672 x 4096 with the
// second operand as here).  The products of a Llama-3.1-8B block's linears
// (symmetric ones counted half) run at 1050 to 1150: the matrix cores are busy 53
// to 74% of the time, at 1.6 to 1.8 GHz.  The whole step of its 218 million weights
// takes 12.8 to 13.9 ms by card, of which the gradients' and moments' passes are 1.1
// (4.7 to 5 TB/s); 4096 x 4096 alone 1.35 to 1.55, busy 50 to 62% at 1.8 to 2.1 GHz: one
// round of the chip, whose first copies and epilogues nothing hides.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <utility>
#include "ortho_kernels.h"

namespace mx {

namespace {

typedef _Float16 half_t;
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

constexpr int kRow = 128;                // bytes of an operand's row in one K step: 64 values
constexpr float kScaleX = 0x1p12f, kScaleA = 0x1p11f;

struct Args {
  OrthoItem item[kOrthoGroup];
  int end[kOrthoGroup];                  // workgroups of items 0 .. i
  int count;
};

// A matrix as the kernels see it.
struct View {
  int m, n;                              // shorter and longer side, in whole K steps
  int lm, ln;                            // and with room for any tile's rest
  double* parts;
  half_t *x0, *x1, *low;                 // x0 and x1 take turns
  half_t *square;                        // three of [lm][lm]
};

__device__ __forceinline__ View view(const OrthoItem& t) {
  View v;
  const int r = (t.rows + kOrthoPad - 1) / kOrthoPad * kOrthoPad, c = (t.cols + kOrthoPad - 1) / kOrthoPad * kOrthoPad;
  v.m = min(r, c);
  v.n = max(r, c);
  v.lm = v.m + kOrthoRest;
  v.ln = v.n + kOrthoRest;
  v.parts = (double*)t.space;
  v.x0 = (half_t*)(t.space + 8 * kOrthoParts);
  const int64_t mn = (int64_t)v.lm * v.ln;
  v.x1 = v.x0 + mn;
  v.low = v.x1 + mn;
  v.square = v.low + mn;
  return v;
}

// the item of a workgroup, and the workgroup's number in it
__device__ __forceinline__ int find(const Args& a, int& id) {
  int i = 0, base = 0;
  while (i < a.count - 1 && (int)blockIdx.x >= a.end[i]) base = a.end[i++];
  id = (int)blockIdx.x - base;
  return i;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
}
__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// 16 bytes wherever a row may start: one access, whatever the row pitch and the width
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <typename T>
__device__ __forceinline__ T* uniform(T* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (T*)(((uint64_t)hi << 32) | lo);
}
// a pointer known to be the same in all lanes and to lie in global memory (not in LDS or scratch)
template <typename T>
__device__ __forceinline__ __attribute__((address_space(1))) T* global(T* p) {
  return (__attribute__((address_space(1))) T*)uniform(p);
}
template <typename V, typename P>
__device__ __forceinline__ V load_at(P p) {
  return *(const __attribute__((address_space(1))) V*)p;
}
template <typename V, typename P>
__device__ __forceinline__ void store_at(P p, const V& x) {
  *(__attribute__((address_space(1))) V*)p = x;
}
template <typename P>
__device__ __forceinline__ void store8(P p, const float (&y)[8]) {
  store_at<u32x4_any>(p, u32x4{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])});
  store_at<u32x4_any>(p + 4, u32x4{__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7])});
}

// ---------------------------------------------------------------------------
// The moment and the sum of squares (4.7 TB/s on a block's weights; element by
// element, with a division each, it was 3.5): m = RN(RN(m mu) + RN(g (1 - mu))), and u =
// RN(RN(g (1 - mu)) + RN(m mu)) (Nesterov) or m.  Squares are added in float64,
// which no float32 overflows or sinks below.
struct Moment {
  float mu, rest, scale;                 // rest = 1 - mu
  bool nesterov;
};

__device__ __forceinline__ float update_of(float g, float m, const Moment& c) {
#pragma clang fp contract(off)
  return c.nesterov ? g * c.rest + m * c.mu : m;
}

__device__ __forceinline__ Moment moment_of(const OrthoStep& s) {
  return Moment{s.momentum, s.rest, s.grad_scale ? *s.grad_scale : 1.0f, s.nesterov};
}

// `count` <= N values of a gradient or moment from p on, as float32; zeros after them
template <int N>
__device__ __forceinline__ void load_values(const float* p, int count, float (&o)[N]) {
#pragma unroll
  for (int q = 0; q < N; q += 4) {
    if (q + 4 <= count) {
      const u32x4 r = *(const u32x4_any*)(p + q);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[q + e] = __uint_as_float(r[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[q + e] = q + e < count ? p[q + e] : 0.0f;
    }
  }
}
template <int N>
__device__ __forceinline__ void load_values(const uint16_t* p, int count, float (&o)[N]) {
  if (count >= N) {
    uint32_t r[N / 2];
    __builtin_memcpy(r, p, sizeof(r));
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = __uint_as_float((e & 1) ? r[e >> 1] & 0xFFFF0000u : r[e >> 1] << 16);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = e < count ? bf16_value(p[e]) : 0.0f;
  }
}
template <int N>
__device__ __forceinline__ void load_gradient(const OrthoItem& t, int64_t at, int count, float scale, float (&o)[N]) {
  if (t.g_bf16) load_values((const uint16_t*)t.g + at, count, o);
  else load_values((const float*)t.g + at, count, o);
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] *= scale;
}

// U's scale 2^12 / (|U| + eps), whose float32 might overflow or sink, in two factors; 0 for a matrix of zeros, where
// that of the smallest eps would be Inf
struct Scale {
  float factor;
  int power;
};
__device__ __forceinline__ Scale scale_of(double sum, double eps) {
  if (sum == 0.0) return Scale{0.0f, 0};
  int power;
  const double f = frexp((double)kScaleX / (sqrt(sum) + eps), &power);
  return Scale{(float)f, power};
}
// the power first: it is exact, takes u to at most 2^13, and makes a subnormal u a normal number before the product rounds
__device__ __forceinline__ float scaled(float u, const Scale& s) { return ldexpf(u, s.power) * s.factor; }

constexpr int kSumThreads = 1024;

__global__ void __launch_bounds__(kSumThreads) ortho_sum(const Args a, const OrthoStep step) {
#pragma clang fp contract(off)
  __shared__ double red[kSumThreads / 64];
  int id;
  const OrthoItem t = a.item[find(a, id)];
  const View v = view(t);
  const Moment c = moment_of(step);
  const int64_t total = (int64_t)t.rows * t.cols, parts = min((int64_t)kOrthoParts, (total + kOrthoRun - 1) / kOrthoRun);
  // a contiguous gradient is one long row, of which a part is a run; otherwise a part is a run of rows
  const bool one = t.ld_g == t.cols;
  const int64_t rows = one ? 1 : t.rows, cols = one ? total : t.cols, units = one ? (total + 7) / 8 : t.rows;
  const int64_t each = (units + parts - 1) / parts, from = min(units, id * each), to = min(units, from + each);
  const int64_t row0 = one ? 0 : from, row1 = one ? 1 : to, col0 = one ? 8 * from : 0, col1 = one ? min(cols, 8 * to) : cols;
  double sum = 0.0;
  for (int64_t row = row0; row < row1; ++row)
    for (int64_t col = col0 + 8 * threadIdx.x; col < col1; col += 8 * kSumThreads) {
      const int count = (int)min((int64_t)8, col1 - col);
      float u[8];
      load_gradient(t, row * t.ld_g + col, count, c.scale, u);
      if (t.moment != nullptr) {               // moments and their gradients are contiguous
        float m[8];
        load_values(t.moment + col, count, m);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          m[e] = m[e] * c.mu + u[e] * c.rest;
          u[e] = update_of(u[e], m[e], c);
        }
        if (count == 8) {
          store8(t.moment + col, m);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < count) t.moment[col + e] = m[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += (double)u[e] * (double)u[e];
    }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kSumThreads / 64; ++i) sum += red[i];
    v.parts[id] = sum;
  }
}

// ---------------------------------------------------------------------------
// X from U: a 64 x 64 piece of X a workgroup, zeros up to whole K steps.  A tall
// U is transposed through LDS.  5.0 TB/s on a block's weights.
__global__ void __launch_bounds__(256) ortho_start(const Args a, const OrthoStep step) {
  __shared__ double red[4];
  __shared__ float piece[64][65];
  int id;
  const OrthoItem t = a.item[find(a, id)];
  const View v = view(t);
  const Moment c = moment_of(step);
  const int64_t total = (int64_t)t.rows * t.cols;
  const int parts = (int)min((int64_t)kOrthoParts, (total + kOrthoRun - 1) / kOrthoRun);
  const double mine = (int)threadIdx.x < parts ? v.parts[threadIdx.x] : 0.0;
  const bool tall = t.rows > t.cols;
  const int across = v.n / 64, m0 = id / across * 64, n0 = id % across * 64;
  const int r0 = tall ? n0 : m0, c0 = tall ? m0 : n0;          // the piece in U
  // a lane takes four neighbouring values of every 16th row, asked for before the sums are added
  const int row = threadIdx.x / 16, col = 4 * (threadIdx.x % 16);
  float u[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + row + 16 * i, count = r < t.rows ? min(4, t.cols - (c0 + col)) : 0;
    if (count <= 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) u[i][e] = 0.0f;
      continue;
    }
    load_gradient(t, (int64_t)r * t.ld_g + c0 + col, count, c.scale, u[i]);
    if (t.moment != nullptr) {
      float m[4];
      load_values(t.moment + (int64_t)r * t.cols + c0 + col, count, m);
#pragma unroll
      for (int e = 0; e < 4; ++e) u[i][e] = update_of(u[i][e], m[e], c);
    }
  }
  double sum = mine;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = (red[0] + red[1]) + (red[2] + red[3]);
  const Scale scale = scale_of(sum, step.eps);
  auto put = [&](int m, int n, const float (&x)[4]) {
    v4h hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hi[e] = (half_t)x[e];
      lo[e] = (half_t)(x[e] - (float)hi[e]);
    }
    const int64_t at = (int64_t)(m0 + m) * v.ln + n0 + n;
    *(v4h*)(v.x0 + at) = hi;
    *(v4h*)(v.low + at) = lo;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) u[i][e] = scaled(u[i][e], scale);
    if (!tall) {
      put(row + 16 * i, col, u[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) piece[col + e][row + 16 * i] = u[i][e];
    }
  }
  if (!tall) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = piece[row + 16 * i][col + e];
    put(row + 16 * i, col, x);
  }
}

// ---------------------------------------------------------------------------
// The products: a workgroup of four waves takes a tile of the result, 64 F by 64
// F, each wave a quarter of it, F x F fragments of the 32x32x16 instruction.
// K advances 64 values (128 bytes of every row) a step, copied global -> LDS by
// DMA into one of a ring of stages while another is consumed.
//
//   kGram  A = X X^T              both operands K-contiguous
//   kPoly  S = f S1 + g L R       the same: squares that are their own transposes
//   kMix   S = f S1 + f2 S2 + g L R
//   kStep  X' = x X + B X         the second operand has K as its rows: LDS reads
//   kLast  O = B X                that transpose (ds_read_b64_tr_b16)
//
// The squares are polynomials of A, hence symmetric, and commute: tiles on and
// below the diagonal are computed, and what is below it is stored twice.
//
// Layout of the instruction: lane l holds row l % 32 of an operand and 8 of its
// 16 k (8 (l / 32) ..); the 32 x 32 result has row 8 (r / 4) + 4 (l / 32) + r % 4 in
// register r and column l % 32.  The columns of the product's tile are passed as
// the instruction's rows, in an order that leaves a lane with columns 8 (l / 32)
// .. + 7 and 16 more of its row (strip_col), so that a wave's 16-byte accesses
// meet 32 bytes of each row.  For a tall matrix's last step the two sides change
// places, so that the result leaves as the rows of O's transpose.
//
// A Llama-3.1-8B block's four kStep products, 1.79 TFLOP with all that they read
// and write of X: 1645 to 1672 us, 1070 to 1090 TFLOP/s, the matrix cores 59% busy
// at 1.74 GHz; the epilogue's 8 bytes an element are a fifth.  Steps on the way:
// copies issued together 1972 us; fragments read two parts ahead 1850; the copies
// spread over three parts 1795; the epilogue's reads two rows ahead, without
// bounds 1708; its low part unscaled 1672.
enum Mode { kGram, kPoly, kMix, kStep, kLast };

// 16-byte piece's place in a 128-byte LDS row: a 16-byte LDS read serves the wave in groups of 16 lanes (0-3, 12-15 and
// 20-27, and so on); with this order each group covers all 64 banks
__device__ __forceinline__ int slot(int row, int piece) { return (piece ^ ((row >> 1) & 7)) * 16; }

// the column that row f of a 32-column strip's fragment holds
__device__ __forceinline__ int strip_col(int f) {
  return 16 * (f >> 4) + 8 * ((f >> 2) & 1) + 4 * ((f >> 3) & 1) + (f & 3);
}

// Global -> LDS copy of 16 bytes per lane: LDS address = M0 + 16 * lane.  Inline asm, so that the compiler places no
// waits of its own for it; it writes no register.  An SALU write of M0 needs one wait state before the copy reads it.
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
// Transposing LDS reads: in each 16 lanes, lane s gives the address of four neighbouring values of row s / 4, and gets
// the four rows' values of column s.
__device__ __forceinline__ v8h read_columns(const uint8_t* rows03, const uint8_t* rows47) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const v4h lo = __builtin_bit_cast(v4h, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)rows03));
  const v4h hi = __builtin_bit_cast(v4h, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)rows47));
  return v8h{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}
template <int... I, typename F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, const F& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(const F& f) {
  each(std::make_integer_sequence<int, N>{}, f);
}

// What the last step writes: eight neighbouring results in row `row` of U's layout, from column `col`, the lane's `own`
// elements on from the wave's element `first`.  `w`: the weights there, read ahead where all eight exist.
__device__ __forceinline__ void finish(const OrthoItem& t, float keep, float rate, int row, int col, int64_t first,
                                       uint32_t own, const float (&o)[8], const u32x4 (&w)[2]) {
#pragma clang fp contract(off)
  if (row >= t.rows || col >= t.cols) return;
  const int left = t.cols - col;
  float y[8];
  if (t.w != nullptr) {
    const auto to = global(t.w + first) + own;
    const auto copy = global(t.copy + first) + own;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float old = left >= 8 ? __uint_as_float(w[e >> 2][e & 3]) : e < left ? to[e] : 0.0f;
      y[e] = old * keep - o[e] * rate;
    }
    const u32x4 h = {pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])};
    if (left >= 8) {
      store8(to, y);
      if (t.copy != nullptr) store_at<u32x4_any>(copy, h);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) {
          to[e] = y[e];
          if (t.copy != nullptr) copy[e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
        }
    }
    return;
  }
  const auto out16 = global((uint16_t*)t.out + first) + own;
  const auto out32 = global((float*)t.out + first) + own;
  const u32x4 h = {pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])};
  if (left >= 8) {
    if (t.out_bf16) {
      store_at<u32x4_any>(out16, h);
    } else {
      store8(out32, o);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) {
        if (t.out_bf16) out16[e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
        else out32[e] = o[e];
      }
  }
}

// what the weights keep, and what they take of the result
__device__ __forceinline__ void rates(const OrthoItem& t, const OrthoStep& step, float& keep, float& rate) {
  keep = 1.0f;
  rate = 0.0f;
  if (t.w == nullptr) return;
  const double lr = step.lr_dev ? (double)*step.lr_dev : step.lr;
  keep = (float)(1.0 - lr * step.weight_decay);
  rate = (float)(lr * t.scale);
}

struct Coef {
  float x, f, f2, g;
  float diagonal;                        // added to a square's diagonal
  int from;                              // which X holds the step's
  int left, right, add, add2, out;       // squares
};

// t: the workgroup's matrix, id: its number in it, lds: room for S stages of both operands
template <int F, int S, int MODE, bool TRANS>
__device__ __forceinline__ void product_tile(const OrthoItem t, int id, const OrthoStep& step, const Coef& c,
                                             uint8_t* lds) {
  constexpr bool kSym = MODE <= kMix;
  constexpr int T = 64 * F, kStage = T * kRow;
  uint8_t *const sP = lds, *const sQ = lds + S * kStage;               // the first operand's stages, the second's
  const View v = view(t);
  // An XCD (workgroup ids are dealt to them in turn, items start at a multiple of 8) takes a contiguous run of tiles.
  const int tm = (v.m + T - 1) / T, tn = kSym ? tm : (v.n + T - 1) / T, tiles = kSym ? tm * (tm + 1) / 2 : tm * tn;
  const int per = (tiles + kXcds - 1) / kXcds, tile = id % kXcds * per + id / kXcds;
  if (id / kXcds >= per || tile >= tiles) return;
  int ti, tj;
  if constexpr (kSym) {
    ti = (int)((sqrtf(8.0f * (float)tile + 1.0f) - 1.0f) * 0.5f);
    while (ti * (ti + 1) / 2 > tile) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= tile) ++ti;
    tj = tile - ti * (ti + 1) / 2;
  } else {
    // bands of four rows of tiles, column by column
    const int band = tile / (4 * tn), in = tile % (4 * tn), rows = min(4, tm - 4 * band);
    ti = 4 * band + in % rows;
    tj = in / rows;
  }
  const int m0 = ti * T, n0 = tj * T;
  const half_t* x = c.from ? v.x1 : v.x0;
  constexpr bool kSquares = MODE == kPoly || MODE == kMix;
  const int64_t square = (int64_t)v.lm * v.lm;
  const half_t* pp = MODE == kGram ? x : v.square + c.left * square;
  const half_t* qq = kSquares ? v.square + c.right * square : x;
  const int ldp = MODE == kGram ? v.ln : v.lm, ldq = kSquares ? v.lm : v.ln;
  const int nk = (MODE == kGram ? v.n : v.m) / 64;

  const int th = threadIdx.x, lane = th & 63, wave = __builtin_amdgcn_readfirstlane(th >> 6);
  const int wm = 32 * F * (wave & 1), wn = 32 * F * (wave >> 1);
  const int l32 = lane & 31, h = lane >> 5;

  // Copies: one instruction moves 1 KB, eight LDS rows of a K-contiguous operand or a run of the other's rows; a wave
  // copies a quarter of each operand.  Rows and columns past the matrix hold anything: each spoils its own row or column of
  // the result, which lies past the matrix too.
  constexpr int kCopies = 2 * F;
  constexpr bool kOdd = F % 2 != 0;        // K rows of an odd number of 128 bytes already part the banks of neighbours
  uint32_t op[kCopies], oq[kCopies];
#pragma unroll
  for (int e = 0; e < kCopies; ++e) {
    const int f = (wave * kCopies + e) * 8 + (lane >> 3);
    const int pr = TRANS ? (f & ~31) + strip_col(f & 31) : f;
    op[e] = (uint32_t)pr * (uint32_t)(2 * ldp) + (uint32_t)(((lane & 7) ^ ((f >> 1) & 7)) * 16);
    if constexpr (kSym) {
      const int qr = (f & ~31) + strip_col(f & 31);
      oq[e] = (uint32_t)qr * (uint32_t)(2 * ldq) + (uint32_t)(((lane & 7) ^ ((f >> 1) & 7)) * 16);
    } else {
      // K row k of T values, its 64-byte pieces in an order that parts four neighbouring rows' banks
      const int at = (wave * kCopies + e) * 1024 + lane * 16, k = at / (2 * T), piece = at % (2 * T) / 16;
      const int turn = kOdd ? (k >> 1) & 1 : k & 3;
      const int col = 8 * ((((piece >> 2) ^ turn) << 2) + (piece & 3));
      oq[e] = (uint32_t)k * (uint32_t)(2 * ldq) + (uint32_t)(2 * col);
    }
  }
  const uint8_t* cp = uniform((const uint8_t*)(pp + (int64_t)m0 * ldp));
  const uint8_t* cq = uniform((const uint8_t*)(kSym ? qq + (int64_t)n0 * ldq : qq + n0));
  const int64_t stepq = kSym ? kRow : (int64_t)128 * ldq;          // 64 values, or 64 rows
  const uint32_t dP = lds_addr(sP + wave * kCopies * 1024), dQ = lds_addr(sQ + wave * kCopies * 1024);
  auto copy = [&](int st, int n) __attribute__((always_inline)) {
    if (n & 1) dma16(cq, oq[n >> 1], dQ + st * kStage + (n >> 1) * 1024);
    else dma16(cp, op[n >> 1], dP + st * kStage + (n >> 1) * 1024);
  };
  auto advance = [&]() __attribute__((always_inline)) {
    cp += kRow;
    cq += stepq;
  };

  // a fragment's place in LDS: rows 32 apart are immediates, the four K parts of a step turn the pieces
  uint32_t rp[4], rq[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) rp[s] = (uint32_t)((wm + l32) * kRow + slot(l32, 2 * s + h));
  const int chunk = 4 * ((lane >> 4) & 1) + (lane & 3), krow = 8 * h + ((lane >> 2) & 3);
  if constexpr (kSym) {
#pragma unroll
    for (int s = 0; s < 4; ++s) rq[s] = (uint32_t)((wn + l32) * kRow + slot(l32, 2 * s + h));
  } else {
    // strip j of the wave: chunk `chunk` of four columns (in fragment order) of K row krow; rows 4, 16 .. on are
    // immediates
    const int col = TRANS ? 4 * chunk : strip_col(4 * chunk);
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const int seg = (wn >> 5) + j, turn = kOdd ? (krow >> 1) & 1 : krow & 3;
      rq[j] = (uint32_t)(krow * 2 * T + (seg ^ turn) * 64 + col * 2);
    }
  }
  auto read_p = [&](int st, int s, int i) __attribute__((always_inline)) { return *(const v8h*)(sP + st * kStage + rp[s] + i * 32 * kRow); };
  auto read_q = [&](int st, int s, int j) __attribute__((always_inline)) {
    if constexpr (kSym) {
      return *(const v8h*)(sQ + st * kStage + rq[s] + j * 32 * kRow);
    } else {
      const uint8_t* p = sQ + st * kStage + rq[j] + s * 16 * 2 * T;
      return read_columns(p, p + 4 * 2 * T);
    }
  };

  v16f acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // A step is four parts of 16 k, each with fragments of its own: part 0 reads those of parts 1 and 2, part 1 those of 3.
  // Then every read of the stage is done, and a barrier frees it for the copies of the step S further on.  A copy occupies
  // the CU's address unit for 16 cycles, so that the waves' 16 F of them would stop the matrix cores if issued together:
  // they are spread over parts 2 and 3 and the next step's part 0.  A second barrier, before part 3 reads the next step's
  // first fragments, waits for the copies that bring them.
  constexpr int kAll = 2 * kCopies, kIn2 = (kAll + 2) / 3, kIn3 = (kAll + 1) / 3;
#pragma unroll
  for (int b = 0; b < S; ++b) {
    if (b >= nk) break;
    // the last stage's batch is left to step 0 in part, as every later batch to the step after
#pragma unroll
    for (int n = 0; n < (b + 1 < S ? kAll : kIn2 + kIn3); ++n) copy(b, n);
    if (b + 1 < S) advance();
  }
  if (nk >= S) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((S - 2) * kAll + kIn2 + kIn3) : "memory");
  else asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  v8h fp[4][F], fq[4][F];
#pragma unroll
  for (int i = 0; i < F; ++i) {
    fp[0][i] = read_p(0, 0, i);
    fq[0][i] = read_q(0, 0, i);
  }
  int st = 0, last = S - 1;              // the step's stage, and the one before it
  auto one_step = [&](auto finish_, auto issue_, auto more_) __attribute__((always_inline)) {
    constexpr bool ends = decltype(finish_)::value, issue = decltype(issue_)::value, more = decltype(more_)::value;
    const int next = st + 1 == S ? 0 : st + 1;
    each<4>([&](auto part) __attribute__((always_inline)) {
      constexpr int s = decltype(part)::value;
      if constexpr (s == 2 && issue) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if constexpr (s == 3 && more) {
        if constexpr (issue) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((S - 2) * kAll + kIn2) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
      }
      each<F * F>([&](auto index) __attribute__((always_inline)) {
        constexpr int n = decltype(index)::value, i = n / F, j = n % F;
        // the fragments that go with this product: 2 F a part to read, 4 F in part 0
        constexpr int reads = s == 0 ? 4 * F : s == 2 ? 0 : 2 * F, from = n * reads / (F * F), to = (n + 1) * reads / (F * F);
        each<to - from>([&](auto k) __attribute__((always_inline)) {
          constexpr int r = from + decltype(k)::value, set = s == 0 ? 1 + r / (2 * F) : s == 1 ? 3 : 0, f = r % (2 * F) / 2;
          if constexpr (s < 2) {
            if constexpr (r & 1) fq[set][f] = read_q(st, set, f);
            else fp[set][f] = read_p(st, set, f);
          } else if constexpr (more) {
            if constexpr (r & 1) fq[0][f] = read_q(next, 0, f);
            else fp[0][f] = read_p(next, 0, f);
          }
        });
        acc[i][j] = TRANS ? __builtin_amdgcn_mfma_f32_32x32x16_f16(fp[s][i], fq[s][j], acc[i][j], 0, 0, 0)
                          : __builtin_amdgcn_mfma_f32_32x32x16_f16(fq[s][j], fp[s][i], acc[i][j], 0, 0, 0);
        // and the copies: [first, first + here) of them in this part
        constexpr bool active = s == 0 ? ends : s >= 2 && issue;
        constexpr int first = s == 2 ? 0 : s == 3 ? kIn2 : kIn2 + kIn3, here = s == 2 ? kIn2 : s == 3 ? kIn3 : kAll - first;
        if constexpr (active) {
          each<(n + 1) * here / (F * F) - n * here / (F * F)>([&](auto k) __attribute__((always_inline)) {
            copy(s == 0 ? last : st, first + n * here / (F * F) + decltype(k)::value);
          });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (s == 0 && ends) advance();
    });
    last = st;
    st = next;
  };
  float keep = 1.0f, rate = 0.0f;
  if constexpr (MODE == kLast) rates(t, step, keep, rate);
  // The epilogue, a row of fragments at a time; what it reads is asked for two rows ahead, the first two before the last
  // step's products.  TRANS: the lane's column is l % 32 of strip j, its rows 8 h .. and 16 + 8 h .. of strip i.  In the
  // result's own rows a lane is always at row l % 32 and columns 8 h .. of a fragment: one offset a lane, and a uniform
  // address for each fragment.
  const int ld = MODE == kLast ? (t.w != nullptr ? t.cols : (int)t.ld_out) : kSym ? v.lm : v.ln;
  const uint32_t own = (uint32_t)l32 * (uint32_t)ld + 8 * h;
  // the first element of fragment (i, j) in rows of ld
  auto first_of = [&](int i, int j) __attribute__((always_inline)) {
    const int64_t m = m0 + wm + 32 * i, n = n0 + wn + 32 * j;
    return TRANS ? n * ld + m : m * ld + n;
  };
  constexpr int kAhead = MODE == kGram ? 1 : MODE == kPoly ? 2 : 4;
  half_t* const out = v.square + (kSym ? c.out * square : 0);
  u32x4 ahead[F < 3 ? F : 3][F][kAhead];
  auto ask = [&](int i, u32x4 (&to)[F][kAhead]) __attribute__((always_inline)) {
    each<F>([&](auto column) __attribute__((always_inline)) {
      constexpr int j = decltype(column)::value;
      if constexpr (kSquares) {
        const auto base = global(v.square + c.add * square + first_of(i, j)) + own;
        to[j][0] = load_at<u32x4>(base);
        to[j][1] = load_at<u32x4>(base + 16);
        if constexpr (MODE == kMix) {
          const auto base2 = global(v.square + c.add2 * square + first_of(i, j)) + own;
          to[j][2] = load_at<u32x4>(base2);
          to[j][3] = load_at<u32x4>(base2 + 16);
        }
      } else if constexpr (MODE == kStep) {
        const auto hi = global(x + first_of(i, j)) + own;
        const auto lo = global(v.low + first_of(i, j)) + own;
        to[j][0] = load_at<u32x4>(hi);
        to[j][1] = load_at<u32x4>(lo);
        to[j][2] = load_at<u32x4>(hi + 16);
        to[j][3] = load_at<u32x4>(lo + 16);
      } else if constexpr (MODE == kLast) {
        const int row = (TRANS ? n0 + wn + 32 * j : m0 + wm + 32 * i) + l32;
        const int col = (TRANS ? m0 + wm + 32 * i : n0 + wn + 32 * j) + 8 * h;
        if (t.w == nullptr || row >= t.rows) return;
        const auto base = global(t.w + first_of(i, j)) + own;
        if (col + 8 <= t.cols) {
          to[j][0] = load_at<u32x4_any>(base);
          to[j][1] = load_at<u32x4_any>(base + 4);
        }
        if (col + 24 <= t.cols) {
          to[j][2] = load_at<u32x4_any>(base + 16);
          to[j][3] = load_at<u32x4_any>(base + 20);
        }
      }
    });
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  int kt = 0;
  for (; kt + S < nk; ++kt) one_step(yes, yes, yes);
  if (nk >= S) {
    one_step(yes, no, yes);
    ++kt;
  }
  for (; kt + 1 < nk; ++kt) one_step(no, no, yes);
  ask(0, ahead[0]);
  if constexpr (F > 1) ask(1, ahead[1]);
  one_step(no, no, no);
  // The other half of a symmetric result goes through LDS, a wave's part [row][column] in its own quarter, and leaves by
  // transposing reads as rows of 16 bytes.
  uint8_t* const turn = lds + wave * (32 * F * 64 * F);
  auto side = [&](int row, int col) __attribute__((always_inline)) {
    // 32-byte pieces in an order that parts the banks of the eight rows of a read
    const int unit = (col >> 4) ^ (F == 4 ? (row & 3) | ((row >> 1) & 4) : 0);
    return row * 64 * F + unit * 32 + 2 * (col & 15);
  };
  if constexpr (kSym) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  each<F>([&](auto row) __attribute__((always_inline)) {
    constexpr int i = decltype(row)::value;
    if constexpr (i + 2 < F) ask(i + 2, ahead[(i + 2) % 3]);
    __builtin_amdgcn_sched_barrier(0);
    const auto& got = ahead[i % 3];
    each<F>([&](auto column) __attribute__((always_inline)) {
      constexpr int j = decltype(column)::value;
      const int64_t first = first_of(i, j);
      const v16f d = acc[i][j];
      each<2>([&](auto half) __attribute__((always_inline)) {
        constexpr int q = decltype(half)::value;
        if constexpr (MODE == kLast) {
          float o[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) o[r] = d[8 * q + r] * (1.0f / kScaleX);
          const u32x4 w[2] = {got[j][2 * q], got[j][2 * q + 1]};
          const int row = (TRANS ? n0 + wn + 32 * j : m0 + wm + 32 * i) + l32;
          const int col = (TRANS ? m0 + wm + 32 * i : n0 + wn + 32 * j) + 16 * q + 8 * h;
          finish(t, keep, rate, row, col, first + 16 * q, own, o, w);
        } else if constexpr (kSym) {
          v8h y;
          if constexpr (MODE == kGram) {
#pragma unroll
            for (int r = 0; r < 8; ++r) y[r] = (half_t)(d[8 * q + r] * (kScaleA / (kScaleX * kScaleX)));
          } else {
            const v8h base = __builtin_bit_cast(v8h, got[j][q]);
            v8h base2 = base;
            if constexpr (MODE == kMix) base2 = __builtin_bit_cast(v8h, got[j][2 + q]);
            // the lane's row less its first column, where the diagonal may pass
            const int off = m0 + wm + 32 * i + l32 - (n0 + wn + 32 * j + 16 * q + 8 * h);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              float o = fmaf(c.f, (float)base[r], d[8 * q + r] * c.g);
              if constexpr (MODE == kMix) o = fmaf(c.f2, (float)base2[r], o);
              if (off == r) o += c.diagonal;
              y[r] = (half_t)o;
            }
          }
          store_at(global(out + first + 16 * q) + own, y);
          if (ti != tj) *(v8h*)(turn + side(32 * i + l32, 32 * j + 16 * q + 8 * h)) = y;
        } else {
          const v8h xh = __builtin_bit_cast(v8h, got[j][2 * q]), xl = __builtin_bit_cast(v8h, got[j][2 * q + 1]);
          v8h nh, nl;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float y = fmaf(c.x, (float)xl[r] + (float)xh[r], d[8 * q + r]);
            nh[r] = (half_t)y;
            nl[r] = (half_t)(y - (float)nh[r]);
          }
          store_at(global((c.from ? v.x0 : v.x1) + first + 16 * q) + own, nh);
          store_at(global(v.low + first + 16 * q) + own, nl);
        }
      });
      __builtin_amdgcn_sched_barrier(0);         // one fragment's registers at a time
    });
  });
  if constexpr (kSym) {
    if (ti == tj) return;
    const int s = lane & 15, g = lane >> 4;
#pragma unroll
    for (int n = 0; n < 32 * F; n += 16)
#pragma unroll
      for (int m = 0; m < 32 * F; m += 32) {
        // 16 columns of 32 rows: a lane takes column n + s and rows m + 8 g ..
        const int row = m + 8 * g + (s >> 2), col = n + 4 * (s & 3);
        const v8h y = read_columns(turn + side(row, col), turn + side(row + 4, col));
        store_at(global(out + (int64_t)(n0 + wn + n) * ld + m0 + wm + m) + ((uint32_t)s * (uint32_t)ld + 8 * g), y);
      }
  }
}

// ---------------------------------------------------------------------------
// Small matrices: a workgroup of sixteen waves takes one through all of its steps
// in LDS: X (its low part in registers, where the last product left it), A and
// B.  What a launch for each product costs (3 to 4 us each, 17 of them) is more
// than the work.  The rows of all three are an odd number of 16 bytes apart, so
// that row reads and transposing reads part the banks.  128 x 256: 43 us (8 waves:
// 53, whose vector instructions and LDS latency hid less behind one another; a
// launch for each product: 66); 64 matrices of 64 x 64: 48 (164).
constexpr int kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64;

constexpr int NF = 2;                      // fragments of X a wave has at most

__global__ void __launch_bounds__(kSmallThreads) ortho_small(const Args a, const OrthoStep step) {
  extern __shared__ __attribute__((aligned(16))) uint8_t mem[];
  const OrthoItem t = a.item[blockIdx.x];
  const View v = view(t);
  const Moment c = moment_of(step);
  const int px = ortho_pitch(v.n), ps = ortho_pitch(v.m);        // bytes between rows
  uint8_t *const sX = mem, *const sA = sX + v.m * px, *const sB = sA + v.m * ps;
  // U and the result, [m][n] in float32, before and after the others
  float* const whole = (float*)mem;
  const int pw = v.n + 4;
  __shared__ double red[kSmallThreads / 64];
  const int th = threadIdx.x, lane = th & 63, wave = __builtin_amdgcn_readfirstlane(th >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const bool tall = t.rows > t.cols;
  const int fm = v.m / 32, fms = fm == 4 ? 2 : 1, frags = fm * (v.n / 32);       // v.m is 64 or 128
  // fragment f of the wave: strips (i, j) of X; a lane has row l % 32 and columns 8 h .. and 16 + 8 h ..
  auto strips = [&](int f, int& i, int& j) {
    const int k = wave + kSmallWaves * f;
    i = k & (fm - 1);
    j = k >> fms;
    return k < frags;
  };
  // U in pieces of four neighbouring values: a wave takes as many rows at a time as 64 lanes hold, kAtOnce times
  const int pieces = (t.cols + 3) / 4, shift = pieces > 32 ? 6 : pieces > 1 ? 32 - __builtin_clz(pieces - 1) : 0, across = 1 << shift;
  const int rows_at_once = 64 >> shift, lane_row = lane >> shift, lane_col = 4 * (lane & (across - 1));
  constexpr int kAtOnce = 4;
  // begin(e, row, column) for the lane's pieces of a batch, which asks for what they need, then end(e, row, column)
  auto batches = [&](auto begin, auto end) {
#pragma unroll 1
    for (int col = lane_col; col - lane_col < t.cols; col += 256)
#pragma unroll 1
      for (int from = wave * rows_at_once; from < t.rows; from += kSmallWaves * kAtOnce * rows_at_once) {
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) begin(e, from + kSmallWaves * e * rows_at_once + lane_row, col);
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) end(e, from + kSmallWaves * e * rows_at_once + lane_row, col);
      }
  };
  auto count_of = [&](int row, int col) { return row < t.rows ? min(4, t.cols - col) : 0; };

  for (int i = th; i < v.m * pw / 4; i += kSmallThreads) ((v4f*)whole)[i] = v4f{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  double sum = 0.0;
  {
#pragma clang fp contract(off)
    float u[kAtOnce][4], x[kAtOnce][4];
    batches(
        [&](int e, int row, int col) {
          const int count = count_of(row, col);
          if (count <= 0) return;
          load_gradient(t, (int64_t)row * t.ld_g + col, count, c.scale, u[e]);
          if (t.moment != nullptr) load_values(t.moment + row * t.cols + col, count, x[e]);
        },
        [&](int e, int row, int col) {
          const int count = count_of(row, col);
          if (count <= 0) return;
          if (t.moment != nullptr) {
            float* to = t.moment + row * t.cols + col;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[e][k] = x[e][k] * c.mu + u[e][k] * c.rest;
              if (k < count) to[k] = x[e][k];
              u[e][k] = update_of(u[e][k], x[e][k], c);
            }
          }
          if (tall) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < count) whole[(col + k) * pw + row] = u[e][k];
          } else {
            // past the last column these are zeros, and inside the padded row
            *(v4f*)(whole + row * pw + col) = v4f{u[e][0], u[e][1], u[e][2], u[e][3]};
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) sum += (double)u[e][k] * (double)u[e][k];
        });
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) red[wave] = sum;
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int i = 1; i < kSmallThreads / 64; ++i) sum += red[i];
  const Scale scale = scale_of(sum, step.eps);

  v8h high[NF][2], low[NF][2];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    int i, j;
    if (!strips(f, i, j)) continue;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const v4f* u = (const v4f*)(whole + (32 * i + l32) * pw + 32 * j + 16 * q + 8 * h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = scaled(u[e / 4][e % 4], scale);
        high[f][q][e] = (half_t)x;
        low[f][q][e] = (half_t)(x - (float)high[f][q][e]);
      }
    }
  }
  auto keep_x = [&]() {
    __syncthreads();                         // what X takes the place of has been read
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      int i, j;
      if (!strips(f, i, j)) continue;
#pragma unroll
      for (int q = 0; q < 2; ++q) *(v8h*)(sX + (32 * i + l32) * px + 2 * (32 * j + 16 * q + 8 * h)) = high[f][q];
    }
    __syncthreads();
  };

  const int order = strip_col(l32);
  const int chunk = strip_col(4 * (4 * ((lane >> 4) & 1) + (lane & 3))), krow = 8 * h + ((lane >> 2) & 3);
  // strip i of a matrix as the second operand, strip j as the first, 16 k from 16 s on
  auto rows_of = [&](const uint8_t* x, int pitch, int i, int s) {
    return *(const v8h*)(x + (32 * i + l32) * pitch + 32 * s + 16 * h);
  };
  auto strip_of = [&](const uint8_t* x, int pitch, int j, int s) {
    return *(const v8h*)(x + (32 * j + order) * pitch + 32 * s + 16 * h);
  };
  auto columns_of = [&](const uint8_t* x, int pitch, int j, int s) {
    const uint8_t* p = x + (16 * s + krow) * pitch + 2 * (32 * j + chunk);
    return read_columns(p, p + 4 * pitch);
  };
  const v16f zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  // A wave's fragments lie in one strip of rows, since the waves are a multiple of the strips: they share the second
  // operand, and their products are independent of one another.  Strips past the last are computed and left.
  const int i = wave & (fm - 1), j0 = wave >> fms, js = kSmallWaves >> fms;      // fragment f is (i, j0 + js f)
  auto square = [&](const uint8_t* x, int pitch, int k16, auto done) {
    if (j0 >= fm) return;
    v16f d = zero;
#pragma unroll 4
    for (int s = 0; s < k16; ++s)
      d = __builtin_amdgcn_mfma_f32_32x32x16_f16(strip_of(x, pitch, j0, s), rows_of(x, pitch, i, s), d, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float o[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) o[r] = d[8 * q + r];
      done(32 * i + l32, 32 * j0 + 16 * q + 8 * h, o);
    }
  };
  auto squares = [&](bool last) {
    // A = X X^T
    square(sX, px, v.n / 16, [&](int m, int n, const float (&o)[8]) {
      v8h y;
#pragma unroll
      for (int r = 0; r < 8; ++r) y[r] = (half_t)(o[r] * (kScaleA / (kScaleX * kScaleX)));
      *(v8h*)(sA + m * ps + 2 * n) = y;
    });
    __syncthreads();
    // B = b A + c A A, and a on its diagonal in the last step
    const float fb = (float)(step.b / kScaleA), fc = (float)(step.c / ((double)kScaleA * kScaleA));
    const float fa = last ? (float)step.a : 0.0f;
    square(sA, ps, v.m / 16, [&](int m, int n, const float (&o)[8]) {
      const v8h base = *(const v8h*)(sA + m * ps + 2 * n);
      v8h y;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        float b = fmaf(fb, (float)base[r], o[r] * fc);
        if (n + r == m) b += fa;
        y[r] = (half_t)b;
      }
      *(v8h*)(sB + m * ps + 2 * n) = y;
    });
    __syncthreads();
  };
  v16f d[NF];
  auto products_of_x = [&]() {
#pragma unroll
    for (int f = 0; f < NF; ++f) d[f] = zero;
#pragma unroll 2
    for (int s = 0; s < v.m / 16; ++s) {
      const v8h p = rows_of(sB, ps, i, s);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int j = j0 + js * f < v.n / 32 ? j0 + js * f : 0;
        d[f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(columns_of(sX, px, j, s), p, d[f], 0, 0, 0);
      }
    }
  };
#pragma unroll 1
  for (int k = 0; k < step.steps; ++k) {
    keep_x();
    squares(k + 1 == step.steps);
    products_of_x();
    // X' = a X + B X
#pragma unroll
    for (int f = 0; f < NF; ++f) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = fmaf((float)step.a, (float)low[f][q][e] + (float)high[f][q][e], d[f][8 * q + e]);
          high[f][q][e] = (half_t)y;
          low[f][q][e] = (half_t)(y - (float)high[f][q][e]);
        }
    }
  }
  // the last step's B X is the result
  __syncthreads();
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    int i, j;
    if (!strips(f, i, j)) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r)
      whole[(32 * i + l32) * pw + 32 * j + 16 * (r / 8) + 8 * h + r % 8] = d[f][r] * (1.0f / kScaleX);
  }
  __syncthreads();
  float keep, rate;
  rates(t, step, keep, rate);
  {
#pragma clang fp contract(off)
    float w[kAtOnce][4];
    batches(
        [&](int e, int row, int col) {
          const int count = count_of(row, col);
          if (t.w != nullptr && count > 0) load_values(t.w + row * t.cols + col, count, w[e]);
        },
        [&](int e, int row, int col) {
          const int count = count_of(row, col);
          if (count <= 0) return;
          float o[4];
          if (tall) {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = k < count ? whole[(col + k) * pw + row] : 0.0f;
          } else {
            const v4f y = *(const v4f*)(whole + row * pw + col);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = y[k];
          }
          const int at = row * t.cols + col;
          const int64_t to = row * t.ld_out + col;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= count) continue;
            if (t.w != nullptr) {
              const float x = w[e][k] * keep - o[k] * rate;
              t.w[at + k] = x;
              if (t.copy != nullptr) t.copy[at + k] = (uint16_t)pack_bf16(x, 0.0f);
            } else if (t.out_bf16) {
              ((uint16_t*)t.out)[to + k] = (uint16_t)pack_bf16(o[k], 0.0f);
            } else {
              ((float*)t.out)[to + k] = o[k];
            }
          }
        });
  }
}

// Whether every item fits ortho_small; launches it if so.
bool small_items(const Args& a, const OrthoStep& step, hipStream_t s) {
  int64_t bytes = 0;
  for (int i = 0; i < a.count; ++i) {
    const OrthoSize z = ortho_size(a.item[i].rows, a.item[i].cols);
    if (!ortho_small_fits(z)) return false;
    const int64_t need = ortho_small_bytes(z);
    bytes = need > bytes ? need : bytes;
  }
  const dim3 g((unsigned)a.count), b(kSmallThreads);
  hipLaunchKernelGGL(ortho_small, g, b, (uint32_t)bytes, s, a, step);
  return true;
}

// a's items by falling `key`, so that the longest tiles start first.
template <typename Key>
void sort_items(Args& a, const Key& key) {
  for (int i = 1; i < a.count; ++i)
    for (int k = i; k > 0 && key(a.item[k - 1]) < key(a.item[k]); --k) std::swap(a.item[k - 1], a.item[k]);
}

// (The item by value: by reference, the tall matrices' last step spilled its accumulators.)
template <int F, int S, int MODE>
__global__ void __launch_bounds__(256, F < 3 ? 2 : 1) ortho_product(const Args a, const OrthoStep step, const Coef c) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * S * 64 * F * kRow];
  int id;
  const OrthoItem t = a.item[find(a, id)];
  if constexpr (MODE == kLast) {
    if (t.rows > t.cols) {
      product_tile<F, S, MODE, true>(t, id, step, c, lds);
      return;
    }
  }
  product_tile<F, S, MODE, false>(t, id, step, c, lds);
}

// Workgroups of each item, `of(item)` of them, as a's table; their number.
template <typename Of>
int deal(Args& a, const Of& of) {
  int total = 0;
  for (int i = 0; i < kOrthoGroup; ++i) {
    if (i < a.count) total += of(a.item[i]);
    a.end[i] = total;
  }
  return total;
}

template <int F, int S, int MODE>
void products(Args& a, const OrthoStep& step, const Coef& c, hipStream_t s) {
  const int total = deal(a, [&](const OrthoItem& t) {
    const OrthoSize z = ortho_size(t.rows, t.cols);
    return (int)((ortho_tiles(z, MODE <= kMix, F) + kXcds - 1) / kXcds * kXcds);
  });
  hipLaunchKernelGGL((ortho_product<F, S, MODE>), dim3((unsigned)total), dim3(256), 0, s, a, step, c);
}

// The tile whose time for these items is the least.
template <int MODE>
OrthoTile tile_of(const Args& a) {
  OrthoSize sizes[kOrthoGroup];
  for (int i = 0; i < a.count; ++i) sizes[i] = ortho_size(a.item[i].rows, a.item[i].cols);
  return ortho_choose(sizes, a.count, MODE <= kMix, MODE == kGram);
}

template <int MODE>
void products_of(Args& a, OrthoTile tile, const OrthoStep& step, const Coef& c, hipStream_t s) {
  switch (tile) {
    case OrthoTile::k64: products<1, 4, MODE>(a, step, c, s); break;
    case OrthoTile::k128: products<2, 3, MODE>(a, step, c, s); break;
    case OrthoTile::k128Two: products<2, 2, MODE>(a, step, c, s); break;
    case OrthoTile::k192: products<3, 3, MODE>(a, step, c, s); break;
    case OrthoTile::k256: products<4, 2, MODE>(a, step, c, s); break;
  }
}

}  // namespace

hipError_t launch_ortho(const OrthoItem* items, int count, const OrthoStep& step, hipStream_t s) {
  Args a;
  a.count = count;
  for (int i = 0; i < kOrthoGroup; ++i) a.item[i] = items[i < count ? i : count - 1];
  if (small_items(a, step, s)) return hipGetLastError();
  int total = deal(a, [](const OrthoItem& t) { return (int)ortho_size(t.rows, t.cols).parts; });
  hipLaunchKernelGGL(ortho_sum, dim3((unsigned)total), dim3(kSumThreads), 0, s, a, step);
  total = deal(a, [](const OrthoItem& t) {
    const OrthoSize z = ortho_size(t.rows, t.cols);
    return (int)(z.m / 64 * (z.n / 64));
  });
  hipLaunchKernelGGL(ortho_start, dim3((unsigned)total), dim3(256), 0, s, a, step);
  // Gram: a tile's K is the longer side; the others: the shorter
  Args by_n = a, by_m = a;
  sort_items(by_n, [](const OrthoItem& t) { return t.rows > t.cols ? t.rows : t.cols; });
  sort_items(by_m, [](const OrthoItem& t) { return t.rows < t.cols ? t.rows : t.cols; });
  const OrthoTile gram = tile_of<kGram>(by_n), poly = tile_of<kPoly>(by_m), next = tile_of<kStep>(by_m);
  Coef c{};
  auto gram_of_x = [&](int from) {
    c.from = from;
    c.out = 0;
    products_of<kGram>(by_n, gram, step, c, s);
  };
  // out = b A + c A A, and a on its diagonal if asked for
  auto poly_of = [&](int of, int out, double diagonal) {
    c.left = c.right = c.add = of;
    c.out = out;
    c.f = (float)(step.b / kScaleA);
    c.g = (float)(step.c / ((double)kScaleA * kScaleA));
    c.diagonal = (float)diagonal;
    products_of<kPoly>(by_m, poly, step, c, s);
    c.diagonal = 0.0f;
  };
  // out = f S + L R
  auto times = [&](double f, int add, int left, int right, int out) {
    c.f = (float)f;
    c.g = 1.0f;
    c.add = add;
    c.left = left;
    c.right = right;
    c.out = out;
    products_of<kPoly>(by_m, poly, step, c, s);
  };
  int k = 0, from = 0;
  // The first two steps in one, where the list's matrices are wide: with P0 = a I + B0 and P1 = a I + B1 their factors, X2
  // = P1 P0 X0, and A1 = P0 A0 P0 comes from squares instead of a second pass over X.  That trades 3 m^2 n products for 3
  // m^3 and a pass of X.  Where roundings are independent it costs up to a fifth of the error (rank 1: 1.4e-3 -> 1.6e-3;
  // noise: 1.5e-3 either way); P1 P0 - a^2 is ten times P1 P0, which doubles the error of a constant matrix (at most
  // 1.5e-2 -> 2.5e-2).  (Three steps in one lose weak directions: 4e-3 off on a matrix of rank 1.)
  if (step.steps >= 3 && ortho_joins(by_m.item, count)) {
    gram_of_x(0);                                    // 0: A0
    poly_of(0, 1, 0.0);                              // 1: B0
    times(step.a, 0, 1, 0, 2);                       // 2: P0 A0
    times(step.a, 2, 1, 2, 0);                       // 0: A1 = P0 (P0 A0)
    poly_of(0, 2, 0.0);                              // 2: B1
    c.f = c.f2 = (float)step.a;                      // 0: P1 P0 - a^2 I = a B0 + a B1 + B1 B0
    c.g = 1.0f;
    c.add = c.left = 1;
    c.add2 = c.right = 2;
    c.out = 0;
    products_of<kMix>(by_m, poly, step, c, s);
    c.left = 0;
    c.x = (float)(step.a * step.a);
    products_of<kStep>(by_m, next, step, c, s);
    k = 2;
    from = 1;
  }
  for (; k < step.steps; ++k, from ^= 1) {
    const bool last = k + 1 == step.steps;
    gram_of_x(from);
    poly_of(0, 1, last ? step.a : 0.0);
    c.left = 1;
    c.x = (float)step.a;
    if (last) products_of<kLast>(by_m, next, step, c, s);
    else products_of<kStep>(by_m, next, step, c, s);
  }
  return hipGetLastError();
}

}  // namespace mx
