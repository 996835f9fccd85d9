// 8-bit block-scaled matrix product on gfx950's matrix cores:
//
//   C[m][n] = sum_b sa[b][m] * sb[b][n] * sum_{k in block b} A[m][k] B[n][k]
//
// A and B are K-contiguous 8-bit operands (E4M3 or E5M2), K in blocks of 128;
// A has a float32 scale per line and block, B one per line and block or one
// per 128 x 128 tile.  The scales are general float32 numbers, which the
// matrix instructions' power-of-two block scales cannot carry, so each block's
// product is formed from a zero accumulator and joins the float32 sum by one
// fused multiply-add per element.
//
// Two matrix instructions, by the output's type.
//  - bf16 output: V_MFMA_F32_16X16X128_F8F6F4, whose K is exactly one block.
//    Within each run of 8 neighbouring k of a lane it aligns the products to
//    the largest and drops what lies below 2^-13 of it (found with one large
//    and one small product; between the runs it adds in float32).  On normal
//    data that is 1.5e-5 of the result's norm, a hundredth of what rounding to
//    bf16 costs.
//  - fp32 output: the codes become bf16 (exact for both formats) after the LDS
//    read and run V_MFMA_F32_16X16X32_BF16: exact products, float32 sums, half
//    the matrix rate.  Whoever asks for float32 gets its accuracy.
//
// Operand layout of the 16x16x128 instruction on 8-bit data: lane l holds row
// l % 16 and 32 bytes of its 128 k (which 32 does not matter, as long as both
// operands agree; the bf16 form takes the same bytes eight at a time); the
// 16 x 16 result has row 4 (l / 16) + r in register r and column l % 16.  B is
// passed as the first operand and A as the second, so a lane's accumulators
// belong to one row m of C (one A scale per lane) and to four neighbouring
// columns n.  Fragment j of a 64-column strip holds the strip's columns
// 16 h + 4 j + i (h = 0..3, i = 0..3) as its rows 4 h + i: a lane then ends with
// the sixteen consecutive columns 16 (l / 16) .. + 15 over j = 0..3, and stores
// them without any exchange between lanes.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include "fp8_kernels.h"

namespace mx {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kKB = 128;      // bytes (values) of a row per K step

// 16-byte piece position in a 128-byte LDS row: lanes of a fragment read (16
// consecutive rows, one piece) or write whole rows without bank conflicts.
__device__ __forceinline__ int slot(int row, int piece) { return (piece ^ ((row >> 1) & 7)) * 16; }

// the strip column that row f of the strip's LDS rows holds (fragment order)
__device__ __forceinline__ int strip_col(int f) { return 16 * ((f >> 2) & 3) + 4 * (f >> 4) + (f & 3); }

__device__ __forceinline__ v8i fragment(const uint8_t* lds, int row, int q) {
  const u32x4 x = *(const u32x4*)(lds + row * kKB + slot(row, 2 * q));
  const u32x4 y = *(const u32x4*)(lds + row * kKB + slot(row, 2 * q + 1));
  return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// An operand fragment as the matrix instruction of the output type takes it.
template <bool EXACT>
struct Operand;

template <>
struct Operand<false> {
  v8i x;
};

template <>
struct Operand<true> {
  bf16x8_t x[4];       // bytes 8 q .. 8 q + 7 of the lane's 32
};

// eight codes of one format as bf16
template <int FMT>
__device__ __forceinline__ bf16x8_t widen(uint32_t lo, uint32_t hi) {
  bf16x2_t v[4];
  if constexpr (FMT == MX_FP8_E4M3) {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  } else {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
  }
  return bf16x8_t{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
}

template <int FMT, bool EXACT>
__device__ __forceinline__ Operand<EXACT> operand(const v8i& x) {
  Operand<EXACT> o;
  if constexpr (EXACT) {
#pragma unroll
    for (int q = 0; q < 4; ++q) o.x[q] = widen<FMT>((uint32_t)x[2 * q], (uint32_t)x[2 * q + 1]);
  } else {
    o.x = x;
  }
  return o;
}

// One block's product of two fragments.  Format codes: 0 E4M3, 1 E5M2; zero scale operands select the
// instruction without block scales.
template <int BF, int AF, bool EXACT>
__device__ __forceinline__ v4f mma(const Operand<EXACT>& b, const Operand<EXACT>& a) {
  v4f d = v4f{0.f, 0.f, 0.f, 0.f};
  if constexpr (EXACT) {
#pragma unroll
    for (int q = 0; q < 4; ++q) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.x[q], a.x[q], d, 0, 0, 0);
  } else {
    d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.x, a.x, d, BF, AF, 0, 0, 0, 0);
  }
  return d;
}

// round to nearest even, NaN quieted
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
}

// 16 bytes at any address that a row of C may start at: one store, whatever the row pitch
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

// Sixteen consecutive columns of one row of C from a lane's accumulators.
template <int OUT>
__device__ __forceinline__ void store16(const Fp8GemmParams& p, int64_t m, int64_t n, const v4f (&acc)[4]) {
  if (m >= p.M || n >= p.N) return;
  const int64_t at = m * p.ldc + n;
  if (n + 16 <= p.N) {
    if constexpr (OUT == MX_OUT_F32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) *(v4f_any*)((float*)p.c + at + 4 * j) = acc[j];
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *(u32x4_any*)((uint16_t*)p.c + at + 8 * h) =
            u32x4{pack_bf16(acc[2 * h][0], acc[2 * h][1]), pack_bf16(acc[2 * h][2], acc[2 * h][3]),
                  pack_bf16(acc[2 * h + 1][0], acc[2 * h + 1][1]), pack_bf16(acc[2 * h + 1][2], acc[2 * h + 1][3])};
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (n + 4 * j + r >= p.N) return;
      if constexpr (OUT == MX_OUT_F32) ((float*)p.c)[at + 4 * j + r] = acc[j][r];
      else ((uint16_t*)p.c)[at + 4 * j + r] = (uint16_t)pack_bf16(acc[j][r], 0.0f);
    }
}

// ---------------------------------------------------------------------------
// Bounds-checked kernel, any shape: a 128 x 128 tile of C per workgroup, four
// waves of 64 x 64, operands through registers into LDS one K block at a time.
constexpr int kGT = 128, kGThreads = 256;

template <int AF, int BF, int KIND, int OUT>
__global__ void __launch_bounds__(kGThreads) fp8_mm_any(const Fp8GemmParams p, int64_t tiles_m) {
  __shared__ __attribute__((aligned(16))) uint8_t sA[kGT * kKB], sB[kGT * kKB];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t m0 = (blockIdx.x % tiles_m) * kGT, n0 = (blockIdx.x / tiles_m) * kGT;
  const int wm = 64 * (wave & 1), wn = 64 * (wave >> 1);
  const int64_t nk = (p.K + kKB - 1) / kKB;
  const int lrow = lane & 15, q = lane >> 4;

  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  const int64_t col = n0 + wn + 16 * q;      // the lane's first column of C
  for (int64_t kb = 0; kb < nk; ++kb) {
    u32x4 ra[4], rb[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 32 * e + (t >> 3), piece = t & 7;
      const int64_t m = m0 + row, n = n0 + (row & 64) + strip_col(row & 63);
      ra[e] = m < p.M ? *(const u32x4*)(p.a_codes + m * p.lda + kb * kKB + piece * 16) : u32x4{0u, 0u, 0u, 0u};
      rb[e] = n < p.N ? *(const u32x4*)(p.b_codes + n * p.ldb + kb * kKB + piece * 16) : u32x4{0u, 0u, 0u, 0u};
    }
    float sa[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + wm + 16 * i + lrow;
      sa[i] = m < p.M ? p.a_scales[kb * p.lda_scales + m] : 0.0f;
    }
    float sb[16];
    if constexpr (KIND == MX_FP8_TILE) {
      sb[0] = n0 < p.N ? p.b_scales[(n0 / kFp8Block) * p.ldb_scales + kb] : 0.0f;
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) sb[e] = col + e < p.N ? p.b_scales[kb * p.ldb_scales + col + e] : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 32 * e + (t >> 3), piece = t & 7;
      *(u32x4*)(sA + row * kKB + slot(row, piece)) = ra[e];
      *(u32x4*)(sB + row * kKB + slot(row, piece)) = rb[e];
    }
    __syncthreads();
    constexpr bool kExact = OUT == MX_OUT_F32;
    Operand<kExact> fb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) fb[j] = operand<BF, kExact>(fragment(sB, wn + 16 * j + lrow, q));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Operand<kExact> fa = operand<AF, kExact>(fragment(sA, wm + 16 * i + lrow, q));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4f d = mma<BF, AF, kExact>(fb[j], fa);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] = fmaf(d[r], sa[i] * (KIND == MX_FP8_TILE ? sb[0] : sb[4 * j + r]), acc[i][j][r]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) store16<OUT>(p, m0 + wm + 16 * i + lrow, col, acc[i]);
}

// ---------------------------------------------------------------------------
// Large products: a persistent grid, one workgroup per CU, each walking 256 x
// 256 tiles of C with eight waves of 128 x 64 (two waves per SIMD).  K advances
// one block (a 128-byte line of every operand row) per step, copied global ->
// LDS by DMA into one of two 64 KB stages while the other is consumed.
//
// A wave holds the step's four B fragments and streams its eight A fragments;
// row i's four matrix instructions run beside the fused multiply-adds of row
// i - 1, so their results are never waited for.  The step's last two rows run
// column by column after the barrier that frees the stage: a B fragment is
// replaced by the next step's as soon as its two instructions are issued, which
// hides the next step's first LDS reads behind the last quarter of this one.
//
// Rows of a tile past the operand's last line read that line again (their
// results are not stored), so every copy stays inside the operand and any M
// and N run here.
constexpr int kBT = 256, kBThreads = 512, kXcds = 8, kGroupM = 4, kGroupN = 8;
constexpr int kStage = kBT * kKB;

// Global -> LDS copy of 16 (4) bytes per lane: LDS address = M0 + size * lane.  Inline asm, so that the
// compiler places no waits of its own for it; it writes no register.  An SALU write of M0 needs one wait
// state before the copy reads it.
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
template <typename T>
__device__ __forceinline__ const T* uniform(const T* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const T*)(((uint64_t)hi << 32) | lo);
}

// Tiles are dealt in groups of 4 (M) x 8 (N) to the 8 XCDs, a group to the 32 CUs of one, so that the tiles
// an XCD computes at once share 4 A strips and 8 B strips in its L2.
struct BigMap {
  int tiles_m, tiles_n, groups_m, groups, rounds;
};

__device__ __forceinline__ int next_tile(const BigMap& t, int r, int& bm, int& bn) {
  const int xcd = blockIdx.x % kXcds, member = blockIdx.x / kXcds;
  for (; r < t.rounds; ++r) {
    const int g = r * kXcds + xcd;
    if (g >= t.groups) return t.rounds;
    bm = (g % t.groups_m) * kGroupM + member % kGroupM;
    bn = (g / t.groups_m) * kGroupN + member / kGroupM;
    if (bm < t.tiles_m && bn < t.tiles_n) return r;
  }
  return t.rounds;
}

template <int AF, int BF, int KIND>
__global__ void __launch_bounds__(kBThreads, 2) fp8_mm_big(const Fp8GemmParams p, const BigMap map) {
  __shared__ __attribute__((aligned(1024))) uint8_t sA[2][kStage], sB[2][kStage];
  __shared__ __attribute__((aligned(1024))) float sSA[2][kBT], sSB[2][kBT];

  int bm = 0, bn = 0;
  int r = next_tile(map, 0, bm, bn);
  if (r >= map.rounds) return;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = 128 * (wave & 1), wn = 64 * (wave >> 1);
  const int lrow = lane & 15, q = lane >> 4;
  const int nk = (int)((p.K + kKB - 1) / kKB);

  // Copies: one instruction moves eight rows (lane i: row i / 8, LDS piece i % 8, which holds the row's piece
  // i % 8 ^ swizzle).  Wave w copies LDS rows 32 w .. 32 w + 31 of A and of B, and the scales of rows
  // 64 (w % 4) .. + 63 of A (w < 4) or B.
  const int l8 = lane >> 3;
  const int piece0 = ((lane & 7) ^ (l8 >> 1)) * 16, piece1 = ((lane & 7) ^ (4 + (l8 >> 1))) * 16;
  const int brow = 16 * (l8 >> 2) + (l8 & 3);              // the lane's part of strip_col
  const uint32_t dA = lds_addr(&sA[0][32 * wave * kKB]), dB = lds_addr(&sB[0][32 * wave * kKB]);
  auto issue = [&](int tm, int tn, int kt, int st) {
    const int64_t m0 = (int64_t)tm * kBT, n0 = (int64_t)tn * kBT;
    const uint32_t ma = (uint32_t)(p.M - 1 - m0 < kBT ? p.M - 1 - m0 : kBT - 1);
    const uint32_t na = (uint32_t)(p.N - 1 - n0 < kBT ? p.N - 1 - n0 : kBT - 1);
    const uint8_t* a = uniform(p.a_codes + m0 * p.lda + (int64_t)kt * kKB);
    const uint8_t* b = uniform(p.b_codes + n0 * p.ldb + (int64_t)kt * kKB);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // LDS row f = 32 w + 8 e + l8; of B it is column 64 (f / 64) + strip_col(f % 64)
      const uint32_t ra = min((uint32_t)(32 * wave + 8 * e + l8), ma);
      const int s8 = 4 * (wave & 1) + e;
      const uint32_t rb = min((uint32_t)(64 * (wave >> 1) + 32 * (s8 & 1) + 4 * (s8 >> 1) + brow), na);
      const uint32_t piece = (uint32_t)((e & 1) ? piece1 : piece0);
      dma16(a, __umul24(ra, (uint32_t)p.lda) + piece, dA + st * kStage + e * 8 * kKB);
      dma16(b, __umul24(rb, (uint32_t)p.ldb) + piece, dB + st * kStage + e * 8 * kKB);
    }
    const uint32_t f = (uint32_t)(64 * (wave & 3) + lane);
    if (wave < 4) {
      dma4(uniform(p.a_scales + (int64_t)kt * p.lda_scales + m0), 4 * min(f, ma), lds_addr(&sSA[st][64 * (wave & 3)]));
    } else if constexpr (KIND == MX_FP8_LINE) {
      dma4(uniform(p.b_scales + (int64_t)kt * p.ldb_scales + n0), 4 * min(f, na), lds_addr(&sSB[st][64 * (wave & 3)]));
    } else if (wave == 4) {
      // a tile's two scales, each for 128 columns: lanes 0 .. 31 copy the first, 32 .. 63 the second
      const uint32_t last = (uint32_t)((p.N - 1) / kFp8Block), first = (uint32_t)(n0 / kFp8Block);
      const uint32_t row = min(first + (uint32_t)(lane >> 5), last) - first;
      dma4(uniform(p.b_scales + (int64_t)first * p.ldb_scales + kt), 4 * row * (uint32_t)p.ldb_scales,
           lds_addr(&sSB[st][0]));
    }
  };

  v4f acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  int nbm = 0, nbn = 0;
  int rn = next_tile(map, r + 1, nbm, nbn);
  issue(bm, bn, 0, 0);
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  if (nk > 1) issue(bm, bn, 1, 1);
  else if (rn < map.rounds) issue(nbm, nbn, 0, 1);

  v8i fb[4], fa[2];
  float sa[8], sb[KIND == MX_FP8_LINE ? 16 : 1];
  int st = 0;
  // a fragment row's two pieces: their place depends on the lane only, rows 16 apart are immediates
  const uint32_t off0 = lrow * kKB + ((2 * q) ^ (lrow >> 1)) * 16, off1 = lrow * kKB + ((2 * q + 1) ^ (lrow >> 1)) * 16;
  auto read = [&](const uint8_t* base, int f) {
    const u32x4 x = *(const u32x4*)(base + off0 + f * 16 * kKB), y = *(const u32x4*)(base + off1 + f * 16 * kKB);
    return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  };
  auto read_scales = [&](int stage) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sa[i] = sSA[stage][wm + 16 * i + lrow];
    if constexpr (KIND == MX_FP8_LINE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4f x = *(const v4f*)&sSB[stage][wn + 16 * q + 4 * j];
#pragma unroll
        for (int e = 0; e < 4; ++e) sb[4 * j + e] = x[e];
      }
    } else {
      const float s = sSB[stage][(wn >> 7) * 32];
#pragma unroll
      for (int i = 0; i < 8; ++i) sa[i] *= s;
    }
  };
  auto join = [&](v4f& c, const v4f& d, int i, int j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = fmaf(d[e], KIND == MX_FP8_LINE ? sa[i] * sb[4 * j + e] : sa[i], c[e]);
    // the sums have no use before the next step: without this they are sunk there, every product kept until then
    asm volatile("" : "+v"(c));
  };
  auto mul = [&](const v8i& b, const v8i& a) {
    Operand<false> x, y;
    x.x = b;
    y.x = a;
    return mma<BF, AF, false>(x, y);
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) fb[j] = read(sB[0] + wn * kKB, j);
  fa[0] = read(sA[0] + wm * kKB, 0);
  read_scales(0);
  for (;;) {
    for (int kt = 0; kt < nk; ++kt) {
      v4f d[2][4];
      const uint8_t* a = sA[st] + wm * kKB;
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        fa[(i + 1) & 1] = read(a, i + 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[i & 1][j] = mul(fb[j], fa[i & 1]);
          if (i > 0) join(acc[i - 1][j], d[(i - 1) & 1][j], i - 1, j);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // rows 6 and 7
      fa[1] = read(a, 7);
      const bool more = kt + 1 < nk || rn < map.rounds;
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (kt + 2 < nk) issue(bm, bn, kt + 2, st);
      else if (rn < map.rounds && kt + 2 - nk < nk) issue(nbm, nbn, kt + 2 - nk, st);
      st ^= 1;
      const uint8_t* b = sB[st] + wn * kKB;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[0][j] = mul(fb[j], fa[0]);
        join(acc[5][j], d[1][j], 5, j);
        d[1][j] = mul(fb[j], fa[1]);
        if (more) fb[j] = read(b, j);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (more) fa[0] = read(sA[st] + wm * kKB, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        join(acc[6][j], d[0][j], 6, j);
        join(acc[7][j], d[1][j], 7, j);
      }
      if (more) read_scales(st);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      store16<MX_OUT_BF16>(p, (int64_t)bm * kBT + wm + 16 * i + lrow, (int64_t)bn * kBT + wn + 16 * q, acc[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    if (rn >= map.rounds) break;
    r = rn;
    bm = nbm;
    bn = nbn;
    rn = next_tile(map, r + 1, nbm, nbn);
  }
}

// The large-product kernel looks two steps ahead, so that K must span two blocks.  Its copies address a tile's rows by 32-bit offsets whose row pitch is a 24-bit factor.
bool big_offsets(const Fp8GemmParams& p) {
  const int64_t lim = int64_t(1) << 24;
  return p.lda < lim && p.ldb < lim && p.lda_scales < lim && p.ldb_scales < lim && p.K < (int64_t(1) << 30);
}

template <int AF, int BF, int KIND, int OUT>
void launch(const Fp8GemmParams& p, hipStream_t s) {
  if constexpr (OUT == MX_OUT_BF16) {
    if (p.M >= kBT && p.N >= kBT && p.K > kKB && big_offsets(p)) {
      BigMap map;
      map.tiles_m = (int)((p.M + kBT - 1) / kBT);
      map.tiles_n = (int)((p.N + kBT - 1) / kBT);
      map.groups_m = (map.tiles_m + kGroupM - 1) / kGroupM;
      map.groups = map.groups_m * ((map.tiles_n + kGroupN - 1) / kGroupN);
      map.rounds = (map.groups + kXcds - 1) / kXcds;
      hipLaunchKernelGGL((fp8_mm_big<AF, BF, KIND>), dim3(kXcds * kGroupM * kGroupN), dim3(kBThreads), 0, s, p, map);
      return;
    }
  }
  const int64_t tm = (p.M + kGT - 1) / kGT, tn = (p.N + kGT - 1) / kGT;
  hipLaunchKernelGGL((fp8_mm_any<AF, BF, KIND, OUT>), dim3((unsigned)(tm * tn)), dim3(kGThreads), 0, s, p, tm);
}

template <int AF, int BF>
void launch_kinds(const Fp8GemmParams& p, int b_kind, int out_kind, hipStream_t s) {
  if (b_kind == MX_FP8_TILE) {
    if (out_kind == MX_OUT_F32) launch<AF, BF, MX_FP8_TILE, MX_OUT_F32>(p, s);
    else launch<AF, BF, MX_FP8_TILE, MX_OUT_BF16>(p, s);
  } else {
    if (out_kind == MX_OUT_F32) launch<AF, BF, MX_FP8_LINE, MX_OUT_F32>(p, s);
    else launch<AF, BF, MX_FP8_LINE, MX_OUT_BF16>(p, s);
  }
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmParams& p, int a_fmt, int b_fmt, int b_kind, int out_kind, hipStream_t s) {
  if (a_fmt == MX_FP8_E4M3 && b_fmt == MX_FP8_E4M3) launch_kinds<MX_FP8_E4M3, MX_FP8_E4M3>(p, b_kind, out_kind, s);
  else if (a_fmt == MX_FP8_E5M2 && b_fmt == MX_FP8_E4M3) launch_kinds<MX_FP8_E5M2, MX_FP8_E4M3>(p, b_kind, out_kind, s);
  else if (a_fmt == MX_FP8_E4M3) launch_kinds<MX_FP8_E4M3, MX_FP8_E5M2>(p, b_kind, out_kind, s);
  else launch_kinds<MX_FP8_E5M2, MX_FP8_E5M2>(p, b_kind, out_kind, s);
  return hipGetLastError();
}

}  // namespace mx
