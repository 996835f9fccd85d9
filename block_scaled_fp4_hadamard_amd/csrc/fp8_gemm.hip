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
// 16 h + 4 j + i (h = 0..3, i = 0..3) as its rows 4 h + i: over j = 0..3 a lane
// then ends with the sixteen consecutive columns 16 (l / 16) .. + 15 of its row.
//
// Three kernels: few rows of A, 128 x 128 tiles, 256 x 256 tiles (fp8_plan says
// which product runs where).
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <utility>
#include "fp8_kernels.h"
#include "fp8_path.h"

namespace mx {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// 16-byte piece position in a 128-byte LDS row.  A 16-byte LDS read serves the
// wave in four groups of 16 lanes, taken from neighbouring 16-lane rows: 0-3,
// 12-15 and 20-27, then the other half, then the same of lanes 32 and up.  A
// fragment's lanes l read piece l / 16 (and l / 16 + 4) of row l % 16: with
// this order of the pieces each group covers all 64 banks.  Reading pieces
// 2 (l / 16) and 2 (l / 16) + 1 instead met every bank twice (45% of the LDS
// cycles of the large kernel).
__device__ __forceinline__ int slot(int row, int piece) { return (piece ^ ((row >> 1) & 7)) * 16; }

// f(0), f(1), ... f(N - 1), each index a constant of its own instance
template <int... I, typename F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, const F& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(const F& f) {
  each(std::make_integer_sequence<int, N>{}, f);
}

// the strip column that row f of the strip's LDS rows holds (fragment order)
__device__ __forceinline__ int strip_col(int f) { return 16 * ((f >> 2) & 3) + 4 * (f >> 4) + (f & 3); }

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Two codes (the low or the high half of a dword) as packed bf16, exact.
template <int FMT>
__device__ __forceinline__ uint32_t widen(uint32_t codes, bool high) {
  if constexpr (FMT == MX_FP8_E4M3)
    return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, false));
  else
    return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, 1.0f, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, 1.0f, false));
}

// A fragment's 32 codes of a lane as bf16, eight for each of four 32-deep instructions.
struct Wide {
  uint32_t w[16];
};

template <int FMT>
__device__ __forceinline__ Wide widen(const v8i& x) {
  Wide o;
#pragma unroll
  for (int c = 0; c < 16; ++c) o.w[c] = widen<FMT>((uint32_t)x[c >> 1], (c & 1) != 0);
  return o;
}

// codes 8 q .. 8 q + 7 of one block's product
__device__ __forceinline__ v4f mma_wide(const Wide& b, const Wide& a, int q, const v4f& d) {
  const u32x4 x = {b.w[4 * q], b.w[4 * q + 1], b.w[4 * q + 2], b.w[4 * q + 3]};
  const u32x4 y = {a.w[4 * q], a.w[4 * q + 1], a.w[4 * q + 2], a.w[4 * q + 3]};
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x), __builtin_bit_cast(bf16x8_t, y), d, 0,
                                                 0, 0);
}

// One block's product of two fragments.  Format codes: 0 E4M3, 1 E5M2; zero scale operands select the
// instruction without block scales.
template <int BF, int AF>
__device__ __forceinline__ v4f mma(const v8i& b, const v8i& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, v4f{0.f, 0.f, 0.f, 0.f}, BF, AF, 0, 0, 0, 0);
}

// round to nearest even, NaN quieted
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
}

// 16 bytes at any address that a row of C may start at: one store, whatever the row pitch
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

// A wave's 16 rows x 64 columns of C from its accumulators: row m0 + l % 16, columns n0 + 16 (l / 16) .. + 15 in
// lane l.  Non-temporal: the output streams past the L2, which keeps the operand rows that the next tiles read.
// bf16: lanes l and l ^ 8 trade halves of their 32 bytes, so that each store writes whole 128-byte pieces of
// eight rows.  fp32: each quad of lanes transposes its 4 x 4 pieces of 16 bytes, so that each store writes
// whole 256-byte pieces of four rows (a lane's own 64 bytes, stored as they are, reached 0.9 TB/s).  The last
// columns of an odd width go one by one.
__device__ __forceinline__ float dpp_xor1(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
}
__device__ __forceinline__ float dpp_xor2(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
}

template <int OUT>
__device__ __forceinline__ void store_rows(const Fp8GemmParams& p, int64_t m0, int64_t n0, int lane,
                                           const v4f (&acc)[4]) {
  const int lrow = lane & 15, q = lane >> 4;
  if constexpr (OUT == MX_OUT_F32) {
    // t[e] of lane 4 y + x: row 4 y + x, piece e; transposed, row 4 y + e, piece x
    v4f t[4] = {acc[0], acc[1], acc[2], acc[3]};
    const bool odd = (lane & 1) != 0, high = (lane & 2) != 0;
#pragma unroll
    for (int r = 0; r < 4; r += 2)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float got = dpp_xor1(odd ? t[r][e] : t[r + 1][e]);
        t[r][e] = odd ? got : t[r][e];
        t[r + 1][e] = odd ? t[r + 1][e] : got;
      }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float got = dpp_xor2(high ? t[r][e] : t[r + 2][e]);
        t[r][e] = high ? got : t[r][e];
        t[r + 2][e] = high ? t[r + 2][e] : got;
      }
    const int64_t n = n0 + 16 * q + 4 * (lrow & 3);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t m = m0 + (lrow & 12) + e;
      if (m >= p.M) continue;
      float* c = (float*)p.c + m * p.ldc + n;
      if (n + 4 <= p.N) {
        __builtin_nontemporal_store(t[e], (v4f_any*)c);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < p.N) c[r] = t[e][r];
      }
    }
  } else {
    u32x4 h[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      h[e] = u32x4{pack_bf16(acc[2 * e][0], acc[2 * e][1]), pack_bf16(acc[2 * e][2], acc[2 * e][3]),
                   pack_bf16(acc[2 * e + 1][0], acc[2 * e + 1][1]), pack_bf16(acc[2 * e + 1][2], acc[2 * e + 1][3])};
    const bool low = lrow < 8;
    u32x4 got;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      got[e] = (uint32_t)__builtin_amdgcn_mov_dpp((int)(low ? h[1][e] : h[0][e]), 0x128, 0xF, 0xF, false);   // l ^ 8
    const int64_t n = n0 + 16 * q + 8 * (lrow >> 3);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t m = m0 + (lrow & 7) + 8 * e;
      const u32x4 x = low == (e == 0) ? h[e] : got;
      if (m >= p.M) continue;
      uint16_t* c = (uint16_t*)p.c + m * p.ldc + n;
      if (n + 8 <= p.N) {
        __builtin_nontemporal_store(x, (u32x4_any*)c);
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (n + r < p.N) c[r] = (uint16_t)(x[r >> 1] >> (16 * (r & 1)));
      }
    }
  }
}

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
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const T*)(((uint64_t)hi << 32) | lo);
}

// ---------------------------------------------------------------------------
// Few rows of A (single tokens, short batches): the operand that matters is
// B, read once.  A workgroup takes 16 J columns of C (fp8_few_columns) and
// all M <= 16 F rows; its waves take the K blocks in turn, straight from memory
// to registers with U blocks in flight, and their sums meet in LDS in the
// waves' order.  Rows past M and columns past N read the last one and are not
// stored.
//
// Memory-bound.  Back to back in a graph, launch included, other weights each
// time (from HBM) and the same weights again (in the 256 MB last-level cache): one
// row takes 8.4 and 6.8 us with 6144 x 4096 (3.0 and 3.7 TB/s), 16.1 and 10.6 us
// with 4096 x 14336 (3.7 and 5.5), 26.7 and 20.0 with 28672 x 4096 (4.4 and 5.9), 74
// us either way with 28672 x 14336 (5.6); sixteen rows 10.0 and 8.0, 19.1 and 15.1,
// 28.1 and 21.1, 76; 32 rows 11.8 and 10.2, 22.5 and 21.5, 32.3 and 27.2, 95.  Eight
// waves rather than a split over workgroups: no second launch joins the parts.
// Sixteen waves took the same or more.
template <int AF, int BF, int KIND, int OUT, int F, int J>
__global__ void __launch_bounds__(64 * kFewWaves) fp8_mm_few(const Fp8GemmParams p) {
  constexpr bool kExact = OUT == MX_OUT_F32;
  // Fewer loads in flight are faster where they suffice: a fragment's two 16-byte pieces of a row are two
  // instructions' halves of one line, and with one block in flight a wave the second still finds it in the L1 (one row,
  // 8192 x 14336: 18.9 us against 22.6 with four blocks).  Where few waves are resident, or the widening and the second
  // A fragment hold up the next loads, more are.
  constexpr int U = F == 2 ? (kExact ? (J == 3 ? 1 : 2) : (J <= 2 ? 1 : 2)) : kExact && J >= 3 ? 4 : 1;
  __shared__ __attribute__((aligned(16))) v4f part[kFewWaves][F * J][64];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lrow = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * J;
  const int64_t nk = (p.K + kKB - 1) / kKB;
  const uint8_t *a[F], *b[J];
  const float *sa[F], *sb[J];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int64_t m = 16 * f + lrow < p.M ? 16 * f + lrow : p.M - 1;
    a[f] = p.a_codes + m * p.lda + q * 16;
    sa[f] = p.a_scales + m;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t n = n0 + 16 * j + lrow < p.N ? n0 + 16 * j + lrow : p.N - 1;
    b[j] = p.b_codes + n * p.ldb + q * 16;
    // a lane's accumulators are columns 4 q .. 4 q + 3 of the fragment
    const int64_t c = n0 + 16 * j < p.N ? n0 + 16 * j : p.N - 1;
    sb[j] = KIND == MX_FP8_LINE ? p.b_scales : p.b_scales + (c / kFp8Block) * p.ldb_scales;
  }
  auto piece2 = [](const uint8_t* x) {
    const u32x4 u = *(const u32x4*)x, v = *(const u32x4*)(x + 64);
    return v8i{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)v.x, (int)v.y, (int)v.z, (int)v.w};
  };
  v4f acc[F][J];
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[f][j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int64_t kb = wave; kb < nk; kb += kFewWaves * U) {
    v8i ra[U][F], rb[U][J];
    float ca[U][F];
    v4f cb[U][J];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a block past the last reads the last again and is left out below
      const int64_t k = kb + u * kFewWaves < nk ? kb + u * kFewWaves : nk - 1;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        rb[u][j] = piece2(b[j] + k * kKB);
        if constexpr (KIND == MX_FP8_TILE) {
          cb[u][j][0] = sb[j][k];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t c = n0 + 16 * j + 4 * q + r;
            cb[u][j][r] = sb[j][k * p.ldb_scales + (c < p.N ? c : p.N - 1)];
          }
        }
      }
#pragma unroll
      for (int f = 0; f < F; ++f) {
        ra[u][f] = piece2(a[f] + k * kKB);
        ca[u][f] = sa[f][k * p.lda_scales];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool counts = kb + u * kFewWaves < nk;
      Wide ob[J];
      if constexpr (kExact) {
#pragma unroll
        for (int j = 0; j < J; ++j) ob[j] = widen<BF>(rb[u][j]);
      }
#pragma unroll
      for (int f = 0; f < F; ++f) {
        Wide oa;
        if constexpr (kExact) oa = widen<AF>(ra[u][f]);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          v4f d = v4f{0.f, 0.f, 0.f, 0.f};
          if constexpr (kExact) {
#pragma unroll
            for (int e = 0; e < 4; ++e) d = mma_wide(ob[j], oa, e, d);
          } else {
            d = mma<BF, AF>(rb[u][j], ra[u][f]);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float s = ca[u][f] * cb[u][j][KIND == MX_FP8_TILE ? 0 : r];
            // chosen, not multiplied by 0: the block may hold Inf
            acc[f][j][r] = counts ? fmaf(d[r], s, acc[f][j][r]) : acc[f][j][r];
          }
        }
      }
    }
  }
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int j = 0; j < J; ++j) part[wave][f * J + j][lane] = acc[f][j];
  __syncthreads();
  if (wave >= F * J) return;
  v4f sum = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) sum += part[w][wave][lane];
  const int64_t m = 16 * (wave / J) + lrow, n = n0 + 16 * (wave % J) + 4 * q;
  if (m >= p.M) return;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n + r < p.N) {
      if constexpr (kExact) ((float*)p.c)[m * p.ldc + n + r] = sum[r];
      else ((uint16_t*)p.c)[m * p.ldc + n + r] = (uint16_t)pack_bf16(sum[r], 0.0f);
    }
}

// ---------------------------------------------------------------------------
// Everything between, and fp32 output: a 128 x 128 tile of C per workgroup,
// four waves of 64 x 64, two workgroups on a CU.  K blocks arrive by DMA in two
// 32 KB LDS stages, as in the large kernel below; a step's 16 fragment
// products run row by row, each joined four products later, and the barrier
// that frees the stage comes before the last row.  Where tiles alone do not
// fill the chip, a tile's K blocks are dealt to `splits` workgroups, whose
// float32 sums go to the workspace and are added in order by a second launch.
// Rows of a tile past the operand's last line read that line again.
//
// 2048 x 4096 x 4096 to bf16 takes 36 us (1900 TFLOP/s): bound by the copies, 64
// KB a K block and CU pair of workgroups, 15 TB/s over the chip.  To fp32,
// 4096 x 14336 x 8001 with line scales takes 818 us (1150 TFLOP/s; a bf16 product
// of the library 1445): the widening and the joins issue 280 vector instructions
// beside 64 matrix instructions, and the chip runs them at 1.6 GHz.
constexpr int kMThreads = 256, kMStage = kMT * kKB;

struct MidMap {
  int tiles_m, tiles_n, splits, total, per_xcd;    // total = tiles_m * tiles_n * splits
  float* parts;                                    // [splits][M][N] where splits > 1
};

template <int AF, int BF, int KIND, int OUT>
__global__ void __launch_bounds__(kMThreads, 2) fp8_mm_mid(const Fp8GemmParams p, const MidMap map) {
  constexpr bool kExact = OUT == MX_OUT_F32;
  __shared__ __attribute__((aligned(1024))) uint8_t sA[2][kMStage], sB[2][kMStage];
  __shared__ __attribute__((aligned(1024))) float sSA[2][kMT], sSB[2][kMT];
  // an XCD (workgroup ids are dealt to them in turn) takes a contiguous run of tiles: split by split, bands of
  // eight tile rows, column by column
  const int id = (int)(blockIdx.x % kXcds) * map.per_xcd + (int)(blockIdx.x / kXcds);
  if ((int)(blockIdx.x / kXcds) >= map.per_xcd || id >= map.total) return;
  const int tiles = map.tiles_m * map.tiles_n, split = id / tiles, tile = id % tiles;
  const int band = tile / (8 * map.tiles_n), in = tile % (8 * map.tiles_n);
  const int rows = min(8, map.tiles_m - 8 * band);
  const int64_t m0 = (int64_t)(8 * band + in % rows) * kMT, n0 = (int64_t)(in / rows) * kMT;
  const int nkb = (int)((p.K + kKB - 1) / kKB);
  const int k0 = (int)((int64_t)nkb * split / map.splits), k1 = (int)((int64_t)nkb * (split + 1) / map.splits);

  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = 64 * (wave & 1), wn = 64 * (wave >> 1);
  const int lrow = lane & 15, q = lane >> 4, l8 = lane >> 3;
  const int64_t ma = p.M - 1 - m0 < kMT ? p.M - 1 - m0 : kMT - 1, na = p.N - 1 - n0 < kMT ? p.N - 1 - n0 : kMT - 1;
  // wave w copies LDS rows 32 w .. 32 w + 31 of both operands, eight rows an instruction
  uint32_t oa[4], ob[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int row = 32 * wave + 8 * e + l8;
    const uint32_t piece = (uint32_t)slot(row, lane & 7);
    oa[e] = (uint32_t)(row < ma ? row : ma) * (uint32_t)p.lda + piece;
    const int col = (row & 64) + strip_col(row & 63);
    ob[e] = (uint32_t)(col < na ? col : na) * (uint32_t)p.ldb + piece;
  }
  const int sr = 64 * (wave & 1) + lane;
  const uint32_t os = 4u * (uint32_t)(wave < 2 ? (sr < ma ? sr : ma) : (KIND == MX_FP8_LINE ? (sr < na ? sr : na) : 0));
  const uint8_t* ca = uniform(p.a_codes + m0 * p.lda + (int64_t)k0 * kKB);
  const uint8_t* cb = uniform(p.b_codes + n0 * p.ldb + (int64_t)k0 * kKB);
  const int64_t step = wave < 2 ? p.lda_scales : (KIND == MX_FP8_LINE ? p.ldb_scales : 1);
  const float* cs = uniform(wave < 2 ? p.a_scales + k0 * p.lda_scales + m0
                                     : (KIND == MX_FP8_LINE ? p.b_scales + k0 * p.ldb_scales + n0
                                                            : p.b_scales + (n0 / kFp8Block) * p.ldb_scales + k0));
  const uint32_t dA = lds_addr(&sA[0][32 * wave * kKB]), dB = lds_addr(&sB[0][32 * wave * kKB]);
  const uint32_t dS = lds_addr(wave < 2 ? &sSA[0][64 * wave] : &sSB[0][64 * (wave & 1)]);
  auto issue = [&](int st) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dma16(ca, oa[e], dA + st * kMStage + e * 8 * kKB);
      dma16(cb, ob[e], dB + st * kMStage + e * 8 * kKB);
    }
    dma4(cs, os, dS + st * kMT * 4);
    ca += kKB;
    cb += kKB;
    cs += step;
  };

  const uint32_t off0 = lrow * kKB + slot(lrow, q), off1 = lrow * kKB + slot(lrow, q + 4);
  auto read = [&](const uint8_t* base, int f) {
    const u32x4 x = *(const u32x4*)(base + off0 + f * 16 * kKB), y = *(const u32x4*)(base + off1 + f * 16 * kKB);
    return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  };
  float sb[KIND == MX_FP8_LINE ? 16 : 1];
  auto read_sb = [&](int stage) {
    if constexpr (KIND == MX_FP8_LINE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4f x = *(const v4f*)&sSB[stage][wn + 16 * q + 4 * j];
#pragma unroll
        for (int e = 0; e < 4; ++e) sb[4 * j + e] = x[e];
      }
    } else {
      sb[0] = sSB[stage][0];
    }
  };
  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  auto join = [&](v4f& c, const v4f& d, float s, int j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = fmaf(d[e], KIND == MX_FP8_LINE ? s * sb[4 * j + e] : s, c[e]);
    asm volatile("" : "+v"(c));      // kept here, not sunk to the next step
  };

  const int nk = k1 - k0;
  issue(0);
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  if (nk > 1) issue(1);
  int st = 0;
  auto row = [&](int i) { return read(sA[st] + wm * kKB, i); };
  auto column = [&](int j) { return read(sB[st] + wn * kKB, j); };
  auto next_stage = [&](int kt) {
    // every read of this stage is done, and the next one has landed
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (kt + 2 < nk) issue(st);
    st ^= 1;
  };
  if constexpr (!kExact) {
    v8i fa[4], fb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) fb[j] = column(j);
#pragma unroll
    for (int i = 0; i < 2; ++i) fa[i] = row(i);
    read_sb(0);
    for (int kt = 0; kt < nk; ++kt) {
      v4f d[4];
      float s[4];
      each<16>([&](auto index) {
        constexpr int n = decltype(index)::value, i = n / 4, j = n % 4;
        if constexpr (j == 0) {
          if constexpr (i == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = sSA[st][wm + 16 * e + lrow];
          }
          if constexpr (i < 2) fa[i + 2] = row(i + 2);
          if constexpr (i == 3) {
            next_stage(kt);
            fa[0] = row(0);
            fa[1] = row(1);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (n >= 4) {
          if constexpr (KIND == MX_FP8_TILE && j == 0) s[i - 1] *= sb[0];
          join(acc[i - 1][j], d[j], s[i - 1], j);
        }
        d[j] = mma<BF, AF>(fb[j], fa[i]);
        if constexpr (i == 3) fb[j] = column(j);
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (KIND == MX_FP8_TILE) s[3] *= sb[0];
#pragma unroll
      for (int j = 0; j < 4; ++j) join(acc[3][j], d[j], s[3], j);
      read_sb(st);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    // Product n of a step is four 32-deep instructions, and beside each of them run one element of an earlier
    // product's join and one widening of the next A fragment (two in row 3, whose next fragment has just been asked
    // for).  The next step's B fragments are widened as this step's are done with, at products 14, 15, 0 and 1.
    v8i fa[2], rb[2];                        // as read: A row i in fa[i % 2], B column j in rb[j % 2]
    Wide ax, an, fb[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) fb[j] = widen<BF>(column(j));
#pragma unroll
    for (int j = 0; j < 2; ++j) rb[j] = column(2 + j);
    ax = widen<AF>(row(0));
    fa[1] = row(1);
    read_sb(0);
    for (int kt = 0; kt < nk; ++kt) {
      v4f d[4];
      float s[4];
      each<16>([&](auto index) {
        constexpr int n = decltype(index)::value, i = n / 4, j = n % 4;
        if constexpr (j == 0) {
          if constexpr (i == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = sSA[st][wm + 16 * e + lrow];
          }
          if constexpr (i < 2) fa[i & 1] = row(i + 2);
          if constexpr (i == 3) {
            next_stage(kt);
            fa[0] = row(0);
            rb[0] = column(0);
            rb[1] = column(1);
            fa[1] = row(1);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        constexpr int m = n - 3, mi = m / 4, mj = m & 3;
        if constexpr (m >= 0 && KIND == MX_FP8_TILE && mj == 0) s[mi] *= sb[0];
        constexpr int bj = n == 14 ? 0 : n == 15 ? 1 : n == 0 ? 2 : n == 1 ? 3 : -1;
        v4f x = v4f{0.f, 0.f, 0.f, 0.f};
        each<4>([&](auto part) {
          constexpr int e = decltype(part)::value;
          x = mma_wide(fb[j], ax, e, x);
          if constexpr (m >= 0) {
            acc[mi][mj][e] = fmaf(d[mj][e], KIND == MX_FP8_LINE ? s[mi] * sb[4 * mj + e] : s[mi], acc[mi][mj][e]);
          }
          if constexpr (i < 3) {
            constexpr int c = 4 * j + e;
            an.w[c] = widen<AF>((uint32_t)fa[(i + 1) & 1][c >> 1], (c & 1) != 0);
          } else if constexpr (j >= 2) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int c = 8 * (j - 2) + 2 * e + z;
              an.w[c] = widen<AF>((uint32_t)fa[0][c >> 1], (c & 1) != 0);
            }
          }
          if constexpr (bj >= 0) {
#pragma unroll
            for (int c = 4 * e; c < 4 * e + 4; ++c)
              fb[bj].w[c] = widen<BF>((uint32_t)rb[bj & 1][c >> 1], (c & 1) != 0);
          }
          __builtin_amdgcn_sched_barrier(0);
        });
        d[j] = x;
        if constexpr (m >= 0) asm volatile("" : "+v"(acc[mi][mj]));
        if constexpr (n == 15) {
          rb[0] = column(2);
          rb[1] = column(3);
        }
        if constexpr (j == 3) ax = an;
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int j = 1; j < 4; ++j) join(acc[3][j], d[j], s[3], j);
      read_sb(st);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (map.splits == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) store_rows<OUT>(p, m0 + wm + 16 * i, n0 + wn, lane, acc[i]);
  } else {
    Fp8GemmParams w = p;
    w.c = map.parts + (int64_t)split * p.M * p.N;
    w.ldc = p.N;
#pragma unroll
    for (int i = 0; i < 4; ++i) store_rows<MX_OUT_F32>(w, m0 + wm + 16 * i, n0 + wn, lane, acc[i]);
  }
}

// C from the splits' sums, added in order; four columns a thread.
template <int OUT>
__global__ void __launch_bounds__(256) fp8_mm_sum(const Fp8GemmParams p, const float* parts, int splits) {
  const int64_t quads = (p.N + 3) / 4, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= p.M * quads) return;
  const int64_t m = at / quads, n = 4 * (at % quads);
  const float* x = parts + m * p.N + n;
  if (n + 4 <= p.N) {
    v4f sum = *(const v4f_any*)x;
    for (int i = 1; i < splits; ++i) sum += *(const v4f_any*)(x + i * p.M * p.N);
    if constexpr (OUT == MX_OUT_F32) {
      *(v4f_any*)((float*)p.c + m * p.ldc + n) = sum;
    } else {
      typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
      typedef u32x2 u32x2_any __attribute__((aligned(2)));
      *(u32x2_any*)((uint16_t*)p.c + m * p.ldc + n) = u32x2{pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
    }
    return;
  }
  for (int r = 0; r < p.N - n; ++r) {
    float sum = x[r];
    for (int i = 1; i < splits; ++i) sum += x[i * p.M * p.N + r];
    if constexpr (OUT == MX_OUT_F32) ((float*)p.c)[m * p.ldc + n + r] = sum;
    else ((uint16_t*)p.c)[m * p.ldc + n + r] = (uint16_t)pack_bf16(sum, 0.0f);
  }
}

// ---------------------------------------------------------------------------
// Large products: a persistent grid, one workgroup per CU, each walking 256 x
// 256 tiles of C with eight waves of 128 x 64 (two waves per SIMD).  K advances
// one block (a 128-byte line of every operand row) per step, copied global ->
// LDS by DMA into one of two 64 KB stages while the other is consumed.
//
// A wave's step is 32 matrix instructions (eight A fragments x four B
// fragments), and each runs beside the four multiply-adds that join the result
// of four instructions earlier, so that nothing waits for a result.  Rows 0 - 4
// run row by row, each A fragment read three rows ahead; then every read of
// the stage is done, and a barrier frees it for the copies of the step after
// next.  Rows 5 - 7 run column by column behind the barrier, so that a B
// fragment is free after its three instructions and the next step's can be
// read: the next step's first LDS reads hide behind the last three eighths of
// this one.  (The two waves of a SIMD do not share its matrix core evenly: the
// older one runs ahead, and the younger finishes the step alone, when only its
// own reads ahead cover the LDS latency.)
//
// Rows of a tile past the operand's last line read that line again (their
// results are not stored), so every copy stays inside the operand and any M
// and N run here.
//
// 8192 x 28672 x 4096 takes 759 to 828 us by card (2540 to 2320 TFLOP/s), 8192 x 4096
// x 14336 353 to 374 us (2730 to 2570) with tile scales, 899 and 425 us with line
// scales, whose joins need two operations an element; an E5M2 gradient with an E4M3
// weight, 8192 x 4096 x 28672, 777 us (2480).  The library's product with one scale
// for each whole operand reaches 2680 to 3100.  The matrix cores are busy 58 to 65%
// of the cycles, and the chip lowers its clock to 1.7 to 2.0 GHz for it.
constexpr int kBThreads = 512;
constexpr int kStage = kBT * kKB;

__device__ __forceinline__ int next_tile(const BigMap& t, int r, int& bm, int& bn) {
  const int xcd = blockIdx.x % kXcds, member = blockIdx.x / kXcds;
  for (; r < t.rounds; ++r) {
    const int g = r * kXcds + xcd;
    if (g >= t.groups) return t.rounds;
    bm = (g % t.groups_m) * t.group_m + member % t.group_m;
    bn = (g / t.groups_m) * (kGroup / t.group_m) + member / t.group_m;
    if (bm < t.tiles_m && bn < t.tiles_n) return r;
  }
  return t.rounds;
}

// the step's order: instruction n works on fragment row row_of(n) and column col_of(n)
__device__ constexpr int row_of(int n) { return n < 20 ? n / 4 : 5 + (n - 20) % 3; }
__device__ constexpr int col_of(int n) { return n < 20 ? n % 4 : (n - 20) / 3; }

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
  // i % 8 ^ swizzle).  The waves w and w ^ 4, which share a SIMD, copy alternate steps, so that one keeps the
  // matrix core busy while the other issues: LDS rows 64 (w % 4) .. + 63 of A and of B and those rows' scales.
  // The cursor walks the steps to copy, tile after tile, ahead of the computation.
  const int l8 = lane >> 3, w4 = wave & 3;
  const int piece0 = ((lane & 7) ^ (l8 >> 1)) * 16, piece1 = ((lane & 7) ^ (4 + (l8 >> 1))) * 16;
  const int brow = 16 * (l8 >> 2) + (l8 & 3);              // the lane's part of strip_col
  const uint32_t la0 = l8 * (uint32_t)p.lda + piece0, la1 = l8 * (uint32_t)p.lda + piece1;
  const uint32_t lb0 = brow * (uint32_t)p.ldb + piece0, lb1 = brow * (uint32_t)p.ldb + piece1;
  const uint32_t dA = lds_addr(&sA[0][64 * w4 * kKB]), dB = lds_addr(&sB[0][64 * w4 * kKB]);
  const uint8_t *ca, *cb;          // the cursor's first byte of this wave's rows of A and B
  const float *csa, *csb;          // and of their scales
  uint32_t ma, na;                 // the tile's last row of A and of B, from its first
  bool edge;
  auto aim = [&](int tm, int tn) {
    const int64_t m0 = (int64_t)tm * kBT, n0 = (int64_t)tn * kBT;
    edge = m0 + kBT > p.M || n0 + kBT > p.N;
    // an edge tile's rows are counted from the tile's first, which exists
    const int64_t first = edge ? 0 : 64 * w4;
    ma = (uint32_t)(p.M - 1 - m0 < kBT ? p.M - 1 - m0 : kBT - 1);
    na = (uint32_t)(p.N - 1 - n0 < kBT ? p.N - 1 - n0 : kBT - 1);
    ca = uniform(p.a_codes + (m0 + first) * p.lda);
    cb = uniform(p.b_codes + (n0 + first) * p.ldb);
    csa = uniform(p.a_scales + m0);
    csb = uniform(KIND == MX_FP8_LINE ? p.b_scales + n0 : p.b_scales + (n0 / kFp8Block) * p.ldb_scales);
  };
  auto copy = [&](int st) {
    const uint32_t a0 = dA + st * kStage, b0 = dB + st * kStage;
    if (!edge) {
      // the pitches are made opaque, so that their multiples are formed here and not kept in registers
      uint32_t pa = (uint32_t)p.lda, pb = (uint32_t)p.ldb;
      asm volatile("" : "+s"(pa), "+s"(pb));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // rows 8 e .. 8 e + 7 of A; of B the strip columns of these LDS rows
        dma16(ca + (uint32_t)(8 * e) * pa, (e & 1) ? la1 : la0, a0 + e * 8 * kKB);
        dma16(cb + (uint32_t)(32 * (e & 1) + 4 * (e >> 1)) * pb, (e & 1) ? lb1 : lb0, b0 + e * 8 * kKB);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t ra = min((uint32_t)(64 * w4 + 8 * e + l8), ma);
        const uint32_t rb = min((uint32_t)(64 * w4 + 32 * (e & 1) + 4 * (e >> 1) + brow), na);
        const uint32_t piece = (uint32_t)((e & 1) ? piece1 : piece0);
        dma16(ca, __umul24(ra, (uint32_t)p.lda) + piece, a0 + e * 8 * kKB);
        dma16(cb, __umul24(rb, (uint32_t)p.ldb) + piece, b0 + e * 8 * kKB);
      }
    }
    const uint32_t f = (uint32_t)(64 * w4 + lane);
    dma4(csa, 4 * min(f, ma), lds_addr(&sSA[st][64 * w4]));
    if constexpr (KIND == MX_FP8_LINE) {
      dma4(csb, 4 * min(f, na), lds_addr(&sSB[st][64 * w4]));
    } else if (w4 == 0) {
      // a tile's two scales, each for 128 columns: lanes 0 .. 31 copy the first, 32 .. 63 the second (if any)
      dma4(csb, na >= kFp8Block ? 4 * (uint32_t)(lane >> 5) * (uint32_t)p.ldb_scales : 0u, lds_addr(&sSB[st][0]));
    }
  };
  auto advance = [&]() {
    ca += kKB;
    cb += kKB;
    csa += p.lda_scales;
    csb += KIND == MX_FP8_LINE ? p.ldb_scales : 1;
  };

  v4f acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // the cursor: next step to copy is ck of its tile, whose round is cr (map.rounds: none is left)
  int cr = r, ck = 0, parity = 0;
  aim(bm, bn);
  auto issue = [&](int st) {
    if (cr >= map.rounds) return;
    if ((wave >> 2) == parity) copy(st);
    parity ^= 1;
    advance();
    if (++ck == nk) {
      int cm = 0, cn = 0;
      ck = 0;
      cr = next_tile(map, cr + 1, cm, cn);
      if (cr < map.rounds) aim(cm, cn);
    }
  };
  int nbm = 0, nbn = 0;
  int rn = next_tile(map, r + 1, nbm, nbn);
  issue(0);
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  issue(1);

  v8i fb[4], fa[4];          // fragment row i in fa[i % 4]
  float sb[KIND == MX_FP8_LINE ? 16 : 1];
  int st = 0;
  // a fragment row's two pieces: their place depends on the lane only, rows 16 apart are immediates
  const uint32_t off0 = lrow * kKB + slot(lrow, q), off1 = lrow * kKB + slot(lrow, q + 4);
  auto read = [&](const uint8_t* base, int f) {
    const u32x4 x = *(const u32x4*)(base + off0 + f * 16 * kKB), y = *(const u32x4*)(base + off1 + f * 16 * kKB);
    return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  };
  auto read_sb = [&](int stage) {
    if constexpr (KIND == MX_FP8_LINE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4f x = *(const v4f*)&sSB[stage][wn + 16 * q + 4 * j];
#pragma unroll
        for (int e = 0; e < 4; ++e) sb[4 * j + e] = x[e];
      }
    } else {
      sb[0] = sSB[stage][(wn >> 7) * 32];
    }
  };
  auto join = [&](v4f& c, const v4f& d, float s, int j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = fmaf(d[e], KIND == MX_FP8_LINE ? s * sb[4 * j + e] : s, c[e]);
    // the sums have no use before the next step: without this they are sunk there, every product kept until then
    asm volatile("" : "+v"(c));
  };
  // Instruction n's result stays in d[n % 4] until instruction n + 4 is due.  A step's last four results are joined
  // in the next step (tile scales), or at its end (line scales, whose columns' scales the next step replaces).
  constexpr bool kCarry = KIND == MX_FP8_TILE;
  v4f d[4];
  float carry[3];                // the scales of rows 5 - 7 of the step before
  auto clear = [&]() {
#pragma unroll
    for (int n = 0; n < 4; ++n) d[n] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < 3; ++n) carry[n] = 0.0f;
  };
  clear();
#pragma unroll
  for (int j = 0; j < 4; ++j) fb[j] = read(sB[0] + wn * kKB, j);
#pragma unroll
  for (int i = 0; i < 3; ++i) fa[i] = read(sA[0] + wm * kKB, i);
  read_sb(0);
  for (;;) {
    for (int kt = 0; kt < nk; ++kt) {
      float s[8];
      each<32>([&](auto index) {
        constexpr int n = decltype(index)::value, i = row_of(n), j = col_of(n);
        if constexpr (n < 20 && j == 0) {
          s[i] = sSA[st][wm + 16 * i + lrow];
          if constexpr (i == 4) {
#pragma unroll
            for (int e = 5; e < 8; ++e) s[e] = sSA[st][wm + 16 * e + lrow];
          }
          fa[(i + 3) & 3] = read(sA[st] + wm * kKB, i + 3);
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (n == 20) {
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
          issue(st);
          st ^= 1;
          fa[0] = read(sA[st] + wm * kKB, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (n >= 4) {
          constexpr int mi = row_of(n - 4), mj = col_of(n - 4);
          if constexpr (KIND == MX_FP8_TILE && mj == 0) s[mi] *= sb[0];
          join(acc[mi][mj], d[n & 3], s[mi], mj);
        } else if constexpr (kCarry) {
          join(acc[row_of(28 + n)][col_of(28 + n)], d[n], carry[row_of(28 + n) - 5], 0);
        }
        d[n & 3] = mma<BF, AF>(fb[j], fa[i & 3]);
        if constexpr (n >= 20 && i == 7) fb[j] = read(sB[st] + wn * kKB, j);
        if constexpr (n == 29) fa[1] = read(sA[st] + wm * kKB, 1);
        if constexpr (n == 30) fa[2] = read(sA[st] + wm * kKB, 2);
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (kCarry) {
#pragma unroll
        for (int e = 0; e < 3; ++e) carry[e] = s[5 + e];
      } else {
#pragma unroll
        for (int n = 28; n < 32; ++n) join(acc[row_of(n)][col_of(n)], d[n & 3], s[row_of(n)], col_of(n));
      }
      read_sb(st);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kCarry) {
#pragma unroll
      for (int n = 28; n < 32; ++n) join(acc[row_of(n)][col_of(n)], d[n & 3], carry[row_of(n) - 5], 0);
      clear();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      store_rows<MX_OUT_BF16>(p, (int64_t)bm * kBT + wm + 16 * i, (int64_t)bn * kBT + wn, lane, acc[i]);
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

template <int AF, int BF, int KIND, int OUT, int F, int J>
void few(const Fp8GemmParams& p, hipStream_t s) {
  hipLaunchKernelGGL((fp8_mm_few<AF, BF, KIND, OUT, F, J>), dim3((unsigned)((p.N + 16 * J - 1) / (16 * J))),
                     dim3(64 * kFewWaves), 0, s, p);
}

template <int AF, int BF, int KIND, int OUT, int F>
void launch_few(const Fp8GemmParams& p, hipStream_t s) {
  for (int64_t m = 0; m < p.M; m += 16 * F) {
    Fp8GemmParams r = p;
    r.a_codes += m * p.lda;
    r.a_scales += m;
    r.M = p.M - m < 16 * F ? p.M - m : 16 * F;
    r.c = (uint8_t*)p.c + m * p.ldc * (OUT == MX_OUT_F32 ? 4 : 2);
    switch (fp8_few_columns(r.M, p.N, OUT == MX_OUT_F32)) {
      case 1: few<AF, BF, KIND, OUT, F, 1>(r, s); break;
      case 2: few<AF, BF, KIND, OUT, F, 2>(r, s); break;
      case 3: few<AF, BF, KIND, OUT, F, 3>(r, s); break;
      default: few<AF, BF, KIND, OUT, F, 4>(r, s);
    }
  }
}

template <int AF, int BF, int KIND, int OUT>
void launch(const Fp8GemmParams& p, float* parts, int64_t parts_bytes, hipStream_t s) {
  Fp8Plan plan = fp8_plan(p.M, p.N, p.K, p.lda, p.ldb, KIND == MX_FP8_TILE ? p.ldb_scales : 0, OUT == MX_OUT_F32);
  if (plan.path == Fp8Path::kFew) {
    if (p.M <= 16) launch_few<AF, BF, KIND, OUT, 1>(p, s);
    else launch_few<AF, BF, KIND, OUT, 2>(p, s);
    return;
  }
  if constexpr (OUT == MX_OUT_BF16) {
    if (plan.path == Fp8Path::kBig) {
      hipLaunchKernelGGL((fp8_mm_big<AF, BF, KIND>), dim3(kXcds * kGroup), dim3(kBThreads), 0, s, p, plan.big);
      return;
    }
  }
  // the workspace holds as many sums as it can
  while (plan.splits > 1 && (parts == nullptr || parts_bytes / 4 / plan.splits / p.M < p.N)) --plan.splits;
  MidMap map;
  map.tiles_m = (int)((p.M + kMT - 1) / kMT);
  map.tiles_n = (int)((p.N + kMT - 1) / kMT);
  map.splits = plan.splits;
  map.total = map.tiles_m * map.tiles_n * map.splits;
  map.per_xcd = (map.total + kXcds - 1) / kXcds;
  map.parts = parts;
  hipLaunchKernelGGL((fp8_mm_mid<AF, BF, KIND, OUT>), dim3((unsigned)(kXcds * map.per_xcd)), dim3(kMThreads), 0, s, p,
                     map);
  if (map.splits > 1) {
    const int64_t quads = p.M * ((p.N + 3) / 4);
    hipLaunchKernelGGL((fp8_mm_sum<OUT>), dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, s, p, parts,
                       map.splits);
  }
}

template <int AF, int BF>
void launch_kinds(const Fp8GemmParams& p, int b_kind, int out_kind, float* w, int64_t bytes, hipStream_t s) {
  if (b_kind == MX_FP8_TILE) {
    if (out_kind == MX_OUT_F32) launch<AF, BF, MX_FP8_TILE, MX_OUT_F32>(p, w, bytes, s);
    else launch<AF, BF, MX_FP8_TILE, MX_OUT_BF16>(p, w, bytes, s);
  } else {
    if (out_kind == MX_OUT_F32) launch<AF, BF, MX_FP8_LINE, MX_OUT_F32>(p, w, bytes, s);
    else launch<AF, BF, MX_FP8_LINE, MX_OUT_BF16>(p, w, bytes, s);
  }
}

}  // namespace

int64_t fp8_gemm_workspace(int64_t M, int64_t N, int64_t K, int out_kind) {
  const int64_t k = ((K + kKB - 1) / kKB) * kKB;
  const Fp8Plan plan = fp8_plan(M, N, K, k, k, 0, out_kind == MX_OUT_F32);
  return plan.splits > 1 ? 4 * plan.splits * M * N : 0;
}

hipError_t launch_fp8_gemm(const Fp8GemmParams& p, int a_fmt, int b_fmt, int b_kind, int out_kind, float* parts,
                           int64_t bytes, hipStream_t s) {
  constexpr int k4 = MX_FP8_E4M3, k5 = MX_FP8_E5M2;
  if (a_fmt == k4 && b_fmt == k4) launch_kinds<k4, k4>(p, b_kind, out_kind, parts, bytes, s);
  else if (b_fmt == k4) launch_kinds<k5, k4>(p, b_kind, out_kind, parts, bytes, s);
  else if (a_fmt == k4) launch_kinds<k4, k5>(p, b_kind, out_kind, parts, bytes, s);
  else launch_kinds<k5, k5>(p, b_kind, out_kind, parts, bytes, s);
  return hipGetLastError();
}

}  // namespace mx
