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

// Sixteen consecutive columns of one row of C from a lane's accumulators.
template <int OUT>
__device__ __forceinline__ void store16(const Fp8GemmParams& p, int64_t m, int64_t n, const v4f (&acc)[4], bool wide) {
  if (m >= p.M || n >= p.N) return;
  const int64_t at = m * p.ldc + n;
  if (wide && n + 16 <= p.N) {
    if constexpr (OUT == MX_OUT_F32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) *(v4f*)((float*)p.c + at + 4 * j) = acc[j];
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *(u32x4*)((uint16_t*)p.c + at + 8 * h) =
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
__global__ void __launch_bounds__(kGThreads) fp8_mm_any(const Fp8GemmParams p, int64_t tiles_m, bool wide) {
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
  for (int i = 0; i < 4; ++i) store16<OUT>(p, m0 + wm + 16 * i + lrow, col, acc[i], wide);
}

// rows of C start 16-byte aligned and are a whole number of 16-byte pieces apart
bool wide_rows(const Fp8GemmParams& p, int out_kind) {
  return (uintptr_t)p.c % 16 == 0 && p.ldc % (out_kind == MX_OUT_F32 ? 4 : 8) == 0;
}

template <int AF, int BF, int KIND, int OUT>
void launch(const Fp8GemmParams& p, hipStream_t s) {
  const int64_t tm = (p.M + kGT - 1) / kGT, tn = (p.N + kGT - 1) / kGT;
  hipLaunchKernelGGL((fp8_mm_any<AF, BF, KIND, OUT>), dim3((unsigned)(tm * tn)), dim3(kGThreads), 0, s, p, tm,
                     wide_rows(p, OUT));
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
