// The 8-bit floating-point cast with a float32 scale for each block of 128:
// per line and 128 values (LINE), or per 128 x 128 tile (TILE), along the rows
// of a bf16 matrix, its columns (the transpose's lines), or both from one read.
//
//   s = max(RN(amax * RN(1 / F)), 2^-126), F = 448 (E4M3) or 57344 (E5M2)
//   r = RN(1 / s), code = RNE8(RN(x * r))
//
// x * r stays within F (1 + 2^-22), which rounds to F, so nothing saturates.
// A block that holds Inf or NaN gets s = NaN and codes 0.
//
// One workgroup casts a 128 x 128 tile: it holds every block it touches whole,
// for both axes and both kinds, and the tile stays in registers between the
// maxima and the cast.  Lane group g = t / 16 takes rows 8g .. 8g + 7, lane
// c = t % 16 of it columns 8c .. 8c + 7, so a wave's load of one row index
// covers four 256-byte row pieces, a row's maximum is a DPP reduction over 16
// lanes, a row's codes are one whole 128-byte line, and a lane's eight rows are
// eight consecutive bytes of each of its columns' output lines.  The column
// codes go through LDS (16 KB, 16-byte pieces XOR-swizzled by column) and leave
// as whole 128-byte lines too.
//
// Memory-bound: 2 bytes read and 1 written per element and output.  Where every
// call has other memory, as in a training step, both axes of 8192 x 4096 take 30
// us (4.5 TB/s), of 28672 x 4096 (tiles) 91 us (5.2); of 8192 x 14336 the rows
// alone 65 us (5.4), the columns alone 77 (4.6).  The same buffers cast again
// and again, part of them in the 256 MB last-level cache: 22, 71, 52 and 53 us.
// HBM's peak is 8 TB/s, a copy of 4 GiB reaches 4.6 to 4.7 here.  The codes leave
// by non-temporal stores, which gained 20% and 3% on the first two: they stay out
// of the way of x, which the operation before may have left in the cache; a
// training step that multiplies the codes next runs the same either way.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include "fp8_kernels.h"

namespace mx {

namespace {

constexpr int kTile = 128;
constexpr int kFqThreads = 256;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}

// max over the 16 lanes of a DPP row (packed 16-bit pairs)
__device__ __forceinline__ uint32_t row_max16(uint32_t v) {
  v = pk_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));    // l ^ 1
  v = pk_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));    // l ^ 2
  v = pk_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));   // 7 - l within 8
  v = pk_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));   // 15 - l within 16
  return v;
}

// max over the wave's four 16-lane rows, lane by lane
__device__ __forceinline__ uint32_t rows4_max(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = pk_max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return pk_max(b[0], b[1]);
}

// Scale and reciprocal of a block whose largest |x| has bf16 magnitude bits
// `mag`; a block with Inf or NaN (mag >= 0x7F80) gets s = NaN and r = 0.
template <int FMT>
__device__ __forceinline__ void block_scale(uint32_t mag, float& s, float& r) {
  constexpr float kLargest = FMT == MX_FP8_E4M3 ? 448.0f : 57344.0f;
  const bool bad = mag >= 0x7F80u;
  s = fmaxf(__uint_as_float(mag << 16) * (1.0f / kLargest), 0x1p-126f);
  r = 1.0f / s;
  if (bad) {
    s = __uint_as_float(0x7FC00000u);
    r = 0.0f;
  }
}

// four codes of y0 .. y3, low byte first
template <int FMT>
__device__ __forceinline__ uint32_t cast4(float y0, float y1, float y2, float y3) {
  int d = 0;
  if constexpr (FMT == MX_FP8_E4M3) {
    d = __builtin_amdgcn_cvt_pk_fp8_f32(y0, y1, d, false);
    d = __builtin_amdgcn_cvt_pk_fp8_f32(y2, y3, d, true);
  } else {
    d = __builtin_amdgcn_cvt_pk_bf8_f32(y0, y1, d, false);
    d = __builtin_amdgcn_cvt_pk_bf8_f32(y2, y3, d, true);
  }
  return (uint32_t)d;
}

template <int FMT, bool TILE, bool ROW, bool COL>
__global__ void __launch_bounds__(kFqThreads) fp8_quant_tiles(const Fp8QuantParams p, int64_t tiles_c) {
  // part[w][d]: wave w's column maxima, two columns per dword; rmax: row maxima, two rows per dword
  __shared__ uint32_t part[4][kTile / 2];
  __shared__ uint32_t rmax[kTile / 2];
  __shared__ float rrow[kTile], rcol[kTile];
  __shared__ __attribute__((aligned(16))) uint8_t tr[COL ? kTile * kTile : 16];

  const int t = threadIdx.x, c = t & 15, g = t >> 4, wave = t >> 6;
  const int64_t rt = blockIdx.x / tiles_c, ct = blockIdx.x % tiles_c;
  const int64_t row0 = rt * kTile + 8 * g, col0 = ct * kTile + 8 * c;
  uint32_t v[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint4 q = uint4{0u, 0u, 0u, 0u};
    if (row0 + i < p.rows && col0 < p.cols) q = *(const uint4*)(p.x + (row0 + i) * p.ld_x + col0);
    v[i][0] = q.x;
    v[i][1] = q.y;
    v[i][2] = q.z;
    v[i][3] = q.w;
  }
  uint32_t m[8], cm[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = 0u;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t a = v[i][d] & 0x7FFF7FFFu;
      m[i] = pk_max(m[i], a);
      cm[d] = pk_max(cm[d], a);
    }
  }
  if constexpr (TILE) {
    uint32_t all = pk_max(pk_max(cm[0], cm[1]), pk_max(cm[2], cm[3]));
    all = rows4_max(row_max16(all));
    if ((t & 63) == 0) part[wave][0] = max(all & 0xFFFFu, all >> 16);
    __syncthreads();
    const uint32_t mag = max(max(part[0][0], part[1][0]), max(part[2][0], part[3][0]));
    float s, r;
    block_scale<FMT>(mag, s, r);
    if (t < kTile) {
      rrow[t] = r;
      rcol[t] = r;
    }
    if (t == 0) {
      if constexpr (ROW) p.row_scales[rt * p.ld_row_scales + ct] = s;
      if constexpr (COL) p.col_scales[ct * p.ld_col_scales + rt] = s;
    }
  } else {
    if constexpr (ROW) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        // rows i (low half) and i + 1 (high half)
        const uint32_t lo = __builtin_amdgcn_perm(m[i + 1], m[i], 0x05040100u);
        const uint32_t hi = __builtin_amdgcn_perm(m[i + 1], m[i], 0x07060302u);
        const uint32_t mm = row_max16(pk_max(lo, hi));
        if (c == 0) rmax[4 * g + i / 2] = mm;
      }
    }
    if constexpr (COL) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t w = rows4_max(cm[d]);
        if ((t & 63) < 16) part[wave][4 * c + d] = w;
      }
    }
    __syncthreads();
    // threads 0 .. 127 take a column each, 128 .. 255 a row each
    const int e = t & (kTile - 1), shift = 16 * (e & 1);
    if (t < kTile) {
      if constexpr (COL) {
        uint32_t w = pk_max(pk_max(part[0][e >> 1], part[1][e >> 1]), pk_max(part[2][e >> 1], part[3][e >> 1]));
        float s, r;
        block_scale<FMT>((w >> shift) & 0xFFFFu, s, r);
        rcol[e] = r;
        if (ct * kTile + e < p.cols) p.col_scales[rt * p.ld_col_scales + ct * kTile + e] = s;
      }
    } else {
      if constexpr (ROW) {
        float s, r;
        block_scale<FMT>((rmax[e >> 1] >> shift) & 0xFFFFu, s, r);
        rrow[e] = r;
        if (rt * kTile + e < p.rows) p.row_scales[ct * p.ld_row_scales + rt * kTile + e] = s;
      }
    }
  }
  __syncthreads();
  auto lo = [](uint32_t d) { return __uint_as_float(d << 16); };
  auto hi = [](uint32_t d) { return __uint_as_float(d & 0xFFFF0000u); };
  if constexpr (ROW) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = rrow[8 * g + i];
      uint32_t q0 = cast4<FMT>(lo(v[i][0]) * r, hi(v[i][0]) * r, lo(v[i][1]) * r, hi(v[i][1]) * r);
      uint32_t q1 = cast4<FMT>(lo(v[i][2]) * r, hi(v[i][2]) * r, lo(v[i][3]) * r, hi(v[i][3]) * r);
      if (r == 0.0f) q0 = q1 = 0u;       // Inf or NaN in the block (a finite block's r is at least 2^-120)
      if (row0 + i < p.rows)
        __builtin_nontemporal_store(u32x2{q0, q1}, (u32x2*)(p.row_codes + (row0 + i) * p.ld_row_codes + col0));
    }
  }
  if constexpr (COL) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float r = rcol[8 * c + j];
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = ((j & 1) ? hi(v[i][j >> 1]) : lo(v[i][j >> 1])) * r;
      uint32_t q0 = cast4<FMT>(y[0], y[1], y[2], y[3]), q1 = cast4<FMT>(y[4], y[5], y[6], y[7]);
      if (r == 0.0f) q0 = q1 = 0u;
      // 8-byte unit g of column 8c + j, its 16-byte piece at g / 2 ^ (c % 8)
      *(uint2*)(tr + (8 * c + j) * kTile + (((g >> 1) ^ (c & 7)) * 16 + (g & 1) * 8)) = uint2{q0, q1};
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int col = 32 * u + (t >> 3), piece = t & 7;
      const u32x4 q = *(const u32x4*)(tr + col * kTile + ((piece ^ ((col >> 3) & 7)) * 16));
      if (ct * kTile + col < p.cols)
        __builtin_nontemporal_store(
            q, (u32x4*)(p.col_codes + (ct * kTile + col) * p.ld_col_codes + rt * kTile + piece * 16));
    }
  }
}

template <int FMT, bool TILE>
void launch_axes(const Fp8QuantParams& p, bool do_row, bool do_col, hipStream_t s) {
  const int64_t tr = (p.rows + kTile - 1) / kTile, tc = (p.cols + kTile - 1) / kTile;
  const dim3 g((unsigned)(tr * tc)), b(kFqThreads);
  if (do_row && do_col) hipLaunchKernelGGL((fp8_quant_tiles<FMT, TILE, true, true>), g, b, 0, s, p, tc);
  else if (do_row) hipLaunchKernelGGL((fp8_quant_tiles<FMT, TILE, true, false>), g, b, 0, s, p, tc);
  else hipLaunchKernelGGL((fp8_quant_tiles<FMT, TILE, false, true>), g, b, 0, s, p, tc);
}

}  // namespace

hipError_t launch_fp8_quant(const Fp8QuantParams& p, int fmt, int kind, bool do_row, bool do_col, hipStream_t s) {
  if (fmt == MX_FP8_E4M3) {
    if (kind == MX_FP8_TILE) launch_axes<MX_FP8_E4M3, true>(p, do_row, do_col, s);
    else launch_axes<MX_FP8_E4M3, false>(p, do_row, do_col, s);
  } else {
    if (kind == MX_FP8_TILE) launch_axes<MX_FP8_E5M2, true>(p, do_row, do_col, s);
    else launch_axes<MX_FP8_E5M2, false>(p, do_row, do_col, s);
  }
  return hipGetLastError();
}

}  // namespace mx
