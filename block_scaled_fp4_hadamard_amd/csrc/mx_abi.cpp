// C ABI of the MX quantizer and GEMM: argument validation, the random sign
// vector of the randomized Hadamard rotation, and the kernel launches.
// Validation happens before any HIP call, so argument errors never touch the
// device.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <math.h>
#include "mx_kernels.h"
#include "fp8_kernels.h"
#include "norm_kernels.h"
#include "ortho_kernels.h"

namespace {

constexpr uint32_t kM0 = 0xD2511F53u, kM1 = 0xCD9E8D57u, kW0 = 0x9E3779B9u, kW1 = 0xBB67AE85u;

// Host Philox4x32-10, word 0 only: the sign vector of the randomized rotation
// is word 0 of the draw with counter (0, 0, 2, 0) under key had_seed.
uint32_t philox_word0(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)c0 * kM0, p1 = (uint64_t)c2 * kM1;
    const uint32_t n0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    const uint32_t n2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)p1;
    c3 = (uint32_t)p0;
    c0 = n0;
    c2 = n2;
    k0 += kW0;
    k1 += kW1;
  }
  return c0;
}

bool aligned16(const void* ptr) { return ((uintptr_t)ptr & 15u) == 0; }

mx_status check_qtensor(const mx_qtensor* q, int64_t lines, int64_t k, int32_t block) {
  if (q == nullptr || q->codes == nullptr || q->scales == nullptr) return MX_ERR_INVALID;
  // the 32-value kernels store 16 code bytes at a time, the 16-value kernel 8
  const int64_t step = block == 16 ? 8 : 16;
  if (((uintptr_t)q->codes % (uintptr_t)step) != 0 || q->ld_codes % step != 0) return MX_ERR_INVALID;
  if (q->ld_codes < k / 2 || q->ld_scales < k / block) return MX_ERR_INVALID;
  if (lines > 1 && (q->ld_codes <= 0 || q->ld_scales <= 0)) return MX_ERR_INVALID;
  return MX_OK;
}

bool out_ok(int type) { return type == MX_OUT_F32 || type == MX_OUT_BF16; }
bool norm_kind_ok(int kind) { return kind == MX_NORM_LAYER || kind == MX_NORM_RMS; }
bool norm_sizes_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows < (int64_t(1) << 40) && cols < (int64_t(1) << 30);
}
bool norm_rows_ok(const void* x, int type, int64_t ld, int64_t cols) {
  return x != nullptr && ((uintptr_t)x & (type == MX_OUT_F32 ? 3u : 1u)) == 0 && ld >= cols;
}

bool ortho_sizes_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows < mx::kOrthoSide && cols < mx::kOrthoSide &&
         (rows < cols ? rows : cols) < mx::kOrthoMinor;
}

// The most that a group of the list needs, over entries of `rows(i)` x `cols(i)`; empty ones take no part.
template <typename T>
int64_t ortho_workspace(const T* list, int32_t count) {
  if (count < 0 || (count > 0 && list == nullptr)) return 0;
  for (int32_t i = 0; i < count; ++i)
    if (!ortho_sizes_ok(list[i].rows, list[i].cols)) return 0;
  int64_t most = 0;
  mx::each_ortho_group(list, count, [&](const int32_t*, int, int64_t bytes) {
    most = bytes > most ? bytes : most;
    return true;
  });
  return most;
}

bool ortho_params_ok(const mx_ortho_params& p) {
  return p.steps >= 1 && p.steps <= 64 && p.eps > 0.0 && isfinite(p.eps) && mx::ortho_fits(p.a, p.b, p.c, p.steps);
}

mx_status quantize_impl(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, int32_t block, int grid,
                        int round, int axis, uint64_t seed, int had_n, int had_kind, uint64_t had_seed,
                        const mx_qtensor* row_out, const mx_qtensor* col_out, void* stream) {
  if (rows < 0 || cols < 0) return MX_ERR_INVALID;
  if (grid != MX_GRID_E2M1 && grid != MX_GRID_E1M2) return MX_ERR_INVALID;
  if (round != MX_ROUND_RTNE && round != MX_ROUND_SR) return MX_ERR_INVALID;
  if (axis != MX_AXIS_ROW && axis != MX_AXIS_COL && axis != MX_AXIS_BOTH) return MX_ERR_INVALID;
  if (had_kind != MX_HAD_NONE && had_kind != MX_HAD_DET && had_kind != MX_HAD_RAND) return MX_ERR_INVALID;
  if (had_kind == MX_HAD_NONE) had_n = 0;
  else if (had_n != 16 && had_n != 32) return MX_ERR_INVALID;
  if (block != 16 && block != 32) return MX_ERR_INVALID;
  if (had_n > block) return MX_ERR_INVALID;
  const bool do_row = (axis & MX_AXIS_ROW) != 0, do_col = (axis & MX_AXIS_COL) != 0;
  if (rows == 0 || cols == 0) return MX_OK;
  if (x == nullptr || !aligned16(x)) return MX_ERR_INVALID;
  if (ld_x < cols || ld_x % 8 != 0 || cols % 8 != 0 || ld_x >= (int64_t(1) << 25)) return MX_ERR_INVALID;
  if (do_row) {
    if (cols % block != 0) return MX_ERR_INVALID;
    mx_status s = check_qtensor(row_out, rows, cols, block);
    if (s != MX_OK) return s;
  }
  if (do_col) {
    if (rows % block != 0) return MX_ERR_INVALID;
    mx_status s = check_qtensor(col_out, cols, rows, block);
    if (s != MX_OK) return s;
  }
  if (block == 16) {
    // 16-value MX blocks: a separate kernel, no rotation
    if (had_n != 0) return MX_ERR_UNSUPPORTED;
    for (int a = 0; a < 2; ++a) {
      const bool col = a == 1;
      if (col ? !do_col : !do_row) continue;
      const mx_qtensor* q = col ? col_out : row_out;
      mx::Block16Params b{};
      b.x = x;
      b.rows = rows;
      b.cols = cols;
      b.ld_x = ld_x;
      b.codes = q->codes;
      b.ld_codes = q->ld_codes;
      b.scales = q->scales;
      b.ld_scales = q->ld_scales;
      b.seed = seed;
      if (mx::launch_block16(b, false, grid, round, col, (hipStream_t)stream) != hipSuccess) return MX_ERR_DEVICE;
    }
    return MX_OK;
  }
  if (block != 32) return MX_ERR_UNSUPPORTED;
  mx::QuantParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ld_x = ld_x;
  if (do_row) {
    p.row_codes = row_out->codes;
    p.ld_row_codes = row_out->ld_codes;
    p.row_scales = row_out->scales;
    p.ld_row_scales = row_out->ld_scales;
  }
  if (do_col) {
    p.col_codes = col_out->codes;
    p.ld_col_codes = col_out->ld_codes;
    p.col_scales = col_out->scales;
    p.ld_col_scales = col_out->ld_scales;
  }
  p.seed = seed;
  p.sign_mask = 0u;
  const bool rht = had_kind == MX_HAD_RAND;
  if (rht) {
    const uint32_t w0 = philox_word0(0u, 0u, 2u, 0u, (uint32_t)had_seed, (uint32_t)(had_seed >> 32));
    p.sign_mask = had_n == 32 ? w0 : (w0 & 0xFFFFu);
  }
  hipError_t e = mx::launch_quant(p, had_n, rht, grid, round, do_row, do_col, (hipStream_t)stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

// mx_gemm's argument checks; on MX_OK with M, N > 0, p holds the problem
mx_status gemm_args(const mx_qtensor* a, const mx_qtensor* b, int64_t M, int64_t N, int64_t K, int grid,
                    int32_t block, void* c, int64_t ldc, int out, mx::GemmParams& p) {
  if (M < 0 || N < 0 || K <= 0) return MX_ERR_INVALID;
  if (grid != MX_GRID_E2M1 && grid != MX_GRID_E1M2) return MX_ERR_INVALID;
  if (out != MX_OUT_F32 && out != MX_OUT_BF16) return MX_ERR_INVALID;
  if (block != 16 && block != 32) return MX_ERR_INVALID;
  if (K % block != 0) return MX_ERR_INVALID;
  if (M == 0 || N == 0) return MX_OK;
  mx_status s = check_qtensor(a, M, K, block);
  if (s != MX_OK) return s;
  s = check_qtensor(b, N, K, block);
  if (s != MX_OK) return s;
  const uintptr_t esize = out == MX_OUT_F32 ? 4u : 2u;
  if (c == nullptr || ((uintptr_t)c % esize) != 0 || ldc < N) return MX_ERR_INVALID;
  if (block != 32) return MX_ERR_UNSUPPORTED;
  p = mx::GemmParams{};
  p.a_codes = a->codes;
  p.a_scales = a->scales;
  p.b_codes = b->codes;
  p.b_scales = b->scales;
  p.lda_codes = a->ld_codes;
  p.lda_scales = a->ld_scales;
  p.ldb_codes = b->ld_codes;
  p.ldb_scales = b->ld_scales;
  p.M = M;
  p.N = N;
  p.K = K;
  p.c = c;
  p.ldc = ldc;
  return MX_OK;
}

int64_t fp8_blocks(int64_t n) { return n / mx::kFp8Block + (n % mx::kFp8Block != 0); }

bool fp8_fmt_ok(int fmt) { return fmt == MX_FP8_E4M3 || fmt == MX_FP8_E5M2; }
bool fp8_kind_ok(int kind) { return kind == MX_FP8_LINE || kind == MX_FP8_TILE; }

mx_status check_fp8(const mx_fp8_tensor* q, int64_t lines, int64_t k, int kind) {
  if (q == nullptr || q->codes == nullptr || q->scales == nullptr) return MX_ERR_INVALID;
  if (!aligned16(q->codes) || ((uintptr_t)q->scales & 3u) != 0) return MX_ERR_INVALID;
  if (q->ld_codes % 16 != 0 || q->ld_codes / mx::kFp8Block < fp8_blocks(k)) return MX_ERR_INVALID;
  if (q->ld_scales < (kind == MX_FP8_LINE ? lines : fp8_blocks(k))) return MX_ERR_INVALID;
  return MX_OK;
}

// 128 x 128 tiles that one launch can take: its grid holds fewer than 2^32 threads, 256 a tile
bool too_many_tiles(int64_t m, int64_t n) {
  constexpr int64_t kMost = int64_t(1) << 23;
  return fp8_blocks(m) >= kMost || fp8_blocks(n) >= kMost || fp8_blocks(m) * fp8_blocks(n) >= kMost;
}

}  // namespace

extern "C" {

mx_status mx_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, int32_t block, mx_grid grid,
                      mx_round round, mx_axis axis, uint64_t seed, const mx_qtensor* row_out,
                      const mx_qtensor* col_out, void* hip_stream) {
  return quantize_impl(x, rows, cols, ld_x, block, grid, round, axis, seed, 0, MX_HAD_NONE, 0, row_out, col_out,
                       hip_stream);
}

mx_status mx_hadamard_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, int32_t block,
                               mx_grid grid, mx_round round, mx_axis axis, uint64_t seed, int32_t had_n,
                               mx_had had_kind, uint64_t had_seed, const mx_qtensor* row_out,
                               const mx_qtensor* col_out, void* hip_stream) {
  if (had_kind == MX_HAD_NONE) return MX_ERR_INVALID;
  return quantize_impl(x, rows, cols, ld_x, block, grid, round, axis, seed, had_n, had_kind, had_seed, row_out,
                       col_out, hip_stream);
}

mx_status mx_gemm(const mx_qtensor* a, const mx_qtensor* b, int64_t M, int64_t N, int64_t K, mx_grid grid,
                  int32_t block, void* c, int64_t ldc, mx_out out, void* hip_stream) {
  mx::GemmParams p{};
  const mx_status s = gemm_args(a, b, M, N, K, grid, block, c, ldc, out, p);
  if (s != MX_OK || M == 0 || N == 0) return s;
  hipError_t e = mx::launch_gemm(p, grid, out, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

mx_status mx_gemm_grouped(const mx_gemm_problem* problems, int32_t count, int64_t K, mx_grid grid, int32_t block,
                          mx_out out, void* hip_stream) {
  if (problems == nullptr || count < 1 || count > MX_GEMM_GROUP_MAX) return MX_ERR_INVALID;
  mx::GemmParams ps[MX_GEMM_GROUP_MAX];
  int n = 0;
  for (int i = 0; i < count; ++i) {
    const mx_gemm_problem& q = problems[i];
    const mx_status s = gemm_args(q.a, q.b, q.M, q.N, K, grid, block, q.c, q.ldc, out, ps[n]);
    if (s != MX_OK) return s;
    if (q.M > 0 && q.N > 0) ++n;
  }
  if (n == 0) return MX_OK;
  hipError_t e = mx::launch_gemm_grouped(ps, n, grid, out, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

mx_status mx_mxnorm_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, int32_t power, float c,
                             mx_grid grid, mx_round round, uint64_t seed, const mx_qtensor* out, float* rho,
                             void* hip_stream) {
  if (rows < 0 || cols < 0) return MX_ERR_INVALID;
  if (power != 1 && power != 2) return MX_ERR_INVALID;
  if (!(c > 0.0f) || c > 3.0e38f) return MX_ERR_INVALID;          // rejects NaN, non-positive and infinite c
  if (grid != MX_GRID_E2M1 && grid != MX_GRID_E1M2) return MX_ERR_INVALID;
  if (round != MX_ROUND_RTNE && round != MX_ROUND_SR) return MX_ERR_INVALID;
  if (rows == 0 || cols == 0) return MX_OK;
  if (cols % 32 != 0 || cols > 65536) return MX_ERR_INVALID;
  if (x == nullptr || !aligned16(x)) return MX_ERR_INVALID;
  if (ld_x < cols || ld_x % 8 != 0) return MX_ERR_INVALID;
  mx_status s = check_qtensor(out, rows, cols, 32);
  if (s != MX_OK) return s;
  if (rho == nullptr || ((uintptr_t)rho & 3u) != 0) return MX_ERR_INVALID;
  mx::MxNormParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ld_x = ld_x;
  p.codes = out->codes;
  p.ld_codes = out->ld_codes;
  p.scales = out->scales;
  p.ld_scales = out->ld_scales;
  p.rho = rho;
  p.c = c;
  p.seed = seed;
  hipError_t e = mx::launch_mxnorm(p, power, grid, round, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

mx_status mx_quant_stats(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, mx_axis axis, mx_grid grid,
                         int32_t had_n, mx_had had_kind, uint64_t had_seed, const mx_qtensor* q,
                         mx_quant_stats_t* stats, void* hip_stream) {
  if (rows < 0 || cols < 0) return MX_ERR_INVALID;
  if (axis != MX_AXIS_ROW && axis != MX_AXIS_COL) return MX_ERR_INVALID;
  if (grid != MX_GRID_E2M1 && grid != MX_GRID_E1M2) return MX_ERR_INVALID;
  if (had_kind != MX_HAD_NONE && had_kind != MX_HAD_DET && had_kind != MX_HAD_RAND) return MX_ERR_INVALID;
  if (had_kind == MX_HAD_NONE) had_n = 0;
  else if (had_n != 16 && had_n != 32) return MX_ERR_INVALID;
  if (stats == nullptr || ((uintptr_t)stats & 7u) != 0) return MX_ERR_INVALID;
  if (rows == 0 || cols == 0) return MX_OK;
  if (x == nullptr || ((uintptr_t)x & 1u) != 0 || ld_x < cols) return MX_ERR_INVALID;
  const bool col = axis == MX_AXIS_COL;
  const int64_t lines = col ? cols : rows, len = col ? rows : cols;
  if (len % 32 != 0) return MX_ERR_INVALID;
  mx_status s = check_qtensor(q, lines, len, 32);
  if (s != MX_OK) return s;
  mx::QuantStatsParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ld_x = ld_x;
  p.codes = q->codes;
  p.ld_codes = q->ld_codes;
  p.scales = q->scales;
  p.ld_scales = q->ld_scales;
  p.axis_col = col ? 1 : 0;
  p.grid = grid;
  p.sign_mask = 0u;
  if (had_kind == MX_HAD_RAND) {
    const uint32_t w0 = philox_word0(0u, 0u, 2u, 0u, (uint32_t)had_seed, (uint32_t)(had_seed >> 32));
    p.sign_mask = had_n == 32 ? w0 : (w0 & 0xFFFFu);
  }
  p.out = stats;
  hipError_t e = mx::launch_quant_stats(p, had_n, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

mx_status mx_nvfp4_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, mx_round round,
                            mx_axis axis, uint64_t seed, const mx_nvfp4_tensor* row_out,
                            const mx_nvfp4_tensor* col_out, void* hip_stream) {
  if (rows < 0 || cols < 0) return MX_ERR_INVALID;
  if (round != MX_ROUND_RTNE && round != MX_ROUND_SR) return MX_ERR_INVALID;
  if (axis != MX_AXIS_ROW && axis != MX_AXIS_COL && axis != MX_AXIS_BOTH) return MX_ERR_INVALID;
  if (rows == 0 || cols == 0) return MX_OK;
  if (x == nullptr || !aligned16(x)) return MX_ERR_INVALID;
  if (ld_x < cols || ld_x % 8 != 0 || cols % 8 != 0) return MX_ERR_INVALID;
  const bool do_row = (axis & MX_AXIS_ROW) != 0, do_col = (axis & MX_AXIS_COL) != 0;
  for (int a = 0; a < 2; ++a) {
    const bool col = a == 1;
    if (col ? !do_col : !do_row) continue;
    const mx_nvfp4_tensor* q = col ? col_out : row_out;
    const int64_t lines = col ? cols : rows, len = col ? rows : cols;
    if (len % 128 != 0) return MX_ERR_INVALID;
    if (q == nullptr || q->codes == nullptr || q->inner == nullptr || q->outer == nullptr) return MX_ERR_INVALID;
    if (!aligned16(q->codes) || q->ld_codes % 16 != 0 || q->ld_codes < len / 2) return MX_ERR_INVALID;
    if (q->ld_inner < len / 16 || q->ld_outer < len / 128 || ((uintptr_t)q->outer & 3u) != 0) return MX_ERR_INVALID;
    if (lines > 1 && (q->ld_inner <= 0 || q->ld_outer <= 0)) return MX_ERR_INVALID;
  }
  for (int a = 0; a < 2; ++a) {
    const bool col = a == 1;
    if (col ? !do_col : !do_row) continue;
    const mx_nvfp4_tensor* q = col ? col_out : row_out;
    mx::Block16Params b{};
    b.x = x;
    b.rows = rows;
    b.cols = cols;
    b.ld_x = ld_x;
    b.codes = q->codes;
    b.ld_codes = q->ld_codes;
    b.scales = q->inner;
    b.ld_scales = q->ld_inner;
    b.outer = q->outer;
    b.ld_outer = q->ld_outer;
    b.seed = seed;
    if (mx::launch_block16(b, true, MX_GRID_E2M1, round, col, (hipStream_t)hip_stream) != hipSuccess)
      return MX_ERR_DEVICE;
  }
  return MX_OK;
}

mx_status mx_hadamard_rotate(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, int32_t had_n,
                             mx_had had_kind, uint64_t had_seed, mx_axis axis, float* y, int64_t ld_y,
                             void* hip_stream) {
  if (rows < 0 || cols < 0) return MX_ERR_INVALID;
  if (had_kind != MX_HAD_DET && had_kind != MX_HAD_RAND) return MX_ERR_INVALID;
  if (had_n != 16 && had_n != 32) return MX_ERR_INVALID;
  if (axis != MX_AXIS_ROW && axis != MX_AXIS_COL) return MX_ERR_INVALID;
  if (rows == 0 || cols == 0) return MX_OK;
  const bool col = axis == MX_AXIS_COL;
  const int64_t len = col ? rows : cols;
  if (len % 32 != 0) return MX_ERR_INVALID;
  if (x == nullptr || !aligned16(x) || ld_x < cols || ld_x % 8 != 0 || cols % 8 != 0) return MX_ERR_INVALID;
  if (y == nullptr || !aligned16(y) || ld_y < len || ld_y % 4 != 0) return MX_ERR_INVALID;
  mx::RotateParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ld_x = ld_x;
  p.y = y;
  p.ld_y = ld_y;
  p.col = col;
  p.sign_mask = 0u;
  const bool rht = had_kind == MX_HAD_RAND;
  if (rht) {
    const uint32_t w0 = philox_word0(0u, 0u, 2u, 0u, (uint32_t)had_seed, (uint32_t)(had_seed >> 32));
    p.sign_mask = had_n == 32 ? w0 : (w0 & 0xFFFFu);
  }
  hipError_t e = mx::launch_rotate(p, had_n, rht, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

mx_status mx_quantize_f32(const float* y, int64_t lines, int64_t len, int64_t ld_y, mx_grid grid, mx_round round,
                          mx_axis axis, uint64_t seed, const mx_qtensor* out, void* hip_stream) {
  if (lines < 0 || len < 0) return MX_ERR_INVALID;
  if (grid != MX_GRID_E2M1 && grid != MX_GRID_E1M2) return MX_ERR_INVALID;
  if (round != MX_ROUND_RTNE && round != MX_ROUND_SR) return MX_ERR_INVALID;
  if (axis != MX_AXIS_ROW && axis != MX_AXIS_COL) return MX_ERR_INVALID;
  if (lines == 0 || len == 0) return MX_OK;
  if (len % 32 != 0) return MX_ERR_INVALID;
  if (y == nullptr || !aligned16(y) || ld_y < len || ld_y % 4 != 0) return MX_ERR_INVALID;
  mx_status s = check_qtensor(out, lines, len, 32);
  if (s != MX_OK) return s;
  mx::QuantF32Params p{};
  p.y = y;
  p.lines = lines;
  p.len = len;
  p.ld_y = ld_y;
  p.codes = out->codes;
  p.ld_codes = out->ld_codes;
  p.scales = out->scales;
  p.ld_scales = out->ld_scales;
  p.seed = seed;
  p.stream = axis == MX_AXIS_COL ? 1u : 0u;
  hipError_t e = mx::launch_quant_f32(p, grid, round, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

mx_status mx_osci_reset(float* w, int64_t rows, int64_t cols, int64_t ld_w, const mx_qtensor* q, mx_grid grid,
                        float* w_prev, float* q_prev, float* dist_m, float* dist_q, int64_t ld_state,
                        mx_osci_mode mode, float threshold, uint64_t* resets, void* hip_stream) {
  if (rows < 0 || cols < 0) return MX_ERR_INVALID;
  if (grid != MX_GRID_E2M1 && grid != MX_GRID_E1M2) return MX_ERR_INVALID;
  if (mode != MX_OSCI_INIT && mode != MX_OSCI_TRACK && mode != MX_OSCI_CHECK) return MX_ERR_INVALID;
  if (mode == MX_OSCI_CHECK && !(threshold >= 0.0f && threshold <= 3.0e38f)) return MX_ERR_INVALID;
  if (rows == 0 || cols == 0) return MX_OK;
  if (cols % 32 != 0) return MX_ERR_INVALID;
  const float* arrays[5] = {w, w_prev, q_prev, dist_m, dist_q};
  for (const float* a : arrays)
    if (a == nullptr || !aligned16(a)) return MX_ERR_INVALID;
  if (ld_w < cols || ld_w % 4 != 0 || ld_state < cols || ld_state % 4 != 0) return MX_ERR_INVALID;
  if (resets != nullptr && ((uintptr_t)resets & 7u) != 0) return MX_ERR_INVALID;
  mx_status s = check_qtensor(q, rows, cols, 32);
  if (s != MX_OK) return s;
  mx::OsciParams p{};
  p.w = w;
  p.rows = rows;
  p.cols = cols;
  p.ld_w = ld_w;
  p.codes = q->codes;
  p.ld_codes = q->ld_codes;
  p.scales = q->scales;
  p.ld_scales = q->ld_scales;
  p.w_prev = w_prev;
  p.q_prev = q_prev;
  p.dist_m = dist_m;
  p.dist_q = dist_q;
  p.ld_s = ld_state;
  p.mode = mode;
  p.threshold = threshold;
  p.resets = (unsigned long long*)resets;
  hipError_t e = mx::launch_osci(p, grid, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

mx_status mx_fp8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, mx_fp8_fmt fmt,
                          mx_fp8_kind kind, mx_axis axis, const mx_fp8_tensor* row_out, const mx_fp8_tensor* col_out,
                          void* hip_stream) {
  if (rows < 0 || cols < 0) return MX_ERR_INVALID;
  if (!fp8_fmt_ok(fmt) || !fp8_kind_ok(kind)) return MX_ERR_INVALID;
  if (axis != MX_AXIS_ROW && axis != MX_AXIS_COL && axis != MX_AXIS_BOTH) return MX_ERR_INVALID;
  if (rows == 0 || cols == 0) return MX_OK;
  if (x == nullptr || !aligned16(x)) return MX_ERR_INVALID;
  if (ld_x < cols || ld_x % 8 != 0 || cols % 8 != 0 || too_many_tiles(rows, cols)) return MX_ERR_INVALID;
  const bool do_row = (axis & MX_AXIS_ROW) != 0, do_col = (axis & MX_AXIS_COL) != 0;
  if (do_row) {
    const mx_status s = check_fp8(row_out, rows, cols, kind);
    if (s != MX_OK) return s;
  }
  if (do_col) {
    const mx_status s = check_fp8(col_out, cols, rows, kind);
    if (s != MX_OK) return s;
  }
  mx::Fp8QuantParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ld_x = ld_x;
  if (do_row) {
    p.row_codes = row_out->codes;
    p.ld_row_codes = row_out->ld_codes;
    p.row_scales = row_out->scales;
    p.ld_row_scales = row_out->ld_scales;
  }
  if (do_col) {
    p.col_codes = col_out->codes;
    p.ld_col_codes = col_out->ld_codes;
    p.col_scales = col_out->scales;
    p.ld_col_scales = col_out->ld_scales;
  }
  const hipError_t e = mx::launch_fp8_quant(p, fmt, kind, do_row, do_col, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

mx_status mx_fp8_gemm(const mx_fp8_tensor* a, mx_fp8_fmt a_fmt, const mx_fp8_tensor* b, mx_fp8_fmt b_fmt,
                      mx_fp8_kind b_kind, int64_t M, int64_t N, int64_t K, void* c, int64_t ldc, mx_out out,
                      void* workspace, int64_t workspace_bytes, void* hip_stream) {
  if (M < 0 || N < 0 || K <= 0) return MX_ERR_INVALID;
  if (!fp8_fmt_ok(a_fmt) || !fp8_fmt_ok(b_fmt) || !fp8_kind_ok(b_kind)) return MX_ERR_INVALID;
  if (out != MX_OUT_F32 && out != MX_OUT_BF16) return MX_ERR_INVALID;
  if (M == 0 || N == 0) return MX_OK;
  mx_status s = check_fp8(a, M, K, MX_FP8_LINE);
  if (s != MX_OK) return s;
  s = check_fp8(b, N, K, b_kind);
  if (s != MX_OK) return s;
  const uintptr_t esize = out == MX_OUT_F32 ? 4u : 2u;
  if (c == nullptr || ((uintptr_t)c % esize) != 0 || ldc < N) return MX_ERR_INVALID;
  // few rows: 512 threads for each 16 to 64 columns (fp8_few_columns keeps the grid below 2^32 threads)
  if (too_many_tiles(M, N) || N >= (int64_t(1) << 27)) return MX_ERR_INVALID;
  if (workspace_bytes < 0 || !aligned16(workspace)) return MX_ERR_INVALID;
  mx::Fp8GemmParams p{};
  p.a_codes = a->codes;
  p.b_codes = b->codes;
  p.a_scales = a->scales;
  p.b_scales = b->scales;
  p.lda = a->ld_codes;
  p.ldb = b->ld_codes;
  p.lda_scales = a->ld_scales;
  p.ldb_scales = b->ld_scales;
  p.M = M;
  p.N = N;
  p.K = K;
  p.c = c;
  p.ldc = ldc;
  const hipError_t e = mx::launch_fp8_gemm(p, a_fmt, b_fmt, b_kind, out, (float*)workspace, workspace_bytes,
                                             (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

int64_t mx_fp8_gemm_workspace(int64_t M, int64_t N, int64_t K, mx_out out) {
  if (out != MX_OUT_F32 && out != MX_OUT_BF16) return 0;
  // sizes that mx_fp8_gemm refuses, or whose rows no memory holds
  if (M <= 0 || N <= 0 || K <= 0 || too_many_tiles(M, N) || K >= (int64_t(1) << 62)) return 0;
  return mx::fp8_gemm_workspace(M, N, K, out);
}

mx_status mx_adamw_step(const mx_adamw_tensor* tensors, int32_t count, int32_t bits, const mx_adamw_params* params,
                        mx_round round, uint64_t seed, void* hip_stream) {
  if (count < 0 || (count > 0 && tensors == nullptr) || params == nullptr) return MX_ERR_INVALID;
  if (bits != 8 && bits != 32) return MX_ERR_INVALID;
  if (round != MX_ROUND_RTNE && round != MX_ROUND_SR) return MX_ERR_INVALID;
  const mx_adamw_params& q = *params;
  if (!(q.beta1 >= 0.0 && q.beta1 < 1.0) || !(q.beta2 >= 0.0 && q.beta2 < 1.0)) return MX_ERR_INVALID;
  if (!(q.eps >= 0.0) || !isfinite(q.eps) || !isfinite(q.weight_decay)) return MX_ERR_INVALID;
  if (q.lr_dev == nullptr ? !isfinite(q.lr) : ((uintptr_t)q.lr_dev & 3u) != 0) return MX_ERR_INVALID;
  if (q.step_dev == nullptr ? q.step < 1 : ((uintptr_t)q.step_dev & 7u) != 0) return MX_ERR_INVALID;
  if (((uintptr_t)q.grad_scale & 3u) != 0) return MX_ERR_INVALID;
  const uintptr_t state = bits == 32 ? 3u : 0u;
  for (int32_t i = 0; i < count; ++i) {
    const mx_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n >= (int64_t(1) << 36)) return MX_ERR_INVALID;
    if (t.grad != MX_OUT_F32 && t.grad != MX_OUT_BF16) return MX_ERR_INVALID;
    if (t.n == 0) continue;
    if (t.w == nullptr || t.g == nullptr || t.m == nullptr || t.v == nullptr) return MX_ERR_INVALID;
    if (((uintptr_t)t.w & 3u) || ((uintptr_t)t.g & (t.grad == MX_OUT_F32 ? 3u : 1u))) return MX_ERR_INVALID;
    if (((uintptr_t)t.m & state) || ((uintptr_t)t.v & state) || ((uintptr_t)t.copy & 1u)) return MX_ERR_INVALID;
    if (bits == 8) {
      if (t.m_scales == nullptr || t.v_scales == nullptr) return MX_ERR_INVALID;
      if (((uintptr_t)t.m_scales & 3u) || ((uintptr_t)t.v_scales & 3u)) return MX_ERR_INVALID;
    }
  }
  mx::AdamwStep step{};
  step.lr = q.lr;
  step.beta1 = q.beta1;
  step.beta2 = q.beta2;
  step.eps = q.eps;
  step.weight_decay = q.weight_decay;
  step.step = q.step;
  step.step_dev = q.step_dev;
  step.lr_dev = q.lr_dev;
  step.grad_scale = q.grad_scale;
  step.seed = seed;
  for (int32_t at = 0; at < count; at += mx::kAdamwGroup) {
    mx::AdamwTensor group[mx::kAdamwGroup];
    bool bf16[mx::kAdamwGroup];
    const int n = count - at < mx::kAdamwGroup ? count - at : mx::kAdamwGroup;
    for (int i = 0; i < n; ++i) {
      const mx_adamw_tensor& t = tensors[at + i];
      group[i] = mx::AdamwTensor{t.w, t.g, t.m, t.v, t.m_scales, t.v_scales, t.copy, t.n};
      bf16[i] = t.grad == MX_OUT_BF16;
    }
    const hipError_t e = mx::launch_adamw(group, bf16, n, at, step, bits, round, (hipStream_t)hip_stream);
    if (e != hipSuccess) return MX_ERR_DEVICE;
  }
  return MX_OK;
}

mx_status mx_layer_norm(const void* x, mx_out type, int64_t rows, int64_t cols, int64_t ld_x, const void* weight,
                        const void* bias, mx_out weight_type, double eps, mx_norm_kind kind, void* y, int64_t ld_y,
                        float* mean, float* rstd, void* hip_stream) {
  if (!out_ok(type) || !out_ok(weight_type) || !norm_kind_ok(kind) || !norm_sizes_ok(rows, cols)) return MX_ERR_INVALID;
  if (!(eps >= 0.0) || !isfinite((float)eps)) return MX_ERR_INVALID;
  if (kind == MX_NORM_RMS && (bias != nullptr || mean != nullptr)) return MX_ERR_INVALID;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!norm_rows_ok(x, type, ld_x, cols) || !norm_rows_ok(y, type, ld_y, cols)) return MX_ERR_INVALID;
  const uintptr_t wmask = weight_type == MX_OUT_F32 ? 3u : 1u;
  if (((uintptr_t)weight & wmask) || ((uintptr_t)bias & wmask)) return MX_ERR_INVALID;
  if (((uintptr_t)mean & 3u) || ((uintptr_t)rstd & 3u)) return MX_ERR_INVALID;
  const mx::NormParams p{x, weight, bias, rows, cols, ld_x, (float)eps, y, ld_y, mean, rstd};
  const hipError_t e = mx::launch_norm(p, type, weight_type, kind, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

int64_t mx_layer_norm_grad_workspace(int64_t rows, int64_t cols, mx_out type, int32_t sums) {
  if (!out_ok(type) || !norm_sizes_ok(rows, cols) || rows == 0 || cols == 0) return 0;
  return mx::norm_grad_workspace(rows, cols, type, sums != 0);
}

mx_status mx_layer_norm_grad(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, mx_out type, int64_t rows,
                             int64_t cols, const void* weight, mx_out weight_type, const float* mean,
                             const float* rstd, mx_norm_kind kind, void* dx, int64_t ld_dx, float* dweight,
                             float* dbias, void* workspace, int64_t workspace_bytes, void* hip_stream) {
  if (!out_ok(type) || !out_ok(weight_type) || !norm_kind_ok(kind) || !norm_sizes_ok(rows, cols)) return MX_ERR_INVALID;
  if (kind == MX_NORM_RMS && mean != nullptr) return MX_ERR_INVALID;
  if (((uintptr_t)dweight & 3u) || ((uintptr_t)dbias & 3u)) return MX_ERR_INVALID;
  if (cols == 0) return MX_OK;
  if (rows > 0) {
    if (!norm_rows_ok(dy, type, ld_dy, cols) || !norm_rows_ok(x, type, ld_x, cols) ||
        !norm_rows_ok(dx, type, ld_dx, cols))
      return MX_ERR_INVALID;
    if ((uintptr_t)weight & (weight_type == MX_OUT_F32 ? 3u : 1u)) return MX_ERR_INVALID;
    if (rstd == nullptr || ((uintptr_t)rstd & 3u) || ((uintptr_t)mean & 3u)) return MX_ERR_INVALID;
    if (kind == MX_NORM_LAYER && mean == nullptr) return MX_ERR_INVALID;
    const bool sums = dweight != nullptr || dbias != nullptr;
    const int64_t need = mx::norm_grad_workspace(rows, cols, type, sums);
    if (need > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need)) return MX_ERR_INVALID;
  }
  const mx::NormGradParams p{dy, x, weight, mean, rstd, rows, cols, ld_dy, ld_x, ld_dx, dx, dweight, dbias};
  const hipError_t e = mx::launch_norm_grad(p, type, weight_type, kind, (float*)workspace, (hipStream_t)hip_stream);
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

int64_t mx_orthogonalize_workspace(const mx_ortho_matrix* matrices, int32_t count) {
  return ortho_workspace(matrices, count);
}

int64_t mx_muon_workspace(const mx_muon_tensor* tensors, int32_t count) { return ortho_workspace(tensors, count); }

mx_status mx_orthogonalize(const mx_ortho_matrix* matrices, int32_t count, const mx_ortho_params* params,
                           void* workspace, int64_t workspace_bytes, void* hip_stream) {
  if (count < 0 || (count > 0 && matrices == nullptr) || params == nullptr) return MX_ERR_INVALID;
  if (!ortho_params_ok(*params)) return MX_ERR_INVALID;
  for (int32_t i = 0; i < count; ++i) {
    const mx_ortho_matrix& t = matrices[i];
    if (!ortho_sizes_ok(t.rows, t.cols) || !out_ok(t.grad) || !out_ok(t.type)) return MX_ERR_INVALID;
    if (t.rows == 0 || t.cols == 0) continue;
    if (!norm_rows_ok(t.g, t.grad, t.ld_g, t.cols) || !norm_rows_ok(t.out, t.type, t.ld_out, t.cols))
      return MX_ERR_INVALID;
    if (t.ld_out >= mx::kOrthoPitch) return MX_ERR_INVALID;
  }
  const int64_t need = ortho_workspace(matrices, count);
  if (need > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need)) return MX_ERR_INVALID;
  mx::OrthoStep step{};
  step.a = params->a;
  step.b = params->b;
  step.c = params->c;
  step.eps = params->eps;
  step.steps = params->steps;
  hipError_t e = hipSuccess;
  mx::each_ortho_group(matrices, count, [&](const int32_t* at, int n, int64_t) {
    mx::OrthoItem items[mx::kOrthoGroup];
    uint8_t* space = (uint8_t*)workspace;
    for (int i = 0; i < n; ++i) {
      const mx_ortho_matrix& t = matrices[at[i]];
      items[i] = mx::OrthoItem{t.g, nullptr, nullptr, nullptr, t.out, space, t.ld_g, t.ld_out, (int)t.rows, (int)t.cols,
                               t.grad == MX_OUT_BF16, t.type == MX_OUT_BF16, 1.0f};
      space += mx::ortho_size(t.rows, t.cols).bytes;
    }
    e = mx::launch_ortho(items, n, step, (hipStream_t)hip_stream);
    return e == hipSuccess;
  });
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

mx_status mx_muon_step(const mx_muon_tensor* tensors, int32_t count, const mx_muon_params* params, void* workspace,
                       int64_t workspace_bytes, void* hip_stream) {
  if (count < 0 || (count > 0 && tensors == nullptr) || params == nullptr) return MX_ERR_INVALID;
  const mx_muon_params& q = *params;
  if (!ortho_params_ok(q.ortho) || !(q.momentum >= 0.0 && q.momentum < 1.0)) return MX_ERR_INVALID;
  // as the float32 that the kernels take
  if (!((float)q.momentum < 1.0f) || !isfinite(q.weight_decay) || (q.nesterov != 0 && q.nesterov != 1))
    return MX_ERR_INVALID;
  if (q.adjust != MX_MUON_PLAIN && q.adjust != MX_MUON_RMS && q.adjust != MX_MUON_SHAPE) return MX_ERR_INVALID;
  if (q.lr_dev == nullptr ? !isfinite(q.lr) : ((uintptr_t)q.lr_dev & 3u) != 0) return MX_ERR_INVALID;
  if (((uintptr_t)q.grad_scale & 3u) != 0) return MX_ERR_INVALID;
  for (int32_t i = 0; i < count; ++i) {
    const mx_muon_tensor& t = tensors[i];
    if (!ortho_sizes_ok(t.rows, t.cols) || !out_ok(t.grad)) return MX_ERR_INVALID;
    if (t.rows == 0 || t.cols == 0) continue;
    if (!norm_rows_ok(t.g, t.grad, t.cols, t.cols) || !norm_rows_ok(t.w, MX_OUT_F32, t.cols, t.cols) ||
        !norm_rows_ok(t.m, MX_OUT_F32, t.cols, t.cols) || ((uintptr_t)t.copy & 1u))
      return MX_ERR_INVALID;
  }
  const int64_t need = ortho_workspace(tensors, count);
  if (need > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need)) return MX_ERR_INVALID;
  mx::OrthoStep step{};
  step.a = q.ortho.a;
  step.b = q.ortho.b;
  step.c = q.ortho.c;
  step.eps = q.ortho.eps;
  step.steps = q.ortho.steps;
  step.momentum = (float)q.momentum;
  step.rest = (float)(1.0 - q.momentum);
  step.nesterov = q.nesterov != 0;
  step.lr = q.lr;
  step.weight_decay = q.weight_decay;
  step.lr_dev = q.lr_dev;
  step.grad_scale = q.grad_scale;
  hipError_t e = hipSuccess;
  mx::each_ortho_group(tensors, count, [&](const int32_t* at, int n, int64_t) {
    mx::OrthoItem items[mx::kOrthoGroup];
    uint8_t* space = (uint8_t*)workspace;
    for (int i = 0; i < n; ++i) {
      const mx_muon_tensor& t = tensors[at[i]];
      const double r = (double)t.rows, c = (double)t.cols;
      const double scale = q.adjust == MX_MUON_RMS     ? 0.2 * sqrt(r > c ? r : c)
                           : q.adjust == MX_MUON_SHAPE ? sqrt(r > c ? r / c : 1.0)
                                                       : 1.0;
      items[i] = mx::OrthoItem{t.g, t.m, t.w, t.copy, nullptr, space, t.cols, 0, (int)t.rows, (int)t.cols,
                               t.grad == MX_OUT_BF16, false, scale};
      space += mx::ortho_size(t.rows, t.cols).bytes;
    }
    e = mx::launch_ortho(items, n, step, (hipStream_t)hip_stream);
    return e == hipSuccess;
  });
  return e == hipSuccess ? MX_OK : MX_ERR_DEVICE;
}

const char* mx_status_str(mx_status status) {
  switch (status) {
    case MX_OK: return "MX_OK";
    case MX_ERR_INVALID: return "MX_ERR_INVALID: invalid argument";
    case MX_ERR_UNSUPPORTED: return "MX_ERR_UNSUPPORTED: valid request not implemented";
    case MX_ERR_DEVICE: return "MX_ERR_DEVICE: HIP runtime error";
  }
  return "unknown mx_status";
}

int32_t mx_version(void) { return 100; }

}  // extern "C"
