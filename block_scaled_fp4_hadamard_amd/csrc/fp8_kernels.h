// Internal interface between the C ABI layer and the 8-bit floating-point and
// optimizer kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include "../../include/mxfp4.h"

namespace mx {

constexpr int64_t kFp8Block = MX_FP8_BLOCK;

// The 8-bit cast of a bf16 matrix along its rows, its columns or both.
struct Fp8QuantParams {
  const uint16_t* x;
  int64_t rows, cols, ld_x;
  uint8_t* row_codes;
  int64_t ld_row_codes;
  float* row_scales;
  int64_t ld_row_scales;
  uint8_t* col_codes;
  int64_t ld_col_codes;
  float* col_scales;
  int64_t ld_col_scales;
};

hipError_t launch_fp8_quant(const Fp8QuantParams& p, int fmt, int kind, bool do_row, bool do_col, hipStream_t s);

struct Fp8GemmParams {
  const uint8_t* a_codes;
  const uint8_t* b_codes;
  const float* a_scales;
  const float* b_scales;
  int64_t lda, ldb;                  // bytes between lines of codes
  int64_t lda_scales, ldb_scales;    // floats
  int64_t M, N, K;
  void* c;
  int64_t ldc;
};

// parts: float32 workspace of `bytes` bytes (may be null)
hipError_t launch_fp8_gemm(const Fp8GemmParams& p, int a_fmt, int b_fmt, int b_kind, int out_kind, float* parts,
                           int64_t bytes, hipStream_t s);
int64_t fp8_gemm_workspace(int64_t M, int64_t N, int64_t K, int out_kind);

// One AdamW step.  Up to kAdamwGroup tensors ride in one launch's arguments.
constexpr int kAdamwGroup = 48;

struct AdamwTensor {
  float* w;
  const void* g;
  void* m;
  void* v;
  float* m_scales;
  float* v_scales;
  uint16_t* copy;
  int64_t n;
};

// What every element of a step uses, in float32 (from float64 arithmetic).
struct AdamwCoef {
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
  float c1;        // lr / (1 - beta1^t)
  float c2;        // 1 / sqrt(1 - beta2^t)
  float keep;      // 1 - lr * weight_decay
};

struct AdamwStep {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
  uint64_t seed;
};

// tensors[0 .. count-1]; a tensor's stochastic-rounding streams go by first + its index
hipError_t launch_adamw(const AdamwTensor* tensors, const bool* grad_bf16, int count, int first, const AdamwStep& step,
                        int bits, int round, hipStream_t s);

}  // namespace mx
