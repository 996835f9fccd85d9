// Internal interface between the C ABI layer and the norm kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include "../../include/mxfp4.h"

namespace mx {

struct NormParams {
  const void* x;                 // [rows][ld_x], of one type with y, dy and dx
  const void* weight;            // [cols], or null: ones
  const void* bias;              // [cols], or null: zeros (forward only)
  int64_t rows, cols, ld_x;
  float eps;
  void* y;
  int64_t ld_y;
  float* mean;                   // [rows], or null
  float* rstd;                   // [rows], or null
};

struct NormGradParams {
  const void* dy;
  const void* x;
  const void* weight;            // or null
  const float* mean;             // layer norm only
  const float* rstd;
  int64_t rows, cols, ld_dy, ld_x, ld_dx;
  void* dx;
  float* dweight;                // [cols], or null
  float* dbias;                  // [cols], or null
};

// type: MX_OUT_F32 or MX_OUT_BF16, of x and y; weight_type: of weight and bias
hipError_t launch_norm(const NormParams& p, int type, int weight_type, int kind, hipStream_t s);
// workspace: norm_grad_workspace bytes
hipError_t launch_norm_grad(const NormGradParams& p, int type, int weight_type, int kind, float* workspace,
                            hipStream_t s);
int64_t norm_grad_workspace(int64_t rows, int64_t cols, int type, bool sums);

}  // namespace mx
