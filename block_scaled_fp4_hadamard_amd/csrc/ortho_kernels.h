// Internal interface between the C ABI layer and the kernels that
// orthogonalize matrices by Newton-Schulz steps.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include "../../include/mxfp4.h"
#include "ortho_path.h"

namespace mx {

// One matrix: orthogonalized into `out`, or (w set) a Muon step of w.
struct OrthoItem {
  const void* g;                 // [rows][ld_g], float32 or bf16
  float* moment;                 // [rows][cols], or null
  float* w;                      // [rows][cols], or null
  uint16_t* copy;                // [rows][cols], or null
  void* out;                     // [rows][ld_out], float32 or bf16, or null
  uint8_t* space;                // its part of the workspace
  int64_t ld_g, ld_out;
  int rows, cols;
  bool g_bf16, out_bf16;
  double scale;                  // of the update (w)
};

struct OrthoStep {
  double a, b, c, eps;
  int steps;
  // Muon
  float momentum, rest;          // of the moment, rest = 1 - momentum; u = g without one
  bool nesterov;
  double lr, weight_decay;
  const float* lr_dev;
  const float* grad_scale;
};

// items: at most kOrthoGroup of them, none empty
hipError_t launch_ortho(const OrthoItem* items, int count, const OrthoStep& step, hipStream_t s);

}  // namespace mx
