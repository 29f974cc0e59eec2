// Layer norm: kernel arguments, plan and launchers (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/flce.h"

namespace flce {

struct NormArgs {
  int64_t rows, ld_x, ld_dy;   // elements between rows
  int cols;
  float eps;
  int dtype, param_dtype;
  const void* x;
  const void* weight;          // NULL = ones
  const void* bias;            // NULL = zeros
  void* y;
  float* mean;                 // of each row, for the backward; NULL: none follows
  float* rstd;
  const void* dy;
  void* dx;                    // NULL where it is not wanted, as dw and db
  void* dw;
  void* db;
  float* part;                 // column sums: [parts][2][cols], of dy xhat and of dy
  int parts;
};

// Row ranges whose column sums are formed apart.
int norm_parts(int64_t rows, int64_t cols);

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t st);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t st);

}  // namespace flce
