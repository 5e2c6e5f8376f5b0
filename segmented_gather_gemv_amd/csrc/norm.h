// Arguments of the root-mean-square norm (passed by value).
#pragma once

#include "common.h"

namespace sgmv {

struct NormArgs {
  const void* x;
  const void* residual;  // may be null
  const void* weight;
  void* residual_out;    // may be null
  void* out;             // may be null
  void* codes;           // may be null
  float* scale;
  int64_t ldx_t, ldx_h, ldr_t, ldr_h, lds_t, lds_h, ldo_t, ldo_h, ldc_t, ldc_h;
  int64_t rows;          // T * heads
  int32_t H, W;
  float eps;
};

// Threads that share a row, and its 16-byte pieces that each of them takes.
struct NormShape {
  int group, per;
};
NormShape norm_shape(int64_t rows, int pieces);

hipError_t launch_norm(const NormArgs& A, int dtype, int format, hipStream_t stream);

}  // namespace sgmv
