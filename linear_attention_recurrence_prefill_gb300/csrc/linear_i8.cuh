// linear_i8.cuh -- kda_linear_i8: arguments and launchers.
#pragma once

#include "linear.cuh"

namespace kda {

// `l` holds what kda_linear has too (x and w of 8 bits, strides in bytes; K, M, N, the
// epilogue's arrays).
struct LinearI8Args {
  LinearArgs l;
  const float* x_scale;
  const float* w_scale;
};

cudaError_t launch_linear_i8_simt(const LinearI8Args& a, int dtype, int sms, cudaStream_t s);

}  // namespace kda
