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

// A sum with its scales and the bias, in two roundings.  Every kernel has it from here, so that a token's
// row is the same to the bit whatever kernel the number of rows chooses (the compiler fused the
// bias's addition in some of them and not in others).
__device__ __forceinline__ float scaled(float sum, float x_scale, float w_scale, float bias) {
  return __fmaf_rn(__fmul_rn(sum, x_scale), w_scale, bias);
}

// K = 0 only: y = act(bias) + residual.
cudaError_t launch_linear_i8_none(const LinearI8Args& a, int dtype, cudaStream_t s);
// Up to eight rows of x; x and w 16-byte aligned, rows a multiple of 16 bytes apart, K > 0.
bool linear_i8_few_takes(const LinearI8Args& a);
cudaError_t launch_linear_i8_few(const LinearI8Args& a, int dtype, int sms, cudaStream_t s);
// Any alignment and number of rows, K > 0.
bool linear_i8_tc_takes(int M, int N);
size_t linear_i8_workspace_bytes(int M, int N, int K);  // whatever the alignment
bool linear_i8_tc_needs_workspace(const LinearArgs& l);
cudaError_t launch_linear_i8_tc(const LinearI8Args& a, int dtype, void* workspace, int sms, int* status,
                                cudaStream_t s);
// linear_tc.cu: l.x and l.w are fp16 arrays that hold the integers, rows 16-byte aligned.
cudaError_t launch_linear_i8_pair(const LinearI8Args& a, int dtype, int sms, int* status, cudaStream_t s);

}  // namespace kda
