// norm.cuh -- kda_rmsnorm and kda_quantize_i8: arguments and launcher.
#pragma once

#include "kda_common.cuh"

namespace kda {

struct NormArgs {
  const void* x;
  const void* residual;  // NULL: none
  const float* w;        // NULL: ones
  void* sum;             // NULL: not wanted; may be x or the residual
  void* y;               // NULL: not wanted
  int8_t* q;             // NULL: not wanted, with scale
  float* scale;
  long long ldx, ldr, lds, ldy, ldq;
  int M, D;
  float eps;
  bool norm;  // false: n = s
};

cudaError_t launch_norm_bf16(const NormArgs& a, int sms, cudaStream_t s);
cudaError_t launch_norm_f32(const NormArgs& a, int sms, cudaStream_t s);
inline cudaError_t launch_norm(const NormArgs& a, int dtype, int sms, cudaStream_t s) {
  return dtype == KDA_BF16 ? launch_norm_bf16(a, sms, s) : launch_norm_f32(a, sms, s);
}

}  // namespace kda
