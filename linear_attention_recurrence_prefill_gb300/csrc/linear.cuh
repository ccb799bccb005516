// linear.cuh -- kda_linear: arguments and the epilogue that its kernels share.
#pragma once

#include "kda_common.cuh"

namespace kda {

struct LinearArgs {
  const void* x;
  const void* w;
  const void* bias;      // NULL: none
  const void* residual;  // NULL: none; may be y
  void* y;
  long long ldx, ldw, ldr, ldy;
  int M, N, K, act;
};

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case KDA_ACT_RELU: return x < 0.f ? 0.f : x;
    case KDA_ACT_SILU: return x / (1.f + expf(-x));
    // x Phi(x) = x erfc(-x / sqrt 2) / 2: no cancellation in the left tail
    case KDA_ACT_GELU: return 0.5f * x * erfcf(-0.70710678118654752f * x);
    // (1 + tanh y) / 2 = 1 / (1 + e^-2y), sqrt(2 / pi) = 0.79788456
    case KDA_ACT_GELU_TANH:
      return x / (1.f + expf(-1.5957691216057308f * (x + 0.044715f * x * x * x)));
    case KDA_ACT_SIGMOID: return sigmoidf_(x);
    default: return x;
  }
}

// What one thread of an epilogue does to the sum of element (m, n).
template <typename T>
__device__ __forceinline__ void finish(const LinearArgs& a, float z, float bias, long long m,
                                       int n) {
  z = activate(z + bias, a.act);
  if (a.residual) z += to_f32(static_cast<const T*>(a.residual)[m * a.ldr + n]);
  static_cast<T*>(a.y)[m * a.ldy + n] = from_f32<T>(z);
}

cudaError_t launch_linear_simt(const LinearArgs& a, int dtype, cudaStream_t s);
// bf16 with x and w 16-byte aligned, rows a multiple of 16 bytes apart, K > 0.
bool linear_tc_takes(const LinearArgs& a, int dtype);
cudaError_t launch_linear_tc(const LinearArgs& a, int* status, cudaStream_t s);

}  // namespace kda
