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

// kFast, for results that are rounded to bf16: the exponential and the division
// by their approximate instructions, off by a few 2^-23, not by half a step of bf16
// (2^-9 and more).
template <bool kFast>
__device__ __forceinline__ float over_1_plus_exp(float x, float y) {  // x / (1 + e^y)
  if constexpr (kFast) {
    const float d = 1.f + __expf(y);
    // __fdividef is 0 for divisors beyond 2^126, where x / d is below 2^-126 x anyway; x
    // infinite there is the quotient's NaN
    return __fdividef(x, d);
  }
  return x / (1.f + expf(y));
}

template <bool kFast>
__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case KDA_ACT_RELU: return x < 0.f ? 0.f : x;
    case KDA_ACT_SILU: return over_1_plus_exp<kFast>(x, -x);
    // x Phi(x) = x erfc(-x / sqrt 2) / 2: no cancellation in the left tail
    case KDA_ACT_GELU: return 0.5f * x * erfcf(-0.70710678118654752f * x);
    // (1 + tanh y) / 2 = 1 / (1 + e^-2y), sqrt(2 / pi) = 0.79788456
    case KDA_ACT_GELU_TANH:
      return over_1_plus_exp<kFast>(x, -1.5957691216057308f * (x + 0.044715f * x * x * x));
    case KDA_ACT_SIGMOID: return over_1_plus_exp<kFast>(1.f, -x);
    default: return x;
  }
}

// What one thread of an epilogue does to the sum of element (m, n).
template <typename T>
__device__ __forceinline__ void finish(const LinearArgs& a, float z, float bias, long long m,
                                       int n) {
  z = activate<sizeof(T) == 2>(z + bias, a.act);
  if (a.residual) z += to_f32(static_cast<const T*>(a.residual)[m * a.ldr + n]);
  static_cast<T*>(a.y)[m * a.ldy + n] = from_f32<T>(z);
}

// Launchers, for a device of `sms` SMs; each returns the launch's cudaError_t.
cudaError_t launch_linear_simt(const LinearArgs& a, int dtype, int sms, cudaStream_t s);
// Up to four rows of x; x and w 16-byte aligned, rows a multiple of 16 bytes apart, K > 0.
bool linear_few_takes(const LinearArgs& a, int dtype);
cudaError_t launch_linear_few(const LinearArgs& a, int dtype, int sms, cudaStream_t s);
// bf16, x and w as above, any number of rows.
bool linear_tc_takes(const LinearArgs& a, int dtype);
cudaError_t launch_linear_tc(const LinearArgs& a, int sms, int* status, cudaStream_t s);

}  // namespace kda
