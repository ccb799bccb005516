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
// by their approximate instructions.  __expf(y) is off by up to 2 + floor(|1.173 y|) units of
// 2^-23, about 100 where y is near 88, which is 2^-16: 128 times less than half a step of
// bf16 (2^-9 and more).
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

// Four neighbouring channels n .. of token m, those below N: as one access where y (and the
// residual) allow it, which `wide` says (rows and addresses a multiple of four elements).
__device__ __forceinline__ bool wide4(const LinearArgs& a, size_t elem) {
  auto ok = [&](const void* p, long long ld) {
    return (reinterpret_cast<uintptr_t>(p) & (4 * elem - 1)) == 0 && (ld & 3) == 0;
  };
  return ok(a.y, a.ldy) && (!a.residual || ok(a.residual, a.ldr));
}
template <typename T>
__device__ __forceinline__ void finish4(const LinearArgs& a, bool wide, float4 z, float4 bias,
                                        long long m, int n) {
  if (wide && n + 3 < a.N) {
    struct alignas(4 * sizeof(T)) V {
      T e[4];
    };
    float v[4] = {z.x + bias.x, z.y + bias.y, z.z + bias.z, z.w + bias.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = activate<sizeof(T) == 2>(v[i], a.act);
    if (a.residual) {
      const V r = *reinterpret_cast<const V*>(static_cast<const T*>(a.residual) + m * a.ldr + n);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += to_f32(r.e[i]);
    }
    V y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y.e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<V*>(static_cast<T*>(a.y) + m * a.ldy + n) = y;
    return;
  }
  if (n < a.N) finish<T>(a, z.x, bias.x, m, n);
  if (n + 1 < a.N) finish<T>(a, z.y, bias.y, m, n + 1);
  if (n + 2 < a.N) finish<T>(a, z.z, bias.z, m, n + 2);
  if (n + 3 < a.N) finish<T>(a, z.w, bias.w, m, n + 3);
}
template <typename T>
__device__ __forceinline__ float4 bias4(const LinearArgs& a, int n) {
  const T* b = static_cast<const T*>(a.bias);
  auto at = [&](int i) { return b && n + i < a.N ? to_f32(b[n + i]) : 0.f; };
  return make_float4(at(0), at(1), at(2), at(3));
}

// Launchers, for a device of `sms` SMs; each returns the launch's cudaError_t.
cudaError_t launch_linear_simt(const LinearArgs& a, int dtype, int sms, cudaStream_t s);
// Up to two rows of x in bf16, four in fp32; x and w 16-byte aligned, rows a multiple of 16 bytes apart, K > 0.
bool linear_few_takes(const LinearArgs& a, int dtype);
cudaError_t launch_linear_few(const LinearArgs& a, int dtype, int sms, cudaStream_t s);
// bf16, any alignment, any number of rows, K > 0.
bool linear_tc_takes(const LinearArgs& a, int dtype);
cudaError_t launch_linear_tc(const LinearArgs& a, int sms, int* status, cudaStream_t s);

}  // namespace kda
