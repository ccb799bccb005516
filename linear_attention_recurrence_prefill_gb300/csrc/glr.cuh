// glr.cuh -- the gated linear recurrence: arguments and the per-element
// arithmetic that its kernels share.
//
//     g = min(la, 0) | -A softplus(la + b) | -A sigmoid(la + b),   a = e^g
//     u = c sigmoid(i) x,   c = 1 | 1 - a | sqrt(1 - a^2)
//     h_t = a_t h_{t-1} + u_t
//
// A decay near one is kept as a - 1, not as a: fp32 spaces values below one by
// 2^-24, which for a state that remembers a thousand tokens is a systematic
// error of 2^-25 x 1000 in it and in every gradient, while a - 1 keeps 24 bits of
// its own.  So a decay is a `Decay`: a number whose sign bit says what it is,
// a - 1 in [-1/2, -0] or a itself in [+0, 1/2..].  (Gradients of A and b, sums of
// terms that nearly cancel, were 2.7e-5 of their size off with a itself.)
#pragma once

#include "gdr.cuh"
#include "umma.cuh"

namespace kda {

constexpr int kGlrTile = KDA_GLR_TILE;  // tokens from one saved state to the next
constexpr int kGlrWarps = 8, kGlrSeg = kGlrTile / kGlrWarps;

struct GlrArgs {
  const void* x;
  const void* la;
  const void* gate;           // NULL: none
  const float* h0;            // NULL: zeros
  float* h_T;
  void* y;
  const int32_t* cu_seqlens;  // NULL: N sequences of T_total / N tokens
  const int32_t* slots;       // NULL: state n belongs to sequence n
  const float* decay_scale;   // NULL: ones
  const float* decay_bias;    // NULL: zeros
  float* checkpoints;         // NULL, or the state before every kGlrTile-th token
  int* status;
  int N, T_total, D, n_slots, decay_from, input_scale;
  long long ldx, ldla, ldg;   // elements between tokens
  // the gradient
  const void* dy;             // NULL: zeros
  const float* dh_T;          // NULL: zeros
  void* dx;
  void* dla;
  void* dgate;                // NULL: not wanted, as the ones below
  float* dh0;
  double2* partial;           // NULL, or [N][ranks][D]: the share of each CTA in dA and db
};

// ---------------------------------------------------------------- a decay
__device__ __forceinline__ bool decay_is_near(float t) { return __float_as_int(t) < 0; }
// e^g - 1 for g in [-0.347, 0]: the Taylor polynomial, the next term below 1.5e-8 of the value.
__device__ __forceinline__ float expm1_near(float g) {
  float p = 1.f / 5040;
  p = fmaf(p, g, 1.f / 720);
  p = fmaf(p, g, 1.f / 120);
  p = fmaf(p, g, 1.f / 24);
  p = fmaf(p, g, 1.f / 6);
  p = fmaf(p, g, 0.5f);
  return fmaf(p * g, g, g);
}
// The decay of log decay g <= 0 (NaN stays).
__device__ __forceinline__ float decay_of(float g) {
  const float near = -fabsf(expm1_near(g)), far = expf(g);
  return g > -0.34657359f ? near : far;
}
__device__ __forceinline__ float decay_value(float t) { return decay_is_near(t) ? 1.f + t : t; }
// a h + u
__device__ __forceinline__ float decay_apply(float t, float h, float u) {
  const float r = fmaf(t, h, u);
  return decay_is_near(t) ? h + r : r;
}

// ---------------------------------------------------------------- the gates
// x's sigmoid and e^-|x|, by the approximate instructions where kFast (data in bf16: their error,
// 2^-20 for |x| up to 10, is far below the 2^-9 that x itself is rounded by).
template <bool kFast>
__device__ __forceinline__ float exp_of(float x) {
  return kFast ? __expf(x) : expf(x);
}
template <bool kFast>
__device__ __forceinline__ float quotient(float x, float y) {
  return kFast ? __fdividef(x, y) : x / y;
}
template <bool kFast>
__device__ __forceinline__ float sigmoid_of(float x) {
  // e^-|x| <= 1: no quotient of infinities
  const float e = exp_of<kFast>(-fabsf(x));
  return quotient<kFast>(x < 0.f ? e : 1.f, 1.f + e);
}
// softplus(x) = max(x, 0) + log1p(e^-|x|), the logarithm as 2 artanh(s) with s = e / (2 + e) <= 1/3
// by its series up to s^13 (the next term below 1.5e-8): no loss where e is small.
template <bool kFast>
__device__ __forceinline__ float softplus_of(float x) {
  const float e = exp_of<kFast>(-fabsf(x));
  const float s = quotient<kFast>(e, 2.f + e), q = s * s;
  float p = 1.f / 13;
  p = fmaf(p, q, 1.f / 11);
  p = fmaf(p, q, 1.f / 9);
  p = fmaf(p, q, 1.f / 7);
  p = fmaf(p, q, 1.f / 5);
  p = fmaf(p, q, 1.f / 3);
  p = fmaf(p * q, s, s);
  return fmaf(2.f, p, fmaxf(x, 0.f));  // (a NaN is one of e)
}
__device__ __forceinline__ float sqrt_fast(float x) {  // off by 2^-23 at most
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// c of the decay t
__device__ __forceinline__ float input_factor(int scale, float t) {
  if (scale == KDA_GLR_INPUT_NONE) return 1.f;
  const bool near = decay_is_near(t);
  if (scale == KDA_GLR_INPUT_COMPLEMENT) return near ? -t : 1.f - t;
  return sqrt_fast(near ? -t * (2.f + t) : fmaf(-t, t, 1.f));
}

// ---------------------------------------------------------------- channels of a thread
// bf16: two neighbouring channels per lane (4 bytes a token, 128 per warp); fp32: one.
template <typename T> struct GlrLane;
template <> struct GlrLane<__nv_bfloat16> {
  static constexpr int kCh = 2;
  static constexpr bool kFast = true;
  using Raw = uint32_t;
  static __device__ __forceinline__ void widen(Raw r, float (&v)[2]) {
    v[0] = __uint_as_float(r << 16);
    v[1] = __uint_as_float(r & 0xffff0000u);
  }
  static __device__ __forceinline__ Raw narrow(const float (&v)[2]) {
    return umma::pack_bf162(v[0], v[1]);
  }
  // kPair: both at once (rows and base a multiple of 4 bytes, D even); else one by one, `n` of them
  template <bool kPair>
  static __device__ __forceinline__ Raw load(const __nv_bfloat16* p, int n) {
    if constexpr (kPair) {
      return n > 0 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
      uint32_t r = n > 0 ? __ldg(q) : 0u;
      if (n > 1) r |= (uint32_t)__ldg(q + 1) << 16;
      return r;
    }
  }
  template <bool kPair>
  static __device__ __forceinline__ void store(__nv_bfloat16* p, Raw r, int n) {
    if constexpr (kPair) {
      if (n > 0) *reinterpret_cast<uint32_t*>(p) = r;
    } else {
      uint16_t* q = reinterpret_cast<uint16_t*>(p);
      if (n > 0) q[0] = (uint16_t)r;
      if (n > 1) q[1] = (uint16_t)(r >> 16);
    }
  }
};
template <> struct GlrLane<float> {
  static constexpr int kCh = 1;
  static constexpr bool kFast = false;
  using Raw = float;
  static __device__ __forceinline__ void widen(Raw r, float (&v)[1]) { v[0] = r; }
  static __device__ __forceinline__ Raw narrow(const float (&v)[1]) { return v[0]; }
  template <bool kPair>
  static __device__ __forceinline__ Raw load(const float* p, int n) {
    return n > 0 ? __ldg(p) : 0.f;
  }
  template <bool kPair>
  static __device__ __forceinline__ void store(float* p, Raw r, int n) {
    if (n > 0) *p = r;
  }
};
// `n` of a thread's fp32 values at p (not __ldg: a state may be written by the same kernel)
template <int kCh>
__device__ __forceinline__ void load_states(float (&v)[kCh], const float* p, int n) {
#pragma unroll
  for (int c = 0; c < kCh; ++c) v[c] = p && c < n ? p[c] : 0.f;
}
template <int kCh>
__device__ __forceinline__ void store_states(float* p, const float (&v)[kCh], int n) {
#pragma unroll
  for (int c = 0; c < kCh; ++c)
    if (c < n) p[c] = v[c];
}

// A channel's parameters.
struct GlrChannel {
  float A, b;
};
__device__ __forceinline__ GlrChannel glr_channel(const GlrArgs& a, int ch, bool in) {
  GlrChannel p;
  p.A = a.decay_scale && in ? a.decay_scale[ch] : 1.f;
  p.b = a.decay_bias && in ? a.decay_bias[ch] : 0.f;
  return p;
}
// The log decay of an element.
template <bool kFast>
__device__ __forceinline__ float glr_log_decay(int from, const GlrChannel& p, float la) {
  if (from == KDA_GLR_LOG) return la > 0.f ? 0.f : la;  // NaN stays
  return -p.A * (from == KDA_GLR_SOFTPLUS ? softplus_of<kFast>(la + p.b) : sigmoid_of<kFast>(la + p.b));
}

// Row of the saved states at which sequence n, whose first token is t0, starts: rows of
// different sequences never meet, since t0' / 64 - t0 / 64 + 1 >= (t0' - t0) / 64 rounded up.
__device__ __forceinline__ size_t glr_checkpoint_row(int t0, int n) {
  return (size_t)(t0 / kGlrTile) + n;
}

// Launchers; each returns the launch's cudaError_t.  pair: see GlrLane.
cudaError_t launch_glr_few(const GlrArgs& a, int dtype, bool pair, cudaStream_t s);
cudaError_t launch_glr_scan(const GlrArgs& a, int dtype, bool pair, int ranks, cudaStream_t s);
cudaError_t launch_glr_backward(const GlrArgs& a, int dtype, bool pair, int ranks, float* dA, float* db,
                                cudaStream_t s);

}  // namespace kda
