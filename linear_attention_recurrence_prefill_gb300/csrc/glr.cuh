// glr.cuh -- the gated linear recurrence: arguments and the arithmetic that its
// kernels share.
//
//     g = min(la, 0) | -A softplus(la + b) | -A sigmoid(la + b),   a = e^g
//     u = c sigmoid(i) x,   c = 1 | 1 - a | sqrt(1 - a^2)
//     h_t = a_t h_{t-1} + u_t
//
// A decay near one is kept as a - 1, not as a: fp32 spaces numbers below one by
// 2^-24, which for a state that remembers a thousand tokens is a systematic
// error of 2^-25 x 1000 in it and in every gradient, while a - 1 keeps 24 bits of
// its own.  So a decay is k + t with k = 1 where it is near one and 0 where not, and
// a h + u = t h + (k h + u).  (Gradients of A and b, sums of terms that nearly cancel,
// were 2.7e-5 of their size off with a itself.)
//
// A thread has two neighbouring channels, and two numbers per instruction wherever
// there is one (packed.cuh): an element takes 44 instructions forward and 104 backward (with
// the input gate; 110 and 251 one number at a time), while HBM brings its 8 and 14 bytes in the
// time of some 40 and 75 at the best rate.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "gdr.cuh"
#include "packed.cuh"
#include "umma.cuh"

namespace kda {

constexpr int kGlrTile = KDA_GLR_TILE;  // tokens from one saved state to the next
constexpr int kGlrMaxRanks = 8;

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

// Tensor maps of the arrays that kernels read in tiles (where TMA takes them).
struct GlrMaps {
  CUtensorMap la, x, gate, dy;
};

// ---------------------------------------------------------------- the gates
// kFast, for data in bf16: the approximate instructions, whose errors (2^-22 of the value, and
// 2^-24 |x| from rounding an exponential's argument) are far below the 2^-9 that x itself is
// rounded by.  Else the functions of CUDA's library.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool kFast>
__device__ __forceinline__ float2 exp_minus(float2 x) {  // e^-x
  if constexpr (kFast) {
    const float2 y = mul2(x, both(-kLog2e));
    return make_float2(ex2_approx(y.x), ex2_approx(y.y));
  }
  return make_float2(expf(-x.x), expf(-x.y));
}
template <bool kFast>
__device__ __forceinline__ float2 inverse(float2 x) {
  return kFast ? make_float2(rcp_approx(x.x), rcp_approx(x.y)) : make_float2(1.f / x.x, 1.f / x.y);
}
template <bool kFast>
__device__ __forceinline__ float2 sigmoid2(float2 x) {  // e^-x may be infinite: 1 / infinity = 0
  return inverse<kFast>(add2(both(1.f), exp_minus<kFast>(x)));
}
// and 1 - sigmoid = e^-x sigmoid, not by a difference
template <bool kFast>
__device__ __forceinline__ float2 sigmoid2(float2 x, float2& rest) {
  const float2 e = exp_minus<kFast>(x), s = inverse<kFast>(add2(both(1.f), e)), r = mul2(e, s);
  rest = make_float2(e.x > 1e30f ? 1.f : r.x, e.y > 1e30f ? 1.f : r.y);
  return s;
}
// softplus(x) = max(x, 0) + log1p(e^-|x|), the logarithm as 2 artanh(s) with s = e / (2 + e) <= 1/3
// by its series up to s^13 (the next term below 1.5e-8): no loss where e is small.  (A NaN is one of e.)
template <bool kFast>
__device__ __forceinline__ float2 softplus2(float2 x) {
  const float2 e = exp_minus<kFast>(make_float2(fabsf(x.x), fabsf(x.y)));
  const float2 s = mul2(e, inverse<kFast>(add2(both(2.f), e))), q = mul2(s, s);
  float2 p = both(1.f / 13);
  p = fma2(p, q, both(1.f / 11));
  p = fma2(p, q, both(1.f / 9));
  p = fma2(p, q, both(1.f / 7));
  p = fma2(p, q, both(1.f / 5));
  p = fma2(p, q, both(1.f / 3));
  p = fma2(mul2(p, q), s, s);
  return fma2(both(2.f), p, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}

// ---------------------------------------------------------------- a decay
struct Decay {
  float2 t, k;
};
// 2^y - 1 for y = g log2 e in [-kNear2, 0], the Taylor polynomial of e^g - 1 in y: the first term left out
// is below 5e-8 of the value (|g| <= 1/8, and 2^-22 beyond it from the exponential, of a decay below
// 0.89) where kFast, else 1.5e-8 (|g| <= 0.347).
template <bool kFast>
struct Near {
  static constexpr float kFrom = kFast ? -0.125f * kLog2e : -0.5f;
  static __device__ __forceinline__ float2 poly(float2 y) {
    constexpr double l = 0.69314718055994531;
    float2 p;
    if constexpr (kFast) {
      p = both((float)(l * l * l * l * l / 120));
    } else {
      p = both((float)(l * l * l * l * l * l * l / 5040));
      p = fma2(p, y, both((float)(l * l * l * l * l * l / 720)));
      p = fma2(p, y, both((float)(l * l * l * l * l / 120)));
    }
    p = fma2(p, y, both((float)(l * l * l * l / 24)));
    p = fma2(p, y, both((float)(l * l * l / 6)));
    p = fma2(p, y, both((float)(l * l / 2)));
    p = fma2(p, y, both((float)l));
    return mul2(p, y);
  }
};
// The decay 2^y (NaN stays).
template <bool kFast>
__device__ __forceinline__ Decay decay_of(float2 y) {
  const float2 near = Near<kFast>::poly(y);
  const bool nx = y.x > Near<kFast>::kFrom, ny = y.y > Near<kFast>::kFrom;
  Decay d;
  d.t.x = nx ? near.x : kFast ? ex2_approx(y.x) : exp2f(y.x);
  d.t.y = ny ? near.y : kFast ? ex2_approx(y.y) : exp2f(y.y);
  d.k = make_float2(nx ? 1.f : 0.f, ny ? 1.f : 0.f);
  return d;
}
__device__ __forceinline__ float2 decay_value(const Decay& d) { return add2(d.k, d.t); }
// a h + u, a h
__device__ __forceinline__ float2 decay_apply(const Decay& d, float2 h, float2 u) {
  return fma2(d.t, h, fma2(d.k, h, u));
}
__device__ __forceinline__ float2 decay_apply(const Decay& d, float2 h) { return fma2(d.t, h, mul2(d.k, h)); }
// As one float per channel between the warps: the sign bit says whether k is 1 (t is then -0 or below).
__device__ __forceinline__ float2 decay_pack(const Decay& d) {
  return make_float2(d.k.x != 0.f ? -fabsf(d.t.x) : d.t.x, d.k.y != 0.f ? -fabsf(d.t.y) : d.t.y);
}
__device__ __forceinline__ Decay decay_unpack(float2 t) {
  Decay d;
  d.t = t;
  d.k = make_float2(__int_as_float((__float_as_int(t.x) >> 31) & 0x3f800000),
                    __int_as_float((__float_as_int(t.y) >> 31) & 0x3f800000));
  return d;
}
// 1 - a
__device__ __forceinline__ float2 decay_rest(const Decay& d) {
  return fma2(both(-1.f), d.t, fma2(both(-1.f), d.k, both(1.f)));
}
// c of a decay, and 1 / c (0 where c is 0)
template <bool kFast, bool kInverse = false>
__device__ __forceinline__ float2 input_factor(int scale, const Decay& d, float2* inv = nullptr) {
  if (scale == KDA_GLR_INPUT_NONE) return both(1.f);
  const float2 r = decay_rest(d);
  if (scale == KDA_GLR_INPUT_COMPLEMENT) return r;
  const float2 sq = mul2(r, fma2(r, both(-1.f), both(2.f)));  // (1 - a) (1 + a)
  // (the bound keeps 0 times infinity out; a NaN is still one of sq)
  float2 i = make_float2(rsqrt_approx(fmaxf(sq.x, 0x1p-126f)), rsqrt_approx(fmaxf(sq.y, 0x1p-126f)));
  if constexpr (!kFast) {  // one step of Newton's for the instruction's 2^-22
    const float2 e = fma2(mul2(mul2(sq, i), i), both(-0.5f), both(0.5f));
    i = fma2(i, e, i);
  }
  if constexpr (kInverse) *inv = make_float2(sq.x > 0x1p-126f ? i.x : 0.f, sq.y > 0x1p-126f ? i.y : 0.f);
  return mul2(sq, i);
}

// ---------------------------------------------------------------- channels of a thread
// Two neighbouring channels of a token: in one access where rows, bases and D allow it (kPair),
// else one by one, n of them.
template <typename T> struct GlrLane;
template <> struct GlrLane<__nv_bfloat16> {
  static constexpr bool kFast = true;
  using Raw = uint32_t;
  static __device__ __forceinline__ float2 widen(Raw r) {
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
  template <bool kPair>
  static __device__ __forceinline__ float2 load(const __nv_bfloat16* p, int n) {
    if constexpr (kPair) return widen(n > 0 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u);
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    return widen((n > 0 ? __ldg(q) : 0u) | (n > 1 ? (uint32_t)__ldg(q + 1) << 16 : 0u));
  }
  template <bool kPair>
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float2 v, int n) {
    const Raw r = umma::pack_bf162(v.x, v.y);
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
  static constexpr bool kFast = false;
  using Raw = float2;
  static __device__ __forceinline__ float2 widen(Raw r) { return r; }
  template <bool kPair>
  static __device__ __forceinline__ float2 load(const float* p, int n) {
    if constexpr (kPair) return n > 0 ? __ldg(reinterpret_cast<const float2*>(p)) : both(0.f);
    return make_float2(n > 0 ? __ldg(p) : 0.f, n > 1 ? __ldg(p + 1) : 0.f);
  }
  template <bool kPair>
  static __device__ __forceinline__ void store(float* p, float2 v, int n) {
    if constexpr (kPair) {
      if (n > 0) *reinterpret_cast<float2*>(p) = v;
    } else {
      if (n > 0) p[0] = v.x;
      if (n > 1) p[1] = v.y;
    }
  }
};

// ---------------------------------------------------------------- tiles
// A tile of 64 tokens by 64 channels of each array on its way to, or in, shared memory: rows of
// [token][channel], of which a warp has eight tokens and a lane two channels.  By TMA where kBytes is
// 16 (rows and bases at 16 bytes), which leaves the threads' registers to the recurrence; else copied
// by the threads in pieces of 4 bytes, or of 2 (bf16 rows at odd places).
constexpr int kGlrSeg = 8, kGlrWarps = kGlrTile / kGlrSeg, kGlrThreads = kGlrWarps * 32, kGlrCols = 64;
constexpr long long kGlrSpins = 4000000000LL;  // ~2 s of clock cycles

template <typename T, int kBytes>
struct GlrTile {
  static constexpr int kRow = kGlrCols * sizeof(T);
  static constexpr int kArray = kGlrTile * kRow;  // bytes
  static constexpr bool kTma = kBytes == 16;
  static constexpr bool kPair = kTma || (kBytes == 4 && sizeof(T) == 2);

  // Rows [0, rows) and columns [0, cols) of p (rows ld apart) to shared memory at `to`; the rest of
  // the tile gets `none` in every element.
  static __device__ __forceinline__ void copy(uint8_t* to, const T* p, long long ld, int rows, int cols, T none) {
    constexpr int kPieces = kRow / kBytes, kElems = kBytes / sizeof(T), kPer = kGlrTile * kPieces / kGlrThreads;
    const int c = threadIdx.x % kPieces, r0 = threadIdx.x / kPieces;
    const T* from = p + r0 * ld + c * kElems;
    uint8_t* dst = to + r0 * kRow + c * kBytes;
    constexpr int kStep = kGlrThreads / kPieces;
    const bool in = c * kElems < cols;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (in && r0 + i * kStep < rows) {
        if constexpr (kBytes == 4) umma::cp_async4(umma::smem_u32(dst), from);
        else *reinterpret_cast<T*>(dst) = *from;
      } else {
#pragma unroll
        for (int e = 0; e < kElems; ++e) reinterpret_cast<T*>(dst)[e] = none;
      }
      from += kStep * ld;
      dst += kStep * kRow;
    }
  }
  // This thread's own elements behind the end of the sequence, of which TMA brings the next one's:
  // `none`, from token `k0` of its segment on.
  static __device__ __forceinline__ void clear(uint8_t* array, int warp, int lane, int k0, T none) {
    for (int k = k0 > 0 ? k0 : 0; k < kGlrSeg; ++k) {
      T* e = reinterpret_cast<T*>(array + (warp * kGlrSeg + k) * kRow) + 2 * lane;
      e[0] = e[1] = none;
    }
  }
  // this thread's channels of token k of its segment
  static __device__ __forceinline__ float2 get(const uint8_t* array, int warp, int lane, int k) {
    using Raw = typename GlrLane<T>::Raw;
    return GlrLane<T>::widen(*reinterpret_cast<const Raw*>(array + (warp * kGlrSeg + k) * kRow + lane * sizeof(Raw)));
  }
};

// n of a thread's states at p, or zeros (not __ldg: they may be written by the same kernel)
__device__ __forceinline__ float2 load_states(const float* p, int n) {
  return make_float2(p && n > 0 ? p[0] : 0.f, p && n > 1 ? p[1] : 0.f);
}
__device__ __forceinline__ void store_states(float* p, float2 v, int n) {
  if (n > 0) p[0] = v.x;
  if (n > 1) p[1] = v.y;
}

// Parameters of a thread's channels.
struct GlrChannels {
  float2 A, b;  // A times -log2 e
};
__device__ __forceinline__ GlrChannels glr_channels(const GlrArgs& a, int ch, int n) {
  GlrChannels p;
  p.A = a.decay_scale ? load_states(a.decay_scale + ch, n) : both(1.f);
  p.A = mul2(p.A, both(-kLog2e));
  p.b = load_states(a.decay_bias ? a.decay_bias + ch : nullptr, n);
  return p;
}
// Log decays to base 2.
template <int kFrom, bool kFast>
__device__ __forceinline__ float2 glr_log_decay(const GlrChannels& p, float2 la) {
  if constexpr (kFrom == KDA_GLR_LOG)  // above 0: 0 (NaN stays)
    return mul2(make_float2(la.x > 0.f ? 0.f : la.x, la.y > 0.f ? 0.f : la.y), both(kLog2e));
  const float2 v = add2(la, p.b);
  return mul2(p.A, kFrom == KDA_GLR_SOFTPLUS ? softplus2<kFast>(v) : sigmoid2<kFast>(v));
}
// A log_alpha whose decay is 1, for tokens behind a sequence's end.
__device__ __forceinline__ float glr_no_decay(int from) { return from == KDA_GLR_LOG ? 0.f : -INFINITY; }

// Row of the saved states at which sequence n, whose first token is t0, starts: rows of
// different sequences never meet, since t0' / 64 - t0 / 64 + 1 >= (t0' - t0) / 64 rounded up.
__device__ __forceinline__ size_t glr_checkpoint_row(int t0, int n) {
  return (size_t)(t0 / kGlrTile) + n;
}

// f(std::integral_constant) of the form of the decays, or of the inputs
template <typename F>
__device__ __forceinline__ void glr_decay_from(int from, const F& f) {
  if (from == KDA_GLR_LOG) f(std::integral_constant<int, KDA_GLR_LOG>());
  else if (from == KDA_GLR_SOFTPLUS) f(std::integral_constant<int, KDA_GLR_SOFTPLUS>());
  else f(std::integral_constant<int, KDA_GLR_SIGMOID>());
}

template <typename F>
__device__ __forceinline__ void glr_input_scale(int scale, const F& f) {
  if (scale == KDA_GLR_INPUT_NONE) f(std::integral_constant<int, KDA_GLR_INPUT_NONE>());
  else if (scale == KDA_GLR_INPUT_COMPLEMENT) f(std::integral_constant<int, KDA_GLR_INPUT_COMPLEMENT>());
  else f(std::integral_constant<int, KDA_GLR_INPUT_NORMALIZED>());
}

// A wait for a tile, or for the other CTAs' totals.  A build of these kernels for tests defines which of
// them give up at once (limits as arguments instead took 3 us of the 105 that nine packed prompts take).
enum GlrWait { kGlrWaitTile, kGlrWaitTotals };
#ifndef KDA_GLR_GIVES_UP
#define KDA_GLR_GIVES_UP(what) false
#endif
template <GlrWait kWhat>
__device__ __forceinline__ bool glr_wait(uint64_t* bar, int parity) {
  return !(KDA_GLR_GIVES_UP(kWhat)) && umma::mbar_wait_soon(bar, parity, kGlrSpins);
}

// ---------------------------------------------------------------- between the CTAs of a cluster
// Decays and states (or gradients) of the tiles of a round, which every CTA sends to every other:
// each write counts on a barrier of the CTA that it goes to, so that nobody waits for more than
// what it needs.  Two sets in turn: a CTA sends those of a round only behind its own reads of the
// round before, and nobody gets to the next round without them.
struct GlrExchange {
  float4 tot[2][kGlrMaxRanks][32];
  uint64_t arrived[2];

  __device__ __forceinline__ void init() {  // one thread; before the cluster's first barrier
    umma::mbar_init(&arrived[0], 1);
    umma::mbar_init(&arrived[1], 1);
    umma::mbar_fence_init();
  }
  // by one warp
  __device__ __forceinline__ void send(int p, int rank, int ranks, int lane, float4 v) {
    if (lane == 0) umma::mbar_arrive_expect_tx(&arrived[p], ranks * 512);
    for (int r = 0; r < ranks; ++r)
      umma::st_async_f32x4(umma::map_to_rank(umma::smem_u32(&tot[p][rank][lane]), r), v,
                           umma::map_to_rank(umma::smem_u32(&arrived[p]), r));
  }
  __device__ __forceinline__ bool wait(int p, int round) {
    return glr_wait<kGlrWaitTotals>(&arrived[p], (round >> 1) & 1);
  }
};

// Behind a wait that gave up, which the whole CTA has agreed on before it expects anything more on a
// barrier: what is still on its way to this CTA's shared memory lands, or has its time, before that is
// released.  `fetched`, `sent`: how often the barriers of either pair, in turn, were told what to expect.
__device__ __forceinline__ void glr_settle(uint64_t (&landed)[2], int fetched, uint64_t (&arrived)[2], int sent) {
  for (int i = fetched > 2 ? fetched - 2 : 0; i < fetched; ++i) umma::mbar_wait(&landed[i & 1], (i >> 1) & 1, kGlrSpins);
  for (int i = sent > 2 ? sent - 2 : 0; i < sent; ++i) umma::mbar_wait(&arrived[i & 1], (i >> 1) & 1, kGlrSpins);
}

// Launchers; each returns the launch's cudaError_t.  bytes: what rows, bases and D allow to move at
// once (GlrTile): 16, 4, or 2.
cudaError_t launch_glr_few(const GlrArgs& a, int dtype, int bytes, cudaStream_t s);
cudaError_t launch_glr_scan(const GlrArgs& a, int dtype, int bytes, int ranks, cudaStream_t s);
cudaError_t launch_glr_backward(const GlrArgs& a, int dtype, int bytes, int ranks, float* dA, float* db,
                                cudaStream_t s);

}  // namespace kda
