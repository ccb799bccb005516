// norm_rows.cuh -- the kernels of the root-mean-square norm with the residual's addition,
// output in the data type or in 8 bits with a scale per token.  Included by one file per
// data type, for the time that they take to compile.
//
//     s = x + residual,  n = s r w with r = 1 / sqrt(mean s^2 + eps)
//     scale = max |n| / 127,  q = n / scale = 127 p / max |p| with p = s w
//
// q does not depend on r, so the squares' sum and the largest |p| are found in one
// reduction over the row, which stays in registers between that and the outputs: each
// array is read once and written once, and HBM is the bound.  q is the integer nearest to
// the quotient as 64 bits have it: the product of p and 127 / max |p| is off by the five roundings of
// s, p, the largest s and p, and the division, 5 * 2^-24 of itself, and its distance to an integer, formed
// by one fma, by 2^-26 more, which is 2^-25 of a quotient of 1/2 or above: 3.28e-7 in all.  So
// only those that are nearer than 3.3e-7 of themselves to the middle between two integers (one in
// 48,000 of normally distributed ones) are taken again in 64 bits, with the largest product, from the
// stored inputs.
//
// 12,001 x 4096 in bf16 with the residual: 65 us (6.0 TB/s, 0.89 of the measured copy rate), 82 us with one
// row at a time; in fp32 129 us (0.90).  In 8 bits, bound by the barriers and instructions of forming the
// integers, 90 us (0.56) with weights that differ, 110 us (0.86) in fp32.  Where bf16 rows have no weights,
// or equal ones, nearly every row has elements of half its largest, whose quotient is 63.5 exactly, and takes some
// of its quotients again: 200 to 215 us (0.24), without a residual 225, kda_quantize_i8 195 (0.11; in fp32,
// where such elements are rare, 68, 0.53).  One row of 4096: 2.8 us.  Rows that are no multiple of 8
// elements, or not at 16 bytes, go element by element: 3000 x 8191 89 us (0.32).  The 8-bit forms for 8,193 to 16,384
// elements spill (up to 704 bytes a thread in bf16, 868 in fp32, whose 1024 threads have 64 registers): 4000 x 12288
// without differing weights 335 and 241 us.
#pragma once

#include "norm.cuh"
#include "umma.cuh"

namespace kda {
namespace {

constexpr float kMiddle = 3.3e-7f;

template <typename T>
__device__ __forceinline__ double exact_product(const NormArgs& a, long long m, int d) {
  double s = (double)to_f32(static_cast<const T*>(a.x)[m * a.ldx + d]);
  if (a.residual) s += (double)to_f32(static_cast<const T*>(a.residual)[m * a.ldr + d]);
  return a.w ? s * (double)a.w[d] : s;
}
// The nearest integer to the quotient of a product next to the middle between two.
__device__ __noinline__ int quantized_exactly(double product, double largest) {
  return (int)rint(127. * product / largest);
}

// What a row's threads know after the reductions.
struct Row {
  float r, scale, inv;  // inv = 127 / largest
  float always;  // 1 where 127 / largest may overflow: every quotient is taken again
};
__device__ __forceinline__ Row row_of(const NormArgs& a, float squares, uint32_t largest_bits) {
  Row o;
  const float v = squares / (float)a.D + a.eps;
  o.r = !a.norm ? 1.f : v > 0.f ? 1.f / sqrtf(v) : v;  // 0 for a row of zeros with eps = 0; NaN stays
  const float big = __uint_as_float(largest_bits);
  const bool finite = largest_bits < 0x7f800000u;
  o.scale = finite ? big * (1.f / 127.f) * o.r : big * o.r;
  if (finite && big < 0x1p-100f) o.scale = (float)((double)big * (double)o.r / 127.);
  o.inv = finite && big > 0.f && o.r != 0.f ? 127.f / big : 0.f;  // (r = 0: the squares vanished)
  o.always = finite && big > 0.f && big < 0x1p-100f ? 1.f : 0.f;
  return o;
}
// What the products are that may be the largest in 64 bits.
__device__ __forceinline__ float next_to(uint32_t largest_bits) {
  return __uint_as_float(largest_bits) * (1.f - 0x1p-21f);
}
__device__ __forceinline__ void take_larger(unsigned long long* largest, double product) {
  atomicMax(largest, (unsigned long long)__double_as_longlong(fabs(product)));
}
// The integer of product p, which is next to the middle between two or may be.
template <typename T>
__device__ __forceinline__ int quantized(const NormArgs& a, const Row& o, double largest, float p, long long m, int d) {
  if (o.inv == 0.f) return 0;
  const float v = p * o.inv, k = rintf(v);
  return !(fabsf(fmaf(p, o.inv, -k)) + kMiddle * fabsf(v) < 0.5f - o.always)
             ? quantized_exactly(exact_product<T>(a, m, d), largest)
             : (int)k;
}

// Rows in registers: kThreads threads per row, each kVecs vectors of eight elements, one in every
// kThreads; a persistent CTA walks over rows and has the next ones on their way while it works.
// kWide: 16-byte accesses (every row and w at 16 bytes, q at 8); else element by element,
// neighbouring threads neighbouring elements.
template <typename T, int kThreads, bool kI8>
struct Norm {
  static constexpr int kRows = kThreads >= 256 ? 1 : 256 / kThreads;  // of a CTA
  static constexpr int kCta = kThreads * kRows;
  // 64 registers per thread, 128 where elements have 32 bits (two rows are held at a time) and where
  // integers are formed
  static constexpr int kPerSm = kCta >= 1024 ? 1 : (sizeof(T) == 2 && !kI8 ? 1024 : 512) / kCta;
};
template <typename T, int kThreads, int kVecs, bool kWide, bool kI8>
__global__ void __launch_bounds__(Norm<T, kThreads, kI8>::kCta, Norm<T, kThreads, kI8>::kPerSm) norm_kernel(NormArgs a) {
  constexpr int kRows = Norm<T, kThreads, kI8>::kRows, kWarps = kThreads / 32;
  constexpr int kRaw = (int)sizeof(T) * 2;  // words of a vector
  __shared__ float squares[2][kRows][kWarps];
  __shared__ uint32_t bits[2][kRows][kWarps];
  __shared__ unsigned long long largest[2][kRows];
  const int row = threadIdx.x / kThreads, tid = threadIdx.x % kThreads, warp = tid >> 5, lane = tid & 31;
  umma::grid_launch_dependents();
  umma::grid_wait_prerequisites();  // what ran before is complete
  auto sync = [] {
    if constexpr (kThreads == 32) __syncwarp();
    else __syncthreads();
  };
  // element e of vector v
  auto index = [&](int v, int e) { return kWide ? (v * kThreads + tid) * 8 + e : (v * 8 + e) * kThreads + tid; };
  auto load = [&](uint32_t (&raw)[kVecs][kRaw], const void* base, long long ld, long long m) {
    const T* p = static_cast<const T*>(base) + m * ld;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if constexpr (kWide) {
        const bool in = m < a.M && index(v, 0) < a.D;
#pragma unroll
        for (int i = 0; i < kRaw / 4; ++i) {
          const uint4 q = in ? *(reinterpret_cast<const uint4*>(p + index(v, 0)) + i) : make_uint4(0, 0, 0, 0);
          raw[v][4 * i] = q.x; raw[v][4 * i + 1] = q.y; raw[v][4 * i + 2] = q.z; raw[v][4 * i + 3] = q.w;
        }
      } else {
        auto at = [&](int e) { return m < a.M && index(v, e) < a.D ? to_f32(p[index(v, e)]) : 0.f; };
#pragma unroll
        for (int e = 0; e < kRaw; ++e)
          raw[v][e] = kRaw == 8 ? __float_as_uint(at(e)) : umma::pack_bf162(at(2 * e), at(2 * e + 1));
      }
    }
  };
  auto widen = [](const uint32_t (&raw)[kRaw], int e) {
    if constexpr (kRaw == 8) return __uint_as_float(raw[e]);
    return __uint_as_float(e & 1 ? raw[e >> 1] & 0xffff0000u : raw[e >> 1] << 16);
  };
  auto store = [&](void* base, long long at, const float (&out)[8], int v) {
    T* p = static_cast<T*>(base) + at;
    if constexpr (kWide) {
      const int d = index(v, 0);
      if (d >= a.D) return;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p + d) = make_uint4(umma::pack_bf162(out[0], out[1]), umma::pack_bf162(out[2], out[3]),
                                                      umma::pack_bf162(out[4], out[5]), umma::pack_bf162(out[6], out[7]));
      } else {
        *reinterpret_cast<float4*>(p + d) = make_float4(out[0], out[1], out[2], out[3]);
        *(reinterpret_cast<float4*>(p + d) + 1) = make_float4(out[4], out[5], out[6], out[7]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (index(v, e) < a.D) p[index(v, e)] = from_f32<T>(out[e]);
    }
  };
  auto weights = [&](float (&w)[8], int v) {
    if constexpr (kWide) {
      const int d = index(v, 0);
      const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
      const bool in = a.w && d < a.D;
      const float4 q0 = in ? __ldg(reinterpret_cast<const float4*>(a.w + d)) : one;
      const float4 q1 = in ? __ldg(reinterpret_cast<const float4*>(a.w + d) + 1) : one;
      w[0] = q0.x; w[1] = q0.y; w[2] = q0.z; w[3] = q0.w;
      w[4] = q1.x; w[5] = q1.y; w[6] = q1.z; w[7] = q1.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = a.w && index(v, e) < a.D ? __ldg(a.w + index(v, e)) : 1.f;
    }
  };

  const long long step = (long long)gridDim.x * kRows;
  uint32_t rx[kVecs][kRaw], rr[kVecs][kRaw];
  long long m = (long long)blockIdx.x * kRows + row;
  load(rx, a.x, a.ldx, m);
  if (a.residual) load(rr, a.residual, a.ldr, m);
  int p = 0;
  for (long long first = (long long)blockIdx.x * kRows; first < a.M; first += step, m += step, p ^= 1) {
    const bool live = m < a.M;
    float s[kVecs][8], sq = 0.f;
    uint32_t big = 0;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[v][e] = widen(rx[v], e);
        if (a.residual) s[v][e] += widen(rr[v], e);
        sq = fmaf(s[v][e], s[v][e], sq);
      }
      if constexpr (kI8) {
        float w[8];
        weights(w, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)  // NaN above infinity above all else
          big = max(big, __float_as_uint(fabsf(s[v][e] * w[e])));
      }
    }
    // the next rows (x and the residual, of which `sum` may be one, are only written at this row)
    if (first + step < a.M) {
      load(rx, a.x, a.ldx, m + step);
      if (a.residual) load(rr, a.residual, a.ldr, m + step);
    }
    const uint32_t mine = big;
    sq = warp_sum(sq);
    if constexpr (kI8) big = __reduce_max_sync(0xffffffffu, big);
    if constexpr (kWarps > 1) {
      if (lane == 0) {
        squares[p][row][warp] = sq;
        bits[p][row][warp] = big;
      }
      if (tid == 0) largest[p][row] = 0;
      sync();
      sq = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        sq += squares[p][row][i];
        if constexpr (kI8) big = max(big, bits[p][row][i]);
      }
    } else if (kI8 && tid == 0) {
      largest[p][row] = 0;
    }
    const Row o = row_of(a, sq, big);
    if constexpr (kI8) {
      if (live && tid == 0) a.scale[m] = o.scale;
      // the nearest integers by adding 1.5 * 2^23, whose low bits they then are
      constexpr float kMagic = 12582912.f;
      uint32_t k[kVecs][8];
      float far = 0.f;
      const float middle = o.inv * kMiddle;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        float w[8];
        weights(w, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = s[v][e] * w[e], t = fmaf(z, o.inv, kMagic);
          k[v][e] = __float_as_uint(t);
          far = fmaxf(far, fabsf(fmaf(z, o.inv, kMagic - t)) + fabsf(z * middle));
        }
      }
      const bool again = live && o.inv != 0.f && !(far < 0.5f - o.always);
      const bool any = kWarps > 1 ? __syncthreads_or(again) : __any_sync(0xffffffffu, again);
      if (any) {
        if (kWarps == 1) __syncwarp();  // `largest` is zero for every lane
        if (live && __uint_as_float(mine) >= next_to(big)) {
#pragma unroll
          for (int v = 0; v < kVecs; ++v) {
            float w[8];
            weights(w, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (fabsf(s[v][e] * w[e]) >= next_to(big) && index(v, e) < a.D)
                take_larger(&largest[p][row], exact_product<T>(a, m, index(v, e)));
          }
        }
        sync();
        if (again) {
          const double exact = __longlong_as_double((long long)largest[p][row]);
#pragma unroll
          for (int v = 0; v < kVecs; ++v) {
            float w[8];
            weights(w, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (index(v, e) < a.D)
                k[v][e] = (uint32_t)quantized<T>(a, o, exact, s[v][e] * w[e], m, index(v, e));
          }
        }
      }
      if (live) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          if (o.inv == 0.f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) k[v][e] = 0;
          }
          if constexpr (kWide) {
            const uint32_t lo =
                __byte_perm(__byte_perm(k[v][0], k[v][1], 0x0040), __byte_perm(k[v][2], k[v][3], 0x0040), 0x5410);
            const uint32_t hi =
                __byte_perm(__byte_perm(k[v][4], k[v][5], 0x0040), __byte_perm(k[v][6], k[v][7], 0x0040), 0x5410);
            if (index(v, 0) < a.D) *reinterpret_cast<uint2*>(a.q + m * a.ldq + index(v, 0)) = make_uint2(lo, hi);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (index(v, e) < a.D) a.q[m * a.ldq + index(v, e)] = (int8_t)k[v][e];
          }
        }
      }
    }
    if (!live) continue;
    if (kI8 && !a.y && !a.sum) continue;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (a.sum) store(a.sum, m * a.lds, s[v], v);  // behind the last read of the inputs, of which it may be one
      if (!kI8 || a.y) {
        float w[8], n[8];
        weights(w, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = s[v][e] * o.r * w[e];
        store(a.y, m * a.ldy, n, v);
      }
    }
  }
}

// Rows that do not fit in registers: a CTA per row, which reads it once per step.
template <typename T>
__global__ void __launch_bounds__(1024) norm_any_kernel(NormArgs a) {
  __shared__ float squares[32];
  __shared__ uint32_t bits[32];
  __shared__ unsigned long long largest;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  umma::grid_launch_dependents();
  umma::grid_wait_prerequisites();  // what ran before is complete
  const long long m = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + m * a.ldx;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + m * a.ldr : nullptr;
  const unsigned width = a.D;  // 1024 beyond it an int would pass 2^31
  auto at = [&](unsigned d) { return to_f32(x[d]) + (res ? to_f32(res[d]) : 0.f); };
  float sq = 0.f;
  uint32_t big = 0;
  for (unsigned d = threadIdx.x; d < width; d += 1024) {
    const float s = at(d), p = a.w ? s * a.w[d] : s;
    sq = fmaf(s, s, sq);
    big = max(big, __float_as_uint(fabsf(p)));
  }
  sq = warp_sum(sq);
  big = __reduce_max_sync(0xffffffffu, big);
  if (lane == 0) {
    squares[warp] = sq;
    bits[warp] = big;
  }
  if (threadIdx.x == 0) largest = 0;
  __syncthreads();
  sq = 0.f;
  for (int w = 0; w < 32; ++w) {
    sq += squares[w];
    big = max(big, bits[w]);
  }
  if (a.q && big < 0x7f800000u) {
    for (unsigned d = threadIdx.x; d < width; d += 1024) {
      const float z = at(d), p = a.w ? z * a.w[d] : z;
      if (fabsf(p) >= next_to(big)) take_larger(&largest, exact_product<T>(a, m, d));
    }
  }
  __syncthreads();
  const Row o = row_of(a, sq, big);
  const double exact = __longlong_as_double((long long)largest);
  if (a.q && threadIdx.x == 0) a.scale[m] = o.scale;
  for (unsigned d = threadIdx.x; d < width; d += 1024) {
    const float z = at(d), w = a.w ? a.w[d] : 1.f;
    if (a.q) a.q[m * a.ldq + d] = (int8_t)quantized<T>(a, o, exact, z * w, m, d);
    if (a.y) static_cast<T*>(a.y)[m * a.ldy + d] = from_f32<T>(z * o.r * w);
    if (a.sum) static_cast<T*>(a.sum)[m * a.lds + d] = from_f32<T>(z);  // last: it may be an input
  }
}

template <typename T, int kThreads, int kVecs, bool kWide, bool kI8>
cudaError_t launch_form(const NormArgs& a, int sms, cudaStream_t s) {
  using N = Norm<T, kThreads, kI8>;
  const long long blocks = (a.M + (long long)N::kRows - 1) / N::kRows, most = (long long)sms * N::kPerSm;
  return launch_early(norm_kernel<T, kThreads, kVecs, kWide, kI8>, dim3((unsigned)(blocks < most ? blocks : most)),
                      N::kCta, 0, 1, s, a);
}
template <typename T, int kThreads, int kVecs>
cudaError_t launch_of(const NormArgs& a, bool wide, int sms, cudaStream_t s) {
  if (a.q)
    return wide ? launch_form<T, kThreads, kVecs, true, true>(a, sms, s)
                : launch_form<T, kThreads, kVecs, false, true>(a, sms, s);
  return wide ? launch_form<T, kThreads, kVecs, true, false>(a, sms, s)
              : launch_form<T, kThreads, kVecs, false, false>(a, sms, s);
}

template <typename T>
cudaError_t launch_t(const NormArgs& a, int sms, cudaStream_t s) {
  auto on16 = [](const void* p, long long ld, size_t e, size_t to) {
    return !p || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * (long long)e)) & (to - 1)) == 0;
  };
  const bool wide = a.D % 8 == 0 && on16(a.x, a.ldx, sizeof(T), 16) && on16(a.residual, a.ldr, sizeof(T), 16) &&
                    on16(a.sum, a.lds, sizeof(T), 16) && on16(a.y, a.ldy, sizeof(T), 16) && on16(a.w, 0, 4, 16) &&
                    on16(a.q, a.ldq, 1, 8);
  // Eight elements per thread where there are few rows, for the latency, sixteen where rows fill the
  // GPU; a warp at least.  (Eight for one row of 512 to 2048 elements would take 2.1 us and not 2.75, for 64 rows
  // the same as sixteen; for one of 8192 3.5 and not 2.8.)
  if (a.D <= 256) return launch_of<T, 32, 1>(a, wide, sms, s);
  if (a.D <= 512) return launch_of<T, 32, 2>(a, wide, sms, s);
  if (a.D <= 1024) return launch_of<T, 64, 2>(a, wide, sms, s);
  if (a.D <= 2048) return launch_of<T, 128, 2>(a, wide, sms, s);
  if (a.D <= 4096) return a.M < 4 * sms ? launch_of<T, 512, 1>(a, wide, sms, s) : launch_of<T, 256, 2>(a, wide, sms, s);
  if (a.D <= 8192) return launch_of<T, 512, 2>(a, wide, sms, s);
  if (a.D <= 16384) return launch_of<T, 1024, 2>(a, wide, sms, s);
  return launch_early(norm_any_kernel<T>, dim3(a.M), 1024, 0, 1, s, a);
}

}  // namespace
}  // namespace kda
