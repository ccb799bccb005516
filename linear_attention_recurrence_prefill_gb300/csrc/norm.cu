// norm.cu -- the root-mean-square norm with the residual's addition, in the data
// type or in 8 bits with a scale per token.
//
//     s = x + residual,  n = s r w with r = 1 / sqrt(mean s^2 + eps)
//     scale = max |n| / 127,  q = n / scale = 127 p / max |p| with p = s w
//
// q does not depend on r, so the squares' sum and the largest |p| are found in one
// reduction over the row, which stays in registers between that and the outputs: each
// array is read once and written once, and HBM is the bound.  q is the integer nearest to
// the quotient without rounding errors: the fp32 quotient is off by at most four
// roundings, 127 * 4 * 2^-24 = 3.1e-5, so only those within 4e-5 of the middle between two
// integers (one in 12,000) are taken again in 64 bits, from the stored inputs.
#include "norm.cuh"
#include "umma.cuh"

namespace kda {
namespace {

constexpr float kMiddle = 4e-5f;

template <typename T>
__device__ __forceinline__ double exact_product(const NormArgs& a, long long m, int d) {
  double s = (double)to_f32(static_cast<const T*>(a.x)[m * a.ldx + d]);
  if (a.residual) s += (double)to_f32(static_cast<const T*>(a.residual)[m * a.ldr + d]);
  return a.w ? s * (double)a.w[d] : s;
}
// The nearest integer to p inv, inv = 127 / largest.
template <typename T>
__device__ __forceinline__ int quantized(const NormArgs& a, float p, float inv, double largest, bool all, long long m,
                                         int d) {
  const float v = p * inv, k = rintf(v);
  if (all || fabsf(fabsf(v - k) - 0.5f) < kMiddle) return (int)rint(127. * exact_product<T>(a, m, d) / largest);
  return (int)k;
}

// What a row's threads know after the reductions.
struct Row {
  float r, scale, inv;
  double largest;
  bool all;  // every quotient in 64 bits: the largest product is so small that 127 / it may overflow
};
__device__ __forceinline__ Row row_of(const NormArgs& a, float squares, uint32_t largest_bits, double largest) {
  Row o;
  const float v = squares / (float)a.D + a.eps;
  o.r = !a.norm ? 1.f : v > 0.f ? 1.f / sqrtf(v) : v;  // 0 for a row of zeros with eps = 0; NaN stays
  o.largest = largest;
  const float big = __uint_as_float(largest_bits);
  const bool finite = largest_bits < 0x7f800000u;
  o.scale = finite ? (float)(largest * (double)o.r / 127.) : big * o.r;
  o.inv = finite && big > 0.f ? 127.f / big : 0.f;
  o.all = finite && big > 0.f && big < 0x1p-100f;
  return o;
}

// Any row length and alignment: a CTA per row, which reads it once per step.
template <typename T>
__global__ void __launch_bounds__(1024) norm_any_kernel(NormArgs a) {
  __shared__ float squares[32];
  __shared__ uint32_t bits[32];
  __shared__ unsigned long long largest;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  umma::grid_launch_dependents();
  umma::grid_wait_prerequisites();  // what ran before is complete
  const long long m = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + m * a.ldx;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + m * a.ldr : nullptr;
  auto at = [&](int d) { return to_f32(x[d]) + (res ? to_f32(res[d]) : 0.f); };
  float sq = 0.f;
  uint32_t big = 0;
  for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
    const float s = at(d), p = a.w ? s * a.w[d] : s;
    sq = fmaf(s, s, sq);
    big = max(big, __float_as_uint(fabsf(p)));  // NaN above infinity above all else
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
  for (int w = 0; w < warps; ++w) {
    sq += squares[w];
    big = max(big, bits[w]);
  }
  if (a.q && big < 0x7f800000u) {  // the largest product in 64 bits, among those next to it
    const float near = __uint_as_float(big) * (1.f - 0x1p-21f);
    for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
      const float s = at(d), p = a.w ? s * a.w[d] : s;
      if (fabsf(p) >= near) atomicMax(&largest, (unsigned long long)__double_as_longlong(fabs(exact_product<T>(a, m, d))));
    }
  }
  __syncthreads();
  const Row o = row_of(a, sq, big, __longlong_as_double((long long)largest));
  if (a.q && threadIdx.x == 0) a.scale[m] = o.scale;
  for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
    const float s = at(d), w = a.w ? a.w[d] : 1.f;
    if (a.q) a.q[m * a.ldq + d] = (int8_t)(o.inv > 0.f ? quantized<T>(a, s * w, o.inv, o.largest, o.all, m, d) : 0);
    if (a.y) static_cast<T*>(a.y)[m * a.ldy + d] = from_f32<T>(s * o.r * w);
    if (a.sum) static_cast<T*>(a.sum)[m * a.lds + d] = from_f32<T>(s);  // last: it may be an input
  }
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int sms, cudaStream_t s) {
  (void)sms;
  int threads = 32;
  while (threads < 1024 && threads * 8 < a.D) threads *= 2;
  if (dtype == KDA_BF16) return launch_early(norm_any_kernel<__nv_bfloat16>, dim3(a.M), threads, 0, 1, s, a);
  return launch_early(norm_any_kernel<float>, dim3(a.M), threads, 0, 1, s, a);
}

}  // namespace kda
