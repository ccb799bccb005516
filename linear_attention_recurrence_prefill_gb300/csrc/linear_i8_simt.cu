// linear_i8_simt.cu -- the 8-bit product on the CUDA cores, any size, stride and
// alignment: four products per instruction, sums in 32-bit integers.
#include "linear_i8.cuh"
#include "umma.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8, kRowsM = 4;

// Four bytes at p, of which `n` exist.
__device__ __forceinline__ int bytes4(const int8_t* p, int n) {
  if (n >= 4 && (reinterpret_cast<uintptr_t>(p) & 3) == 0) return *reinterpret_cast<const int*>(p);
  uint32_t v = 0;
  for (int i = 0; i < 4 && i < n; ++i) v |= (uint32_t)(uint8_t)p[i] << (8 * i);
  return (int)v;
}

// A warp per channel and four tokens.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) linear_i8_simt_kernel(LinearI8Args a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  umma::grid_launch_dependents();
  umma::grid_wait_prerequisites();  // what ran before is complete
  const LinearArgs& l = a.l;
  const long long blocks = (l.N + kWarps - 1LL) / kWarps;
  const long long n = blockIdx.x % blocks * kWarps + warp, m0 = blockIdx.x / blocks * kRowsM;
  if (n >= l.N) return;
  const int8_t* w = static_cast<const int8_t*>(l.w) + n * l.ldw;
  const int8_t* x = static_cast<const int8_t*>(l.x);
  long long sum[kRowsM] = {};
  for (long long k0 = 0; k0 < l.K; k0 += 65536) {  // parts whose sums fit in 32 bits
    const int end = l.K - k0 < 65536 ? (int)(l.K - k0) : 65536;
    int part[kRowsM] = {};
    for (int k = lane * 4; k < end; k += 128) {
      const int wv = bytes4(w + k0 + k, end - k);
#pragma unroll
      for (int i = 0; i < kRowsM; ++i)
        if (m0 + i < l.M) part[i] = __dp4a(wv, bytes4(x + (m0 + i) * l.ldx + k0 + k, end - k), part[i]);
    }
#pragma unroll
    for (int i = 0; i < kRowsM; ++i) sum[i] += __reduce_add_sync(0xffffffffu, part[i]);
  }
  if (lane < kRowsM && m0 + lane < l.M) {
    const long long m = m0 + lane;
    const long long z = lane == 0 ? sum[0] : lane == 1 ? sum[1] : lane == 2 ? sum[2] : sum[3];
    const float b = l.bias ? to_f32(static_cast<const T*>(l.bias)[n]) : 0.f;
    finish<T>(l, (float)z * a.x_scale[m] * a.w_scale[n], b, m, (int)n);
  }
}

}  // namespace

cudaError_t launch_linear_i8_simt(const LinearI8Args& a, int dtype, int sms, cudaStream_t s) {
  (void)sms;
  const long long blocks = (a.l.N + kWarps - 1LL) / kWarps * ((a.l.M + kRowsM - 1LL) / kRowsM);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (dtype == KDA_BF16)
    return launch_early(linear_i8_simt_kernel<__nv_bfloat16>, dim3((unsigned)blocks), kWarps * 32, 0, 1, s, a);
  return launch_early(linear_i8_simt_kernel<float>, dim3((unsigned)blocks), kWarps * 32, 0, 1, s, a);
}

}  // namespace kda
