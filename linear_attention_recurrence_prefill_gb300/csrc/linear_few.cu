// linear_few.cu -- y = act(x w^T + bias) + residual for up to two rows of x in bf16, four in fp32
// (the next token of a few sequences), where reading w is all the time there is: fp32 sums on the
// CUDA cores, w streamed in 16-byte loads.
//
// A warp takes kRows neighbouring rows of w; a lane its vectors of 16 bytes, kUnroll of them per
// row in flight (4 KB per warp).  Where w has too few rows to give every SM 16 warps, the warps of
// a CTA share rows, each takes a part of K, and their sums meet in shared memory, added in the
// order of the warps.  x comes from L1.  One row with 4096 x 4096 weights takes 8.3 us (4.0 TB/s, of
// which some 3 us are the launch and the first loads' latency), with 4096 x 12288 19.6 us (5.1 TB/s).
#include "linear.cuh"
#include "umma.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8, kRows = 2, kUnroll = 4, kMaxM = 4;

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
template <typename T>
__device__ __forceinline__ void widen(const uint4& v, float (&x)[16 / sizeof(T)]) {
  const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(e[i]);
    } else {
      x[2 * i] = __uint_as_float(e[i] << 16);
      x[2 * i + 1] = __uint_as_float(e[i] & 0xffff0000u);
    }
  }
}

// `parts` warps share a group of kRows rows (1, 2, 4 or 8).
template <int M, typename T>
__global__ void __launch_bounds__(kWarps * 32) linear_few_kernel(LinearArgs a, int parts) {
  constexpr int V = 16 / sizeof(T);
  __shared__ float sums[kWarps][kRows * M];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % parts;
  umma::grid_launch_dependents();
  umma::grid_wait_prerequisites();  // what ran before is complete
  const long long n0 = ((long long)blockIdx.x * (kWarps / parts) + warp / parts) * kRows;
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);
  float acc[kRows][M] = {};
  // vectors [v0, v1) of this warp, then the K % V elements behind the last vector
  const int vectors = a.K / V;
  const int v0 = (int)((long long)vectors * part / parts), v1 = (int)((long long)vectors * (part + 1) / parts);
  const T* row[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) row[r] = w + (n0 + r < a.N ? n0 + r : a.N - 1) * a.ldw;

  auto add = [&](const uint4 (&q)[kRows], int v) {
    float wf[kRows][V];
#pragma unroll
    for (int r = 0; r < kRows; ++r) widen<T>(q[r], wf[r]);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float xf[V];
      widen<T>(*reinterpret_cast<const uint4*>(x + m * a.ldx + (long long)v * V), xf);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[r][m] = fmaf(wf[r][i], xf[i], acc[r][m]);
    }
  };
  int v = v0 + lane;
  for (; v + (kUnroll - 1) * 32 < v1; v += kUnroll * 32) {
    uint4 q[kUnroll][kRows];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int r = 0; r < kRows; ++r) q[u][r] = load_once(row[r] + (long long)(v + u * 32) * V);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) add(q[u], v + u * 32);
  }
  for (; v < v1; v += 32) {
    uint4 q[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) q[r] = load_once(row[r] + (long long)v * V);
    add(q, v);
  }
  if (part == parts - 1 && vectors * V + lane < a.K) {
    const int k = vectors * V + lane;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int m = 0; m < M; ++m) acc[r][m] = fmaf(to_f32(row[r][k]), to_f32(x[m * a.ldx + k]), acc[r][m]);
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      acc[r][m] = warp_sum(acc[r][m]);
      if (lane == 0) sums[warp][r * M + m] = acc[r][m];
    }
  __syncthreads();
  if (part == 0 && lane < kRows * M) {
    const int r = lane / M, m = lane % M;
    const long long n = n0 + r;
    if (n < a.N) {
      float z = 0.f;
      for (int p = 0; p < parts; ++p) z += sums[warp + p][lane];
      finish<T>(a, z, a.bias ? to_f32(static_cast<const T*>(a.bias)[n]) : 0.f, m, (int)n);
    }
  }
}

template <int M, typename T>
cudaError_t launch_m(const LinearArgs& a, int sms, cudaStream_t s) {
  const long long groups = ((long long)a.N + kRows - 1) / kRows;
  int parts = 1;
  while (parts < kWarps && groups * parts < 16LL * sms) parts *= 2;
  const long long blocks = (groups + kWarps / parts - 1) / (kWarps / parts);
  return launch_early(linear_few_kernel<M, T>, dim3((unsigned)blocks), kWarps * 32, 0, 1, s, a, parts);
}

template <typename T>
cudaError_t launch_t(const LinearArgs& a, int sms, cudaStream_t s) {
  switch (a.M) {
    case 1: return launch_m<1, T>(a, sms, s);
    case 2: return launch_m<2, T>(a, sms, s);
  }
  if constexpr (sizeof(T) == 4) return a.M == 3 ? launch_m<3, T>(a, sms, s) : launch_m<4, T>(a, sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace

bool linear_few_takes(const LinearArgs& a, int dtype) {
  // bf16 rows from the third on are cheaper on the tensor cores: 4096 x 4096 weights took 8.5, 8.6,
  // 9.4, 10.9 us for 1 to 4 rows here, 8.9, 8.9, 8.9, 9.4 us there
  if (a.M > (dtype == KDA_BF16 ? 2 : kMaxM) || a.K < 1) return false;
  const int v = dtype == KDA_BF16 ? 8 : 4;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w);
  return (at & 15) == 0 && (a.ldx % v == 0 || a.M == 1) && (a.ldw % v == 0 || a.N == 1);
}

cudaError_t launch_linear_few(const LinearArgs& a, int dtype, int sms, cudaStream_t s) {
  return dtype == KDA_BF16 ? launch_t<__nv_bfloat16>(a, sms, s) : launch_t<float>(a, sms, s);
}

}  // namespace kda
