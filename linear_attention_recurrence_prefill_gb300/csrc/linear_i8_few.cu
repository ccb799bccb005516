// linear_i8_few.cu -- the 8-bit product for up to eight rows of x (the next token of a few
// sequences), where reading w is all the time there is: sums in 32-bit integers on the CUDA
// cores, four products per instruction, w streamed in 16-byte loads.
//
// A warp takes kRows neighbouring rows of w; a lane its vectors of 16 bytes, kUnroll of them per
// row in flight (4 KB per warp).  Where w has too few rows to give every SM 16 warps, the warps of
// a CTA share rows, each takes a part of K, and their sums meet in shared memory.  x comes from L1.
#include "linear_i8.cuh"
#include "umma.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8, kRows = 2, kUnroll = 4, kMaxM = 8;

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// `parts` warps share a group of kRows rows (1, 2, 4 or 8).
template <int M, typename T>
__global__ void __launch_bounds__(kWarps * 32) linear_i8_few_kernel(LinearI8Args a, int parts) {
  __shared__ int sums[kWarps][kRows * M];
  const LinearArgs& l = a.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % parts;
  umma::grid_launch_dependents();
  umma::grid_wait_prerequisites();  // what ran before is complete
  const long long n0 = ((long long)blockIdx.x * (kWarps / parts) + warp / parts) * kRows;
  const int8_t* x = static_cast<const int8_t*>(l.x);
  const int8_t* w = static_cast<const int8_t*>(l.w);
  int acc[kRows][M] = {};
  // vectors [v0, v1) of this warp, then the K % 16 integers behind the last vector
  const int vectors = l.K / 16;
  const int v0 = (int)((long long)vectors * part / parts), v1 = (int)((long long)vectors * (part + 1) / parts);
  const int8_t* row[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) row[r] = w + (n0 + r < l.N ? n0 + r : l.N - 1) * l.ldw;

  auto add = [&](const uint4 (&q)[kRows], int v) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const uint4 xv = __ldg(reinterpret_cast<const uint4*>(x + m * l.ldx + (long long)v * 16));
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        acc[r][m] = __dp4a((int)q[r].x, (int)xv.x, acc[r][m]);
        acc[r][m] = __dp4a((int)q[r].y, (int)xv.y, acc[r][m]);
        acc[r][m] = __dp4a((int)q[r].z, (int)xv.z, acc[r][m]);
        acc[r][m] = __dp4a((int)q[r].w, (int)xv.w, acc[r][m]);
      }
    }
  };
  int v = v0 + lane;
  for (; v + (kUnroll - 1) * 32 < v1; v += kUnroll * 32) {
    uint4 q[kUnroll][kRows];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int r = 0; r < kRows; ++r) q[u][r] = load_once(row[r] + (long long)(v + u * 32) * 16);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) add(q[u], v + u * 32);
  }
  for (; v < v1; v += 32) {
    uint4 q[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) q[r] = load_once(row[r] + (long long)v * 16);
    add(q, v);
  }
  if (part == parts - 1 && vectors * 16 + lane < l.K) {
    const int k = vectors * 16 + lane;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int m = 0; m < M; ++m) acc[r][m] += (int)row[r][k] * (int)x[m * l.ldx + k];
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int z = __reduce_add_sync(0xffffffffu, acc[r][m]);
      if (lane == 0) sums[warp][r * M + m] = z;
    }
  __syncthreads();
  if (part == 0 && lane < kRows * M) {
    const int r = lane / M, m = lane % M;
    const long long n = n0 + r;
    if (n < l.N) {
      int z = 0;
      for (int p = 0; p < parts; ++p) z += sums[warp + p][lane];
      const float bias = l.bias ? to_f32(static_cast<const T*>(l.bias)[n]) : 0.f;
      finish<T>(l, scaled((float)z, a.x_scale[m], a.w_scale[n], bias), 0.f, m, (int)n);
    }
  }
}

template <int M, typename T>
cudaError_t launch_m(const LinearI8Args& a, int sms, cudaStream_t s) {
  const long long groups = ((long long)a.l.N + kRows - 1) / kRows;
  int parts = 1;
  while (parts < kWarps && groups * parts < 16LL * sms) parts *= 2;
  const long long blocks = (groups + kWarps / parts - 1) / (kWarps / parts);
  return launch_early(linear_i8_few_kernel<M, T>, dim3((unsigned)blocks), kWarps * 32, 0, 1, s, a, parts);
}
template <typename T>
cudaError_t launch_t(const LinearI8Args& a, int sms, cudaStream_t s) {
  switch (a.l.M) {
    case 1: return launch_m<1, T>(a, sms, s);
    case 2: return launch_m<2, T>(a, sms, s);
    case 3: return launch_m<3, T>(a, sms, s);
    case 4: return launch_m<4, T>(a, sms, s);
    case 5: return launch_m<5, T>(a, sms, s);
    case 6: return launch_m<6, T>(a, sms, s);
    case 7: return launch_m<7, T>(a, sms, s);
    default: return launch_m<8, T>(a, sms, s);
  }
}

}  // namespace

bool linear_i8_few_takes(const LinearI8Args& a) {
  const LinearArgs& l = a.l;
  // sums of up to 131,071 products fit in 32 bits
  if (l.M > kMaxM || l.K < 1 || l.K > 131071) return false;
  const uintptr_t at = reinterpret_cast<uintptr_t>(l.x) | reinterpret_cast<uintptr_t>(l.w);
  return (at & 15) == 0 && (l.ldx % 16 == 0 || l.M == 1) && (l.ldw % 16 == 0 || l.N == 1);
}

cudaError_t launch_linear_i8_few(const LinearI8Args& a, int dtype, int sms, cudaStream_t s) {
  return dtype == KDA_BF16 ? launch_t<__nv_bfloat16>(a, sms, s) : launch_t<float>(a, sms, s);
}

}  // namespace kda
