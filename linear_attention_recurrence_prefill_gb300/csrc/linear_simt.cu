// linear_simt.cu -- y = act(x w^T + bias) + residual on the CUDA cores: fp32 data, and bf16 data
// without columns (K = 0).
//
// A CTA of 128 threads per 64 x 64 tile of y, 8 x 4 sums per thread as pairs of rows
// (fma.rn.f32x2): three 16-byte reads of shared memory for 32 products.  x and w pass through shared memory 16 columns at
// a time, the next ones fetched into registers meanwhile.  Where there are too few tiles to give
// every SM two CTAs, the CTAs of a cluster share a tile, each takes a part of K, and the sums meet
// in distributed shared memory, added in the order of the ranks.  1024^3 takes 70 us
// (31 TFLOP/s, under half of the CUDA cores' rate: 256 tiles are 1.7 waves of 152 SMs, with two warps
// per scheduler and one step fetched ahead); small products are bound by latency (200 x 512 x 640:
// 10.5 us).
#include "linear.cuh"
#include "umma.cuh"

namespace kda {
namespace {

using umma::cluster_ctarank;
using umma::cluster_sync;
using umma::ld_cluster_f32;
using umma::map_to_rank;
using umma::smem_u32;

constexpr int kTile = 64, kStep = 16, kThreads = 128, kPitch = kTile + 4;
typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 both(float x) {
  const uint32_t b = __float_as_uint(x);
  return ((f32x2)b << 32) | b;
}

// kVec: fp32 rows of x and w that 16-byte loads can fetch (K, too, a multiple of four).
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) linear_simt_kernel(LinearArgs a) {
  // the tiles, [column][row]; then the partial sums [row of y][column]
  __shared__ __align__(16) union {
    struct {
      float x[2][kStep][kPitch], w[2][kStep][kPitch];
    };
    float part[kTile][kTile];
  } s;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const uint32_t rank = cluster_ctarank(), ranks = gridDim.z;
  const long long n0 = (long long)blockIdx.x * kTile, m0 = (long long)blockIdx.y * kTile;
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);
  const int steps = (a.K + kStep - 1) / kStep;
  const int s0 = (int)((long long)steps * rank / ranks), s1 = (int)((long long)steps * (rank + 1) / ranks);

  // a thread fetches column c of rows r, r + 8, ..., or columns c .. c + 3 of rows r and r + 32
  constexpr int kFetch = 8, kApart = kVec ? 32 : 8, kWide = kVec ? 4 : 1;
  const int c = kVec ? (tid & 3) * 4 : tid & 15, r = kVec ? tid >> 2 : tid >> 4;
  float fx[kFetch], fw[kFetch];
  auto fetch = [&](int step) {
    const int k = step * kStep + c;
#pragma unroll
    for (int i = 0; i < kFetch / kWide; ++i) {
      const long long m = m0 + r + i * kApart, n = n0 + r + i * kApart;
      const bool mi = k < a.K && m < a.M, ni = k < a.K && n < a.N;
      if constexpr (kVec) {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(&fx[4 * i]) = mi ? *reinterpret_cast<const float4*>(&x[m * a.ldx + k]) : zero;
        *reinterpret_cast<float4*>(&fw[4 * i]) = ni ? *reinterpret_cast<const float4*>(&w[n * a.ldw + k]) : zero;
      } else {
        fx[i] = mi ? to_f32(x[m * a.ldx + k]) : 0.f;
        fw[i] = ni ? to_f32(w[n * a.ldw + k]) : 0.f;
      }
    }
  };
  auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < kFetch / kWide; ++i)
#pragma unroll
      for (int j = 0; j < kWide; ++j) {
        s.x[b][c + j][r + i * kApart] = fx[i * kWide + j];
        s.w[b][c + j][r + i * kApart] = fw[i * kWide + j];
      }
  };
  f32x2 acc[4][4] = {};  // rows ty * 8 + 2 i, + 1, column tx * 4 + j
  if (s0 < s1) {
    fetch(s0);
    put(0);
  }
  __syncthreads();
  for (int step = s0; step < s1; ++step) {
    const int b = (step - s0) & 1;
    if (step + 1 < s1) fetch(step + 1);
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      const ulonglong2 x0 = *reinterpret_cast<const ulonglong2*>(&s.x[b][k][ty * 8]);
      const ulonglong2 x1 = *reinterpret_cast<const ulonglong2*>(&s.x[b][k][ty * 8 + 4]);
      const float4 w4 = *reinterpret_cast<const float4*>(&s.w[b][k][tx * 4]);
      const f32x2 xs[4] = {x0.x, x0.y, x1.x, x1.y}, ws[4] = {both(w4.x), both(w4.y), both(w4.z), both(w4.w)};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i][j]) : "l"(xs[i]), "l"(ws[j]));
    }
    if (step + 1 < s1) put(b ^ 1);
    __syncthreads();
  }
  auto sum = [&](int i, int j) { return __uint_as_float((uint32_t)(acc[i >> 1][j] >> (32 * (i & 1)))); };
  const T* bias = static_cast<const T*>(a.bias);
  auto out = [&](float z, int row, int col) {
    const long long m = m0 + row, n = n0 + col;
    if (m < a.M && n < a.N) finish<T>(a, z, bias ? to_f32(bias[n]) : 0.f, m, (int)n);
  };
  if (ranks == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        out(sum(i, j), ty * 8 + i, tx * 4 + j);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<float4*>(&s.part[ty * 8 + i][tx * 4]) = make_float4(sum(i, 0), sum(i, 1), sum(i, 2), sum(i, 3));
  cluster_sync();
  uint32_t from[8];
#pragma unroll
  for (uint32_t q = 0; q < 8; ++q) from[q] = map_to_rank(smem_u32(&s.part[0][0]), q < ranks ? q : 0);
  // rank q finishes rows q, q + ranks, ..
  for (int i = tid; i < kTile / (int)ranks * kTile; i += kThreads) {
    const int row = i / kTile * (int)ranks + (int)rank, col = i % kTile;
    float v[8];
#pragma unroll
    for (uint32_t q = 0; q < 8; ++q) v[q] = q < ranks ? ld_cluster_f32(from[q] + (row * kTile + col) * 4) : 0.f;
    float z = v[0];
#pragma unroll
    for (uint32_t q = 1; q < 8; ++q) z += v[q];
    out(z, row, col);
  }
  cluster_sync();  // no CTA leaves while its sums are read
}

template <typename T>
cudaError_t launch_t(const LinearArgs& a, int sms, cudaStream_t s) {
  // gridDim.y holds 65,535 tiles of rows: more rows go in several launches
  constexpr int kRows = 65535 * kTile;
  for (long long m = 0; m < a.M; m += kRows) {
    LinearArgs b = a;
    b.x = static_cast<const T*>(a.x) + m * a.ldx;
    if (a.residual) b.residual = static_cast<const T*>(a.residual) + m * a.ldr;
    b.y = static_cast<T*>(a.y) + m * a.ldy;
    b.M = a.M - m < kRows ? (int)(a.M - m) : kRows;
    const long long nt = (b.N + kTile - 1LL) / kTile, mt = (b.M + kTile - 1LL) / kTile;
    const int steps = (b.K + kStep - 1) / kStep;
    int split = 1;
    while (split < 8 && split * 8 <= steps && nt * mt * split * 2 <= 4LL * sms) split *= 2;
    // an ordinary launch: behind each other, started early, 200 x 512 x 640 took 13.1 us, not 9.7
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nt, (unsigned)mt, split);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = split;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if constexpr (sizeof(T) == 4) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(b.x) | reinterpret_cast<uintptr_t>(b.w);
      const bool vec = (at & 15) == 0 && b.ldx % 4 == 0 && b.ldw % 4 == 0 && b.K % 4 == 0;
      e = cudaLaunchKernelEx(&cfg, vec ? linear_simt_kernel<T, true> : linear_simt_kernel<T, false>, b);
    } else {
      e = cudaLaunchKernelEx(&cfg, linear_simt_kernel<T, false>, b);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_linear_simt(const LinearArgs& a, int dtype, int sms, cudaStream_t s) {
  return dtype == KDA_BF16 ? launch_t<__nv_bfloat16>(a, sms, s) : launch_t<float>(a, sms, s);
}

}  // namespace kda
