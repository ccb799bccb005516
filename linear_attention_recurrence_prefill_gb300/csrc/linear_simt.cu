// linear_simt.cu -- y = act(x w^T + bias) + residual on the CUDA cores: fp32
// data, and bf16 data whose rows the tensor-core path cannot fetch (addresses
// or strides that are not multiples of 16 bytes).
//
// One CTA of 256 threads per 64 x 64 tile of y, 4 x 4 sums per thread, x and w
// taken through shared memory 16 columns at a time.  Every sum runs over k in
// ascending order in fp32.
#include "linear.cuh"

namespace kda {
namespace {

constexpr int kTile = 64, kStep = 16;

template <typename T>
__global__ void __launch_bounds__(256) linear_simt_kernel(LinearArgs a) {
  __shared__ float sx[kStep][kTile + 4], sw[kStep][kTile + 4];
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int n0 = blockIdx.x * kTile;
  const long long m0 = (long long)blockIdx.y * kTile;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kStep) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (tid >> 4) + 16 * i, c = tid & 15;
      const bool kin = k0 + c < a.K;
      sx[c][r] = kin && m0 + r < a.M ? to_f32(x[(m0 + r) * a.ldx + k0 + c]) : 0.f;
      sw[c][r] = kin && n0 + r < a.N ? to_f32(w[(long long)(n0 + r) * a.ldw + k0 + c]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kStep; ++c) {
      const float4 xa = *reinterpret_cast<const float4*>(&sx[c][ty * 4]);
      const float4 wb = *reinterpret_cast<const float4*>(&sw[c][tx * 4]);
      const float xs[4] = {xa.x, xa.y, xa.z, xa.w}, ws[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ws[j], acc[i][j]);
    }
    __syncthreads();
  }
  const T* bias = static_cast<const T*>(a.bias);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long m = m0 + ty * 4 + i;
    if (m >= a.M) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= a.N) break;
      finish<T>(a, acc[i][j], bias ? to_f32(bias[n]) : 0.f, m, n);
    }
  }
}

template <typename T>
cudaError_t launch_t(const LinearArgs& a, cudaStream_t s) {
  // gridDim.y holds 65,535 tiles of rows: more rows go in several launches
  constexpr int kRows = 65535 * kTile;
  for (long long m = 0; m < a.M; m += kRows) {
    LinearArgs b = a;
    b.x = static_cast<const T*>(a.x) + m * a.ldx;
    if (a.residual) b.residual = static_cast<const T*>(a.residual) + m * a.ldr;
    b.y = static_cast<T*>(a.y) + m * a.ldy;
    b.M = a.M - m < kRows ? (int)(a.M - m) : kRows;
    const dim3 grid((a.N + kTile - 1) / kTile, (b.M + kTile - 1) / kTile);
    linear_simt_kernel<T><<<grid, 256, 0, s>>>(b);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_linear_simt(const LinearArgs& a, int dtype, cudaStream_t s) {
  return dtype == KDA_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace kda
