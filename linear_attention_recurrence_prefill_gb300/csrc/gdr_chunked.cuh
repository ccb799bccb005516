// gdr_chunked.cuh -- the chunked gated delta rule: the workspace between its kernels, and the
// bf16 parts that fp32 operands are split into.
#pragma once

#include "gdr.cuh"
#include "umma.cuh"

namespace kda {

constexpr int kC = 64;                 // tokens per chunk
constexpr long long kGdrSpins = 4000000000LL;  // ~2 s of clock cycles

// One (chunk, value head) of the workspace: the bf16 parts of T and P as tiles [row][64] of
// 128-byte rows whose 16-byte groups are XORed with the row's low three bits, then vectors.  The
// 16 x 16 blocks above the diagonal ones are neither written nor read.
constexpr uint32_t kTile = kC * kC * 2;
constexpr uint32_t kT = 0, kP = 3 * kTile;  // T: three parts, P: two
constexpr uint32_t kVec = 5 * kTile;        // floats: a[64], b[64], ku[64], e^{g_C}
constexpr uint32_t kBlock = kVec + 1024;

__host__ __device__ constexpr uint32_t tile_at(uint32_t row, uint32_t col) {
  return row * 128u + ((((col >> 3) ^ row) & 7u) << 4) + (col & 7u) * 2u;
}

// Chunk c of sequence n has block (t0 / 64 + n) + c: floor((t0 + len) / 64) + 1 is at
// least floor(t0 / 64) + ceil(len / 64), so that sequences never share a block, and no
// prefix sum over the sequences is needed.
__host__ __device__ constexpr int block_base(int t0, int n) { return t0 / kC + n; }

// x, y as sums of bf16 parts, packed
__device__ __forceinline__ uint32_t part(float& x, float& y) {  // takes the next part off
  const uint32_t p = umma::pack_bf162(x, y);
  x -= __uint_as_float(p << 16);
  y -= __uint_as_float(p & 0xffff0000u);
  return p;
}
template <int kParts>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[kParts]) {
#pragma unroll
  for (int i = 0; i < kParts - 1; ++i) p[i] = part(x, y);
  p[kParts - 1] = umma::pack_bf162(x, y);
}

// The same for three parts, by cutting instead of rounding: 8 + 8 + 8 bits hold all of fp32's 24,
// so the sum of the parts is exact.
__device__ __forceinline__ unsigned long long f2(float x, float y) {
  return ((unsigned long long)__float_as_uint(y) << 32) | __float_as_uint(x);
}
__device__ __forceinline__ void split3(float x, float y, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  const unsigned long long kMinus = f2(-1.f, -1.f);
  const uint32_t m = 0xffff0000u;
  uint32_t xi = __float_as_uint(x), yi = __float_as_uint(y);
  unsigned long long r = f2(x, y), h;
  p0 = __byte_perm(xi, yi, 0x7632);
  h = ((unsigned long long)(yi & m) << 32) | (xi & m);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(r) : "l"(h), "l"(kMinus));
  xi = (uint32_t)r; yi = (uint32_t)(r >> 32);
  p1 = __byte_perm(xi, yi, 0x7632);
  h = ((unsigned long long)(yi & m) << 32) | (xi & m);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(r) : "l"(h), "l"(kMinus));
  p2 = __byte_perm((uint32_t)r, (uint32_t)(r >> 32), 0x7632);
}

// The sequence that the walk takes as its `place`-th: the longest first (ties by index), so that the
// grid's last CTAs have little to do; up to 32 sequences, in their own order beyond.  By a whole warp.
__device__ __forceinline__ int longest_first(const GdrArgs& a, int place) {
  if (!a.cu_seqlens || a.N == 1 || a.N > 32) return place;
  const int lane = threadIdx.x & 31;
  const int len = lane < a.N ? a.cu_seqlens[lane + 1] - a.cu_seqlens[lane] : 0;
  int before = 0;
  for (int i = 0; i < a.N; ++i) {
    const int other = __shfl_sync(0xffffffffu, len, i);
    before += other > len || (other == len && i < lane);
  }
  return __ffs(__ballot_sync(0xffffffffu, lane < a.N && before == place)) - 1;
}

// The walk over the chunks on tcgen05: d_k in {64, 128}, d_v a multiple of 128.
bool gdr_chain_tc_takes(const GdrArgs& a);
cudaError_t launch_gdr_chain_tc(const GdrArgs& a, const uint8_t* ws, cudaStream_t s);

}  // namespace kda
