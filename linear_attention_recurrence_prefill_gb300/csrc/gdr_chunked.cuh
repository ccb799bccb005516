// gdr_chunked.cuh -- the chunked gated delta rule: the workspace between its kernels, and the
// bf16 parts that fp32 operands are split into.
#pragma once

#include "gdr.cuh"
#include "umma.cuh"

namespace kda {

constexpr int kC = 64;                 // tokens per chunk
constexpr long long kGdrSpins = 4000000000LL;  // ~2 s of clock cycles

// One (chunk, value head) of the workspace: the bf16 parts of T and P as tiles [row][64] of
// 128-byte rows whose 16-byte groups are XORed with the row's low three bits, then vectors.
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

// The same for three parts, the middle one cut to 8 bits by r' = (c r) - (c r - r), c = 2^16 + 1
// (Veltkamp), as packed fp32 operations: conversions and integer operations run at half the
// rate of fp32 multiplications and additions.
__device__ __forceinline__ unsigned long long f2(float x, float y) {
  return ((unsigned long long)__float_as_uint(y) << 32) | __float_as_uint(x);
}
__device__ __forceinline__ void split3(float x, float y, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  const unsigned long long kMinus = f2(-1.f, -1.f), kC16 = f2(65537.f, 65537.f);
  unsigned long long r = f2(x, y), t, h;
  p0 = umma::pack_bf162(x, y);
  h = f2(__uint_as_float(p0 << 16), __uint_as_float(p0 & 0xffff0000u));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(r) : "l"(h), "l"(kMinus));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(r), "l"(kC16));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(h) : "l"(r), "l"(kMinus), "l"(t));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(h) : "l"(kMinus), "l"(t));
  p1 = __byte_perm((uint32_t)h, (uint32_t)(h >> 32), 0x7632);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(r) : "l"(h), "l"(kMinus));
  p2 = umma::pack_bf162(__uint_as_float((uint32_t)r), __uint_as_float((uint32_t)(r >> 32)));
}

// The walk over the chunks on tcgen05: d_k in {64, 128}, d_v a multiple of 128.
bool gdr_chain_tc_takes(const GdrArgs& a);
cudaError_t launch_gdr_chain_tc(const GdrArgs& a, const uint8_t* ws, cudaStream_t s);

}  // namespace kda
