// gdr_chunked.cuh -- the chunked gated delta rule: the workspace between its kernels, and the
// bf16 parts that fp32 operands are split into.
#pragma once

#include "gdr.cuh"
#include "umma.cuh"

namespace kda {

constexpr int kC = 64;                 // tokens per chunk
constexpr long long kGdrSpins = 4000000000LL;  // ~2 s of clock cycles

// One (chunk, value head) of the workspace: the bf16 parts of T and P as tiles [row][64] of
// 128-byte rows whose 16-byte groups are XORed with the row's low three bits, then vectors.  T has
// three tiles, P two: the 16 x 16 blocks above the diagonal ones are zeros that no product reads, and
// P's third part lies there in its two tiles (third_of_p).
constexpr uint32_t kTile = kC * kC * 2;
constexpr uint32_t kT = 0, kP = 3 * kTile;
constexpr uint32_t kVec = 5 * kTile;        // floats: a[64], b[64], ku[64], e^{g_C}
constexpr uint32_t kBlock = kVec + 1024;

__host__ __device__ constexpr uint32_t tile_at(uint32_t row, uint32_t col) {
  return row * 128u + ((((col >> 3) ^ row) & 7u) << 4) + (col & 7u) * 2u;
}

// Where the 16 x 16 block (i, j), j <= i, of P's third part lies: the tile of P, and the block in it.
// The blocks of a column stay below each other, so that one product takes them, but for (0, 0): no
// tile has four above its diagonal.
struct PlaceOfP {
  int tile, row, col;
};
__host__ __device__ constexpr PlaceOfP third_of_p(int i, int j) {
  return j == 0 ? (i == 0 ? PlaceOfP{1, 0, 1} : PlaceOfP{0, i - 1, 3})
                : PlaceOfP{j == 1 ? 1 : 0, i - j, 4 - j};
}

// Chunk c of sequence n has block (t0 / 64 + n) + c: floor((t0 + len) / 64) + 1 is at
// least floor(t0 / 64) + ceil(len / 64), so that sequences never share a block, and no
// prefix sum over the sequences is needed.
__host__ __device__ constexpr int block_base(int t0, int n) { return t0 / kC + n; }

// x and y as sums of three bf16 parts, packed.  Each part is rounded to nearest: what the first two
// leave is at most 2^-17 of the value, of either sign, and has at most 8 bits, so that the sum of
// the three is exact.  (Parts cut off instead would leave up to 2^-15, always toward zero, in the
// products that take two of them: by emulation o off by 1e-5 of its size, not 3e-6, with states of
// 30 times v's.)
__device__ __forceinline__ unsigned long long f2(float x, float y) {
  return ((unsigned long long)__float_as_uint(y) << 32) | __float_as_uint(x);
}
__device__ __forceinline__ void split3(float x, float y, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  const unsigned long long kMinus = f2(-1.f, -1.f);
  unsigned long long r = f2(x, y);
  auto take = [&](float lo, float hi) {
    const uint32_t p = umma::pack_bf162(lo, hi);
    const unsigned long long h = ((unsigned long long)(p & 0xffff0000u) << 32) | (p << 16);
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(r) : "l"(h), "l"(kMinus));
    return p;
  };
  p0 = take(x, y);
  p1 = take(__uint_as_float((uint32_t)r), __uint_as_float((uint32_t)(r >> 32)));
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
cudaError_t launch_gdr_chain_tc(const GdrArgs& a, const uint8_t* ws, cudaStream_t s);

}  // namespace kda
