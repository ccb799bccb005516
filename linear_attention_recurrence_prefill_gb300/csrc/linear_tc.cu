// linear_tc.cu -- y = act(x w^T + bias) + residual on the tcgen05 tensor cores
// (bf16 data).
//
// The product is taken transposed: D[n][m] = sum_k w[n][k] x[m][k], 128 rows of
// w (the M of the MMA, the lanes of TMEM) by BN rows of x (its N, the columns),
// from a ring of stages of 64 columns of w and x each, with a 128-byte swizzle.
//
// Two kernels; each starts its set-up while the kernel before it in the stream ends.
//  * linear_pair_kernel: pairs of CTAs (cta_group::2) share tiles of 256 rows of w by BN tokens, a
//    persistent pair per two SMs walking the tiles, two accumulators in TMEM so that a tile's
//    epilogue runs beside the next tile's products.  Alone, a CTA would fetch 128 + 256 rows for
//    each 128 x 256 products, 96 bytes per clock from L2 at the tensor cores' full rate, more than
//    an SM gets; a pair fetches 64.  Ten warps: 0-7 the epilogue, a lane per output channel (its
//    bias is one register, and for every token a warp writes 32 neighbouring elements of y and reads
//    those of the residual, whatever their alignment), 8 loads, 9 issues the MMAs.
//    4096 x 4096 x 12288: 234 to 242 us, 1.70 to 1.76
//    PFLOP/s, 0.89 to 0.92 of the measured bf16 rate (with bias, GELU and residual 251 to 262 us;
//    the library's plain product 208 us); 8192^3: 571 us (the library's 542).  The
//    tensor pipe is active in 79 % of the cycles of the former; the rest is 768 tiles in waves of 76,
//    the last one of eight tiles.  It also takes operands in fp16 that hold 8-bit integers, whose scales
//    the epilogue applies (those of the tokens from shared memory: from global memory it was the epilogue
//    that bound the product, 340 us).
//  * linear_split_kernel, where there are too few tiles to fill the GPU (few tokens, or a small
//    product): the CTAs of a cluster share one tile, each takes a part of K, and the partial sums
//    meet in distributed shared memory, added in the order of the ranks, so that results repeat
//    to the bit; four neighbouring channels per lane, a token per warp, which is one access where y's
//    and the residual's rows are multiples of four elements and four where not.  Six warps: 0-3 read
//    the sums, 4 loads, 5 issues the MMAs.  It also takes arrays that TMA cannot (rows that are no
//    multiple of 16 bytes apart): 0-3 and four more warps then fill the ring, from aligned 16-byte
//    loads that they shift into place.  Bound by reading w: 64 x 12288 -> 4096 takes 21.5 us, 4.8 TB/s with its set-up
//    and joining; 4096 x 4095 x 4097, shifted by every CTA that uses a tile, 584 us.
#include <initializer_list>

#include "linear_i8.cuh"
#include "linear_join.cuh"
#include "tensor_map.cuh"
#include "umma.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kThreads = 192, kFillThreads = 320;
constexpr int kWarpLoad = 4, kWarpMma = 5;
constexpr uint32_t kRowsA = 128, kBlockK = 64;
constexpr long long kSpins = 4000000000LL;  // ~2 s of clock cycles

struct Tc {
  CUtensorMap tm_w, tm_x;
  LinearArgs a;
  const float* x_scale;  // of an 8-bit product, whose integers are the operands
  const float* w_scale;
  int* status;
  int n_tiles, m_tiles, k_blocks;
};

// The epilogue of output channel n for the 32 tokens from m on, of which `cols` exist: the
// residual, fetched ahead of the sums, then the rest behind the bias.  T: the type of residual and y.
template <typename T>
__device__ __forceinline__ void load_residual(const LinearArgs& a, T (&add)[32], long long m, int n, int cols) {
  const T* res = static_cast<const T*>(a.residual) + m * a.ldr + n;
#pragma unroll
  for (int j = 0; j < 32; ++j) add[j] = a.residual && j < cols ? res[j * a.ldr] : from_f32<T>(0.f);
}

template <typename T>
__device__ __forceinline__ void finish32(const LinearArgs& a, float (&z)[32], const T (&add)[32], long long m, int n,
                                         int cols) {
  constexpr bool kFast = sizeof(T) == 2;
  // the activation chosen once for all
  auto all = [&](auto f) {
#pragma unroll
    for (int j = 0; j < 32; ++j) z[j] = f(z[j]);
  };
  switch (a.act) {
    case KDA_ACT_RELU: all([](float x) { return activate<kFast>(x, KDA_ACT_RELU); }); break;
    case KDA_ACT_SILU: all([](float x) { return activate<kFast>(x, KDA_ACT_SILU); }); break;
    case KDA_ACT_GELU: all([](float x) { return activate<kFast>(x, KDA_ACT_GELU); }); break;
    case KDA_ACT_GELU_TANH:
      all([](float x) { return activate<kFast>(x, KDA_ACT_GELU_TANH); });
      break;
    case KDA_ACT_SIGMOID: all([](float x) { return activate<kFast>(x, KDA_ACT_SIGMOID); }); break;
    default: break;
  }
  T* y = static_cast<T*>(a.y) + m * a.ldy + n;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < cols) y[j * a.ldy] = from_f32<T>(z[j] + to_f32(add[j]));
}

constexpr uint32_t kAlign = 1024;  // the swizzled tiles' alignment

template <int BN>
struct Pair {
  static constexpr uint32_t kStage = (kRowsA + BN / 2) * kBlockK * 2;
  static constexpr int kStages = BN > 192 ? 6 : 7;
  static constexpr uint32_t kSmem = kStages * kStage + kAlign;
  static constexpr uint32_t kAcc = 256;  // columns from one accumulator to the next
};

constexpr int kPairThreads = 320, kPairOut = 8, kPairLoad = 8, kPairMma = 9;

// Tile i as its rows of w and its tokens: eight rows of tiles at a time, so that the tiles in work
// at once share both and what they read stays in L2.
__device__ __forceinline__ void tile_of(const Tc& t, int i, int& n, int& m) {
  const int full = 8 * t.m_tiles, group = i / full, in = i - group * full;
  const int rows = min(8, t.n_tiles - group * 8);
  m = in / rows;
  n = group * 8 + in - m * rows;
}

// kI8: operands in fp16, which hold integers, and scales in the epilogue; else bf16.
template <int BN, typename T, bool kI8>
__global__ void __launch_bounds__(kPairThreads) __cluster_dims__(2, 1, 1)
    linear_pair_kernel(const __grid_constant__ Tc t) {
  using P = Pair<BN>;
  constexpr int kStages = P::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + ((kAlign - (smem_u32(raw) & (kAlign - 1))) & (kAlign - 1));
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_base;
  __shared__ __align__(16) float scales[kI8 ? kPairOut : 1][32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kPairOut);
    }
    mbar_init(&drained, 1);
    mbar_fence_init();
  }
  if (warp == kPairMma) {
    pair_tmem_alloc(&tmem_base, 512);
    pair_tmem_relinquish();
  }
  fence_before_sync();
  cluster_sync();
  fence_after_sync();
  const uint32_t tmem = tmem_base;
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  const int tiles = t.n_tiles * t.m_tiles, first = blockIdx.x / 2, step = gridDim.x / 2;

  bool ok = true;
  if (warp == kPairLoad && lane == 0) {
    // each CTA its rows of w and half of the tokens; all arrive on the even CTA's barrier
    int it = 0;
    for (int tile = first; tile < tiles && ok; tile += step) {
      int tn, tm;
      tile_of(t, tile, tn, tm);
      const int n0 = tn * 256 + (int)rank * 128, m0 = tm * BN + (int)rank * (BN / 2);
      for (int kb = 0; kb < t.k_blocks; ++kb, ++it) {
        const int s = it % kStages;
        if (it >= kStages && !mbar_wait_soon(&empty[s], (it / kStages - 1) & 1, kSpins)) {
          ok = false;
          break;
        }
        uint8_t* dst = ring + s * P::kStage;
        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * P::kStage);
        const uint32_t bar = map_to_rank(smem_u32(&full[s]), 0);
        pair_tma_load_2d(dst, &t.tm_w, kb * (int)kBlockK, n0, bar);
        pair_tma_load_2d(dst + kRowsA * kBlockK * 2, &t.tm_x, kb * (int)kBlockK, m0, bar);
      }
    }
    // The last signals to either CTA arrive before it leaves: those of the products that read the
    // stages, or, after a wait that gave up, of the loads in flight.
    for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
      if (ok) ok = mbar_wait(&empty[j % kStages], (j / kStages) & 1, kSpins);
      else if (rank == 0) mbar_wait(&full[j % kStages], (j / kStages) & 1, kSpins);
    // (the odd CTA issues no products, but is signalled to all the same)
    if (rank == 1 && !mbar_wait(&drained, 0, 2 * kSpins)) ok = false;
  } else if (warp == kPairMma && rank == 0) {
    const uint32_t lead = elect_leader();
    constexpr uint32_t idesc = idesc_f16(256, BN, !kI8);
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_soon(bar, parity, kSpins));
      fence_after_sync();
      return ok;
    };
    int it = 0, n = 0;
    for (int tile = first; tile < tiles; tile += step, ++n) {
      const int acc = n & 1;
      if (n >= 2 && !wait(&acc_empty[acc], (n / 2 - 1) & 1)) break;
      const uint32_t d = tmem + acc * P::kAcc;
      for (int kb = 0; kb < t.k_blocks; ++kb, ++it) {
        const int s = it % kStages;
        if (!wait(&full[s], (it / kStages) & 1)) break;
        const uint32_t at = smem_u32(ring + s * P::kStage);
        const uint64_t wd = desc_k_sw128(at, 0), xd = desc_k_sw128(at + kRowsA * kBlockK * 2, 0);
#pragma unroll
        for (uint32_t k = 0; k < kBlockK / 16; ++k)
          pair_mma_ss_if(lead, d, wd + (k * 32 >> 4), xd + (k * 32 >> 4), idesc, kb > 0 || k > 0);
        pair_commit_if(lead, &empty[s]);
      }
      if (!ok) break;
      pair_commit_if(lead, &acc_full[acc]);
    }
    // products in flight end before shared memory and TMEM are released
    pair_commit_if(lead, &drained);
    mbar_wait(&drained, 0, kSpins);
  } else if (warp < kPairOut) {
    // two warps per quarter of the lanes, every other 32 tokens each
    const T* bias = static_cast<const T*>(t.a.bias);
    const int quarter = warp & 3, half = warp >> 2;
    int i = 0;
    for (int tile = first; tile < tiles; tile += step, ++i) {
      const int acc = i & 1;
      int tn, tm;
      tile_of(t, tile, tn, tm);
      const int n = tn * 256 + (int)rank * 128 + quarter * 32 + lane;
      const long long m0 = (long long)tm * BN;
      const int cols = t.a.M - m0 < BN ? (int)(t.a.M - m0) : BN;
      const bool in = n < t.a.N;
      const float b = bias && in ? to_f32(bias[n]) : 0.f;
      const float scale = kI8 && in ? t.w_scale[n] : 0.f;
      float scale_m = kI8 && half * 32 + lane < cols ? t.x_scale[m0 + half * 32 + lane] : 0.f;
      T add[32], next[32];
      if (in) load_residual(t.a, add, m0 + half * 32, n, cols - half * 32);
      ok = __all_sync(0xffffffffu, mbar_wait_soon(&acc_full[acc], (i / 2) & 1, kSpins));
      if (!ok) break;
      fence_after_sync();
      const uint32_t d = taddr(tmem, quarter * 32, acc * P::kAcc);
#pragma unroll 1
      for (int c = half * 32; c < cols; c += 64) {
        uint32_t r[32];
        tmem_ld32(d + c, r);
        if (in && c + 64 < cols) load_residual(t.a, next, m0 + c + 64, n, cols - c - 64);
        float z[32];
        tmem_wait_ld();
        if constexpr (kI8) {
          // the tokens' scales, a lane each, to all lanes
          __syncwarp();
          scales[warp][lane] = scale_m;
          __syncwarp();
          if (c + 64 + lane < cols) scale_m = t.x_scale[m0 + c + 64 + lane];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 xs = *reinterpret_cast<const float4*>(&scales[warp][j]);
            z[j] = scaled(__uint_as_float(r[j]), xs.x, scale, b);
            z[j + 1] = scaled(__uint_as_float(r[j + 1]), xs.y, scale, b);
            z[j + 2] = scaled(__uint_as_float(r[j + 2]), xs.z, scale, b);
            z[j + 3] = scaled(__uint_as_float(r[j + 3]), xs.w, scale, b);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(r[j]) + b;
        }
        if (in) finish32(t.a, z, add, m0 + c, n, cols - c);
#pragma unroll
        for (int j = 0; j < 32; ++j) add[j] = next[j];
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&acc_empty[acc]), 0));
    }
  }
  if (!ok && lane == 0) atomicExch(t.status, KDA_ERR_TIMEOUT);
  fence_before_sync();
  cluster_sync();  // no CTA leaves while the other reads its shared memory or signals to it
  fence_after_sync();
  if (warp == kPairMma) pair_tmem_dealloc(tmem, 512);
}

template <int BN, int kStages>
constexpr uint32_t split_smem() {
  return kAlign + kStages * (kRowsA + BN) * kBlockK * 2;
}

// The aligned 16 bytes at `at`, as far as they lie in the array [lo, hi).
__device__ __forceinline__ uint4 part_of_array(uintptr_t at, uintptr_t lo, uintptr_t hi) {
  uint32_t w[4] = {0, 0, 0, 0};
  for (int i = 0; i < 8; ++i) {
    const uintptr_t e = at + 2 * i;
    if (e >= lo && e < hi) w[i >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(e) << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 16 bytes from byte `off` (even) of a and b on.
__device__ __forceinline__ uint4 shift_pieces(const uint4& a, const uint4& b, uint32_t off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = off & 2 ? __byte_perm(w[i], w[i + 1], 0x5432) : w[i];
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// kRows rows of 64 columns, from row r0 and column k0 on, into a tile of the ring, by 256 threads:
// eight per row, 16 bytes each, from two aligned loads; zeros outside the array.
template <int kRows>
__device__ __forceinline__ void fill_tile(uint8_t* tile, const void* base, long long ld, int rows, int K,
                                          long long r0, int k0, int tid) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(base), hi = lo + ((rows - 1) * ld + K) * 2;
  const int g = tid & 7, k = k0 + g * 8;
  // everything that the loads below touch lies in the array, except at its very ends
  const long long last = r0 + kRows < rows ? r0 + kRows - 1 : rows - 1;
  const bool inside = ((lo + (r0 * ld + k0) * 2) & ~(uintptr_t)15) >= lo && lo + (last * ld + k0 + 64) * 2 + 32 <= hi;
  constexpr int kPasses = kRows < 32 ? 1 : kRows / 32, kBatch = kPasses < 4 ? kPasses : 4;
#pragma unroll 1
  for (int i0 = 0; i0 < kPasses; i0 += kBatch) {
    uint4 v[kBatch][2];
    uint32_t off[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const long long r = r0 + (tid >> 3) + (i0 + i) * 32;
      const uintptr_t at = lo + ((r < rows ? r : last) * ld + k) * 2;
      off[i] = (uint32_t)at & 15;
      const uintptr_t from = at - off[i];
      if (inside) {
        v[i][0] = *reinterpret_cast<const uint4*>(from);
        v[i][1] = *reinterpret_cast<const uint4*>(from + 16);
      } else {
        v[i][0] = part_of_array(from, lo, hi);
        v[i][1] = part_of_array(from + 16, lo, hi);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = (tid >> 3) + (i0 + i) * 32;
      uint4 z = shift_pieces(v[i][0], v[i][1], off[i]);
      uint32_t* w = &z.x;
      const int left = r0 + row < rows ? K - k : 0;  // columns from here on that exist
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = left > 2 * e + 1 ? w[e] : left > 2 * e ? w[e] & 0xffffu : 0;
      if (kRows >= 32 || row < kRows) *reinterpret_cast<uint4*>(tile + sw128_chunk(row, g, kRows)) = z;
    }
  }
}

template <int BN, int kStages, bool kTma>
__global__ void __launch_bounds__(kTma ? kThreads : kFillThreads) linear_split_kernel(const __grid_constant__ Tc t) {
  constexpr uint32_t kStage = (kRowsA + BN) * kBlockK * 2;
  constexpr uint32_t kCols = BN <= 32 ? 32 : BN <= 64 ? 64 : 128;
  static_assert(kStages * kStage >= BN * kRowsA * 4, "the partial sums fit in the ring");
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + ((kAlign - (smem_u32(raw) & (kAlign - 1))) & (kAlign - 1));
  __shared__ uint64_t full[kStages], empty[kStages], done;
  __shared__ uint32_t tmem_base;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), ranks = gridDim.z;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], kTma ? 1 : 8);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    mbar_fence_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&tmem_base, kCols);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_base;
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  // this CTA's part of K: every ranks-th block (one at least), so that the cluster reads rows of w
  // in pieces of ranks * 128 bytes
  const int blocks = (t.k_blocks - (int)rank + (int)ranks - 1) / (int)ranks;

  const int n0 = blockIdx.x % t.n_tiles * (int)kRowsA, m0 = blockIdx.x / t.n_tiles * BN;

  bool ok = true;
  if (kTma && warp == kWarpLoad && lane == 0) {
    int it = 0;
    for (; it < blocks; ++it) {
      const int s = it % kStages, x = (it * (int)ranks + (int)rank) * (int)kBlockK;
      if (it >= kStages && !mbar_wait_soon(&empty[s], (it / kStages - 1) & 1, kSpins)) {
        ok = false;
        break;
      }
      uint8_t* dst = ring + s * kStage;
      mbar_arrive_expect_tx(&full[s], kStage);
      tma_load_2d(dst, &t.tm_w, x, n0, &full[s]);
      tma_load_2d(dst + kRowsA * kBlockK * 2, &t.tm_x, x, m0, &full[s]);
    }
    // a wait that gave up: the loads in flight land before shared memory is released
    if (!ok)
      for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
        mbar_wait(&full[j % kStages], (j / kStages) & 1, kSpins);
  } else if (warp == kWarpMma) {
    const uint32_t lead = elect_leader();
    constexpr uint32_t idesc = idesc_f16(kRowsA, BN, true);
    for (int it = 0; it < blocks; ++it) {
      const int s = it % kStages;
      ok = __all_sync(0xffffffffu, mbar_wait_soon(&full[s], (it / kStages) & 1, kSpins));
      if (!ok) break;
      fence_after_sync();
      const uint32_t at = smem_u32(ring + s * kStage);
      const uint64_t wd = desc_k_sw128(at, 0), xd = desc_k_sw128(at + kRowsA * kBlockK * 2, 0);
#pragma unroll
      for (uint32_t k = 0; k < kBlockK / 16; ++k)
        mma_ss_if(lead, tmem, wd + (k * 32 >> 4), xd + (k * 32 >> 4), idesc, it > 0 || k > 0);
      mma_commit_if(lead, &empty[s]);
    }
    // everything issued is complete before the ring or TMEM is used again, or released
    mma_commit_if(lead, &done);
    mbar_wait(&done, 0, kSpins);
  } else if (warp < 4 || warp > kWarpMma) {
    if constexpr (!kTma) {
      const int tid = threadIdx.x - (warp < 4 ? 0 : 64);
      for (int it = 0; it < blocks && ok; ++it) {
        const int s = it % kStages, x = (it * (int)ranks + (int)rank) * (int)kBlockK;
        if (it >= kStages)
          ok = __all_sync(0xffffffffu, mbar_wait_soon(&empty[s], (it / kStages - 1) & 1, kSpins));
        if (!ok) break;
        uint8_t* dst = ring + s * kStage;
        fill_tile<kRowsA>(dst, t.a.w, t.a.ldw, t.a.N, t.a.K, n0, x, tid);
        fill_tile<BN>(dst + kRowsA * kBlockK * 2, t.a.x, t.a.ldx, t.a.M, t.a.K, m0, x, tid);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
    }
    // Done behind all of this CTA's blocks, each of which has a wait of its own that gives up (the
    // MMA warp then signals all the same): a block takes some 300 to 5,000 cycles.
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&done, 0, 3 * kSpins + (long long)blocks * 65536));
    fence_after_sync();
    if (ok && warp < 4) {
      // partial sums [column][channel] over the ring, whose loads and products are done
      const uint32_t d = taddr(tmem, warp * 32, 0);
      float* part = reinterpret_cast<float*>(ring) + warp * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < BN; c += 16) {
        uint32_t r[16];
        tmem_ld16(d + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * (int)kRowsA] = __uint_as_float(r[j]);
      }
    }
  }
  if (!ok && lane == 0) atomicExch(t.status, KDA_ERR_TIMEOUT);

  // every rank adds up its share of the tile's columns over all ranks; a CTA that gave up takes
  // part in the barriers all the same
  cluster_sync();
  if (warp < 4) {
    // four neighbouring channels per thread, a column per warp
    const int n = n0 + lane * 4;
    const int cols = t.a.M - m0 < BN ? t.a.M - m0 : BN;
    const bool wide = wide4(t.a, 2);
    const float4 b = bias4<__nv_bfloat16>(t.a, n);
    const uint32_t part = smem_u32(ring) + lane * 16;
    join(ranks, part, rank, warp, cols,
         [&](const float4& z, int c) { finish4<__nv_bfloat16>(t.a, wide, z, b, m0 + c, n); });
  }
  fence_before_sync();
  cluster_sync();  // no CTA leaves while its sums are read
  fence_after_sync();
  if (warp == kWarpMma) tmem_dealloc(tmem, kCols);
}

// Tensor map of a [rows][K] array in bf16 (or fp16), rows ld elements apart: boxes of 64
// columns by `box` rows, 128-byte swizzle, zeros outside.
bool encode(CUtensorMap* m, const void* base, int rows, int K, long long ld, int box, bool half = false) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t boxes[2] = {kBlockK, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool fill(Tc& t, const LinearArgs& a, bool tma, int* status, int rows_w, int box_w, int rows_x, int box_x,
          bool half = false) {
  t.a = a;
  t.x_scale = t.w_scale = nullptr;
  t.status = status;
  t.n_tiles = (a.N + rows_w - 1) / rows_w;
  t.m_tiles = (int)(((long long)a.M + rows_x - 1) / rows_x);
  t.k_blocks = (a.K + (int)kBlockK - 1) / (int)kBlockK;
  return !tma || (encode(&t.tm_w, a.w, a.N, a.K, a.ldw, box_w, half) &&
                  encode(&t.tm_x, a.x, a.M, a.K, a.ldx, box_x, half));
}

template <int BN, typename T, bool kI8>
cudaError_t launch_pair_of(const LinearI8Args& i, int pairs, int* status, cudaStream_t s) {
  constexpr auto kern = linear_pair_kernel<BN, T, kI8>;
  const cudaError_t e = allow_smem<kern>(Pair<BN>::kSmem);
  if (e != cudaSuccess) return e;
  Tc t;
  if (!fill(t, i.l, true, status, 256, kRowsA, BN, BN / 2, kI8)) return cudaErrorInvalidValue;
  t.x_scale = i.x_scale;
  t.w_scale = i.w_scale;
  const long long tiles = (long long)t.n_tiles * t.m_tiles;
  return launch_early(kern, dim3(2 * (unsigned)(tiles < pairs ? tiles : pairs)), kPairThreads, Pair<BN>::kSmem, 1, s,
                      t);
}
template <int BN>
cudaError_t launch_pair(const LinearArgs& a, int pairs, int* status, cudaStream_t s) {
  return launch_pair_of<BN, __nv_bfloat16, false>({a, nullptr, nullptr}, pairs, status, s);
}

// The width of tile, of those given (widest first), whose waves of tiles cost least.  A tile's
// time hardly falls with its width, since the rows of w have to come all the same: at
// 8192 x 8192 x 8192 a wave took 41.5, 38.5, 36.6, 35.8, 35.2 us for 256, 224, 192, 160, 128.
int pair_width(const LinearArgs& a, int pairs, std::initializer_list<int> widths) {
  const long long rows = (a.N + 255LL) / 256;
  long long best = 0;
  int width = 0;
  for (int bn : widths) {
    const long long tiles = rows * ((a.M + bn - 1LL) / bn);
    const long long cost = (tiles + pairs - 1) / pairs * (448 + bn);
    if (!width || cost < best) {
      best = cost;
      width = bn;
    }
  }
  return width;
}

template <int BN, int kStages, bool kTma>
cudaError_t launch_split_of(const LinearArgs& a, int* status, int split, cudaStream_t s) {
  constexpr auto kern = linear_split_kernel<BN, kStages, kTma>;
  const cudaError_t e = allow_smem<kern>(split_smem<BN, kStages>());
  if (e != cudaSuccess) return e;
  Tc t;
  if (!fill(t, a, kTma, status, kRowsA, kRowsA, BN, BN)) return cudaErrorInvalidValue;
  return launch_early(kern, dim3((unsigned)((long long)t.n_tiles * t.m_tiles), 1, split),
                      kTma ? kThreads : kFillThreads, split_smem<BN, kStages>(), split, s, t);
}

bool tma_takes(const LinearArgs& a) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w);
  return (at & 15) == 0 && a.ldx % 8 == 0 && a.ldw % 8 == 0 && a.ldx < (1LL << 38) &&
         a.ldw < (1LL << 38);
}

template <int BN, int kStages>
cudaError_t launch_split(const LinearArgs& a, bool tma, int* status, int split, cudaStream_t s) {
  return tma ? launch_split_of<BN, kStages, true>(a, status, split, s)
             : launch_split_of<BN, kStages, false>(a, status, split, s);
}

}  // namespace

bool linear_tc_takes(const LinearArgs& a, int dtype) {
  return dtype == KDA_BF16 && a.K > 0 &&
         (a.N + 127LL) / 128 * ((a.M + 15LL) / 16) <= 0x7fffffffLL;  // tiles in a grid
}


cudaError_t launch_linear_tc(const LinearArgs& a, int sms, int* status, cudaStream_t s) {
  const int k_blocks = (a.K + 63) / 64;
  // Pairs of CTAs where their tiles fill half of the SMs at least (4096 x 4096 weights: 25 against
  // 34 us with 512 tokens, 25 against 21 us with 256).
  const int pairs = sms / 2;
  const bool tma = tma_takes(a);
  if (tma && (a.N + 255LL) / 256 * ((a.M + 127LL) / 128) >= pairs / 2) {
    switch (pair_width(a, pairs, {256, 224, 192, 160, 128})) {
      case 256: return launch_pair<256>(a, pairs, status, s);
      case 224: return launch_pair<224>(a, pairs, status, s);
      case 192: return launch_pair<192>(a, pairs, status, s);
      case 160: return launch_pair<160>(a, pairs, status, s);
      default: return launch_pair<128>(a, pairs, status, s);
    }
  }
  // Else K split over the CTAs of a cluster until there are two CTAs per SM.
  const int bn = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
  const long long tiles = (a.N + 127LL) / 128 * ((a.M + bn - 1LL) / bn);
  int split = 1;
  while (split < 8 && split * 2 <= k_blocks && tiles * split * 2 <= 2LL * sms) split *= 2;
  switch (bn) {
    case 16: return launch_split<16, 6>(a, tma, status, split, s);
    case 32: return launch_split<32, 5>(a, tma, status, split, s);
    case 64: return launch_split<64, 4>(a, tma, status, split, s);
    default: return launch_split<128, 3>(a, tma, status, split, s);
  }
}

cudaError_t launch_linear_i8_pair(const LinearI8Args& a, int dtype, int sms, int* status, cudaStream_t s) {
  const int pairs = sms / 2;
  const bool f32 = dtype == KDA_F32;
  switch (pair_width(a.l, pairs, {256, 192, 128})) {
    case 256:
      return f32 ? launch_pair_of<256, float, true>(a, pairs, status, s)
                 : launch_pair_of<256, __nv_bfloat16, true>(a, pairs, status, s);
    case 192:
      return f32 ? launch_pair_of<192, float, true>(a, pairs, status, s)
                 : launch_pair_of<192, __nv_bfloat16, true>(a, pairs, status, s);
    default:
      return f32 ? launch_pair_of<128, float, true>(a, pairs, status, s)
                 : launch_pair_of<128, __nv_bfloat16, true>(a, pairs, status, s);
  }
}

}  // namespace kda
