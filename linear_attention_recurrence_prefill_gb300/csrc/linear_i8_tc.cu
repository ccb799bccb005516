// linear_i8_tc.cu -- y = act(x_scale w_scale (x w^T) + bias) + residual for 8-bit
// integers x and w, on the tcgen05 tensor cores.
//
// This GPU multiplies 8-bit integers far below its rate for 16-bit floats, and every such
// integer is an fp16 number: the products are taken in fp16 with fp32 sums, which are exact below
// 2^24 and lose up to 2^-23 of themselves in each of K / 16 additions beyond (the header gives the
// bound).  So what 8 bits save is memory, and the integers are widened on their way:
//  * few tiles (few tokens, or a small product; bound by reading w): linear_i8_kernel.  w's rows go
//    from shared memory through registers, where they are widened, into TMEM, from which the MMAs take
//    them: a lane of TMEM is a row, so a thread widens 64 neighbouring integers of its row and
//    stores them at once.  x, of which there is less, is widened into tiles of shared memory by
//    warps of its own.  The CTAs of a cluster share a tile of 128 channels, each takes a part of K.
//    64 x 12288 -> 4096: 20.4 us (2.5 TB/s; both widened into shared memory, with its fences, 26 us).
//    Widening nothing changes that by 1 us and a longer ring by nothing: it is the loads of 256 CTAs,
//    two to an SM, on 128 of the SMs, 0.47 us per block, and 5 to 9 us to set up and to join.
//  * many: both arrays are widened into the workspace first, once, and the product is that of
//    kda_linear's pairs of CTAs.  Widened in the product, w would be taken through shared memory
//    once more for every 256 tokens, which the tensor cores' own reads leave no room for.
//    4096 x 4096 -> 12288 with bias, GELU and residual: 282 to 297 us, of which the widening 38 (201 MB, a part of
//    which stays in L2) and the product 250 (1.65 PFLOP/s, as kda_linear's).
// So 8 bits are faster than kda_linear in bf16 up to some 16 to 64 rows and save memory beyond (with the
// residual, 8 bits and bf16, us: 4096 -> 12288, 1, 16, 64, 512, 4096 rows 10.6 and 18.2, 18.9 and 22.0, 24.9 and 22.7,
// 83 and 48, 275 and 248; 12288 -> 4096 12.1 and 21.4, 16.3 and 19.1, 19.4 and 21.3, 69 and 59, 300 and 237).
// linear_i8_kernel has 72 or 80 registers a thread, two CTAs to an SM, and spills 20 to 88 bytes of them, widen_kernel
// 16, the pairs' kernel 12.
#include "linear_i8.cuh"
#include "linear_join.cuh"
#include "tensor_map.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr uint32_t kRowsA = kJoinRows, kBlockK = 64;
// Warps 0-7 widen w, the even blocks of 64 columns by 0-3 and the odd ones by 4-7; then come those
// that widen x, half of them the even blocks, one that issues the MMAs and, where TMA can take the
// arrays, one that loads.
constexpr int kFillW = 8;
constexpr uint32_t kAlign = 1024;                      // the swizzled tiles' alignment
constexpr long long kSpins = 4000000000LL;             // ~2 s of clock cycles

struct I8 {
  CUtensorMap tm_w, tm_x;
  LinearI8Args a;
  int* status;
  int n_tiles, k_blocks;
};

// Four integers as fp16: a byte b + 128 below the exponent of 1024 is 1152 + b.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off), y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}
// 16 bytes from byte `off` of a and b on.
__device__ __forceinline__ uint4 shift_bytes(const uint4& a, const uint4& b, uint32_t off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
  const uint32_t bits = (off & 3) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kTma: rows and bases at 16 bytes.  A block's integers then land in shared memory, in rows of 64
// bytes (w's with TMA's swizzle of 64 bytes: each thread reads a row of its own); else the threads
// read them where they are, four neighbours a row, and those of w pass through a place of each
// warp's own to the thread that has their row (100 x 4095 -> 4096: 30.5 us, 33.3 with a row a
// thread; 150 x 2047 -> 1021: 15.0 and 16.5; but 12 x 1000 -> 1499: 8.9 and 8.3).
template <int BN, bool kTma>
struct Fill {
  static constexpr int kFillX = BN > 32 ? 4 : 2, kFill = (kFillW + kFillX) / 2;  // the latter of a block
  static constexpr int kMma = kFillW + kFillX;
  static constexpr int kThreads = (kMma + (kTma ? 2 : 1)) * 32;
  static constexpr int kTiles = 4;                                // widened blocks
  static constexpr int kRaw = kTma ? (BN > 64 ? 2 : 4) : 0;       // blocks on their way or landed
  static constexpr uint32_t kRawBlock = (kRowsA + BN) * kBlockK;
  static constexpr uint32_t kPass = kTma ? 0 : kFillW * 32 * kBlockK;  // bytes
  static constexpr uint32_t kTile = BN * kBlockK * 2;             // x's part of a widened block
  static constexpr uint32_t kUsed = kTiles * kTile + kRaw * kRawBlock + kPass, kSums = BN * kRowsA * 4;
  static constexpr uint32_t kSmem = kAlign + (kUsed > kSums ? kUsed : kSums);
  static constexpr uint32_t kAcc = BN <= 32 ? 32 : BN <= 64 ? 64 : 128;  // columns of TMEM
  static constexpr uint32_t kA = kBlockK / 2;                            // of w's part of a block
};

// 16 integers from p on, of which `left` exist (zeros behind them), `first`: of the array's first byte.
__device__ __forceinline__ uint4 load16(const int8_t* p, long long left, const int8_t* first) {
  const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15;
  const int8_t* from = p - off;
  if (left >= 16 && from >= first && (off == 0 || left >= 32)) {
    const uint4 a = *reinterpret_cast<const uint4*>(from);
    const uint4 b = off ? *reinterpret_cast<const uint4*>(from + 16) : a;
    return shift_bytes(a, b, off);
  }
  uint4 v = make_uint4(0, 0, 0, 0);
  uint32_t* z = &v.x;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (e < left) z[e >> 2] |= (uint32_t)(uint8_t)p[e] << (8 * (e & 3));
  return v;
}

template <int BN, bool kTma, typename T>
__global__ void __launch_bounds__(Fill<BN, kTma>::kThreads, 2) linear_i8_kernel(const __grid_constant__ I8 t) {
  using F = Fill<BN, kTma>;
  constexpr int kRawSlots = kTma ? F::kRaw : 1;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* tiles = raw_smem + ((kAlign - (smem_u32(raw_smem) & (kAlign - 1))) & (kAlign - 1));
  uint8_t* raw = tiles + F::kTiles * F::kTile;
  __shared__ uint64_t full[F::kTiles], empty[F::kTiles], landed[kRawSlots], taken[kRawSlots], done;
  __shared__ uint32_t tmem_base;

  const LinearArgs& l = t.a.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), ranks = gridDim.z;
  if (threadIdx.x == 0) {
    for (int i = 0; i < F::kTiles; ++i) {
      mbar_init(&full[i], F::kFill);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kRawSlots; ++i) {
      mbar_init(&landed[i], 1);
      mbar_init(&taken[i], F::kFill);
    }
    mbar_init(&done, 1);
    mbar_fence_init();
  }
  if (warp == F::kMma) {
    tmem_alloc(&tmem_base, 256);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_base;
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  // this CTA's part of K: every ranks-th block (one at least)
  const int blocks = (t.k_blocks - (int)rank + (int)ranks - 1) / (int)ranks;
  const int n0 = blockIdx.x % t.n_tiles * (int)kRowsA, m0 = blockIdx.x / t.n_tiles * BN;
  auto column = [&](int it) { return (it * (long long)ranks + rank) * kBlockK; };

  bool ok = true;
  if (warp < kFillW) {
    const int quarter = warp & 3, r = quarter * 32 + lane;
    // where they are: four neighbouring lanes a row, eight rows at a time
    uint8_t* pass = raw + warp * 32 * kBlockK;
    const int c4 = lane & 3;
    uint4 next[4];
    auto fetch = [&](int it) {
      const long long k = column(it) + c4 * 16;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long n = (long long)n0 + quarter * 32 + j * 8 + (lane >> 2);
        const bool in = n < l.N && it < blocks;
        next[j] = load16(static_cast<const int8_t*>(l.w) + (in ? n : 0) * l.ldw + k, in ? l.K - k : 0,
                         static_cast<const int8_t*>(l.w));
      }
    };
    if (!kTma) fetch(warp >> 2);
    for (int it = warp >> 2; it < blocks; it += 2) {
      const int s = it % F::kTiles;
      uint32_t half[32];
      if constexpr (kTma) {
        const int slot = it % F::kRaw;
        ok = __all_sync(0xffffffffu, mbar_wait_soon(&landed[slot], (it / F::kRaw) & 1, kSpins));
        if (!ok) break;
        const uint8_t* from = raw + slot * F::kRawBlock + r * kBlockK;
#pragma unroll
        for (int c = 0; c < 4; ++c) next[c] = *reinterpret_cast<const uint4*>(from + ((c ^ (r >> 1 & 3)) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(&taken[slot]);
      }
      if constexpr (!kTma) {
        __syncwarp();  // the block before has been read
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = j * 8 + (lane >> 2);
          *reinterpret_cast<uint4*>(pass + at * kBlockK + ((c4 ^ (at >> 1 & 3)) << 4)) = next[j];
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c)
          next[c] = *reinterpret_cast<const uint4*>(pass + lane * kBlockK + ((c ^ (lane >> 1 & 3)) << 4));
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        widen4(next[c].x, half[8 * c], half[8 * c + 1]);
        widen4(next[c].y, half[8 * c + 2], half[8 * c + 3]);
        widen4(next[c].z, half[8 * c + 4], half[8 * c + 5]);
        widen4(next[c].w, half[8 * c + 6], half[8 * c + 7]);
      }
      if (!kTma) fetch(it + 2);
      if (it >= F::kTiles)
        ok = __all_sync(0xffffffffu, mbar_wait_soon(&empty[s], (it / F::kTiles - 1) & 1, kSpins));
      if (!ok) break;
      fence_after_sync();
      tmem_st32(taddr(tmem, quarter * 32, F::kAcc + s * F::kA), half);
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
    }
  } else if (warp < F::kMma) {
    constexpr int kThreadsX = F::kFillX * 16, kChunks = (BN * 4 + kThreadsX - 1) / kThreadsX;
    const int tid = ((int)threadIdx.x - kFillW * 32) % kThreadsX, c = tid % 4;
    for (int it = (warp - kFillW) / (F::kFillX / 2); it < blocks; it += 2) {
      const int s = it % F::kTiles;
      uint4 v[kChunks];
      if constexpr (kTma) {
        const int slot = it % F::kRaw;
        ok = __all_sync(0xffffffffu, mbar_wait_soon(&landed[slot], (it / F::kRaw) & 1, kSpins));
        if (!ok) break;
        const uint8_t* from = raw + slot * F::kRawBlock + kRowsA * kBlockK;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) v[i] = *reinterpret_cast<const uint4*>(from + (tid + i * kThreadsX) * 16);
        __syncwarp();
        if (lane == 0) mbar_arrive(&taken[slot]);
      } else {
        const long long k = column(it) + c * 16;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const long long m = (long long)m0 + (tid + i * kThreadsX) / 4;
          const bool in = m < l.M && (tid + i * kThreadsX) / 4 < BN;
          v[i] = load16(static_cast<const int8_t*>(l.x) + (in ? m : 0) * l.ldx + k, in ? l.K - k : 0,
                        static_cast<const int8_t*>(l.x));
        }
      }
      if (it >= F::kTiles)
        ok = __all_sync(0xffffffffu, mbar_wait_soon(&empty[s], (it / F::kTiles - 1) & 1, kSpins));
      if (!ok) break;
      uint8_t* tile = tiles + s * F::kTile;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const uint32_t r = (tid + i * kThreadsX) / 4;
        if (kChunks * kThreadsX != BN * 4 && r >= BN) break;
        uint4 a, b;
        widen4(v[i].x, a.x, a.y);
        widen4(v[i].y, a.z, a.w);
        widen4(v[i].z, b.x, b.y);
        widen4(v[i].w, b.z, b.w);
        *reinterpret_cast<uint4*>(tile + sw128_chunk(r, 2 * c, 0)) = a;
        *reinterpret_cast<uint4*>(tile + sw128_chunk(r, 2 * c + 1, 0)) = b;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
    }
  } else if (warp == F::kMma) {
    const uint32_t lead = elect_leader();
    constexpr uint32_t idesc = idesc_f16(kRowsA, BN, false);
    for (int it = 0; it < blocks; ++it) {
      const int s = it % F::kTiles;
      ok = __all_sync(0xffffffffu, mbar_wait_soon(&full[s], (it / F::kTiles) & 1, kSpins));
      if (!ok) break;
      fence_after_sync();
      const uint64_t xd = desc_k_sw128(smem_u32(tiles + s * F::kTile), 0);
#pragma unroll
      for (uint32_t k = 0; k < kBlockK / 16; ++k)
        mma_ts_if(lead, tmem, tmem + F::kAcc + s * F::kA + k * 8, xd + (k * 32 >> 4), idesc, it > 0 || k > 0);
      mma_commit_if(lead, &empty[s]);
    }
    // everything issued is complete before the tiles or TMEM are used again, or released
    mma_commit_if(lead, &done);
    mbar_wait(&done, 0, kSpins);
  } else if (kTma) {
    if (lane == 0) {
      int it = 0;
      for (; it < blocks; ++it) {
        const int s = it % kRawSlots, x = (int)column(it);
        if (it >= kRawSlots && !mbar_wait_soon(&taken[s], (it / kRawSlots - 1) & 1, kSpins)) {
          ok = false;
          break;
        }
        uint8_t* to = raw + s * F::kRawBlock;
        mbar_arrive_expect_tx(&landed[s], F::kRawBlock);
        tma_load_2d(to, &t.tm_w, x, n0, &landed[s]);
        tma_load_2d(to + kRowsA * kBlockK, &t.tm_x, x, m0, &landed[s]);
      }
      // a wait that gave up, here or of the warps that widen: the loads in flight land before shared
      // memory is released
      for (int j = it > kRawSlots ? it - kRawSlots : 0; j < it; ++j)
        mbar_wait(&landed[j % kRawSlots], (j / kRawSlots) & 1, kSpins);
    }
    __syncwarp();
  }
  // Done behind all of this CTA's blocks, each of which has a wait of its own that gives up (the
  // MMA warp then signals all the same): a block takes some 300 to 5,000 cycles.
  if (warp < 4) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&done, 0, 3 * kSpins + (long long)blocks * 65536));
    fence_after_sync();
  }
  __syncthreads();  // no thread widens any more, and nothing is on its way to shared memory
  if (ok && warp < 4) {
    // partial sums [column][channel] over the tiles, whose products are done
    const uint32_t d = taddr(tmem, warp * 32, 0);
    float* part = reinterpret_cast<float*>(tiles) + warp * 32 + lane;
#pragma unroll 1
    for (int c = 0; c < BN; c += 16) {
      uint32_t r[16];
      tmem_ld16(d + c, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c + j) * (int)kRowsA] = __uint_as_float(r[j]);
    }
  }
  if (!ok && lane == 0) atomicExch(t.status, KDA_ERR_TIMEOUT);

  // every rank adds up its share of the tile's columns over all ranks; a CTA that gave up takes
  // part in the barriers all the same
  cluster_sync();
  if (warp < 4) {
    const int n = n0 + lane * 4;
    const int cols = l.M - m0 < BN ? l.M - m0 : BN;
    const bool wide = wide4(l, sizeof(T));
    const float4 b = bias4<T>(l, n);
    float4 ws;
    ws.x = n < l.N ? t.a.w_scale[n] : 0.f;
    ws.y = n + 1 < l.N ? t.a.w_scale[n + 1] : 0.f;
    ws.z = n + 2 < l.N ? t.a.w_scale[n + 2] : 0.f;
    ws.w = n + 3 < l.N ? t.a.w_scale[n + 3] : 0.f;
    join(ranks, smem_u32(tiles) + lane * 16, rank, warp, cols, [&](float4 z, int c) {
      const float xs = t.a.x_scale[(long long)m0 + c];
      z.x = scaled(z.x, xs, ws.x, b.x);
      z.y = scaled(z.y, xs, ws.y, b.y);
      z.z = scaled(z.z, xs, ws.z, b.z);
      z.w = scaled(z.w, xs, ws.w, b.w);
      finish4<T>(l, wide, z, make_float4(0.f, 0.f, 0.f, 0.f), (long long)m0 + c, n);
    });
  }
  fence_before_sync();
  cluster_sync();  // no CTA leaves while its sums are read
  fence_after_sync();
  if (warp == F::kMma) tmem_dealloc(tmem, 256);
}

// [rows][K] integers, rows ld bytes apart, as fp16 with rows of Kp elements (a multiple of 16, zeros
// behind K), x's rows and then w's: a thread takes 16 columns of two rows at a time.
__global__ void __launch_bounds__(256, 8) widen_kernel(const int8_t* x, long long ldx, long long rows_x, const int8_t* w,
                                                    long long ldw, long long rows_w, int K, int Kp, uint4* to) {
  constexpr int kFlight = 2;
  grid_launch_dependents();
  grid_wait_prerequisites();
  const long long rows = rows_x + rows_w;
  const int chunks = Kp / 16;
  for (long long r0 = (long long)blockIdx.x * kFlight; r0 < rows; r0 += (long long)gridDim.x * kFlight) {
    for (int c = threadIdx.x; c < chunks; c += 256) {
      const int k = c * 16;
      uint4 v[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const long long r = r0 + i;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r >= rows) continue;
        const int8_t* p = (r < rows_x ? x + r * ldx : w + (r - rows_x) * ldw) + k;
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        if (k + 16 <= K && (at & 15) == 0) {
          v[i] = *reinterpret_cast<const uint4*>(p);
        } else if (k + 20 <= K && (k > 0 || (r != 0 && r != rows_x))) {
          // the five aligned words around the 16 bytes begin up to three bytes before them, which an
          // array's first row has not
          uint32_t q[5];
          const uint32_t* a = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
          const uint32_t bits = (uint32_t)(at & 3) * 8;
#pragma unroll
          for (int j = 0; j < 5; ++j) q[j] = a[j];
          v[i] = make_uint4(__funnelshift_r(q[0], q[1], bits), __funnelshift_r(q[1], q[2], bits),
                            __funnelshift_r(q[2], q[3], bits), __funnelshift_r(q[3], q[4], bits));
        } else {
          uint32_t* z = &v[i].x;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (k + e < K) z[e >> 2] |= (uint32_t)(uint8_t)p[e] << (8 * (e & 3));
        }
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        if (r0 + i >= rows) break;
        uint4 a, b;
        widen4(v[i].x, a.x, a.y);
        widen4(v[i].y, a.z, a.w);
        widen4(v[i].z, b.x, b.y);
        widen4(v[i].w, b.z, b.w);
        uint4* out = to + (r0 + i) * (chunks * 2LL) + c * 2;
        out[0] = a;
        out[1] = b;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) no_columns_kernel(LinearI8Args a) {
  grid_launch_dependents();
  grid_wait_prerequisites();
  const LinearArgs& l = a.l;
  const long long total = (long long)l.M * l.N;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const int n = (int)(i % l.N);
    // (scales that are not finite spoil a sum of no products as well)
    finish<T>(l, 0.f * a.x_scale[i / l.N] * a.w_scale[n], l.bias ? to_f32(static_cast<const T*>(l.bias)[n]) : 0.f,
              i / l.N, n);
  }
}

// Tensor map of [rows][K] integers, rows ld bytes apart: boxes of 64 columns by `box` rows, zeros
// outside.
bool encode(CUtensorMap* m, const void* base, int rows, int K, long long ld, int box, CUtensorMapSwizzle swizzle) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? ld : (K + 15LL) / 16 * 16)};  // (one row's says nothing)
  const cuuint32_t boxes[2] = {kBlockK, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool tma_takes(const LinearArgs& l) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(l.x) | reinterpret_cast<uintptr_t>(l.w);
  auto row = [](long long ld, int rows) { return rows == 1 || (ld % 16 == 0 && ld < (1LL << 40)); };
  return (at & 15) == 0 && row(l.ldx, l.M) && row(l.ldw, l.N);
}

template <int BN, bool kTma, typename T>
cudaError_t launch_of(const LinearI8Args& a, int* status, int split, cudaStream_t s) {
  using F = Fill<BN, kTma>;
  constexpr auto kern = linear_i8_kernel<BN, kTma, T>;
  const cudaError_t e = allow_smem<kern>(F::kSmem);
  if (e != cudaSuccess) return e;
  I8 t;
  t.a = a;
  t.status = status;
  t.n_tiles = (a.l.N + (int)kRowsA - 1) / (int)kRowsA;
  t.k_blocks = (a.l.K + (int)kBlockK - 1) / (int)kBlockK;
  if (kTma && !(encode(&t.tm_w, a.l.w, a.l.N, a.l.K, a.l.ldw, kRowsA, CU_TENSOR_MAP_SWIZZLE_64B) &&
                encode(&t.tm_x, a.l.x, a.l.M, a.l.K, a.l.ldx, BN, CU_TENSOR_MAP_SWIZZLE_NONE)))
    return cudaErrorInvalidValue;
  const long long tiles = (long long)t.n_tiles * ((a.l.M + BN - 1LL) / BN);
  return launch_early(kern, dim3((unsigned)tiles, 1, split), F::kThreads, F::kSmem, split, s, t);
}
template <int BN, bool kTma>
cudaError_t launch(const LinearI8Args& a, int dtype, int* status, int split, cudaStream_t s) {
  return dtype == KDA_F32 ? launch_of<BN, kTma, float>(a, status, split, s)
                          : launch_of<BN, kTma, __nv_bfloat16>(a, status, split, s);
}

// Whether both arrays are widened first.  That costs by M + N and pays by M N, and the other way goes in
// waves of 304 CTAs, two to each of 152 SMs (constants, since the workspace's size must not depend on the
// device).  All with inputs that were not in L2, us, widened first and not:
//  * Rows and bases at 16 bytes: from M N / (M + N) = 544 on (columns 4096, channels 4096: 512 and 640 rows
//    36.4 and 40.1, 33.5 and 59.2; channels 8192: 54.8 and 70.7, 59.2 and 103), from 400 on where the tiles of
//    128 x 128 take a second wave (12288 channels, 384 and 512 rows: 76.6 and 82.5, 60.2 and 117; 24576:
//    134 and 140, 121 and 179).  Few channels of many columns would stay longer (2048 of 12288,
//    1024 rows: 91 and 68), 1024 columns go sooner (4096 channels, 320 rows: 15.5 and 20.6).
//  * Else, where a thread reads its own integers and tiles have 64 tokens: from 65 rows on with more
//    tiles than give four CTAs each, 76 (4095 columns, 12288 channels, 96 and 128 rows: 58 and 59, 122 and 122;
//    4096 channels, 128 and 160 rows, 64 and 96 tiles: 36.8 and 37.0, 36.9 and 65.7; 1499 channels of 1000, 333 and 400
//    rows, 72 and 84 tiles: 15.3 and 14.8, 18.9 and 28.8; 100 channels of 1000, 20,000 rows: 45 and 90).  Up to 64 rows the widened weights would
//    pass through memory for at most a quarter of the time (12288 channels, 64 rows: 55.6 and 70.9).
// What the first rule takes the second takes too: the workspace's size goes by the second.
bool widened(long long M, long long N, bool tma) {
  if (!tma) return M > 64 && (N + 127) / 128 * ((M + 63) / 64) > 76;
  return M * N >= 544 * (M + N) || (M * N >= 400 * (M + N) && (N + 127) / 128 * ((M + 127) / 128) > 304);
}
long long padded(int K) { return (K + 15LL) / 16 * 16; }

}  // namespace

bool linear_i8_tc_takes(int M, int N) { return (N + 127LL) / 128 * ((M + 15LL) / 16) <= 0x7fffffffLL; }

bool linear_i8_tc_needs_workspace(const LinearArgs& l) { return widened(l.M, l.N, tma_takes(l)); }

size_t linear_i8_workspace_bytes(int M, int N, int K) {
  return K > 0 && widened(M, N, false) ? ((size_t)M + N) * padded(K) * 2 : 0;
}

cudaError_t launch_linear_i8_none(const LinearI8Args& a, int dtype, cudaStream_t s) {
  const long long total = (long long)a.l.M * a.l.N, blocks = (total + 255) / 256;
  const unsigned grid = (unsigned)(blocks < 65536 ? blocks : 65536);
  return dtype == KDA_F32 ? launch_early(no_columns_kernel<float>, dim3(grid), 256, 0, 1, s, a)
                          : launch_early(no_columns_kernel<__nv_bfloat16>, dim3(grid), 256, 0, 1, s, a);
}

cudaError_t launch_linear_i8_tc(const LinearI8Args& a, int dtype, void* workspace, int sms, int* status,
                                cudaStream_t s) {
  const LinearArgs& l = a.l;
  const bool tma = tma_takes(l);
  if (widened(l.M, l.N, tma)) {
    const long long Kp = padded(l.K), blocks = ((long long)l.M + l.N + 1) / 2, most = 8LL * sms;
    const cudaError_t e = launch_early(
        widen_kernel, dim3((unsigned)(blocks < most ? blocks : most)), 256, 0, 1, s, static_cast<const int8_t*>(l.x),
        l.ldx, (long long)l.M, static_cast<const int8_t*>(l.w), l.ldw, (long long)l.N, l.K, (int)Kp,
        static_cast<uint4*>(workspace));
    if (e != cudaSuccess) return e;
    LinearI8Args h = a;
    h.l.x = workspace;
    h.l.w = static_cast<char*>(workspace) + (size_t)l.M * Kp * 2;
    h.l.ldx = h.l.ldw = Kp;
    return launch_linear_i8_pair(h, dtype, sms, status, s);
  }
  // K split over the CTAs of a cluster until there are two CTAs per SM.  Tiles of 64 tokens at most
  // where threads read the integers where they are.
  const int k_blocks = (l.K + 63) / 64;
  const int bn = l.M <= 16 ? 16 : l.M <= 32 ? 32 : l.M <= 64 || !tma ? 64 : 128;
  const long long tiles = (l.N + 127LL) / 128 * ((l.M + bn - 1LL) / bn);
  int split = 1;
  while (split < 8 && split * 2 <= k_blocks && tiles * split * 2 <= 2LL * sms) split *= 2;
  switch (bn) {
    case 16: return tma ? launch<16, true>(a, dtype, status, split, s) : launch<16, false>(a, dtype, status, split, s);
    case 32: return tma ? launch<32, true>(a, dtype, status, split, s) : launch<32, false>(a, dtype, status, split, s);
    case 64: return tma ? launch<64, true>(a, dtype, status, split, s) : launch<64, false>(a, dtype, status, split, s);
    default: return launch<128, true>(a, dtype, status, split, s);
  }
}

}  // namespace kda
