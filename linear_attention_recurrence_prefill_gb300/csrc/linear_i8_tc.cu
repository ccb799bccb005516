// linear_i8_tc.cu -- y = act(x_scale w_scale (x w^T) + bias) + residual for 8-bit
// integers x and w, on the tcgen05 tensor cores.
//
// This GPU multiplies 8-bit integers far below its rate for 16-bit floats, and every such
// integer is an fp16 number: the products are taken in fp16 with fp32 sums, which are exact below
// 2^24.  So what 8 bits save is memory, and the integers are widened on their way:
//  * few tiles (few tokens, or a small product; bound by reading w): linear_i8_kernel, where
//    eight warps fetch the integers into shared memory, widen them there and lay them out as the
//    tiles that the MMAs read.  The CTAs of a cluster share a tile of 128 channels, each takes a
//    part of K.
//  * many: both arrays are widened into the workspace first, once, and the product is that of
//    kda_linear's pairs of CTAs.  Widened in the product, w would be taken through shared memory
//    once more for every 256 tokens, which the tensor cores' own reads leave no room for.
#include "linear_i8.cuh"
#include "linear_join.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr uint32_t kRowsA = kJoinRows, kBlockK = 64;
constexpr int kFill = 8, kThreads = (kFill + 1) * 32;  // warps that widen, and one that issues the MMAs
constexpr uint32_t kAlign = 1024;                      // the swizzled tiles' alignment
constexpr long long kSpins = 4000000000LL;             // ~2 s of clock cycles

struct I8 {
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

// What a CTA's 256 filling threads fetch per block of 64 columns: the 16 bytes of a row of w or x,
// four neighbouring threads a row; in pieces of 16 aligned bytes, two where rows are not aligned.
template <int BN, bool kAligned>
struct Fill {
  static constexpr int kChunks = ((int)kRowsA + BN + 63) / 64;  // per thread
  static constexpr int kPieces = kAligned ? 1 : 2;
  static constexpr int kRaw = kAligned ? (BN > 64 ? 3 : 4) : 2;  // blocks on their way or landed
  static constexpr uint32_t kRawBlock = kChunks * kPieces * kFill * 32 * 16;
  static constexpr uint32_t kTile = (kRowsA + BN) * kBlockK * 2;
  static constexpr int kTiles = 2;  // widened blocks
  static constexpr uint32_t kSmem = kAlign + kTiles * kTile + kRaw * kRawBlock;
};

template <int BN, bool kAligned, typename T>
__global__ void __launch_bounds__(kThreads) linear_i8_kernel(const __grid_constant__ I8 t) {
  using F = Fill<BN, kAligned>;
  constexpr uint32_t kCols = BN <= 32 ? 32 : BN <= 64 ? 64 : 128;
  static_assert(F::kTiles * F::kTile >= BN * kRowsA * 4, "the partial sums fit in the tiles");
  extern __shared__ uint8_t raw_smem[];
  uint8_t* tiles = raw_smem + ((kAlign - (smem_u32(raw_smem) & (kAlign - 1))) & (kAlign - 1));
  uint8_t* raw = tiles + F::kTiles * F::kTile;
  __shared__ uint64_t full[F::kTiles], empty[F::kTiles], done;
  __shared__ uint32_t tmem_base;

  const LinearArgs& l = t.a.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), ranks = gridDim.z;
  if (threadIdx.x == 0) {
    for (int i = 0; i < F::kTiles; ++i) {
      mbar_init(&full[i], kFill);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    mbar_fence_init();
  }
  if (warp == kFill) {
    tmem_alloc(&tmem_base, kCols);
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

  bool ok = true;
  if (warp < kFill) {
    const int tid = threadIdx.x;
    // this thread's rows, by chunk: the address of their column 16 (tid % 4), whether they exist,
    // and the place of their two pieces of eight columns in a tile
    const int8_t* row[F::kChunks];
    bool in[F::kChunks];
#pragma unroll
    for (int i = 0; i < F::kChunks; ++i) {
      const int r = (tid + i * kFill * 32) / 4;
      const bool of_x = r >= (int)kRowsA;
      const long long at = of_x ? (long long)m0 + r - (int)kRowsA : (long long)n0 + r;
      in[i] = r < (int)kRowsA + BN && at < (of_x ? l.M : l.N);
      row[i] = (of_x ? static_cast<const int8_t*>(l.x) + at * l.ldx : static_cast<const int8_t*>(l.w) + at * l.ldw) +
               tid % 4 * 16;
    }
    const uint32_t mine = smem_u32(raw) + tid * 16;
    auto fetch = [&](int it) {
      if (it < blocks) {
        const long long k = (it * (long long)ranks + rank) * kBlockK;
        const int left = (int)min(16LL, l.K - k - tid % 4 * 16);  // columns of this thread's that exist
        const uint32_t to = mine + it % F::kRaw * F::kRawBlock;
#pragma unroll
        for (int i = 0; i < F::kChunks; ++i) {
          if (kAligned) {
            const bool some = in[i] && left > 0;
            cp_async16(to + i * kFill * 32 * 16, some ? row[i] + k : static_cast<const int8_t*>(l.w), some ? left : 0);
          } else {
            // the aligned pieces around the 16 bytes, up to the end of the row (zeros behind it): their
            // bytes before the 16 are not used, but those before the array are not touched either
            const int8_t* p = row[i] + k;
            const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15;
            const bool of_x = (tid + i * kFill * 32) / 4 >= (int)kRowsA;
            const int8_t* lo = static_cast<const int8_t*>(of_x ? l.x : l.w);
            const int have = in[i] && left > 0 ? (int)off + left : 0;
            const uint32_t at = to + i * 2 * kFill * 32 * 16;
            if (have > 0 && p - off < lo) {
              for (int e = 0; e < 16; ++e)
                raw[at - smem_u32(raw) + e] = e < have && p - off + e >= lo ? (uint8_t)p[e - (int)off] : 0;
            } else {
              cp_async16(at, have > 0 ? p - off : reinterpret_cast<const int8_t*>(reinterpret_cast<uintptr_t>(l.w) & ~(uintptr_t)15),
                         have > 16 ? 16 : have);
            }
            cp_async16(at + kFill * 32 * 16,
                       have > 16 ? p - off + 16 : reinterpret_cast<const int8_t*>(reinterpret_cast<uintptr_t>(l.w) & ~(uintptr_t)15),
                       have > 16 ? have - 16 : 0);
          }
        }
      }
      cp_async_commit();
    };
    for (int it = 0; it < F::kRaw - 1; ++it) fetch(it);
    for (int it = 0; it < blocks; ++it) {
      const int s = it % F::kTiles;
      fetch(it + F::kRaw - 1);
      cp_async_wait_group<F::kRaw - 1>();  // this thread's own pieces of block `it`
      if (it >= F::kTiles)
        ok = __all_sync(0xffffffffu, mbar_wait_soon(&empty[s], (it / F::kTiles - 1) & 1, kSpins));
      if (!ok) break;
      const uint8_t* from = raw + it % F::kRaw * F::kRawBlock + tid * 16;
      uint8_t* tile = tiles + s * F::kTile;
      const long long k = (it * (long long)ranks + rank) * kBlockK;
#pragma unroll
      for (int i = 0; i < F::kChunks; ++i) {
        const int r = (tid + i * kFill * 32) / 4;
        if (((int)kRowsA + BN) % 64 != 0 && r >= (int)kRowsA + BN) break;
        const bool of_x = r >= (int)kRowsA;
        uint4 v = *reinterpret_cast<const uint4*>(from + i * F::kPieces * kFill * 32 * 16);
        if (!kAligned) {
          const uint4 w = *reinterpret_cast<const uint4*>(from + (2 * i + 1) * kFill * 32 * 16);
          v = shift_bytes(v, w, (uint32_t)(reinterpret_cast<uintptr_t>(row[i]) + k) & 15);
        }
        uint4 a, b;
        widen4(v.x, a.x, a.y);
        widen4(v.y, a.z, a.w);
        widen4(v.z, b.x, b.y);
        widen4(v.w, b.z, b.w);
        const uint32_t rr = of_x ? r - kRowsA : r;
        uint8_t* to = tile + (of_x ? kRowsA * kBlockK * 2 : 0);
        const uint32_t c = tid % 4 * 2;
        *reinterpret_cast<uint4*>(to + sw128_chunk(rr, c, 0)) = a;
        *reinterpret_cast<uint4*>(to + sw128_chunk(rr, c + 1, 0)) = b;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
    }
    cp_async_wait_all();
    // Done behind all of this CTA's blocks, each of which has a wait of its own that gives up (the
    // MMA warp then signals all the same): a block takes some 300 to 5,000 cycles.
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&done, 0, 3 * kSpins + (long long)blocks * 65536));
    fence_after_sync();
  } else {
    const uint32_t lead = elect_leader();
    constexpr uint32_t idesc = idesc_f16(kRowsA, BN, false);
    for (int it = 0; it < blocks; ++it) {
      const int s = it % F::kTiles;
      ok = __all_sync(0xffffffffu, mbar_wait_soon(&full[s], (it / F::kTiles) & 1, kSpins));
      if (!ok) break;
      fence_after_sync();
      const uint32_t at = smem_u32(tiles + s * F::kTile);
      const uint64_t wd = desc_k_sw128(at, 0), xd = desc_k_sw128(at + kRowsA * kBlockK * 2, 0);
#pragma unroll
      for (uint32_t k = 0; k < kBlockK / 16; ++k)
        mma_ss_if(lead, tmem, wd + (k * 32 >> 4), xd + (k * 32 >> 4), idesc, it > 0 || k > 0);
      mma_commit_if(lead, &empty[s]);
    }
    // everything issued is complete before the tiles or TMEM are used again, or released
    mma_commit_if(lead, &done);
    mbar_wait(&done, 0, kSpins);
  }
  __syncthreads();  // no thread widens into the tiles any more
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
      z.x = z.x * xs * ws.x;
      z.y = z.y * xs * ws.y;
      z.z = z.z * xs * ws.z;
      z.w = z.w * xs * ws.w;
      finish4<T>(l, wide, z, b, (long long)m0 + c, n);
    });
  }
  fence_before_sync();
  cluster_sync();  // no CTA leaves while its sums are read
  fence_after_sync();
  if (warp == kFill) tmem_dealloc(tmem, kCols);
}

// [rows][K] integers, rows ld bytes apart, as fp16 with rows of Kp elements (a multiple of 8, zeros
// behind K): a thread takes eight columns at a time.
__global__ void __launch_bounds__(256) widen_kernel(const int8_t* x, long long ldx, long long rows_x, const int8_t* w,
                                                    long long ldw, long long rows_w, int K, int Kp, uint4* to) {
  grid_launch_dependents();
  grid_wait_prerequisites();
  const int groups = Kp / 8;
  const long long total = (rows_x + rows_w) * groups;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long r = i / groups;
    const int k = (int)(i - r * groups) * 8;
    const int8_t* p = (r < rows_x ? x + r * ldx : w + (r - rows_x) * ldw) + k;
    uint32_t v[2] = {0, 0};
    if (k + 8 <= K && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      v[0] = q.x;
      v[1] = q.y;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < K) v[e >> 2] |= (uint32_t)(uint8_t)p[e] << (8 * (e & 3));
    }
    uint4 z;
    widen4(v[0], z.x, z.y);
    widen4(v[1], z.z, z.w);
    to[i] = z;
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

template <int BN, bool kAligned, typename T>
cudaError_t launch_of(const LinearI8Args& a, int* status, int split, cudaStream_t s) {
  using F = Fill<BN, kAligned>;
  constexpr auto kern = linear_i8_kernel<BN, kAligned, T>;
  const cudaError_t e = allow_smem<kern>(F::kSmem);
  if (e != cudaSuccess) return e;
  I8 t;
  t.a = a;
  t.status = status;
  t.n_tiles = (a.l.N + (int)kRowsA - 1) / (int)kRowsA;
  t.k_blocks = (a.l.K + (int)kBlockK - 1) / (int)kBlockK;
  const long long tiles = (long long)t.n_tiles * ((a.l.M + BN - 1LL) / BN);
  return launch_early(kern, dim3((unsigned)tiles, 1, split), kThreads, F::kSmem, split, s, t);
}
template <int BN>
cudaError_t launch(const LinearI8Args& a, int dtype, bool is_aligned, int* status, int split, cudaStream_t s) {
  if (dtype == KDA_F32)
    return is_aligned ? launch_of<BN, true, float>(a, status, split, s) : launch_of<BN, false, float>(a, status, split, s);
  return is_aligned ? launch_of<BN, true, __nv_bfloat16>(a, status, split, s)
                    : launch_of<BN, false, __nv_bfloat16>(a, status, split, s);
}

// Whether both arrays are widened first: where pairs of CTAs have tiles for half of the SMs at least.
bool widened(int M, int N, int sms) { return (N + 255LL) / 256 * ((M + 127LL) / 128) >= sms / 4; }
long long padded(int K) { return (K + 7LL) / 8 * 8; }

}  // namespace

bool linear_i8_tc_takes(int M, int N) { return (N + 127LL) / 128 * ((M + 15LL) / 16) <= 0x7fffffffLL; }

size_t linear_i8_workspace_bytes(int M, int N, int K, int sms) {
  return K > 0 && widened(M, N, sms) ? ((size_t)M + N) * padded(K) * 2 : 0;
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
  if (widened(l.M, l.N, sms)) {
    const long long Kp = padded(l.K), total = ((long long)l.M + l.N) * (Kp / 8);
    const long long blocks = (total + 255) / 256, most = 8LL * sms;
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
  const uintptr_t at = reinterpret_cast<uintptr_t>(l.x) | reinterpret_cast<uintptr_t>(l.w);
  const bool is_aligned = (at & 15) == 0 && (l.ldx % 16 == 0 || l.M == 1) && (l.ldw % 16 == 0 || l.N == 1);
  // K split over the CTAs of a cluster until there are two CTAs per SM
  const int k_blocks = (l.K + 63) / 64;
  const int bn = l.M <= 16 ? 16 : l.M <= 32 ? 32 : l.M <= 64 ? 64 : 128;
  const long long tiles = (l.N + 127LL) / 128 * ((l.M + bn - 1LL) / bn);
  int split = 1;
  while (split < 8 && split * 2 <= k_blocks && tiles * split * 2 <= 2LL * sms) split *= 2;
  switch (bn) {
    case 16: return launch<16>(a, dtype, is_aligned, status, split, s);
    case 32: return launch<32>(a, dtype, is_aligned, status, split, s);
    case 64: return launch<64>(a, dtype, is_aligned, status, split, s);
    default: return launch<128>(a, dtype, is_aligned, status, split, s);
  }
}

}  // namespace kda
