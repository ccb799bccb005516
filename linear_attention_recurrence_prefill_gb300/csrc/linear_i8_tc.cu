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
#include "tensor_map.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr uint32_t kRowsA = kJoinRows, kBlockK = 64;
// warps that widen, one that issues the MMAs and, where TMA can take the arrays, one that loads
constexpr int kFill = 8, kMma = 8, kLoad = 9;
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

// The integers of a block of 64 columns: rows of w, then of x, in chunks of 16 bytes, four to a row;
// thread t of the 256 that widen has chunks t, t + 256, ...  By TMA where it takes the arrays (rows
// and bases at 16 bytes); else each thread copies its own, in two aligned pieces around each.
template <int BN, bool kTma>
struct Fill {
  static constexpr int kThreads = (kFill + (kTma ? 2 : 1)) * 32;
  static constexpr int kChunks = ((int)kRowsA + BN + 63) / 64;  // per thread
  static constexpr int kPieces = kTma ? 1 : 2;
  static constexpr int kRaw = kTma ? (BN > 64 ? 3 : 4) : 2;  // blocks on their way or landed
  static constexpr uint32_t kRawBlock = kChunks * kPieces * kFill * 32 * 16;
  static constexpr uint32_t kTile = (kRowsA + BN) * kBlockK * 2;
  static constexpr int kTiles = 2;  // widened blocks
  static constexpr uint32_t kSmem = kAlign + kTiles * kTile + kRaw * kRawBlock;
};

template <int BN, bool kTma, typename T>
__global__ void __launch_bounds__(Fill<BN, kTma>::kThreads) linear_i8_kernel(const __grid_constant__ I8 t) {
  using F = Fill<BN, kTma>;
  constexpr uint32_t kCols = BN <= 32 ? 32 : BN <= 64 ? 64 : 128;
  static_assert(F::kTiles * F::kTile >= BN * kRowsA * 4, "the partial sums fit in the tiles");
  extern __shared__ uint8_t raw_smem[];
  uint8_t* tiles = raw_smem + ((kAlign - (smem_u32(raw_smem) & (kAlign - 1))) & (kAlign - 1));
  uint8_t* raw = tiles + F::kTiles * F::kTile;
  __shared__ uint64_t full[F::kTiles], empty[F::kTiles], landed[F::kRaw], taken[F::kRaw], done;
  __shared__ uint32_t tmem_base;

  const LinearArgs& l = t.a.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), ranks = gridDim.z;
  if (threadIdx.x == 0) {
    for (int i = 0; i < F::kTiles; ++i) {
      mbar_init(&full[i], kFill);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < F::kRaw; ++i) {
      mbar_init(&landed[i], 1);
      mbar_init(&taken[i], kFill);
    }
    mbar_init(&done, 1);
    mbar_fence_init();
  }
  if (warp == kMma) {
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
    // this thread's rows, by chunk: the address of their column 16 (tid % 4), and whether they exist
    const int8_t* row[F::kChunks];
    bool in[F::kChunks];
    auto fetch = [&](int it) {
      if constexpr (!kTma) {
        if (it < blocks) {
          const long long k = (it * (long long)ranks + rank) * kBlockK;
          const int left = (int)min(16LL, l.K - k - tid % 4 * 16);  // columns of this thread's that exist
          const uint32_t to = smem_u32(raw) + tid * 16 + it % F::kRaw * F::kRawBlock;
          const int8_t* const nothing =
              reinterpret_cast<const int8_t*>(reinterpret_cast<uintptr_t>(l.w) & ~(uintptr_t)15);
#pragma unroll
          for (int i = 0; i < F::kChunks; ++i) {
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
              cp_async16(at, have > 0 ? p - off : nothing, have > 16 ? 16 : have);
            }
            cp_async16(at + kFill * 32 * 16, have > 16 ? p - off + 16 : nothing, have > 16 ? have - 16 : 0);
          }
        }
        cp_async_commit();
      }
    };
    if constexpr (!kTma) {
#pragma unroll
      for (int i = 0; i < F::kChunks; ++i) {
        const int r = (tid + i * kFill * 32) / 4;
        const bool of_x = r >= (int)kRowsA;
        const long long at = of_x ? (long long)m0 + r - (int)kRowsA : (long long)n0 + r;
        in[i] = r < (int)kRowsA + BN && at < (of_x ? l.M : l.N);
        row[i] = (of_x ? static_cast<const int8_t*>(l.x) + at * l.ldx : static_cast<const int8_t*>(l.w) + at * l.ldw) +
                 tid % 4 * 16;
      }
    }
    for (int it = 0; it < F::kRaw - 1; ++it) fetch(it);
    for (int it = 0; it < blocks; ++it) {
      const int s = it % F::kTiles;
      if constexpr (kTma) {
        ok = mbar_wait_soon(&landed[it % F::kRaw], (it / F::kRaw) & 1, kSpins);
      } else {
        fetch(it + F::kRaw - 1);
        cp_async_wait_group<F::kRaw - 1>();  // this thread's own pieces of block `it`
      }
      if (ok && it >= F::kTiles) ok = mbar_wait_soon(&empty[s], (it / F::kTiles - 1) & 1, kSpins);
      ok = __all_sync(0xffffffffu, ok);
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
        if (!kTma) {
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
      if (lane == 0) {
        mbar_arrive(&full[s]);
        if (kTma) mbar_arrive(&taken[it % F::kRaw]);
      }
    }
    cp_async_wait_all();
    // Done behind all of this CTA's blocks, each of which has a wait of its own that gives up (the
    // MMA warp then signals all the same): a block takes some 300 to 5,000 cycles.
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&done, 0, 3 * kSpins + (long long)blocks * 65536));
    fence_after_sync();
  } else if (kTma && warp == kLoad) {
    if (lane == 0) {
      int it = 0;
      for (; it < blocks; ++it) {
        const int s = it % F::kRaw, x = (it * (int)ranks + (int)rank) * (int)kBlockK;
        if (it >= F::kRaw && !mbar_wait_soon(&taken[s], (it / F::kRaw - 1) & 1, kSpins)) {
          ok = false;
          break;
        }
        uint8_t* to = raw + s * F::kRawBlock;
        mbar_arrive_expect_tx(&landed[s], (kRowsA + BN) * kBlockK);
        tma_load_2d(to, &t.tm_w, x, n0, &landed[s]);
        tma_load_2d(to + kRowsA * kBlockK, &t.tm_x, x, m0, &landed[s]);
      }
      // a wait that gave up, here or of the warps that widen: the loads in flight land before shared
      // memory is released
      for (int j = it > F::kRaw ? it - F::kRaw : 0; j < it; ++j)
        mbar_wait(&landed[j % F::kRaw], (j / F::kRaw) & 1, kSpins);
    }
    __syncwarp();
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
  if (warp == kMma) tmem_dealloc(tmem, kCols);
}

// [rows][K] integers, rows ld bytes apart, as fp16 with rows of Kp elements (a multiple of 16, zeros
// behind K), x's rows and then w's: a thread takes 16 columns of four rows at a time.
__global__ void __launch_bounds__(256) widen_kernel(const int8_t* x, long long ldx, long long rows_x, const int8_t* w,
                                                    long long ldw, long long rows_w, int K, int Kp, uint4* to) {
  constexpr int kFlight = 4;
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
bool encode(CUtensorMap* m, const void* base, int rows, int K, long long ld, int box) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? ld : (K + 15LL) / 16 * 16)};  // (one row's says nothing)
  const cuuint32_t boxes[2] = {kBlockK, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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
  if (kTma && !(encode(&t.tm_w, a.l.w, a.l.N, a.l.K, a.l.ldw, kRowsA) &&
                encode(&t.tm_x, a.l.x, a.l.M, a.l.K, a.l.ldx, BN)))
    return cudaErrorInvalidValue;
  const long long tiles = (long long)t.n_tiles * ((a.l.M + BN - 1LL) / BN);
  return launch_early(kern, dim3((unsigned)tiles, 1, split), F::kThreads, F::kSmem, split, s, t);
}
template <int BN, bool kTma>
cudaError_t launch(const LinearI8Args& a, int dtype, int* status, int split, cudaStream_t s) {
  return dtype == KDA_F32 ? launch_of<BN, kTma, float>(a, status, split, s)
                          : launch_of<BN, kTma, __nv_bfloat16>(a, status, split, s);
}

// Whether both arrays are widened first: where pairs of CTAs have tiles for half of the SMs at least.
bool widened(int M, int N, int sms) { return (N + 255LL) / 256 * ((M + 127LL) / 128) >= sms / 4; }
long long padded(int K) { return (K + 15LL) / 16 * 16; }

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
    const long long Kp = padded(l.K), blocks = ((long long)l.M + l.N + 3) / 4, most = 8LL * sms;
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
  // where threads copy the integers, so that two CTAs fit on an SM.
  const bool tma = tma_takes(l);
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
