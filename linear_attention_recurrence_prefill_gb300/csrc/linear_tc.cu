// linear_tc.cu -- y = act(x w^T + bias) + residual on the tcgen05 tensor cores
// (bf16 data).
//
// The product is taken transposed: D[n][m] = sum_k w[n][k] x[m][k], 128 rows of
// w (the M of the MMA, the lanes of TMEM) by BN rows of x (its N, the columns).
// A lane of the epilogue then owns one output channel n: its bias is one
// register, and for every token the 32 lanes of a warp write 32 neighbouring
// elements of y, and read those of the residual, whatever their alignment.
//
// Six warps: 0-3 the epilogue (each its quarter of the TMEM lanes), 4 issues the
// TMA loads of a ring of stages (64 columns of w and x each, 128-byte swizzle),
// 5 issues the MMAs.
//
// Two forms.
//  * kSplit = false: a persistent grid, one CTA per SM walking the tiles, two
//    accumulators in TMEM so that a tile's epilogue runs beside the next tile's
//    products.
//  * kSplit = true, where there are too few tiles to fill the GPU (few tokens,
//    or a small product): the CTAs of a cluster share one tile, each takes a part
//    of K, and the partial sums meet in distributed shared memory, added in the
//    order of the ranks, so that results repeat to the bit.
#include <cuda.h>

#include <mutex>

#include "linear.cuh"
#include "umma.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kThreads = 192;
constexpr int kWarpLoad = 4, kWarpMma = 5;
constexpr uint32_t kRowsA = 128, kBlockK = 64;
constexpr long long kSpins = 4000000000LL;  // ~2 s of clock cycles

struct Tc {
  CUtensorMap tm_w, tm_x;
  LinearArgs a;
  int* status;
  int n_tiles, m_tiles, k_blocks;
};

// The epilogue of output channel n for the 32 tokens from m on, of which `cols` exist.
// All of the residual is fetched before the first store: y may be the residual, so the
// compiler would not move a load over a store by itself.
__device__ __forceinline__ void finish32(const LinearArgs& a, const uint32_t (&r)[32], float bias,
                                         long long m, int n, int cols) {
  const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(a.residual) + m * a.ldr + n;
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + m * a.ldy + n;
  __nv_bfloat16 add[32];
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < cols) add[j] = res[j * a.ldr];
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) add[j] = __ushort_as_bfloat16(0);
  }
  float z[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(r[j]) + bias;
  // the activation chosen once for all
  auto all = [&](auto f) {
#pragma unroll
    for (int j = 0; j < 32; ++j) z[j] = f(z[j]);
  };
  switch (a.act) {
    case KDA_ACT_RELU: all([](float x) { return activate<true>(x, KDA_ACT_RELU); }); break;
    case KDA_ACT_SILU: all([](float x) { return activate<true>(x, KDA_ACT_SILU); }); break;
    case KDA_ACT_GELU: all([](float x) { return activate<true>(x, KDA_ACT_GELU); }); break;
    case KDA_ACT_GELU_TANH:
      all([](float x) { return activate<true>(x, KDA_ACT_GELU_TANH); });
      break;
    case KDA_ACT_SIGMOID: all([](float x) { return activate<true>(x, KDA_ACT_SIGMOID); }); break;
    default: break;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < cols) y[j * a.ldy] = __float2bfloat16_rn(z[j] + __bfloat162float(add[j]));
}

template <int BN, int kStages>
constexpr uint32_t smem_bytes() {
  return 1024 + kStages * (kRowsA + BN) * kBlockK * 2;
}

template <int BN, int kStages, bool kSplit>
__global__ void __launch_bounds__(kThreads) linear_tc_kernel(const __grid_constant__ Tc t) {
  constexpr uint32_t kStage = (kRowsA + BN) * kBlockK * 2;
  constexpr int kAcc = kSplit ? 1 : 2;  // accumulators in TMEM
  constexpr uint32_t kCols = kAcc * BN <= 32 ? 32 : kAcc * BN <= 64 ? 64 : kAcc * BN <= 128 ? 128
                             : kAcc * BN <= 256 ? 256 : 512;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[kAcc], acc_empty[kAcc], drained;
  __shared__ uint32_t tmem_base;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kSplit ? cluster_ctarank() : 0, ranks = kSplit ? gridDim.z : 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(&drained, 1);
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

  // tiles of this CTA, and its part of K
  const int tiles = t.n_tiles * t.m_tiles;
  const int first = kSplit ? blockIdx.x + t.n_tiles * blockIdx.y : blockIdx.x;
  const int step = kSplit ? tiles : gridDim.x;
  const int kb0 = (int)((long long)t.k_blocks * rank / ranks);
  const int kb1 = (int)((long long)t.k_blocks * (rank + 1) / ranks);

  bool ok = true;
  if (warp == kWarpLoad && lane == 0) {
    int it = 0;
    for (int tile = first; tile < tiles && ok; tile += step) {
      const int n0 = tile % t.n_tiles * (int)kRowsA, m0 = tile / t.n_tiles * BN;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % kStages;
        if (it >= kStages && !mbar_wait(&empty[s], (it / kStages - 1) & 1, kSpins)) {
          ok = false;
          break;
        }
        uint8_t* dst = ring + s * kStage;
        mbar_arrive_expect_tx(&full[s], kStage);
        tma_load_2d(dst, &t.tm_w, kb * (int)kBlockK, n0, &full[s]);
        tma_load_2d(dst + kRowsA * kBlockK * 2, &t.tm_x, kb * (int)kBlockK, m0, &full[s]);
      }
    }
    // a wait that gave up: the loads in flight land before shared memory is released
    if (!ok)
      for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
        mbar_wait(&full[j % kStages], (j / kStages) & 1, kSpins);
  } else if (warp == kWarpMma && lane == 0) {
    constexpr uint32_t idesc = idesc_f16(kRowsA, BN, true);
    int it = 0, n = 0;
    for (int tile = first; tile < tiles && ok; tile += step, ++n) {
      const int acc = n % kAcc;
      if (n >= kAcc && !mbar_wait(&acc_empty[acc], (n / kAcc - 1) & 1, kSpins)) {
        ok = false;
        break;
      }
      fence_after_sync();
      const uint32_t d = tmem + acc * BN;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % kStages;
        if (!mbar_wait(&full[s], (it / kStages) & 1, kSpins)) {
          ok = false;
          break;
        }
        fence_after_sync();
        const uint32_t wa = smem_u32(ring + s * kStage), xa = wa + kRowsA * kBlockK * 2;
#pragma unroll
        for (uint32_t k = 0; k < kBlockK / 16; ++k)
          mma_ss(d, desc_k_sw128(wa, k * 32), desc_k_sw128(xa, k * 32), idesc,
                 kb > kb0 || k > 0);
        mma_commit(&empty[s]);
      }
      if (!ok) break;
      mma_commit(&acc_full[acc]);
    }
    if (!ok) {  // products in flight end before shared memory and TMEM are released
      mma_commit(&drained);
      mbar_wait(&drained, 0, kSpins);
    }
  } else if (warp < 4) {
    const __nv_bfloat16* bias = static_cast<const __nv_bfloat16*>(t.a.bias);
    int i = 0;
    for (int tile = first; tile < tiles; tile += step, ++i) {
      const int acc = i % kAcc;
      const int n = tile % t.n_tiles * (int)kRowsA + warp * 32 + lane;
      const long long m0 = (long long)(tile / t.n_tiles) * BN;
      const int cols = t.a.M - m0 < BN ? (int)(t.a.M - m0) : BN;
      ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[acc], (i / kAcc) & 1, kSpins));
      if (!ok) break;
      fence_after_sync();
      const uint32_t d = taddr(tmem, warp * 32, acc * BN);
      if constexpr (kSplit) {
        // partial sums [column][channel] over the ring, whose loads and products are done
        float* part = reinterpret_cast<float*>(ring) + warp * 32 + lane;
#pragma unroll 1
        for (int c = 0; c < BN; c += 16) {
          uint32_t r[16];
          tmem_ld16(d + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) part[(c + j) * (int)kRowsA] = __uint_as_float(r[j]);
        }
      } else {
        const float b = bias && n < t.a.N ? to_f32(bias[n]) : 0.f;
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          uint32_t r[32];
          tmem_ld32(d + c, r);
          tmem_wait_ld();
          if (c + 32 >= cols) {  // the accumulator is in registers: its place is free
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
          }
          if (n < t.a.N) finish32(t.a, r, b, m0 + c, n, cols - c);
        }
      }
    }
  }
  if (!ok && lane == 0) atomicExch(t.status, KDA_ERR_TIMEOUT);

  if constexpr (kSplit) {
    // every rank adds up its share of the tile's elements over all ranks; a CTA that gave up
    // takes part in the barriers all the same
    __syncwarp();
    cluster_sync();
    if (warp < 4) {
      const __nv_bfloat16* bias = static_cast<const __nv_bfloat16*>(t.a.bias);
      const int n = blockIdx.x * (int)kRowsA + warp * 32 + lane;
      const long long m0 = (long long)blockIdx.y * BN;
      const int cols = t.a.M - m0 < BN ? (int)(t.a.M - m0) : BN;
      const float b = bias && n < t.a.N ? to_f32(bias[n]) : 0.f;
      const uint32_t part = smem_u32(ring) + (warp * 32 + lane) * 4;
      for (int c = rank; c < cols; c += ranks) {
        float z = 0.f;
        for (uint32_t r = 0; r < ranks; ++r)
          z += ld_cluster_f32(map_to_rank(part + c * kRowsA * 4, r));
        if (n < t.a.N) finish<__nv_bfloat16>(t.a, z, b, m0 + c, n);
      }
    }
    cluster_sync();  // no CTA leaves while its sums are read
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kWarpMma) tmem_dealloc(tmem, kCols);
}

// cuTensorMapEncodeTiled, reached through the runtime (no link against the
// driver library).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// Tensor map of a [rows][K] bf16 array, rows ld elements apart: boxes of 64
// columns by `box` rows, 128-byte swizzle, zeros outside.
bool encode(CUtensorMap* m, const void* base, int rows, int K, long long ld, int box) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t boxes[2] = {kBlockK, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  static int count[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (count[dev] == 0) cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev);
  return count[dev] > 0 ? count[dev] : 152;
}

template <int BN, int kStages, bool kSplit>
cudaError_t launch(const LinearArgs& a, int* status, int split, cudaStream_t s) {
  constexpr auto kern = linear_tc_kernel<BN, kStages, kSplit>;
  static_assert(!kSplit || kStages * (kRowsA + BN) * kBlockK * 2 >= BN * kRowsA * 4,
                "the partial sums fit in the ring");
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes<BN, kStages>());
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
  Tc t;
  t.a = a;
  t.status = status;
  t.n_tiles = (a.N + (int)kRowsA - 1) / (int)kRowsA;
  t.m_tiles = (a.M + BN - 1) / BN;
  t.k_blocks = (a.K + (int)kBlockK - 1) / (int)kBlockK;
  if (!encode(&t.tm_w, a.w, a.N, a.K, a.ldw, kRowsA) || !encode(&t.tm_x, a.x, a.M, a.K, a.ldx, BN))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<BN, kStages>();
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (kSplit) {
    cfg.gridDim = dim3(t.n_tiles, t.m_tiles, split);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = split;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  } else {
    const long long tiles = (long long)t.n_tiles * t.m_tiles;
    const int sms = sm_count();
    cfg.gridDim = dim3((unsigned)(tiles < sms ? tiles : sms));
  }
  return cudaLaunchKernelEx(&cfg, kern, t);
}

}  // namespace

bool linear_tc_takes(const LinearArgs& a, int dtype) {
  if (dtype != KDA_BF16 || a.K < 1) return false;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w);
  return (at & 15) == 0 && a.ldx % 8 == 0 && a.ldw % 8 == 0 && a.ldx < (1LL << 38) &&
         a.ldw < (1LL << 38);
}

cudaError_t launch_linear_tc(const LinearArgs& a, int* status, cudaStream_t s) {
  const long long n_tiles = (a.N + 127LL) / 128;
  const int k_blocks = (a.K + 63) / 64, sms = sm_count();
  // Tiles of 256 tokens where they fill the SMs; else smaller ones, K split over the CTAs of a
  // cluster until there are two CTAs per SM.
  if (n_tiles * ((a.M + 255LL) / 256) >= sms) return launch<256, 4, false>(a, status, 1, s);
  const int bn = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
  const long long tiles = n_tiles * ((a.M + bn - 1) / bn);
  int split = 1;
  while (split < 8 && split * 2 <= k_blocks && tiles * split * 2 <= 2LL * sms) split *= 2;
  switch (bn) {
    case 16: return launch<16, 6, true>(a, status, split, s);
    case 32: return launch<32, 5, true>(a, status, split, s);
    case 64: return launch<64, 4, true>(a, status, split, s);
    default: return launch<128, 3, true>(a, status, split, s);
  }
}

}  // namespace kda
