// gdr_chain_tc.cu -- the state's walk over the chunks of a sequence on tcgen05, for d_k of 64 or
// 128 and 128 columns of the state (d_v) per CTA.  The algebra and the parts that operands are
// split into are those of gdr_chunked.cu; everything is held transposed, lanes of TMEM = d_v:
//     X^T = S^T K^T,  Y^T = S^T Q^T,  U^T = (V - a X)^T T^T,
//     O^T = b Y^T + U^T P^T,          S^T <- e^{g_C} S^T + (ku U)^T K.
//
// S^T stays in the registers of eight warps (thread = lane of TMEM = row of S^T, two warpgroups
// for the two halves of d_k); the A operands of every product are written to TMEM, the B
// operands lie in shared memory as prep and TMA put them there.  A chunk is a chain of four
// dependent steps, each a conversion by the eight warps and products by the tensor cores:
//     S -> parts | X (then Y) | V - a X -> parts | U | ku U -> parts | S's update
// While the tensor cores work on X the warps store the last chunk's o, while they work on U
// the warps scale Y, and P U runs behind the update.
//
// TMEM columns: the parts of S, whose place the update's product takes when X and Y are done;
// X; two regions that Y and U take in turn (the parts of U lie in U's own place; the last
// chunk's o is read from its Y while the next Y is built in the other); the parts of V - a X,
// then of ku U.  Warpgroup h writes and reads only its own columns of each, so that no barrier
// between the warps is needed.
#include <cuda.h>

#include <mutex>

#include "gdr_chunked.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kStateWarps = 8, kWarpLoad = 8, kWarpMma = 9;
constexpr int kThreads = 320;
constexpr uint32_t kDv = 128;
constexpr uint32_t kXCol = 192, kYuCol = 256, kWCol = 384;  // X; two of 64; 96

template <int DK>
struct Layout {
  static constexpr uint32_t kHalf = DK / 2;            // channels of a warpgroup
  static constexpr uint32_t kSpHalf = 3 * kHalf / 2;   // its columns of S's parts
  // the update's product: 128 channels in the places of the parts, 64 beside them
  static constexpr uint32_t kDCol = DK == 128 ? 0 : 96, kDHalf = DK == 128 ? kSpHalf : kHalf;
  static constexpr uint32_t kRows = kC * DK * 2;        // bytes of a K or Q tile
  static constexpr uint32_t kKAt = kBlock, kQAt = kKAt + kRows, kVAt = kQAt + kRows;
  static constexpr uint32_t kStage = kVAt + kC * kDv * 2;
  static constexpr uint32_t kSmem = 2 * kStage + 1024;
};

struct Chain {
  CUtensorMap tm_q, tm_k, tm_v;
  GdrArgs a;
  const uint8_t* ws;
};

template <int N>
__device__ __forceinline__ void tmem_store(uint32_t col, const uint32_t (&r)[N]) {
  if constexpr (N == 32) tmem_st32(col, r);
  else if constexpr (N == 16) tmem_st16(col, r);
  else tmem_st8(col, r);
}

// TMEM stores of this warp -> the thread that issues the products
__device__ __forceinline__ void hand_over(uint64_t* bar, int lane) {
  tmem_wait_st();
  fence_before_sync();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// 2 N values as parts of N columns each, kStep columns apart
template <int kParts, int N>
__device__ __forceinline__ void store_parts(uint32_t col, uint32_t step, const float* x) {
  uint32_t p[kParts][N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t w[kParts];
    split2<kParts>(x[2 * i], x[2 * i + 1], w);
#pragma unroll
    for (int k = 0; k < kParts; ++k) p[k][i] = w[k];
  }
#pragma unroll
  for (int k = 0; k < kParts; ++k) tmem_store<N>(col + k * step, p[k]);
}

template <int DK>
__global__ void __launch_bounds__(kThreads, 1) gdr_chain_tc_kernel(const __grid_constant__ Chain t) {
  using L = Layout<DK>;
  extern __shared__ uint8_t raw[];
  uint8_t* stages = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[2], empty[2], sp[2], x_done, y_done, v_ready, u_done, y_scaled, ku_ready,
      u_ready, d_done, o_done, drained;
  __shared__ uint32_t tmem_base;

  const GdrArgs& a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = a.dv / (int)kDv;
  const int slice = blockIdx.x % slices, h = blockIdx.x / slices % a.Hv, n = blockIdx.x / slices / a.Hv;
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;  // every warp finds the same
  const int chunks = (t1 - t0 + kC - 1) / kC, base = block_base(t0, n);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
      mbar_init(&sp[i], kStateWarps);
    }
    for (uint64_t* b : {&x_done, &y_done, &u_done, &d_done, &o_done, &drained}) mbar_init(b, 1);
    for (uint64_t* b : {&v_ready, &y_scaled, &ku_ready, &u_ready}) mbar_init(b, kStateWarps);
    mbar_fence_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_base;
  bool ok = true;

  if (warp == kWarpLoad && lane == 0) {
    const int hk = h / (a.Hv / a.Hk);
    int c = 0;
    for (; c < chunks; ++c) {
      const int b = c & 1;
      if (c >= 2 && !mbar_wait(&empty[b], (c / 2 - 1) & 1, kGdrSpins)) {
        ok = false;
        break;
      }
      uint8_t* st = stages + b * L::kStage;
      mbar_arrive_expect_tx(&full[b], L::kStage);
      const int row = t0 + c * kC;
#pragma unroll
      for (int i = 0; i < DK / 64; ++i)
        tma_load_3d(st + L::kKAt + i * 8192, &t.tm_k, i * 64, hk, row, &full[b]);
      bulk_g2s(st, t.ws + ((size_t)(base + c) * a.Hv + h) * kBlock, kBlock, &full[b]);
#pragma unroll
      for (int i = 0; i < DK / 64; ++i)
        tma_load_3d(st + L::kQAt + i * 8192, &t.tm_q, i * 64, hk, row, &full[b]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        tma_load_3d(st + L::kVAt + i * 8192, &t.tm_v, slice * (int)kDv + i * 64, h, row, &full[b]);
    }
    // loads in flight land before shared memory is released
    if (!ok)
      for (int j = max(0, c - 2); j < c; ++j) mbar_wait(&full[j & 1], (j / 2) & 1, kGdrSpins);
  } else if (warp == kWarpMma && lane == 0) {
    constexpr uint32_t idesc = idesc_f16(128, 64, true), idesc_d = idesc_f16(128, 64, true, false, true);
    constexpr uint32_t kSteps = DK / 16;
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && mbar_wait(bar, parity, kGdrSpins);
      fence_after_sync();
      return ok;
    };
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, ph = c & 1;
      const uint32_t st = smem_u32(stages + b * L::kStage);
      const uint32_t ycol = tmem + kYuCol + (c & 1) * 64, ucol = tmem + kYuCol + (1 - (c & 1)) * 64;
      if (!wait(&full[b], (c / 2) & 1)) break;
      // X and Y: K step s = channels 16 s ..; half the channels of each warpgroup at a time
      auto product = [&](uint32_t d, uint32_t rows, uint32_t s, uint32_t k, bool add) {
        const uint32_t half = s / (kSteps / 2), col = half * L::kSpHalf + k * (L::kHalf / 2) + (s % (kSteps / 2)) * 8;
        mma_ts(d, tmem + col, desc_k_sw128(st + rows + (s >> 2) * 8192, (s & 3) * 32), idesc, add);
      };
      bool first = true;
      for (int part_of = 0; part_of < 2 && ok; ++part_of) {
        if (!wait(&sp[part_of], ph)) break;
        for (uint32_t half = 0; half < 2; ++half)
          for (uint32_t i = 0; i < kSteps / 4; ++i)
            for (uint32_t k = 0; k < 3; ++k) {
              product(tmem + kXCol, L::kKAt, half * (kSteps / 2) + part_of * (kSteps / 4) + i, k, !first);
              first = false;
            }
      }
      if (!ok) break;
      mma_commit(&x_done);
      for (uint32_t s = 0; s < kSteps; ++s)
        for (uint32_t k = 0; k < 2; ++k) product(ycol, L::kQAt, s, k, s + k > 0);
      mma_commit(&y_done);
      // U: tokens 16 s .. of V - a X against T's columns
      if (!wait(&v_ready, ph)) break;
      for (uint32_t s = 0; s < 4; ++s)
        for (uint32_t j = 0; j < 3; ++j)
          for (uint32_t k = 0; k < 3 - j; ++k)
            mma_ts(ucol, tmem + kWCol + (s >> 1) * 48 + k * 16 + (s & 1) * 8,
                   desc_k_sw128(st + kT + j * kTile, s * 32), idesc, s + j + k > 0);
      mma_commit(&u_done);
      // the update: ku U against K, tokens contracted
      if (!wait(&ku_ready, ph)) break;
      for (uint32_t half = 0; half < DK / 64; ++half)
        for (uint32_t s = 0; s < 4; ++s)
          for (uint32_t k = 0; k < 3; ++k)
            mma_ts(tmem + L::kDCol + half * L::kDHalf, tmem + kWCol + (s >> 1) * 48 + k * 16 + (s & 1) * 8,
                   desc_mn_sw128(st + L::kKAt + half * 8192, s, 8192), idesc_d, s + k > 0);
      mma_commit(&d_done);
      // P U onto b Y
      if (!wait(&y_scaled, ph) || !wait(&u_ready, ph)) break;
      for (uint32_t s = 0; s < 4; ++s)
        for (uint32_t j = 0; j < 2; ++j)
          for (uint32_t k = 0; k < 2 - j; ++k)
            mma_ts(ycol, ucol + (s >> 1) * 32 + k * 16 + (s & 1) * 8,
                   desc_k_sw128(st + kP + j * kTile, s * 32), idesc, 1);
      mma_commit(&o_done);
      mma_commit(&empty[b]);
    }
    // products in flight end before shared memory and TMEM are released
    mma_commit(&drained);
    mbar_wait(&drained, 0, kGdrSpins);
  } else if (warp < kStateWarps) {
    const int quarter = warp & 3, half = warp >> 2;
    const int dv = quarter * 32 + lane;  // this thread's row of S^T
    const uint32_t lanes = taddr(tmem, quarter * 32, 0);
    const size_t mat = ((size_t)slot * a.Hv + h) * DK * a.dv + (size_t)(half * L::kHalf) * a.dv +
                       slice * kDv + dv;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + (size_t)h * a.dv + slice * kDv + dv;
    const size_t token = (size_t)a.Hv * a.dv;
    float S[L::kHalf];
#pragma unroll
    for (uint32_t i = 0; i < L::kHalf; ++i) S[i] = a.S0 ? a.S0[mat + (size_t)i * a.dv] : 0.f;
    float eG = 1.f;
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, kGdrSpins));
      fence_after_sync();
      return ok;
    };
    // S <- e^{g_C} S + the update's product, 32 (or 16) channels from i on
    auto update = [&](uint32_t i) {
      if constexpr (DK == 128) {
        uint32_t r[32];
        tmem_ld32(lanes + L::kDCol + half * L::kDHalf + i, r);
        tmem_wait_ld();
#pragma unroll
        for (uint32_t j = 0; j < 32; ++j) S[i + j] = fmaf(eG, S[i + j], __uint_as_float(r[j]));
      } else {
        uint32_t r[16];
        tmem_ld16(lanes + L::kDCol + half * L::kDHalf + i, r);
        tmem_wait_ld();
#pragma unroll
        for (uint32_t j = 0; j < 16; ++j) S[i + j] = fmaf(eG, S[i + j], __uint_as_float(r[j]));
      }
    };
    // o of chunk c: this warpgroup's 32 tokens, lanes = neighbouring channels
    auto write_o = [&](int c) {
      uint32_t r[32];
      tmem_ld32(lanes + kYuCol + (c & 1) * 64 + half * 32, r);
      tmem_wait_ld();
      const int row = t0 + c * kC + half * 32;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (row + i < t1) o[(size_t)(row + i) * token] = __float2bfloat16_rn(__uint_as_float(r[i]));
    };

    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, ph = c & 1;
      uint8_t* st = stages + b * L::kStage;
      const float* vec = reinterpret_cast<const float*>(st + kVec) + half * 32;
      const int len = min(kC, t1 - t0 - c * kC);
      if (c > 0 && !wait(&d_done, (c - 1) & 1)) break;
      if (len < kC) {
        // rows behind the last token belong to the next sequence: zeros in their place, seen by
        // the products behind the hand-over below
        if (!wait(&full[b], (c / 2) & 1)) break;
        for (int i = threadIdx.x; i < (kC - len) * 8 * (DK / 64) * 2; i += kStateWarps * 32) {
          const int tile = i / ((kC - len) * 8), j = i % ((kC - len) * 8);
          *reinterpret_cast<uint4*>(st + L::kKAt + tile * 8192 + (len + (j >> 3)) * 128 + (j & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
      }
      // the whole product is read before the parts take its place
      if (c > 0) {
        update(0);
        update(L::kHalf / 2);
      }
      // S as parts, in two halves so that the products start on the first
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        store_parts<3, L::kHalf / 4>(lanes + half * L::kSpHalf + i * (L::kHalf / 4), L::kHalf / 2,
                                     &S[i * L::kHalf / 2]);
        hand_over(&sp[i], lane);
      }
      if (c > 0) {
        if (!wait(&o_done, (c - 1) & 1)) break;
        write_o(c - 1);
      }
      // V - a X
      if (!wait(&full[b], (c / 2) & 1)) break;
      float v[32];
      {
        const __nv_bfloat16* vs = reinterpret_cast<const __nv_bfloat16*>(st + L::kVAt + (dv >> 6) * 8192) +
                                  half * 32 * 64 + (dv & 63);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = half * 32 + i < len ? __bfloat162float(vs[i * 64]) : 0.f;
      }
      if (!wait(&x_done, ph)) break;
      {
        uint32_t r[32];
        tmem_ld32(lanes + kXCol + half * 32, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 va = *reinterpret_cast<const float4*>(vec + i);
          v[i] = fmaf(-va.x, __uint_as_float(r[i]), v[i]);
          v[i + 1] = fmaf(-va.y, __uint_as_float(r[i + 1]), v[i + 1]);
          v[i + 2] = fmaf(-va.z, __uint_as_float(r[i + 2]), v[i + 2]);
          v[i + 3] = fmaf(-va.w, __uint_as_float(r[i + 3]), v[i + 3]);
        }
      }
      store_parts<3, 16>(lanes + kWCol + half * 48, 16, v);
      hand_over(&v_ready, lane);
      // b Y
      if (!wait(&y_done, ph)) break;
      {
        const uint32_t ycol = lanes + kYuCol + (c & 1) * 64 + half * 32;
        uint32_t r[32];
        tmem_ld32(ycol, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 vb = *reinterpret_cast<const float4*>(vec + 64 + i);
          r[i] = __float_as_uint(vb.x * __uint_as_float(r[i]));
          r[i + 1] = __float_as_uint(vb.y * __uint_as_float(r[i + 1]));
          r[i + 2] = __float_as_uint(vb.z * __uint_as_float(r[i + 2]));
          r[i + 3] = __float_as_uint(vb.w * __uint_as_float(r[i + 3]));
        }
        tmem_st32(ycol, r);
        hand_over(&y_scaled, lane);
      }
      // ku U and U
      if (!wait(&u_done, ph)) break;
      {
        const uint32_t ucol = lanes + kYuCol + (1 - (c & 1)) * 64 + half * 32;
        uint32_t r[32];
        tmem_ld32(ucol, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 ku = *reinterpret_cast<const float4*>(vec + 128 + i);
          v[i] = ku.x * __uint_as_float(r[i]);
          v[i + 1] = ku.y * __uint_as_float(r[i + 1]);
          v[i + 2] = ku.z * __uint_as_float(r[i + 2]);
          v[i + 3] = ku.w * __uint_as_float(r[i + 3]);
        }
        eG = vec[192 - half * 32];
        store_parts<3, 16>(lanes + kWCol + half * 48, 16, v);
        hand_over(&ku_ready, lane);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
        store_parts<2, 16>(ucol, 16, v);
        hand_over(&u_ready, lane);
      }
    }
    if (ok && chunks > 0) {
      if (wait(&d_done, (chunks - 1) & 1)) {
        update(0);
        update(L::kHalf / 2);
      }
      if (wait(&o_done, (chunks - 1) & 1)) write_o(chunks - 1);
    }
    if (ok) {
#pragma unroll
      for (uint32_t i = 0; i < L::kHalf; ++i) a.S_T[mat + (size_t)i * a.dv] = S[i];
    }
  }
  if (!ok && lane == 0) atomicExch(a.status, KDA_ERR_TIMEOUT);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// cuTensorMapEncodeTiled, reached through the runtime (no link against the driver library).
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

// Tensor map of [T][H][d] bf16 rows, tokens ld elements apart: boxes of 64 channels of one head
// by 64 tokens.
bool encode(CUtensorMap* m, const void* base, int T, int H, int d, long long ld, bool swizzle) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, 1, kC};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK>
cudaError_t launch(const GdrArgs& a, const uint8_t* ws, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(
      gdr_chain_tc_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<DK>::kSmem);
  if (e != cudaSuccess) return e;
  Chain t;
  t.a = a;
  t.ws = ws;
  if (!encode(&t.tm_k, a.k, a.T_total, a.Hk, DK, a.ldk, true) ||
      !encode(&t.tm_q, a.q, a.T_total, a.Hk, DK, a.ldq, true) ||
      !encode(&t.tm_v, a.v, a.T_total, a.Hv, a.dv, a.ldv, false))
    return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)a.N * a.Hv * (a.dv / (int)kDv);
  gdr_chain_tc_kernel<DK><<<grid, kThreads, Layout<DK>::kSmem, s>>>(t);
  return cudaGetLastError();
}

}  // namespace

bool gdr_chain_tc_takes(const GdrArgs& a) {
  return (a.dk == 64 || a.dk == 128) && a.dv % (int)kDv == 0;
}

cudaError_t launch_gdr_chain_tc(const GdrArgs& a, const uint8_t* ws, cudaStream_t s) {
  return a.dk == 128 ? launch<128>(a, ws, s) : launch<64>(a, ws, s);
}

}  // namespace kda
