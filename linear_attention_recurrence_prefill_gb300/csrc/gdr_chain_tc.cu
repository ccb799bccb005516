// gdr_chain_tc.cu -- the state's walk over the chunks of a sequence on tcgen05, for d_k of 64 or
// 128 and 128 columns of the state (d_v) per CTA.  The algebra and the parts that operands are
// split into are those of gdr_chunked.cu; everything is held transposed, lanes of TMEM = d_v:
//     X^T = S^T K^T,  Y^T = S^T Q^T,  U^T = (V - a X)^T T^T,
//     O^T = b Y^T + U^T P^T,          S^T <- e^{g_C} S^T + (ku U)^T K.
//
// S^T stays in the registers of eight warps (thread = lane of TMEM = row of S^T, two warpgroups
// for the two halves of d_k); the A operands of every product are written to TMEM, the B
// operands lie in shared memory as prep and TMA put them there.  A chunk is a chain of
// dependent steps, conversions by the eight warps and products by the tensor cores in turn:
//     S -> parts | X and Y | V - a X -> parts | U | ku U -> parts | S's update
// While the tensor cores work on X and Y the warps store the last chunk's o, while they work on
// U the warps scale Y, and P U runs behind the update.  A product costs what its A operand takes to be fetched, N = 64 as much
// as N = 128, so X and Y are one product against [K; Q].
//
// TMEM columns (d_k = 128): 0-191 the parts of S, the first two of which lie where the same
// warpgroup's half of the update's product comes (0-127), the third (128-191) where V - a X and
// ku U go with 192-223; from 224 two regions in turn: X, then U, then its parts; Y, then o.
// A warpgroup writes and reads only its own columns, so that no barrier between the warps is
// needed.
#include <cuda.h>

#include <mutex>

#include "gdr_chunked.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kStateWarps = 8, kWarpLoad = 8, kWarpMma = 9;
constexpr int kThreads = 320;
constexpr uint32_t kDv = 128;
constexpr uint32_t kVCol = 128, kVCol2 = 192, kXyCol = 224;

template <int DK>
struct Layout {
  static constexpr uint32_t kHalf = DK / 2;        // channels of a warpgroup
  static constexpr uint32_t kPart = kHalf / 2;     // TMEM columns of one part of them
  static constexpr uint32_t kThird = 2 * DK / 2;   // where the third parts of S begin
  static constexpr uint32_t kRows = kC * 128;      // bytes of 64 rows of 64 channels
  static constexpr uint32_t kKqAt = kBlock;        // 64 channels of K, then of Q; the next 64
  static constexpr uint32_t kVAt = kKqAt + 2 * (DK / 64) * kRows;
  static constexpr uint32_t kStage = kVAt + 2 * kRows;
  static constexpr uint32_t kOAt = 2 * kStage;     // o [token][channel], bf16
  static constexpr uint32_t kSmem = kOAt + kC * kDv * 2 + 1024;
  // column of part k of the channels from 16 s on
  static constexpr uint32_t s_col(uint32_t s, uint32_t k) {
    const uint32_t half = s / (DK / 32), at = s % (DK / 32) * 8;
    return (k < 2 ? half * 2 * kPart + k * kPart : kThird + half * kPart) + at;
  }
};
// column of part k of V - a X or ku U, tokens from 16 s on
__host__ __device__ constexpr uint32_t v_col(uint32_t s, uint32_t k) {
  return (k < 2 ? kVCol + (s >> 1) * 32 + k * 16 : kVCol2 + (s >> 1) * 16) + (s & 1) * 8;
}

struct Chain {
  CUtensorMap tm_q, tm_k, tm_v, tm_o;
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

// 2 N values as three parts of N columns each
template <int N>
__device__ __forceinline__ void store_parts3(uint32_t col0, uint32_t col1, uint32_t col2, const float* x) {
  uint32_t p[3][N];
#pragma unroll
  for (int i = 0; i < N; ++i) split3(x[2 * i], x[2 * i + 1], p[0][i], p[1][i], p[2][i]);
  tmem_store<N>(col0, p[0]);
  tmem_store<N>(col1, p[1]);
  tmem_store<N>(col2, p[2]);
}

template <int DK>
__global__ void __launch_bounds__(kThreads, 1) gdr_chain_tc_kernel(const __grid_constant__ Chain t) {
  using L = Layout<DK>;
  extern __shared__ uint8_t raw[];
  uint8_t* stages = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[2], empty[2], sp[2], xy_done, v_ready, u_done, y_scaled, ku_ready, u_ready,
      d_done, o_done, drained;
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
    for (uint64_t* b : {&xy_done, &u_done, &d_done, &o_done, &drained}) mbar_init(b, 1);
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
      for (int i = 0; i < DK / 64; ++i) {
        tma_load_3d(st + L::kKqAt + 2 * i * L::kRows, &t.tm_k, i * 64, hk, row, &full[b]);
        tma_load_3d(st + L::kKqAt + (2 * i + 1) * L::kRows, &t.tm_q, i * 64, hk, row, &full[b]);
      }
      bulk_g2s(st, t.ws + ((size_t)(base + c) * a.Hv + h) * kBlock, kBlock, &full[b]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        tma_load_3d(st + L::kVAt + i * L::kRows, &t.tm_v, slice * (int)kDv + i * 64, h, row, &full[b]);
    }
    // loads in flight land before shared memory is released
    if (!ok)
      for (int j = max(0, c - 2); j < c; ++j) mbar_wait(&full[j & 1], (j / 2) & 1, kGdrSpins);
  } else if (warp == kWarpMma) {
    const uint32_t lead = elect_leader();
    constexpr uint32_t idesc_xy = idesc_f16(128, 128, true), idesc = idesc_f16(128, 64, true),
                       idesc_d = idesc_f16(128, DK, true, false, true);
    constexpr uint32_t kSteps = DK / 16;
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, kGdrSpins));
      fence_after_sync();
      return ok;
    };
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, ph = c & 1;
      const uint32_t st = smem_u32(stages + b * L::kStage);
      const uint32_t xcol = tmem + kXyCol + (c & 1) * 128, ycol = xcol + 64;
      // descriptors: the address is their low 14 bits, in units of 16 bytes
      const uint64_t kq = desc_k_sw128(st + L::kKqAt, 0), tt = desc_k_sw128(st + kT, 0),
                     pp = desc_k_sw128(st + kP, 0), km = desc_mn_sw128(st + L::kKqAt, 0, 2 * L::kRows);
      if (!wait(&full[b], (c / 2) & 1)) break;
      // X and Y, half of each warpgroup's channels at a time
#pragma unroll
      for (uint32_t part_of = 0; part_of < 2; ++part_of) {
        if (!wait(&sp[part_of], ph)) break;
#pragma unroll
        for (uint32_t half = 0; half < 2; ++half)
#pragma unroll
          for (uint32_t i = 0; i < kSteps / 4; ++i)
#pragma unroll
            for (uint32_t k = 0; k < 3; ++k) {
              const uint32_t s = half * (kSteps / 2) + part_of * (kSteps / 4) + i;
              mma_ts_if(lead, xcol, tmem + L::s_col(s, k), kq + (((s >> 2) * 2 * L::kRows + (s & 3) * 32) >> 4),
                     idesc_xy, part_of + half + i + k > 0);
            }
      }
      if (!ok) break;
      mma_commit_if(lead, &xy_done);
      // U: tokens 16 s .. of V - a X against T's columns
      if (!wait(&v_ready, ph)) break;
#pragma unroll
      for (uint32_t s = 0; s < 4; ++s)
#pragma unroll
        for (uint32_t j = 0; j < 3; ++j)
#pragma unroll
          for (uint32_t k = 0; k < 3 - j; ++k)
            mma_ts_if(lead, xcol, tmem + v_col(s, k), tt + ((j * kTile + s * 32) >> 4), idesc, s + j + k > 0);
      mma_commit_if(lead, &u_done);
      // the update: ku U against K, tokens contracted
      if (!wait(&ku_ready, ph)) break;
#pragma unroll
      for (uint32_t s = 0; s < 4; ++s)
#pragma unroll
        for (uint32_t k = 0; k < 3; ++k)
          mma_ts_if(lead, tmem, tmem + v_col(s, k), km + (s * 2048 >> 4), idesc_d, s + k > 0);
      mma_commit_if(lead, &d_done);
      // P U onto b Y
      if (!wait(&y_scaled, ph) || !wait(&u_ready, ph)) break;
#pragma unroll
      for (uint32_t s = 0; s < 4; ++s)
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j)
#pragma unroll
          for (uint32_t k = 0; k < 2 - j; ++k)
            mma_ts_if(lead, ycol, xcol + (s >> 1) * 32 + k * 16 + (s & 1) * 8, pp + ((j * kTile + s * 32) >> 4),
                   idesc, 1);
      mma_commit_if(lead, &o_done);
      mma_commit_if(lead, &empty[b]);
    }
    // products in flight end before shared memory and TMEM are released
    mma_commit_if(lead, &drained);
    mbar_wait(&drained, 0, kGdrSpins);
  } else if (warp < kStateWarps) {
    const int quarter = warp & 3, half = warp >> 2;
    const int dv = quarter * 32 + lane;  // this thread's row of S^T
    const uint32_t lanes = taddr(tmem, quarter * 32, 0);
    const size_t mat = ((size_t)slot * a.Hv + h) * DK * a.dv + (size_t)(half * L::kHalf) * a.dv +
                       slice * kDv + dv;
    float S[L::kHalf];
#pragma unroll
    for (uint32_t i = 0; i < L::kHalf; ++i) S[i] = a.S0 ? a.S0[mat + (size_t)i * a.dv] : 0.f;
    float eG = 1.f;
    // A wait that gave up: the warp goes on without waiting, so that it meets the others at the
    // named barriers, and stores nothing more to global memory.
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, kGdrSpins));
      fence_after_sync();
    };
    // S <- e^{g_C} S + the update's product
    auto update = [&] {
#pragma unroll
      for (uint32_t i = 0; i < L::kHalf; i += 32) {
        uint32_t r[32];
        tmem_ld32(lanes + half * L::kHalf + i, r);
        tmem_wait_ld();
#pragma unroll
        for (uint32_t j = 0; j < 32; ++j) S[i + j] = fmaf(eG, S[i + j], __uint_as_float(r[j]));
      }
    };
    // o of chunk c, this warpgroup's 32 tokens, through shared memory: two boxes of 64 channels,
    // or row by row where the sequence ends among them (what follows is another's)
    uint8_t* so = stages + L::kOAt + half * 2 * 4096;
    auto write_o = [&](int c) {
      uint32_t r[32];
      tmem_ld32(lanes + kXyCol + (c & 1) * 128 + 64 + half * 32, r);
      if (quarter == 0) bulk_wait_read();  // the rows before have left
      named_sync(1 + half, 128);
      tmem_wait_ld();
      __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(so + (dv >> 6) * 4096) + (dv & 63);
#pragma unroll
      for (int i = 0; i < 32; ++i) to[i * 64] = __float2bfloat16_rn(__uint_as_float(r[i]));
      fence_proxy_async();
      named_sync(1 + half, 128);
      const int row = t0 + c * kC + half * 32;
      if (quarter == 0 && ok) {
        if (row + 32 <= t1) {
          if (lane < 2) tma_store_3d(&t.tm_o, so + lane * 4096, slice * (int)kDv + lane * 64, h, row);
        } else if (row + lane < t1) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + ((size_t)(row + lane) * a.Hv + h) * a.dv + slice * kDv;
          bulk_s2g(o, so + lane * 128, 128);
          bulk_s2g(o + 64, so + 4096 + lane * 128, 128);
        }
        bulk_commit();
      }
    };
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, ph = c & 1;
      uint8_t* st = stages + b * L::kStage;
      const float* vec = reinterpret_cast<const float*>(st + kVec) + half * 32;
      const int len = min(kC, t1 - t0 - c * kC);
      // V, and zeros behind the last token: there the rows are the next sequence's (the products
      // see them behind the hand-over below)
      wait(&full[b], (c / 2) & 1);
      uint32_t vp[16];
      {
        const uint16_t* vs = reinterpret_cast<const uint16_t*>(st + L::kVAt + (dv >> 6) * L::kRows) +
                             half * 32 * 64 + (dv & 63);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const uint32_t lo = half * 32 + i < len ? vs[i * 64] : 0, hi = half * 32 + i + 1 < len ? vs[i * 64 + 64] : 0;
          vp[i / 2] = lo | hi << 16;
        }
      }
      if (len < kC) {
        for (int i = threadIdx.x; i < (kC - len) * 8 * (DK / 64) * 2; i += kStateWarps * 32) {
          const int tile = i / ((kC - len) * 8), j = i % ((kC - len) * 8);
          *reinterpret_cast<uint4*>(st + L::kKqAt + tile * L::kRows + (len + (j >> 3)) * 128 + (j & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
      }
      // S as parts, in two halves so that the products start on the first; the update's whole
      // product is read before the parts take its place
      if (c > 0) {
        wait(&d_done, (c - 1) & 1);
        update();
      }
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        store_parts3<L::kHalf / 4>(lanes + half * 2 * L::kPart + i * (L::kPart / 2),
                                   lanes + half * 2 * L::kPart + L::kPart + i * (L::kPart / 2),
                                   lanes + L::kThird + half * L::kPart + i * (L::kPart / 2),
                                   &S[i * L::kHalf / 2]);
        hand_over(&sp[i], lane);
      }
      if (c > 0) {
        wait(&o_done, (c - 1) & 1);
        write_o(c - 1);
      }
      // V - a X
      wait(&xy_done, ph);
      float v[32];
      {
        uint32_t r[32];
        tmem_ld32(lanes + kXyCol + (c & 1) * 128 + half * 32, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 va = *reinterpret_cast<const float4*>(vec + i);
          v[i] = fmaf(-va.x, __uint_as_float(r[i]), __uint_as_float(vp[i / 2] << 16));
          v[i + 1] = fmaf(-va.y, __uint_as_float(r[i + 1]), __uint_as_float(vp[i / 2] & 0xffff0000u));
          v[i + 2] = fmaf(-va.z, __uint_as_float(r[i + 2]), __uint_as_float(vp[i / 2 + 1] << 16));
          v[i + 3] = fmaf(-va.w, __uint_as_float(r[i + 3]), __uint_as_float(vp[i / 2 + 1] & 0xffff0000u));
        }
      }
      const uint32_t w0 = lanes + kVCol + half * 32, w2 = lanes + kVCol2 + half * 16;
      store_parts3<16>(w0, w0 + 16, w2, v);
      hand_over(&v_ready, lane);
      // b Y
      {
        const uint32_t ycol = lanes + kXyCol + (c & 1) * 128 + 64 + half * 32;
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
      wait(&u_done, ph);
      {
        const uint32_t ucol = lanes + kXyCol + (c & 1) * 128 + half * 32;
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
        store_parts3<16>(w0, w0 + 16, w2, v);
        hand_over(&ku_ready, lane);
        uint32_t p[2][16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t w[2];
          split2<2>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), w);
          p[0][i] = w[0];
          p[1][i] = w[1];
        }
        tmem_st16(ucol, p[0]);
        tmem_st16(ucol + 16, p[1]);
        hand_over(&u_ready, lane);
      }
    }
    if (chunks > 0) {
      wait(&d_done, (chunks - 1) & 1);
      update();
      wait(&o_done, (chunks - 1) & 1);
      write_o(chunks - 1);
      if (quarter == 0) bulk_wait_all();
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
// by `rows` tokens.
bool encode(CUtensorMap* m, const void* base, int T, int H, int d, long long ld, int rows,
            bool swizzle) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
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
  if (!encode(&t.tm_k, a.k, a.T_total, a.Hk, DK, a.ldk, kC, true) ||
      !encode(&t.tm_q, a.q, a.T_total, a.Hk, DK, a.ldq, kC, true) ||
      !encode(&t.tm_v, a.v, a.T_total, a.Hv, a.dv, a.ldv, kC, false) ||
      !encode(&t.tm_o, a.o, a.T_total, a.Hv, a.dv, (long long)a.Hv * a.dv, 32, false))
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
