// gdr_chain_tc.cu -- the state's walk over the chunks of a sequence on tcgen05, for d_k of 64 or
// 128 and 128 columns of the state (d_v) per CTA.  The algebra and the parts that operands are
// split into are those of gdr_chunked.cu; everything is held transposed, lanes of TMEM = d_v:
//     X^T = S^T K^T,  Y^T = S^T Q^T,  U^T = V^T T^T - (a X)^T T^T,
//     O^T = b Y^T + U^T P^T,          S^T <- e^{g_C} S^T + (ku U)^T K.
//
// S^T stays in the registers of eight warps (thread = lane of TMEM = row of S^T, two warpgroups
// for the two halves of d_k).  What they make of it is written to TMEM as A operands; V^T is an
// A operand as it lies in shared memory, and so are the B operands, as prep and TMA put them
// there.  A chunk is a chain of dependent steps, conversions by the eight warps and products by
// the tensor cores in turn,
//     S -> parts | X | -a X -> parts | U | ku U -> parts | S's update,
// each handed over in pieces of 16 channels or tokens, so that the products of the first run
// beside the conversion of the next.  The rest fills the gaps: Y runs beside the conversion of
// X, V T of the next chunk beside that of U, P U beside that of S; the warps scale Y while the
// tensor cores work on U and hand the last chunk's o to another warp, which stores it, while
// they work on X.
//
// A chunk of 128 x 128 heads takes 6,000 cycles (4096 tokens x 96 heads: 202 us on 96 SMs), of which
// the products need 5,300: 101 MMAs of N = 64, 45 cycles each whatever N is below 128, and 12 of
// N = 128, 64 each.  (X and Y as one product against [K; Q] need fewer cycles, but X comes 460 later.)
//
// TMEM columns (d_k = 128): 0-191 the parts of S, the first two of which lie where the same
// warpgroup's half of the update's product comes (0-127), the third (128-191) where -a X and
// ku U go with 192-223; 224 and 288 in turn X and U, then U's first two parts; 352 and 416 in turn
// Y, then o; 480-511 U's third part.  A warpgroup writes and reads only its own columns, so that no
// barrier between the warps is needed.
#include "gdr_chunked.cuh"
#include "tensor_map.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kStateWarps = 8, kWarpLoad = 8, kWarpMma = 9, kWarpStore = 10;
constexpr int kThreads = 352;
constexpr uint32_t kDv = 128;
constexpr uint32_t kVCol = 128, kVCol2 = 192, kXuCol = 224, kYCol = 352, kUCol2 = 480;

template <int DK>
struct Layout {
  static constexpr uint32_t kHalf = DK / 2;        // channels of a warpgroup
  static constexpr uint32_t kPart = kHalf / 2;     // TMEM columns of one part of them
  static constexpr uint32_t kThird = 2 * DK / 2;   // where the third parts of S begin
  static constexpr uint32_t kRows = kC * 128;      // bytes of 64 rows of 64 channels
  static constexpr uint32_t kSteps = DK / 16, kSub = DK / 32;  // 16-channel steps, and of a half
  static constexpr uint32_t kKAt = kBlock, kQAt = kKAt + DK / 64 * kRows;
  static constexpr uint32_t kVAt = kQAt + DK / 64 * kRows;
  static constexpr uint32_t kStage = kVAt + 2 * kRows;
  static constexpr uint32_t kOAt = 2 * kStage;     // o [token][channel], bf16
  static constexpr uint32_t kSmem = kOAt + kC * kDv * 2 + 1024;
  // column of part k of the channels from 16 s on
  static constexpr uint32_t s_col(uint32_t s, uint32_t k) {
    const uint32_t half = s / kSub, at = s % kSub * 8;
    return (k < 2 ? half * 2 * kPart + k * kPart : kThird + half * kPart) + at;
  }
};
// column of part k of -a X or ku U, tokens from 16 s on
__host__ __device__ constexpr uint32_t v_col(uint32_t s, uint32_t k) {
  return (k < 2 ? kVCol + (s >> 1) * 32 + k * 16 : kVCol2 + (s >> 1) * 16) + (s & 1) * 8;
}

// column of part k of U, tokens from 16 s on: the first two in place of U itself
__device__ __forceinline__ uint32_t u_col(uint32_t ucol, uint32_t tmem, uint32_t s, uint32_t k) {
  return (k < 2 ? ucol + (s >> 1) * 32 + k * 16 : tmem + kUCol2 + (s >> 1) * 16) + (s & 1) * 8;
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
  __shared__ uint64_t full[2], empty[2], s_ready[4], x_done, y_done, v_ready[2], u_done, y_scaled,
      ku_ready[2], u_ready, d_done, o_done, o_ready, o_free, drained;
  __shared__ uint32_t tmem_base;

  const GdrArgs& a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = a.dv / (int)kDv;
  const int slice = blockIdx.x % slices, h = blockIdx.x / slices % a.Hv;
  const int n = longest_first(a, blockIdx.x / slices / a.Hv);
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;  // every warp finds the same
  const int chunks = (t1 - t0 + kC - 1) / kC, base = block_base(t0, n);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
      mbar_init(&v_ready[i], kStateWarps);
      mbar_init(&ku_ready[i], kStateWarps);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&s_ready[i], kStateWarps);
    for (uint64_t* b : {&x_done, &y_done, &u_done, &d_done, &o_done, &o_free, &drained}) mbar_init(b, 1);
    for (uint64_t* b : {&y_scaled, &u_ready, &o_ready}) mbar_init(b, kStateWarps);
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
        tma_load_3d(st + L::kKAt + i * L::kRows, &t.tm_k, i * 64, hk, row, &full[b]);
        tma_load_3d(st + L::kQAt + i * L::kRows, &t.tm_q, i * 64, hk, row, &full[b]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        tma_load_3d(st + L::kVAt + i * L::kRows, &t.tm_v, slice * (int)kDv + i * 64, h, row, &full[b]);
      bulk_g2s(st, t.ws + ((size_t)(base + c) * a.Hv + h) * kBlock, kBlock, &full[b]);
    }
    // loads in flight land before shared memory is released
    if (!ok)
      for (int j = max(0, c - 2); j < c; ++j) mbar_wait(&full[j & 1], (j / 2) & 1, kGdrSpins);
  } else if (warp == kWarpMma) {
    const uint32_t lead = elect_leader();
    // products with the columns of T or P from 16 s on meet their rows from 16 s on only
    constexpr uint32_t kBelow = 16 * 128 >> 4;  // 16 rows, in a descriptor's units
    constexpr uint32_t idesc = idesc_f16(128, 64, true), idesc_d = idesc_f16(128, DK, true, false, true);
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_soon(bar, parity, kGdrSpins));
      fence_after_sync();
      return ok;
    };
    auto len_of = [&](int c) { return min(kC, t1 - t0 - c * kC); };
    // V T of chunk c: the beginning of its U
    auto v_products = [&](int c) {
      const uint32_t st = smem_u32(stages + (c & 1) * L::kStage);
      const uint64_t vv = desc_mn_sw128(st + L::kVAt, 0, L::kRows), tt = desc_k_sw128(st + kT, 0);
#pragma unroll
      for (uint32_t j = 2; j < 3; --j)
#pragma unroll
        for (uint32_t s = 0; s < 4; ++s)
          mma_ss_if(lead, tmem + kXuCol + (c & 1) * 64 + 16 * s, vv + (s * 2048 >> 4),
                    tt + ((j * kTile + s * 32) >> 4) + s * kBelow, idesc_f16(128, 64 - 16 * s, true, true),
                    s + 2 - j > 0);
    };
    // Sums are cut, not rounded, as products are added: those of the smaller parts go first, while
    // a sum is small.
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, ph = c & 1;
      const uint32_t st = smem_u32(stages + b * L::kStage);
      const uint32_t ucol = tmem + kXuCol + (c & 1) * 64, xcol = tmem + kXuCol + (1 - (c & 1)) * 64,
                     ycol = tmem + kYCol + (c & 1) * 64;
      // descriptors: the address is their low 14 bits, in units of 16 bytes
      const uint64_t kk = desc_k_sw128(st + L::kKAt, 0), qq = desc_k_sw128(st + L::kQAt, 0),
                     tt = desc_k_sw128(st + kT, 0), pp = desc_k_sw128(st + kP, 0),
                     km = desc_mn_sw128(st + L::kKAt, 0, L::kRows);
      if (!wait(&full[b], (c / 2) & 1)) break;
      if (c == 0 && len_of(0) == kC) v_products(0);
      // X, 16 channels of each warpgroup at a time
#pragma unroll
      for (uint32_t i = 0; i < L::kSub; ++i) {
        if (!wait(&s_ready[i], ph)) break;
#pragma unroll
        for (uint32_t k = 2; k < 3; --k)
#pragma unroll
          for (uint32_t half = 0; half < 2; ++half) {
            const uint32_t s = half * L::kSub + i;
            mma_ts_if(lead, xcol, tmem + L::s_col(s, k), kk + (((s >> 2) * L::kRows + (s & 3) * 32) >> 4),
                      idesc, i + half + 2 - k > 0);
          }
      }
      if (!ok) break;
      mma_commit_if(lead, &x_done);
      if (!wait(&x_done, ph)) break;
#pragma unroll
      for (uint32_t k = 1; k < 2; --k)
#pragma unroll
        for (uint32_t s = 0; s < L::kSteps; ++s)
          mma_ts_if(lead, ycol, tmem + L::s_col(s, k), qq + (((s >> 2) * L::kRows + (s & 3) * 32) >> 4),
                    idesc, s + 1 - k > 0);
      mma_commit_if(lead, &y_done);
      // in a chunk that is not full V's last rows are cleared by the time S is handed over
      if (len_of(c) < kC) v_products(c);
      // U: tokens 16 s .. of -a X against T's columns
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        if (!wait(&v_ready[i], ph)) break;
#pragma unroll
        for (uint32_t order = 2; order < 3; --order)
#pragma unroll
          for (uint32_t j = 0; j <= order; ++j)
#pragma unroll
            for (uint32_t s = i, k = order - j; s < 4; s += 2)
              mma_ts_if(lead, ucol + 16 * s, tmem + v_col(s, k), tt + ((j * kTile + s * 32) >> 4) + s * kBelow,
                        idesc_f16(128, 64 - 16 * s, true), 1);
      }
      if (!ok) break;
      mma_commit_if(lead, &u_done);
      if (c + 1 < chunks && len_of(c + 1) == kC) {
        if (!wait(&full[b ^ 1], ((c + 1) / 2) & 1)) break;
        v_products(c + 1);
      }
      // the update: ku U against K, tokens contracted
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        if (!wait(&ku_ready[i], ph)) break;
#pragma unroll
        for (uint32_t k = 2; k < 3; --k)
#pragma unroll
          for (uint32_t s = i; s < 4; s += 2)
            mma_ts_if(lead, tmem, tmem + v_col(s, k), km + (s * 2048 >> 4), idesc_d, s + 2 - k > 0);
      }
      if (!ok) break;
      mma_commit_if(lead, &d_done);
      // P U onto b Y, behind the update: S waits for that.  When it is done the place of o in
      // shared memory is free too: the warps that write it wait for the one only.
      if (!wait(&y_scaled, ph) || !wait(&u_ready, ph)) break;
      if (c > 0 && !wait(&o_free, (c - 1) & 1)) break;
      if (!wait(&d_done, ph)) break;
#pragma unroll
      for (int i = 4; i >= 0; --i) {  // P's third part: column i (0: rows 16 on), then the first block
        const uint32_t s = i < 4 ? i : 0, row = i == 0 ? 1 : s;
        const PlaceOfP at = third_of_p(row, s);
        mma_ts_if(lead, ycol + 16 * row, u_col(ucol, tmem, s, 0), pp + ((at.tile * kTile + at.col * 32) >> 4),
                  idesc_f16(128, i < 4 ? 64 - 16 * row : 16, true), 1);
      }
#pragma unroll
      for (uint32_t order = 2; order < 3; --order)
#pragma unroll
        for (uint32_t j = 0; j <= (order < 1 ? order : 1); ++j)
#pragma unroll
          for (uint32_t s = 0, k = order - j; s < 4; ++s)
            mma_ts_if(lead, ycol + 16 * s, u_col(ucol, tmem, s, k),
                      pp + ((j * kTile + s * 32) >> 4) + s * kBelow, idesc_f16(128, 64 - 16 * s, true), 1);
      mma_commit_if(lead, &o_done);
      mma_commit_if(lead, &empty[b]);
    }
    // products in flight end before shared memory and TMEM are released
    mma_commit_if(lead, &drained);
    mbar_wait(&drained, 0, kGdrSpins);
  } else if (warp == kWarpStore) {
    // o from shared memory: boxes of 64 channels, or by plain stores in a last chunk that is not
    // full (what follows its rows is another sequence's)
    const uint8_t* so = stages + L::kOAt;
    for (int c = 0; c < chunks && ok; ++c) {
      ok = __all_sync(0xffffffffu, mbar_wait_soon(&o_ready, c & 1, kGdrSpins));
      if (!ok) break;
      const int row = t0 + c * kC;
      if (row + kC <= t1) {
        if (lane < 2) tma_store_3d(&t.tm_o, so + lane * L::kRows, slice * (int)kDv + lane * 64, h, row);
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + ((size_t)row * a.Hv + h) * a.dv + slice * kDv;
        for (int i = lane; i < (t1 - row) * 16; i += 32) {  // 16-byte groups
          const int r = i >> 4, g = i & 15;
          *reinterpret_cast<uint4*>(o + (size_t)r * a.Hv * a.dv + g * 8) =
              *reinterpret_cast<const uint4*>(so + (g >> 3) * L::kRows + r * 128 + (((g ^ r) & 7) << 4));
        }
      }
      bulk_commit();
      bulk_wait_read();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free);
    }
    bulk_wait_all();
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
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_soon(bar, parity, kGdrSpins));
      fence_after_sync();
      return ok;
    };
    // S <- e^{g_C} S + the update's product
    auto update = [&] {
      uint32_t r[L::kHalf / 32][32];
#pragma unroll
      for (uint32_t i = 0; i < L::kHalf / 32; ++i) tmem_ld32(lanes + half * L::kHalf + i * 32, r[i]);
      tmem_wait_ld();
#pragma unroll
      for (uint32_t i = 0; i < L::kHalf; ++i) S[i] = fmaf(eG, S[i], __uint_as_float(r[i / 32][i % 32]));
    };
    // o of chunk c, this warpgroup's 32 tokens: 8 x 8 tiles transposed into rows of tokens
    auto write_o = [&](int c) {
      if (!wait(&o_done, c & 1)) return;
      uint32_t r[2][16];
#pragma unroll
      for (int h16 = 0; h16 < 2; ++h16)
        tmem_ld_frag4(taddr(lanes, h16 * 16, kYCol + (c & 1) * 64 + half * 32), r[h16]);
      tmem_wait_ld();
      const uint32_t row = half * 32 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
      for (int h16 = 0; h16 < 2; ++h16) {
        const uint32_t group = quarter * 4 + h16 * 2 + ((lane >> 3) & 1);  // of 8 channels
        const uint32_t at = smem_u32(stages + L::kOAt) + (group >> 3) * L::kRows + row * 128 +
                            (((group ^ row) & 7) << 4);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t* x = &r[h16][p * 8];
          const uint32_t m[4] = {pack_bf162(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                 pack_bf162(__uint_as_float(x[2]), __uint_as_float(x[3])),
                                 pack_bf162(__uint_as_float(x[4]), __uint_as_float(x[5])),
                                 pack_bf162(__uint_as_float(x[6]), __uint_as_float(x[7]))};
          stsm4t(at + p * 16 * 128, m);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_ready);
    };
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, ph = c & 1;
      uint8_t* st = stages + b * L::kStage;
      const float* vec = reinterpret_cast<const float*>(st + kVec) + half * 32;
      const int len = min(kC, t1 - t0 - c * kC);
      if (!wait(&full[b], (c / 2) & 1)) break;
      if (len < kC) {
        // rows behind the last token are the next sequence's: zeros in their place, which the
        // products see behind the hand-over below
        for (int i = threadIdx.x; i < (kC - len) * 8 * (2 * DK / 64 + 2); i += kStateWarps * 32) {
          const int tile = i / ((kC - len) * 8), j = i % ((kC - len) * 8);  // of K, Q and V
          *reinterpret_cast<uint4*>(st + L::kKAt + tile * L::kRows + (len + (j >> 3)) * 128 + (j & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
      }
      // the update's whole product is read before the parts take its place
      if (c > 0) {
        if (!wait(&d_done, (c - 1) & 1)) break;
        update();
      }
#pragma unroll
      for (uint32_t i = 0; i < L::kSub; ++i) {
        const uint32_t at = lanes + half * 2 * L::kPart + i * 8;
        store_parts3<8>(at, at + L::kPart, lanes + L::kThird + half * L::kPart + i * 8, &S[i * 16]);
        hand_over(&s_ready[i], lane);
      }
      if (c > 0) write_o(c - 1);
      // -a X, 16 tokens at a time
      const uint32_t w0 = lanes + kVCol + half * 32, w2 = lanes + kVCol2 + half * 16;
      if (!wait(&x_done, ph)) break;
      {
        uint32_t r[32];
        tmem_ld32(lanes + kXuCol + (1 - (c & 1)) * 64 + half * 32, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 va = *reinterpret_cast<const float4*>(vec + j * 16 + i);
            v[i] = -va.x * __uint_as_float(r[j * 16 + i]);
            v[i + 1] = -va.y * __uint_as_float(r[j * 16 + i + 1]);
            v[i + 2] = -va.z * __uint_as_float(r[j * 16 + i + 2]);
            v[i + 3] = -va.w * __uint_as_float(r[j * 16 + i + 3]);
          }
          store_parts3<8>(w0 + j * 8, w0 + 16 + j * 8, w2 + j * 8, v);
          hand_over(&v_ready[j], lane);
        }
      }
      // b Y
      if (!wait(&y_done, ph)) break;
      {
        const uint32_t ycol = lanes + kYCol + (c & 1) * 64 + half * 32;
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
      // ku U, then U
      if (!wait(&u_done, ph)) break;
      {
        const uint32_t ucol = lanes + kXuCol + (c & 1) * 64 + half * 32;
        uint32_t r[32];
        tmem_ld32(ucol, r);
        tmem_wait_ld();
        eG = vec[192 - half * 32];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 ku = *reinterpret_cast<const float4*>(vec + 128 + j * 16 + i);
            v[i] = ku.x * __uint_as_float(r[j * 16 + i]);
            v[i + 1] = ku.y * __uint_as_float(r[j * 16 + i + 1]);
            v[i + 2] = ku.z * __uint_as_float(r[j * 16 + i + 2]);
            v[i + 3] = ku.w * __uint_as_float(r[j * 16 + i + 3]);
          }
          store_parts3<8>(w0 + j * 8, w0 + 16 + j * 8, w2 + j * 8, v);
          hand_over(&ku_ready[j], lane);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float u[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = __uint_as_float(r[j * 16 + i]);
          store_parts3<8>(ucol + j * 8, ucol + 16 + j * 8, lanes + kUCol2 + half * 16 + j * 8, u);
        }
        hand_over(&u_ready, lane);
      }
    }
    if (ok && chunks > 0 && wait(&d_done, (chunks - 1) & 1)) {
      update();
      write_o(chunks - 1);
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

// Tensor map of [T][H][d] bf16 rows, tokens ld elements apart: boxes of 64 channels of one head
// by `rows` tokens.
bool encode(CUtensorMap* m, const void* base, int T, int H, int d, long long ld, int rows) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK>
cudaError_t launch(const GdrArgs& a, const uint8_t* ws, cudaStream_t s) {
  const cudaError_t e = allow_smem<gdr_chain_tc_kernel<DK>>(Layout<DK>::kSmem);
  if (e != cudaSuccess) return e;
  Chain t;
  t.a = a;
  t.ws = ws;
  if (!encode(&t.tm_k, a.k, a.T_total, a.Hk, DK, a.ldk, kC) ||
      !encode(&t.tm_q, a.q, a.T_total, a.Hk, DK, a.ldq, kC) ||
      !encode(&t.tm_v, a.v, a.T_total, a.Hv, a.dv, a.ldv, kC) ||
      !encode(&t.tm_o, a.o, a.T_total, a.Hv, a.dv, (long long)a.Hv * a.dv, kC))
    return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)a.N * a.Hv * (a.dv / (int)kDv);
  // An ordinary launch: started early by programmatic dependent launch, the CTAs settle on the SMs
  // that prep leaves first, and 4096 tokens x 96 heads took 298 us in place of 283.
  gdr_chain_tc_kernel<DK><<<grid, kThreads, Layout<DK>::kSmem, s>>>(t);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_chain_tc(const GdrArgs& a, const uint8_t* ws, cudaStream_t s) {
  return a.dk == 128 ? launch<128>(a, ws, s) : launch<64>(a, ws, s);
}

}  // namespace kda
