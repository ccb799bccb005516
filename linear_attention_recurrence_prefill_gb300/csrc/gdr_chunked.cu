// gdr_chunked.cu -- the gated delta rule in chunks of 64 tokens on the tensor
// cores (bf16 data).
//
// For one value head, S the state before the chunk, g_i the running sum of the
// log decays, k and q the normalised rows:
//     A_ij = beta_i e^{g_i - g_j} k_i.k_j (j < i),   T = (I + A)^-1 Diag(beta)
//     P_ij = e^{g_i - g_j} q_i.k_j (j <= i)
//     U    = T (V - e^g K S),     O = e^g Q S + P U,
//     S   <- e^{g_C} S + (e^{g_C - g} K)^T U
// which is the recurrence taken over the chunk at once.  Every exponent is <= 0,
// so nothing needs rescaling, whatever the decays.
//
// Two kernels.  prep: T, P and the vectors of every chunk, all chunks in
// parallel.  chain: the state's walk over the chunks of a sequence.
//
// Precision: the final states are fp32 results, so no operand may be rounded to
// bf16.  K, Q and V are bf16 as they come and enter the products unscaled (norms
// and decays multiply rows of results or fp32 operands); everything else (the state,
// V - e^g K S, U, T, P) enters as two bf16 parts, x = hi + lo to 2^-16, one product for
// each pair of parts but lo * lo.
#include "gdr.cuh"
#include "umma.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kC = 64;                 // tokens per chunk
constexpr long long kSpins = 4000000000LL;  // ~2 s of clock cycles

// One (chunk, value head) of the workspace: T and P as bf16 parts [row][64], 128-byte
// rows whose 16-byte groups are XORed with the row's low three bits, then the vectors.
constexpr uint32_t kTile = kC * kC * 2;
constexpr uint32_t kTHi = 0, kTLo = kTile, kPHi = 2 * kTile, kPLo = 3 * kTile;
constexpr uint32_t kVec = 4 * kTile;  // floats: a[64], b[64], ku[64], e^{g_C}
constexpr uint32_t kBlock = kVec + 1024;

__host__ __device__ constexpr uint32_t tile_at(uint32_t row, uint32_t col) {
  return row * 128u + ((((col >> 3) ^ row) & 7u) << 4) + (col & 7u) * 2u;
}

// Chunk c of sequence n has block (t0 / 64 + n) + c: floor((t0 + len) / 64) + 1 is at
// least floor(t0 / 64) + ceil(len / 64), so that sequences never share a block, and no
// prefix sum over the sequences is needed.
__host__ __device__ constexpr int block_base(int t0, int n) { return t0 / kC + n; }

// ------------------------------------------------------------------ fragments
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
               :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// c += a b: a 16 x 16 (rows g = lane / 4 and g + 8), b 16 x 8, bf16, fp32 sums
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x, y as two bf16 parts each
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf162(x, y);
  lo = pack_bf162(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}
// The accumulators of two neighbouring 16 x 8 tiles as the parts of a 16 x 16 A operand: the
// layouts agree element by element.
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4],
                                        uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split2(c0[0], c0[1], hi[0], lo[0]);
  split2(c0[2], c0[3], hi[1], lo[1]);
  split2(c1[0], c1[1], hi[2], lo[2]);
  split2(c1[2], c1[3], hi[3], lo[3]);
}

// ------------------------------------------------------------------ prep
constexpr int kPrepThreads = 128;
constexpr int kAtPitch = kC + 4;

template <int DK>
struct PrepSmem {
  static constexpr int kPitch = DK * 2 + 16;  // bytes: rows 16 bytes past a multiple of 128
  __nv_bfloat16 k[kC * kPitch / 2], q[kC * kPitch / 2];
  float at[2][kC][kAtPitch];                  // A transposed, two heads
  float ik[kC], iq[kC];
  float ghi[2][kC], glo[2][kC], beta[2][kC];
  int n, c, t0, t1;
};

// Column j of (I + A)^-1, rows k0 on (rows before k0 are zero: j >= k0), in x[.] as pairs:
// x_j = 1, then as soon as x_k is known it leaves every later sum.
template <int kK0>
__device__ __forceinline__ void solve_column(const float (*at)[kAtPitch], int j,
                                             unsigned long long (&x)[kC / 2]) {
#pragma unroll
  for (int i = 0; i < kC / 2; ++i)
    x[i] = ((unsigned long long)__float_as_uint(j == 2 * i + 1 ? 1.f : 0.f) << 32) |
           __float_as_uint(j == 2 * i ? 1.f : 0.f);
#pragma unroll
  for (int k = kK0; k < kC - 1; ++k) {
    const uint32_t xk = k & 1 ? (uint32_t)(x[k / 2] >> 32) : (uint32_t)x[k / 2];
    const uint32_t m = xk ^ 0x80000000u;
    const unsigned long long m2 = ((unsigned long long)m << 32) | m;
#pragma unroll
    for (int i = (k + 1) & ~3; i < kC; i += 4) {  // entries up to row k are zero
      const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(&at[k][i]);
      asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(x[i / 2]) : "l"(a.x), "l"(m2));
      asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(x[i / 2 + 1]) : "l"(a.y), "l"(m2));
    }
  }
}

__device__ __forceinline__ void store_parts(uint8_t* hi_tile, uint8_t* lo_tile, uint32_t at,
                                            float v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  *reinterpret_cast<__nv_bfloat16*>(hi_tile + at) = h;
  *reinterpret_cast<__nv_bfloat16*>(lo_tile + at) = __float2bfloat16_rn(v - __bfloat162float(h));
}

template <int DK>
__global__ void __launch_bounds__(kPrepThreads) gdr_prep_kernel(GdrArgs a, uint8_t* ws) {
  using Smem = PrepSmem<DK>;
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int blk = blockIdx.x, hk = blockIdx.y, G = a.Hv / a.Hk;

  if (warp == 0) {
    // the sequence of this block: the last one whose base is not behind it, as far as the
    // offsets do not decrease (later sequences are left out)
    int n = -1;
    for (int i0 = 0; i0 < a.N; i0 += 32) {
      const int i = i0 + lane;
      const int off = i < a.N ? gdr_offset(a, i) : 0;
      const bool down = i < a.N && off > gdr_offset(a, i + 1);
      const uint32_t downs = __ballot_sync(0xffffffffu, down);
      uint32_t in = __ballot_sync(0xffffffffu, i < a.N && block_base(off, i) <= blk);
      if (downs) in &= (2u << (__ffs(downs) - 1)) - 1u;
      n += __popc(in);
      if (downs || in != 0xffffffffu) break;
    }
    int t0 = 0, t1 = 0, slot = 0, c = 0;
    if (n >= 0 && gdr_sequence(a, n, t0, t1, slot)) {
      c = blk - block_base(t0, n);
      if (c < 0 || (long long)t0 + (long long)c * kC >= t1) n = -1;
    } else {
      n = -1;
    }
    if (lane == 0) {
      s.n = n;
      s.t0 = t0 + c * kC;
      s.t1 = t1;
    }
  }
  __syncthreads();
  if (s.n < 0) return;
  const int t0 = s.t0, len = min(kC, s.t1 - t0);

  // K and Q rows, zeros behind the last token
  {
    constexpr int kGroups = DK / 8;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + (size_t)hk * DK;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (size_t)hk * DK;
    for (int i = tid; i < kC * kGroups; i += kPrepThreads) {
      const int r = i / kGroups, g = i % kGroups;
      const size_t t = (size_t)(t0 + (r < len ? r : 0));
      cp_async16(smem_u32(s.k) + r * Smem::kPitch + g * 16, k + t * a.ldk + g * 8, r < len ? 16 : 0);
      cp_async16(smem_u32(s.q) + r * Smem::kPitch + g * 16, q + t * a.ldq + g * 8, r < len ? 16 : 0);
    }
    cp_async_commit();
    cp_async_wait_all();
  }
  __syncthreads();

  // norms: two threads per row
  {
    const int r = tid >> 1;
    const uint4* kr = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(s.k) + r * Smem::kPitch) + (tid & 1);
    const uint4* qr = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(s.q) + r * Smem::kPitch) + (tid & 1);
    float kk = 0.f, qq = 0.f;
    auto add = [](float& x, uint4 w) {
      const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(e[i] << 16), hi = __uint_as_float(e[i] & 0xffff0000u);
        x = fmaf(lo, lo, x);
        x = fmaf(hi, hi, x);
      }
    };
#pragma unroll
    for (int g = 0; g < DK / 16; ++g) {
      add(kk, kr[g * 2]);
      add(qq, qr[g * 2]);
    }
    kk += __shfl_xor_sync(0xffffffffu, kk, 1);
    qq += __shfl_xor_sync(0xffffffffu, qq, 1);
    if ((tid & 1) == 0) {
      s.ik[r] = a.l2norm_qk ? gdr_inv_norm(kk, a.eps_l2) : 1.f;
      s.iq[r] = a.q_scale * (a.l2norm_qk ? gdr_inv_norm(qq, a.eps_l2) : 1.f);
    }
  }

  // K K^T and Q K^T, 16 rows per warp, columns up to the diagonal block
  float kk[8][4] = {}, qk[8][4] = {};
  {
    const uint32_t row = warp * 16 + (lane & 15), col = (lane >> 4) * 16;
    const uint32_t ka = smem_u32(s.k) + row * Smem::kPitch + col;
    const uint32_t qa = smem_u32(s.q) + row * Smem::kPitch + col;
    // B of two column tiles: lanes 0-7 rows of the first, k 0-7; 8-15 k 8-15; then the second
    const uint32_t kb = smem_u32(s.k) + ((lane & 7) + ((lane >> 4) << 3)) * Smem::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int x = 0; x < DK / 16; ++x) {
      uint32_t fk[4], fq[4];
      ldsm4(fk, ka + x * 32);
      ldsm4(fq, qa + x * 32);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (p > warp) break;
        uint32_t b[4];
        ldsm4(b, kb + p * 16 * Smem::kPitch + x * 32);
        mma(kk[2 * p], fk, b[0], b[1]);
        mma(kk[2 * p + 1], fk, b[2], b[3]);
        mma(qk[2 * p], fq, b[0], b[1]);
        mma(qk[2 * p + 1], fq, b[2], b[3]);
      }
    }
  }
  __syncthreads();

  const __nv_bfloat16* beta = static_cast<const __nv_bfloat16*>(a.beta);
  for (int h0 = 0; h0 < G; h0 += 2) {
    if (warp < 2 && h0 + warp < G) {
      // running sums of the log decays, in 64 bits: differences of them are taken
      const int h = hk * G + h0 + warp;
      uint8_t* out = ws + ((size_t)blk * a.Hv + h) * kBlock;
      double g2[2];
      float be[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = lane * 2 + i;
        const size_t at = (size_t)(t0 + r) * a.Hv + h;
        g2[i] = r < len ? (double)gdr_log_decay(a, a.log_alpha[at], h) : 0.0;
        const float b = r < len ? to_f32(beta[at]) : 0.f;
        be[i] = r < len && a.beta_is_logit ? sigmoidf_(b) : b;
      }
      double sum = g2[0] + g2[1];
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const double other = __shfl_up_sync(0xffffffffu, sum, m);
        if (lane >= m) sum += other;
      }
      const double last = __shfl_sync(0xffffffffu, sum, 31);
      const double g[2] = {sum - g2[1], sum};
      float* vec = reinterpret_cast<float*>(out + kVec);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = lane * 2 + i;
        const float hi = (float)g[i];
        s.ghi[warp][r] = hi;
        s.glo[warp][r] = (float)(g[i] - (double)hi);
        s.beta[warp][r] = be[i];
        const float e = expf(hi);
        vec[r] = e * s.ik[r];
        vec[64 + r] = e * s.iq[r];
        vec[128 + r] = expf((float)(last - g[i])) * s.ik[r];
      }
      if (lane == 0) vec[192] = expf((float)last);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (h0 + x >= G) break;
      uint8_t* out = ws + ((size_t)blk * a.Hv + hk * G + h0 + x) * kBlock;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = warp * 16 + (lane >> 2) + half * 8;
        const float gh = s.ghi[x][i], gl = s.glo[x][i], ak = s.beta[x][i] * s.ik[i], pq = s.iq[i];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
          if (nt > 2 * warp + 1) break;
          float p[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = nt * 8 + (lane & 3) * 2 + e;
            const float d = (gh - s.ghi[x][j]) + (gl - s.glo[x][j]);
            const float w = j <= i ? expf(fminf(d, 0.f)) * s.ik[j] : 0.f;
            s.at[x][j][i] = j < i ? ak * w * kk[nt][half * 2 + e] : 0.f;
            p[e] = j <= i ? pq * w * qk[nt][half * 2 + e] : 0.f;
          }
          uint32_t hi, lo;
          split2(p[0], p[1], hi, lo);
          const uint32_t at = tile_at(i, nt * 8 + (lane & 3) * 2);
          *reinterpret_cast<uint32_t*>(out + kPHi + at) = hi;
          *reinterpret_cast<uint32_t*>(out + kPLo + at) = lo;
        }
      }
    }
    __syncthreads();
    {
      const int x = warp >> 1, j = (warp & 1) * 32 + lane;
      if (h0 + x < G) {
        uint8_t* out = ws + ((size_t)blk * a.Hv + hk * G + h0 + x) * kBlock;
        unsigned long long col[kC / 2];
        if (warp & 1) solve_column<32>(s.at[x], j, col);
        else solve_column<0>(s.at[x], j, col);
        const float b = s.beta[x][j];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const float v = b * __uint_as_float(i & 1 ? (uint32_t)(col[i / 2] >> 32) : (uint32_t)col[i / 2]);
          if (i >= (j & ~15)) store_parts(out + kTHi, out + kTLo, tile_at(i, j), v);
        }
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ chain
template <int DK, int W>
struct ChainSmem {
  static constexpr int kDv = 16 * W;
  static constexpr int kPitch = DK * 2 + 16, kPitchV = kDv * 2 + 16;
  struct Stage {
    alignas(128) uint8_t block[kBlock];
    uint8_t k[kC * kPitch], q[kC * kPitch], v[kC * kPitchV];
  };
  Stage stage[2];
  uint8_t out[W][kC * 32];  // a warp's 16 columns of o, 32 bytes per token
  uint64_t full[2], empty[2];
};

// One CTA per (sequence, value head, 16 W columns of the state).  Columns never meet, so each
// of W warps owns 16 of them: S^T [16][DK] in registers as fp32 accumulators, which are the A
// operand of the next product as they lie.  No warp waits for another, only for the loads,
// which an extra warp issues two chunks ahead.
template <int DK, int W>
__global__ void __launch_bounds__(W * 32 + 32) gdr_chain_kernel(GdrArgs a, const uint8_t* ws) {
  using Smem = ChainSmem<DK, W>;
  extern __shared__ __align__(128) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = a.dv / Smem::kDv;
  const int unit = blockIdx.x;
  const int slice = unit % slices, h = unit / slices % a.Hv, n = unit / slices / a.Hv;
  const int hk = h / (a.Hv / a.Hk);
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;  // every warp finds the same
  const int chunks = (t1 - t0 + kC - 1) / kC, base = block_base(t0, n);

  // rows behind the last token are not loaded: what lies there must be finite
  for (int i = threadIdx.x; i < (int)sizeof(s.stage) / 16; i += W * 32 + 32)
    reinterpret_cast<uint4*>(s.stage)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], W);
    }
    mbar_fence_init();
  }
  fence_proxy_async();
  __syncthreads();

  if (warp == W) {  // loads
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + (size_t)hk * DK;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (size_t)hk * DK;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + (size_t)h * a.dv + slice * Smem::kDv;
    bool ok = true;
    int c = 0;
    for (; c < chunks; ++c) {
      const int b = c & 1;
      if (c >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&s.empty[b], (c / 2 - 1) & 1, kSpins));
      if (!ok) break;
      auto& st = s.stage[b];
      const int len = min(kC, t1 - t0 - c * kC);
      if (lane == 0)
        mbar_arrive_expect_tx(&s.full[b], kBlock + len * (2 * DK * 2 + Smem::kDv * 2));
      __syncwarp();
      if (lane == 0)
        bulk_g2s(st.block, ws + ((size_t)(base + c) * a.Hv + h) * kBlock, kBlock, &s.full[b]);
      for (int r = lane; r < len; r += 32) {
        const size_t t = (size_t)(t0 + c * kC + r);
        bulk_g2s(st.k + r * Smem::kPitch, k + t * a.ldk, DK * 2, &s.full[b]);
        bulk_g2s(st.q + r * Smem::kPitch, q + t * a.ldq, DK * 2, &s.full[b]);
        bulk_g2s(st.v + r * Smem::kPitchV, v + t * a.ldv, Smem::kDv * 2, &s.full[b]);
      }
    }
    // loads in flight land before shared memory is released
    for (int j = max(0, c - 2); j < c; ++j) mbar_wait(&s.full[j & 1], (j / 2) & 1, kSpins);
    if (!ok && lane == 0) atomicExch(a.status, KDA_ERR_TIMEOUT);
    return;
  }

  const int g = lane >> 2, t = lane & 3;
  const int col0 = slice * Smem::kDv + warp * 16;  // this warp's columns of the state
  // S^T: tile x holds rows (d_v) col0 + g, + 8 and columns (d_k) 8 x + 2 t, + 1
  float S[DK / 8][4];
  const size_t mat = ((size_t)slot * a.Hv + h) * DK * a.dv;
#pragma unroll
  for (int x = 0; x < DK / 8; ++x)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      S[x][e] = a.S0 ? a.S0[mat + (size_t)(x * 8 + t * 2 + (e & 1)) * a.dv + col0 + g + (e >> 1) * 8] : 0.f;

  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + (size_t)h * a.dv + col0;
  // lane parts of the fragment addresses: B from rows of tokens (plain) or columns (trans)
  const uint32_t nb = (lane & 7) + ((lane >> 4) << 3), kb = (lane >> 3) & 1;
  const uint32_t tr = (lane & 7) + (((lane >> 3) & 1) << 3), tc = lane >> 4;
  const uint32_t out = smem_u32(s.out[warp]);
  bool ok = true;
  for (int c = 0; c < chunks; ++c) {
    const int b = c & 1;
    ok = __all_sync(0xffffffffu, mbar_wait(&s.full[b], (c / 2) & 1, kSpins));
    if (!ok) break;
    auto& st = s.stage[b];
    const uint32_t sk = smem_u32(st.k), sq = smem_u32(st.q), sv = smem_u32(st.v);
    const uint32_t sb = smem_u32(st.block);
    const float* vec = reinterpret_cast<const float*>(st.block + kVec);

    // X^T = S^T K^T, Y^T = S^T Q^T
    float X[8][4] = {}, Y[8][4] = {};
#pragma unroll
    for (int x = 0; x < DK / 16; ++x) {
      uint32_t hi[4], lo[4];
      split_a(S[2 * x], S[2 * x + 1], hi, lo);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t fk[4], fq[4];
        const uint32_t at = (p * 16 + nb) * Smem::kPitch + x * 32 + kb * 16;
        ldsm4(fk, sk + at);
        ldsm4(fq, sq + at);
        mma(X[2 * p], hi, fk[0], fk[1]);
        mma(X[2 * p + 1], hi, fk[2], fk[3]);
        mma(Y[2 * p], hi, fq[0], fq[1]);
        mma(Y[2 * p + 1], hi, fq[2], fq[3]);
        mma(X[2 * p], lo, fk[0], fk[1]);
        mma(X[2 * p + 1], lo, fk[2], fk[3]);
        mma(Y[2 * p], lo, fq[0], fq[1]);
        mma(Y[2 * p + 1], lo, fq[2], fq[3]);
      }
    }
    // V^T - e^g X^T (ik in a); e^g Y^T
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t fv[4];  // tokens 16 p + (0-7, 8-15) x columns (0-7, 8-15): r = token half + 2 column half
      ldsm4t(fv, sv + (p * 16 + tr) * Smem::kPitchV + warp * 32 + tc * 16);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float2 va = *reinterpret_cast<const float2*>(vec + p * 16 + u * 8 + t * 2);
        const float2 vb = *reinterpret_cast<const float2*>(vec + 64 + p * 16 + u * 8 + t * 2);
        float(&xx)[4] = X[2 * p + u];
        float(&yy)[4] = Y[2 * p + u];
        xx[0] = fmaf(-va.x, xx[0], __uint_as_float(fv[u] << 16));
        xx[1] = fmaf(-va.y, xx[1], __uint_as_float(fv[u] & 0xffff0000u));
        xx[2] = fmaf(-va.x, xx[2], __uint_as_float(fv[u + 2] << 16));
        xx[3] = fmaf(-va.y, xx[3], __uint_as_float(fv[u + 2] & 0xffff0000u));
        yy[0] *= vb.x; yy[1] *= vb.y; yy[2] *= vb.x; yy[3] *= vb.y;
      }
    }
    // U^T = X^T T^T, the blocks of T on and below its diagonal
    float U[8][4] = {};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t hi[4], lo[4];
      split_a(X[2 * x], X[2 * x + 1], hi, lo);
#pragma unroll
      for (int p = x; p < 4; ++p) {
        uint32_t fh[4], fl[4];
        const uint32_t at = tile_at(p * 16 + nb, x * 16 + kb * 8);
        ldsm4(fh, sb + kTHi + at);
        ldsm4(fl, sb + kTLo + at);
        mma(U[2 * p], hi, fh[0], fh[1]);
        mma(U[2 * p + 1], hi, fh[2], fh[3]);
        mma(U[2 * p], lo, fh[0], fh[1]);
        mma(U[2 * p + 1], lo, fh[2], fh[3]);
        mma(U[2 * p], hi, fl[0], fl[1]);
        mma(U[2 * p + 1], hi, fl[2], fl[3]);
      }
    }
    // O^T = e^g Y^T + U^T P^T
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t hi[4], lo[4];
      split_a(U[2 * x], U[2 * x + 1], hi, lo);
#pragma unroll
      for (int p = x; p < 4; ++p) {
        uint32_t fh[4], fl[4];
        const uint32_t at = tile_at(p * 16 + nb, x * 16 + kb * 8);
        ldsm4(fh, sb + kPHi + at);
        ldsm4(fl, sb + kPLo + at);
        mma(Y[2 * p], hi, fh[0], fh[1]);
        mma(Y[2 * p + 1], hi, fh[2], fh[3]);
        mma(Y[2 * p], lo, fh[0], fh[1]);
        mma(Y[2 * p + 1], lo, fh[2], fh[3]);
        mma(Y[2 * p], hi, fl[0], fl[1]);
        mma(Y[2 * p + 1], hi, fl[2], fl[3]);
      }
    }
    // S^T <- e^{g_C} S^T + (e^{g_C - g} U)^T K
    {
      const float eG = vec[192];
#pragma unroll
      for (int x = 0; x < DK / 8; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[x][e] *= eG;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float2 ku = *reinterpret_cast<const float2*>(vec + 128 + x * 16 + u * 8 + t * 2);
          float(&uu)[4] = U[2 * x + u];
          uu[0] *= ku.x; uu[1] *= ku.y; uu[2] *= ku.x; uu[3] *= ku.y;
        }
        uint32_t hi[4], lo[4];
        split_a(U[2 * x], U[2 * x + 1], hi, lo);
#pragma unroll
        for (int p = 0; p < DK / 16; ++p) {
          uint32_t f[4];  // tokens 16 x + (0-7, 8-15) x channels 16 p + (0-7, 8-15)
          ldsm4t(f, sk + (x * 16 + tr) * Smem::kPitch + p * 32 + tc * 16);
          mma(S[2 * p], hi, f[0], f[1]);
          mma(S[2 * p + 1], hi, f[2], f[3]);
          mma(S[2 * p], lo, f[0], f[1]);
          mma(S[2 * p + 1], lo, f[2], f[3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.empty[b]);

    // o: the tiles transposed through shared memory, then 32 bytes per token
    const int len = min(kC, t1 - t0 - c * kC);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t r[4] = {pack_bf162(Y[2 * p][0], Y[2 * p][1]), pack_bf162(Y[2 * p + 1][0], Y[2 * p + 1][1]),
                             pack_bf162(Y[2 * p][2], Y[2 * p][3]), pack_bf162(Y[2 * p + 1][2], Y[2 * p + 1][3])};
      const uint32_t row = p * 16 + tr;  // the 16-byte halves swapped every four rows: no bank conflicts
      stsm4t(out + row * 32 + ((tc ^ ((row >> 2) & 1)) << 4), r);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 16 + (lane >> 1), half = lane & 1;
      const uint4 w = *reinterpret_cast<const uint4*>(s.out[warp] + row * 32 + ((half ^ ((row >> 2) & 1)) << 4));
      if (row < len)
        *reinterpret_cast<uint4*>(o + (size_t)(t0 + c * kC + row) * a.Hv * a.dv + half * 8) = w;
    }
    __syncwarp();
  }
  if (!ok) {
    if (lane == 0) atomicExch(a.status, KDA_ERR_TIMEOUT);
    return;
  }
#pragma unroll
  for (int x = 0; x < DK / 8; ++x)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      a.S_T[mat + (size_t)(x * 8 + t * 2 + (e & 1)) * a.dv + col0 + g + (e >> 1) * 8] = S[x][e];
}

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK, int W>
cudaError_t launch_chain(const GdrArgs& a, const uint8_t* ws, cudaStream_t s) {
  const size_t bytes = sizeof(ChainSmem<DK, W>);
  const cudaError_t e = allow_smem(gdr_chain_kernel<DK, W>, bytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)a.N * a.Hv * (a.dv / (16 * W));
  gdr_chain_kernel<DK, W><<<grid, W * 32 + 32, bytes, s>>>(a, ws);
  return cudaGetLastError();
}

template <int DK>
cudaError_t launch_dk(const GdrArgs& a, uint8_t* ws, cudaStream_t s) {
  const size_t bytes = sizeof(PrepSmem<DK>);
  cudaError_t e = allow_smem(gdr_prep_kernel<DK>, bytes);
  if (e != cudaSuccess) return e;
  gdr_prep_kernel<DK><<<dim3(a.T_total / kC + a.N, a.Hk), kPrepThreads, bytes, s>>>(a, ws);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.dv % 128 == 0) return launch_chain<DK, 8>(a, ws, s);
  if (a.dv == 64) return launch_chain<DK, 4>(a, ws, s);
  return launch_chain<DK, 2>(a, ws, s);
}

}  // namespace

bool gdr_chunked_supported(int d_k, int d_v, int dtype) {
  return dtype == KDA_BF16 && (d_k == 32 || d_k == 64 || d_k == 128) && d_v % 32 == 0;
}

size_t gdr_chunked_workspace_bytes(int T_total, int N, int Hv) {
  return ((size_t)(T_total / kC) + N) * Hv * kBlock;
}

cudaError_t launch_gdr_chunked(const GdrArgs& a, void* workspace, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  switch (a.dk) {
    case 32: return launch_dk<32>(a, ws, s);
    case 64: return launch_dk<64>(a, ws, s);
    case 128: return launch_dk<128>(a, ws, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kda
