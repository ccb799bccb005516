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
// Precision: the final states are fp32 results, so no operand on the state's way may be
// rounded to bf16.  K, Q and V are bf16 as they come and enter the products unscaled (norms
// and decays multiply rows of results or fp32 operands).  Everything else enters as a sum of
// bf16 parts: the state, V - e^g K S, U and T as three (24 bits, an fp32 value), of whose
// products those of order 2^-24 are left out; what only o sees (Q S and P U, rounded to bf16
// in the end) as two.
#include "gdr_chunked.cuh"

namespace kda {
namespace {

using namespace umma;

// ------------------------------------------------------------------ fragments
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
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
// The accumulators of two neighbouring 16 x 8 tiles as the parts of a 16 x 16 A operand: the
// layouts agree element by element.
template <int kParts>
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4],
                                        uint32_t (&p)[kParts][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[kParts];
    split2<kParts>((i < 2 ? c0 : c1)[2 * (i & 1)], (i < 2 ? c0 : c1)[2 * (i & 1) + 1], w);
#pragma unroll
    for (int k = 0; k < kParts; ++k) p[k][i] = w[k];
  }
}

// ------------------------------------------------------------------ prep
// One CTA per (chunk, query / key head): the two Grams once, then for each value head its
// decays, A, P and the inverse of I + A:
//   the four 16 x 16 diagonal blocks by forward substitution (a warp each, a lane per column),
//   then twice [X00 0; X10 X11] with X10 = -X11 (A10 X00), from 16 to 32 and from 32 to 64,
// all in fp32.  The operands are laid out in shared memory as the chain reads them and leave by
// bulk copies.
constexpr int kPrepThreads = 128;
constexpr int kPitchA = kC + 4;  // floats
constexpr int kScan = 4;         // heads whose decays are summed up at once, one per warp

template <int DK>
struct PrepSmem {
  static constexpr int kPitch = DK * 2 + 16;  // bytes: rows 16 bytes past a multiple of 128
  union {
    struct {
      __nv_bfloat16 k[kC * kPitch / 2], q[kC * kPitch / 2];
    };
    struct {
      float A[kC][kPitchA], X[kC][kPitchA];  // behind the Grams
    };
  };
  // staging: T's first two parts take A's place, the rest of the block lies here
  alignas(16) uint8_t rest[kBlock - 2 * kTile];
  float ik[kC], iq[kC];
  float ghi[kScan][kC], glo[kScan][kC], beta[kScan][kC];
  int n, t0, t1;
};

template <int DK>
__global__ void __launch_bounds__(kPrepThreads, 3) gdr_prep_kernel(GdrArgs a, uint8_t* ws) {
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
  }
  // running sums of the log decays of heads h0 .., one per warp, in 64 bits: differences of
  // them are taken
  const __nv_bfloat16* beta = static_cast<const __nv_bfloat16*>(a.beta);
  auto scan = [&](int h0) {
    if (h0 + warp >= G) return;
    const int h = hk * G + h0 + warp;
    double g2[2];
    float be[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = lane * 2 + i;
      const size_t at = (size_t)(t0 + (r < len ? r : 0)) * a.Hv + h;
      const float la = a.log_alpha[at], b = to_f32(beta[at]);
      g2[i] = r < len ? (double)gdr_log_decay(a, la, h) : 0.0;
      be[i] = r < len ? (a.beta_is_logit ? sigmoidf_(b) : b) : 0.f;
    }
    double sum = g2[0] + g2[1];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const double other = __shfl_up_sync(0xffffffffu, sum, m);
      if (lane >= m) sum += other;
    }
    const double g[2] = {sum - g2[1], sum};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = lane * 2 + i;
      const float hi = (float)g[i];
      s.ghi[warp][r] = hi;
      s.glo[warp][r] = (float)(g[i] - (double)hi);
      s.beta[warp][r] = be[i];
    }
  };
  scan(0);
  // the blocks of P above its diagonal stay zero
  for (int i = tid; i < (int)sizeof(s.rest) / 16; i += kPrepThreads)
    reinterpret_cast<uint4*>(s.rest)[i] = make_uint4(0, 0, 0, 0);
  cp_async_wait_all();
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

  for (int hg = 0; hg < G; ++hg) {
    const int x = hg % kScan;
    uint8_t* out = ws + ((size_t)blk * a.Hv + hk * G + hg) * kBlock;
    if (hg > 0) {
      if (tid == 0) bulk_wait_read();  // the last head's block has left shared memory
      if (x == 0) scan(hg);
      __syncthreads();
    }
    // A and P, from the Grams in registers; the vectors
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = warp * 16 + (lane >> 2) + half * 8;
      const float gh = s.ghi[x][i], gl = s.glo[x][i], ak = s.beta[x][i] * s.ik[i], pq = s.iq[i];
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        if (nt > 2 * warp + 1) break;
        float m[2], p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = nt * 8 + (lane & 3) * 2 + e;
          const float d = (gh - s.ghi[x][j]) + (gl - s.glo[x][j]);
          const float w = j <= i ? expf(fminf(d, 0.f)) * s.ik[j] : 0.f;
          m[e] = j < i ? ak * w * kk[nt][half * 2 + e] : 0.f;
          p[e] = j <= i ? pq * w * qk[nt][half * 2 + e] : 0.f;
        }
        const int j0 = nt * 8 + (lane & 3) * 2;
        *reinterpret_cast<float2*>(&s.A[i][j0]) = make_float2(m[0], m[1]);
        uint32_t w[2];
        split2<2>(p[0], p[1], w);
        uint8_t* dst = s.rest + (kP - 2 * kTile) + tile_at(i, j0);
        *reinterpret_cast<uint32_t*>(dst) = w[0];
        *reinterpret_cast<uint32_t*>(dst + kTile) = w[1];
      }
    }
    if (tid < kC) {
      float* vec = reinterpret_cast<float*>(s.rest + (kVec - 2 * kTile));
      const float gh = s.ghi[x][tid], gl = s.glo[x][tid], e = expf(gh);
      const float Gh = s.ghi[x][kC - 1], Gl = s.glo[x][kC - 1];
      vec[tid] = e * s.ik[tid];
      vec[64 + tid] = e * s.iq[tid];
      vec[128 + tid] = expf((Gh - gh) + (Gl - gl)) * s.ik[tid];
      if (tid == 0) vec[192] = expf(Gh);
    }
    __syncthreads();

    // diagonal blocks: column c of block `warp`, x_i = -sum_k A_ik x_k
    if (lane < 16) {
      const int b0 = warp * 16;
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float sum = i == lane ? 1.f : 0.f;
#pragma unroll
        for (int k = 0; k < i; ++k) sum = fmaf(-s.A[b0 + i][b0 + k], v[k], sum);
        v[i] = sum;
        s.X[b0 + i][b0 + lane] = sum;
      }
    }
    __syncthreads();
    // 16 -> 32: blocks (1, 0) and (3, 2), 64 threads each, four columns of a row per thread;
    // A10 X00 lies for the time being in the block above the diagonal
    {
      const int b0 = (tid >> 6) * 32, r = (tid >> 2) & 15, c = (tid & 3) * 4;
      float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float m = s.A[b0 + 16 + r][b0 + k];
        const float4 y = *reinterpret_cast<const float4*>(&s.X[b0 + k][b0 + c]);
        z.x = fmaf(m, y.x, z.x); z.y = fmaf(m, y.y, z.y);
        z.z = fmaf(m, y.z, z.z); z.w = fmaf(m, y.w, z.w);
      }
      *reinterpret_cast<float4*>(&s.X[b0 + r][b0 + 16 + c]) = z;
      __syncthreads();
      z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float m = -s.X[b0 + 16 + r][b0 + 16 + k];
        const float4 y = *reinterpret_cast<const float4*>(&s.X[b0 + k][b0 + 16 + c]);
        z.x = fmaf(m, y.x, z.x); z.y = fmaf(m, y.y, z.y);
        z.z = fmaf(m, y.z, z.z); z.w = fmaf(m, y.w, z.w);
      }
      *reinterpret_cast<float4*>(&s.X[b0 + 16 + r][b0 + c]) = z;
    }
    __syncthreads();
    // 32 -> 64, eight columns of a row per thread; entries above the diagonals count as zero
    {
      const int r = tid >> 2, c = (tid & 3) * 8;
      float z[8] = {};
      auto step = [&](float m, const float* y) {
        const float4 y0 = *reinterpret_cast<const float4*>(y);
        const float4 y1 = *reinterpret_cast<const float4*>(y + 4);
        z[0] = fmaf(m, y0.x, z[0]); z[1] = fmaf(m, y0.y, z[1]);
        z[2] = fmaf(m, y0.z, z[2]); z[3] = fmaf(m, y0.w, z[3]);
        z[4] = fmaf(m, y1.x, z[4]); z[5] = fmaf(m, y1.y, z[5]);
        z[6] = fmaf(m, y1.z, z[6]); z[7] = fmaf(m, y1.w, z[7]);
      };
      if (c < 16)
#pragma unroll 8
        for (int k = 0; k < 16; ++k) step(s.A[32 + r][k], &s.X[k][c]);
#pragma unroll 8
      for (int k = 16; k < 32; ++k) step(s.A[32 + r][k], &s.X[k][c]);
      *reinterpret_cast<float4*>(&s.X[r][32 + c]) = make_float4(z[0], z[1], z[2], z[3]);
      *reinterpret_cast<float4*>(&s.X[r][36 + c]) = make_float4(z[4], z[5], z[6], z[7]);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = 0.f;
#pragma unroll 8
      for (int k = 0; k < 16; ++k) step(-s.X[32 + r][32 + k], &s.X[k][32 + c]);
      if (r >= 16)
#pragma unroll 8
        for (int k = 16; k < 32; ++k) step(-s.X[32 + r][32 + k], &s.X[k][32 + c]);
      *reinterpret_cast<float4*>(&s.X[32 + r][c]) = make_float4(z[0], z[1], z[2], z[3]);
      *reinterpret_cast<float4*>(&s.X[32 + r][c + 4]) = make_float4(z[4], z[5], z[6], z[7]);
    }
    __syncthreads();
    // T = (I + A)^-1 Diag(beta) in three parts, eight columns at a time; A is done with
#pragma unroll 1
    for (int i = tid; i < kC * 8; i += kPrepThreads) {
      const int r = i >> 3, c = (i & 7) * 8;
      uint4 w[3] = {};
      if (c <= r) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 y = *reinterpret_cast<const float4*>(&s.X[r][c + e]);
          const float4 be = *reinterpret_cast<const float4*>(&s.beta[x][c + e]);
          v[e] = y.x * be.x; v[e + 1] = y.y * be.y; v[e + 2] = y.z * be.z; v[e + 3] = y.w * be.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e <= r ? v[e] : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t p[3];
          split2<3>(v[2 * e], v[2 * e + 1], p);
#pragma unroll
          for (int k = 0; k < 3; ++k) (&w[k].x)[e] = p[k];
        }
      }
      uint8_t* t01 = reinterpret_cast<uint8_t*>(s.A) + tile_at(r, c);
      *reinterpret_cast<uint4*>(t01) = w[0];
      *reinterpret_cast<uint4*>(t01 + kTile) = w[1];
      *reinterpret_cast<uint4*>(s.rest + tile_at(r, c)) = w[2];
    }
    fence_proxy_async();
    __syncthreads();
    if (tid == 0) {
      bulk_s2g(out, s.A, 2 * kTile);
      bulk_s2g(out + 2 * kTile, s.rest, kBlock - 2 * kTile);
      bulk_commit();
    }
  }
  if (tid == 0) bulk_wait_all();
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
      if (c >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&s.empty[b], (c / 2 - 1) & 1, kGdrSpins));
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
    for (int j = max(0, c - 2); j < c; ++j) mbar_wait(&s.full[j & 1], (j / 2) & 1, kGdrSpins);
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
    ok = __all_sync(0xffffffffu, mbar_wait(&s.full[b], (c / 2) & 1, kGdrSpins));
    if (!ok) break;
    auto& st = s.stage[b];
    const uint32_t sk = smem_u32(st.k), sq = smem_u32(st.q), sv = smem_u32(st.v);
    const uint32_t sb = smem_u32(st.block);
    const float* vec = reinterpret_cast<const float*>(st.block + kVec);

    // X^T = S^T K^T, Y^T = S^T Q^T
    float X[8][4] = {}, Y[8][4] = {};
#pragma unroll
    for (int x = 0; x < DK / 16; ++x) {
      uint32_t f[3][4];
      split_a<3>(S[2 * x], S[2 * x + 1], f);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t fk[4], fq[4];
        const uint32_t at = (p * 16 + nb) * Smem::kPitch + x * 32 + kb * 16;
        ldsm4(fk, sk + at);
        ldsm4(fq, sq + at);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          mma(X[2 * p], f[i], fk[0], fk[1]);
          mma(X[2 * p + 1], f[i], fk[2], fk[3]);
          if (i == 2) break;
          mma(Y[2 * p], f[i], fq[0], fq[1]);
          mma(Y[2 * p + 1], f[i], fq[2], fq[3]);
        }
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
      uint32_t f[3][4];
      split_a<3>(X[2 * x], X[2 * x + 1], f);
#pragma unroll
      for (int p = x; p < 4; ++p) {
        const uint32_t at = sb + kT + tile_at(p * 16 + nb, x * 16 + kb * 8);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          uint32_t m[4];
          ldsm4(m, at + j * kTile);
#pragma unroll
          for (int i = 0; i < 3 - j; ++i) {
            mma(U[2 * p], f[i], m[0], m[1]);
            mma(U[2 * p + 1], f[i], m[2], m[3]);
          }
        }
      }
    }
    // O^T = e^g Y^T + U^T P^T
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t f[2][4];
      split_a<2>(U[2 * x], U[2 * x + 1], f);
#pragma unroll
      for (int p = x; p < 4; ++p) {
        const uint32_t at = sb + kP + tile_at(p * 16 + nb, x * 16 + kb * 8);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t m[4];
          ldsm4(m, at + j * kTile);
#pragma unroll
          for (int i = 0; i < 2 - j; ++i) {
            mma(Y[2 * p], f[i], m[0], m[1]);
            mma(Y[2 * p + 1], f[i], m[2], m[3]);
          }
        }
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
        uint32_t f[3][4];
        split_a<3>(U[2 * x], U[2 * x + 1], f);
#pragma unroll
        for (int p = 0; p < DK / 16; ++p) {
          uint32_t m[4];  // tokens 16 x + (0-7, 8-15) x channels 16 p + (0-7, 8-15)
          ldsm4t(m, sk + (x * 16 + tr) * Smem::kPitch + p * 32 + tc * 16);
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            mma(S[2 * p], f[i], m[0], m[1]);
            mma(S[2 * p + 1], f[i], m[2], m[3]);
          }
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
  if (gdr_chain_tc_takes(a)) return launch_gdr_chain_tc(a, ws, s);
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
