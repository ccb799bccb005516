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
// parallel.  chain: the state's walk over the chunks of a sequence (gdr_chain_tc.cu; here
// the one for d_v of 32 and 64 and d_k of 32).  4096 tokens x 96 heads of 128 x 128: 100 and
// 202 us.
//
// Precision: the final states are fp32 results, so no operand on the state's way may be
// rounded to bf16.  K, Q and V are bf16 as they come and enter the products unscaled (norms
// and decays multiply rows of results or fp32 operands).  Everything else enters as a sum of
// three bf16 parts (24 bits, an fp32 value), of whose products those of order 2^-24 are left
// out.  Only Q S, which o alone sees, takes the first two of the state's parts: 2^-17 at most,
// and in the walk on tcgen05 the third part has to make room for what X becomes meanwhile.
// With P and U in two parts too, o would be off by 4.4e-6 of its size before it is rounded, not by
// 7e-7 (by emulation, sums exact); 4096 tokens x 96 heads took 22 us less so.
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
__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
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
// The accumulators of two neighbouring 16 x 8 tiles as the parts of a 16 x 16 A operand: the
// layouts agree element by element.
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4],
                                        uint32_t (&p)[3][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = (i < 2 ? c0 : c1)[2 * (i & 1)], y = (i < 2 ? c0 : c1)[2 * (i & 1) + 1];
    split3(x, y, p[0][i], p[1][i], p[2][i]);
  }
}

// ------------------------------------------------------------------ prep
// One CTA per (chunk, query / key head).  All four warps form the two Grams, K K^T and Q K^T, in
// fp32 in shared memory.  Then each pair of warps takes every other value head, on its own: the
// running sums of its decays, the inverse of I + A, T, P and the vectors.
//
// The inverse X, in 16 x 16 blocks: the diagonal ones by forward substitution (a lane per
// column), then column by column X_ij = -X_ii sum_k A_ik X_kj on the tensor cores, transposed, so
// that each result is the A operand of the next product as it lies:
//     tmp^T = sum_k X_kj^T A_ik^T,   X_ij^T = -tmp^T X_ii^T,
// every operand in three bf16 parts.  One warp takes column 0, the other 1 and 2
// and the first rows of P.
//
// No one thing bounds it: 16 warps per SM issue in 40 % of the cycles, shared memory is busy in
// half of them, 104 MB are read and 193 MB written in 100 us (151 MB to DRAM by its end), and taking
// any one step out saves 4 to 30 us.
//
// e^{g_i - g_j} off the diagonal blocks is e^{g_i - g_r} e^{g_r - g_j}, r the first row of i's
// block: both exponents are <= 0, and the factors are vectors.
constexpr int kPrepThreads = 128;
constexpr int kPitchG = kC + 8;          // floats, Grams: pairs of four rows meet no bank twice
constexpr int kPitchD = 20, kDiag = 324;  // floats, diagonal blocks and from one to the next
struct PrepHead {
  float ghi[kC], glo[kC], beta[kC];
  float e1[kC];      // e^{g_i - g_r}
  float e2[96];      // e^{g_r - g_j} ik_j, j < 16 x, of row blocks x = 1, 2, 3: from 0, 16, 48 on
};

__host__ __device__ constexpr int e2_at(int x) { return 8 * x * (x - 1); }

template <int DK>
struct PrepSmem {
  static constexpr int kPitch = DK * 2 + 16;  // bytes: rows 16 bytes past a multiple of 128
  union {
    struct {
      __nv_bfloat16 k[kC * kPitch / 2], q[kC * kPitch / 2];
    };
    struct {
      float kk[kC][kPitchG], qk[kC][kPitchG];
    };
  };
  float diag[2][4 * kDiag];          // A's diagonal blocks, then their inverses, per pair
  alignas(16) uint8_t out[4][1536];  // three 16 x 16 blocks of bf16 per warp
  PrepHead head[2];
  float ik[kC], iq[kC];
  int n, t0, t1;
};

// Differences of running sums are taken, so the sums are kept as hi + lo, exact to about 2^-48.
struct Sum2 {
  float hi, lo;
};
__device__ __forceinline__ Sum2 add2(Sum2 a, Sum2 b) {
  const float s = __fadd_rn(a.hi, b.hi), v = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, v)), __fsub_rn(b.hi, v));
  const float lo = __fadd_rn(e, __fadd_rn(a.lo, b.lo)), hi = __fadd_rn(s, lo);
  return {hi, __fsub_rn(lo, __fsub_rn(hi, s))};
}
// e^{g_i - g_j}, j <= i
__device__ __forceinline__ float decay_factor(float hi_i, float lo_i, float hi_j, float lo_j) {
  const float d = (hi_i - hi_j) + (lo_i - lo_j);
  return expf(d > 0.f ? 0.f : d);  // rounding apart, d <= 0; NaN stays
}

// Three 16 x 16 blocks of bf16, parts of T (kTrans: from their transposes) or of P, from 8 x 8 tiles w
// to 32-byte rows of the tiles from `tile` on: through shared memory, 16 bytes per lane.
template <bool kTrans>
__device__ __forceinline__ void store_blocks(uint8_t* tile, int row0, int col0, uint8_t* buf, int lane,
                                             const uint32_t (&w)[3][4]) {
  constexpr int kN = 3;
  // lane l names row l & 7 of tile l >> 3; halves are swapped every four rows against conflicts
  const uint32_t r = (lane & 7) + ((lane >> (kTrans ? 4 : 3)) & 1) * 8, h = (lane >> (kTrans ? 3 : 4)) & 1;
  const uint32_t at = smem_u32(buf) + r * 32 + ((h ^ ((r >> 2) & 1)) << 4);
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    if constexpr (kTrans) stsm4t(at + k * 512, w[k]);
    else stsm4(at + k * 512, w[k]);
  }
  __syncwarp();
  const int row = lane >> 1, half = lane & 1;
  const uint8_t* from = buf + row * 32 + ((half ^ ((row >> 2) & 1)) << 4);
  uint8_t* to = tile + tile_at(row0 + row, col0 + half * 8);
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    uint8_t* at = to + k * kTile;
    if (!kTrans && k == 2) {
      const PlaceOfP p = third_of_p(row0 / 16, col0 / 16);
      at = tile + p.tile * kTile + tile_at(p.row * 16 + row, p.col * 16 + half * 8);
    }
    *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(from + k * 512);
  }
  __syncwarp();
}

// One column of the inverse below its diagonal block, and T's blocks of that column.
template <int J, int DK>
__device__ __forceinline__ void invert_column(const PrepSmem<DK>& s, const PrepHead& hd, const float* diag,
                                              int lane, uint8_t* buf, uint8_t* out) {
  const int g = lane >> 2, t = lane & 3;
  const float b0 = hd.beta[J * 16 + g], b1 = hd.beta[J * 16 + g + 8];
  // c: a block of X^T (rows: X's columns), as two 16 x 8 tiles; its parts as an A operand, and T's
  auto finish = [&](const float (&c)[2][4], int i, uint32_t (&f)[3][4]) {
    split_a(c[0], c[1], f);
    float z[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      z[x][0] = c[x][0] * b0; z[x][1] = c[x][1] * b0;
      z[x][2] = c[x][2] * b1; z[x][3] = c[x][3] * b1;
    }
    uint32_t w[3][4];
    split_a(z[0], z[1], w);
    store_blocks<true>(out + kT, i * 16, J * 16, buf, lane, w);
  };
  // six products of parts, smaller ones first
  auto product = [&](float (&c)[2][4], const uint32_t (&f)[3][4], const uint32_t (&m)[3][4]) {
#pragma unroll
    for (int order = 2; order >= 0; --order)
#pragma unroll
      for (int j = 0; j <= order; ++j) {
        mma(c[0], f[order - j], m[j][0], m[j][1]);
        mma(c[1], f[order - j], m[j][2], m[j][3]);
      }
  };
  uint32_t X[3][3][4];  // parts of X_kJ^T, k from J on
  {
    const float* d = diag + J * kDiag;
    float c[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[x][e] = d[(x * 8 + t * 2 + (e & 1)) * kPitchD + g + (e >> 1) * 8];
    finish(c, J, X[0]);
  }
#pragma unroll
  for (int i = J + 1; i < 4; ++i) {
    float c[2][4] = {};
    // A_ik^T as B operands: rows 16 i + 8 x + g of A
    float row[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = i * 16 + x * 8 + g;
      row[x] = hd.beta[r] * s.ik[r] * hd.e1[r];
    }
#pragma unroll
    for (int k = J; k < i; ++k) {
      uint32_t m[3][4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int col = k * 16 + y * 8 + t * 2;
        const float2 e2 = *reinterpret_cast<const float2*>(&hd.e2[e2_at(i) + col]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 kk = *reinterpret_cast<const float2*>(&s.kk[i * 16 + x * 8 + g][col]);
          split3(row[x] * (e2.x * kk.x), row[x] * (e2.y * kk.y), m[0][x * 2 + y], m[1][x * 2 + y], m[2][x * 2 + y]);
        }
      }
      product(c, X[k - J], m);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[x][e] = -c[x][e];
    uint32_t f[3][4], m[3][4];
    split_a(c[0], c[1], f);
    const float* d = diag + i * kDiag;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float2 v = *reinterpret_cast<const float2*>(&d[(x * 8 + g) * kPitchD + y * 8 + t * 2]);
        split3(v.x, v.y, m[0][x * 2 + y], m[1][x * 2 + y], m[2][x * 2 + y]);
      }
    float z[2][4] = {};
    product(z, f, m);
    uint32_t last[3][4];
    if (i < 3) finish(z, i, X[i - J]);
    else finish(z, i, last);
  }
}

template <int DK>
__global__ void __launch_bounds__(kPrepThreads, 4) gdr_prep_kernel(GdrArgs a, uint8_t* ws) {
  using Smem = PrepSmem<DK>;
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int blk = blockIdx.x, hk = blockIdx.y, G = a.Hv / a.Hk;

  if (warp == 0) {
    // the sequence of this block: the last one whose base is not behind it, as far as the
    // offsets do not decrease (later sequences are left out)
    int n = a.N == 1 ? 0 : -1;
    for (int i0 = 0; i0 < a.N && a.N > 1; i0 += 32) {
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
  const int pair = warp >> 1, second = warp & 1;
  PrepHead& hd = s.head[pair];
  // running sums of the log decays of head hg, by one warp: two tokens per lane
  const __nv_bfloat16* beta = static_cast<const __nv_bfloat16*>(a.beta);
  float la[2], be[2];
  auto fetch_decays = [&](int hg) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = lane * 2 + i;
      const size_t at = (size_t)(t0 + (r < len ? r : 0)) * a.Hv + hk * G + hg;
      la[i] = a.log_alpha[at];
      be[i] = to_f32(beta[at]);
    }
  };
  auto scan = [&](int hg, PrepHead& to) {
    Sum2 g[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = lane * 2 + i < len;
      g[i] = {in ? gdr_log_decay(a, la[i], hk * G + hg) : 0.f, 0.f};
      to.beta[lane * 2 + i] = in ? (a.beta_is_logit ? sigmoidf_(be[i]) : be[i]) : 0.f;
    }
    g[1] = add2(g[0], g[1]);
    Sum2 before = {0.f, 0.f}, sum = g[1];  // of the lanes before this one
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const Sum2 other = {__shfl_up_sync(0xffffffffu, sum.hi, m), __shfl_up_sync(0xffffffffu, sum.lo, m)};
      if (lane >= m) {
        sum = add2(other, sum);
        before = add2(other, before);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Sum2 x = add2(before, g[i]);
      to.ghi[lane * 2 + i] = x.hi;
      to.glo[lane * 2 + i] = x.lo;
    }
  };
  // the factors of e^{g_i - g_j}, when the sums and the norms are there
  auto factors = [&] {
    const int r = lane + second * 32, r0 = r & ~15;
    const float hi = hd.ghi[r], lo = hd.glo[r], ik = s.ik[r];
    const float e1 = decay_factor(hi, lo, hd.ghi[r0], hd.glo[r0]);
    float e2[3];
#pragma unroll
    for (int x = 1; x < 4; ++x) e2[x - 1] = ik * decay_factor(hd.ghi[16 * x], hd.glo[16 * x], hi, lo);
    hd.e1[r] = e1;
#pragma unroll
    for (int x = 1; x < 4; ++x)
      if (r < 16 * x) hd.e2[e2_at(x) + r] = e2[x - 1];
  };
  // the first two heads: warps 0 and 1, which have the fewest tiles of the Grams
  const bool scans = warp < 2 && warp < G;
  if (scans) fetch_decays(warp);
  cp_async_wait_all();
  __syncthreads();
  if (scans) scan(warp, s.head[warp]);

  // K K^T and Q K^T, 16 rows per warp, columns up to the diagonal block
  {
    float kk[8][4] = {}, qk[8][4] = {}, qq[2] = {};
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
      for (int i = 0; i < 4; ++i) {  // |q|^2 of rows g and g + 8
        const float lo = __uint_as_float(fq[i] << 16), hi = __uint_as_float(fq[i] & 0xffff0000u);
        qq[i & 1] = fmaf(lo, lo, fmaf(hi, hi, qq[i & 1]));
      }
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
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      qq[x] += __shfl_xor_sync(0xffffffffu, qq[x], 1);
      qq[x] += __shfl_xor_sync(0xffffffffu, qq[x], 2);
      if ((lane & 3) == 0)
        s.iq[warp * 16 + (lane >> 2) + x * 8] = a.q_scale * (a.l2norm_qk ? gdr_inv_norm(qq[x], a.eps_l2) : 1.f);
    }
    // |k|^2: the diagonal, in the two column tiles of this warp's diagonal block
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = warp * 16 + (lane >> 2) + (e >> 1) * 8;
        if (nt >> 1 == warp && r == nt * 8 + (lane & 3) * 2 + (e & 1))
          s.ik[r] = a.l2norm_qk ? gdr_inv_norm(kk[nt][e], a.eps_l2) : 1.f;
      }
    __syncthreads();  // K and Q are done with
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt > 2 * warp + 1) break;
      const int r = warp * 16 + (lane >> 2), c = nt * 8 + (lane & 3) * 2;
      *reinterpret_cast<float2*>(&s.kk[r][c]) = make_float2(kk[nt][0], kk[nt][1]);
      *reinterpret_cast<float2*>(&s.kk[r + 8][c]) = make_float2(kk[nt][2], kk[nt][3]);
      *reinterpret_cast<float2*>(&s.qk[r][c]) = make_float2(qk[nt][0], qk[nt][1]);
      *reinterpret_cast<float2*>(&s.qk[r + 8][c]) = make_float2(qk[nt][2], qk[nt][3]);
    }
    if (pair < G) factors();
  }
  __syncthreads();

  const int g = lane >> 2, t = lane & 3;
  uint8_t* buf = s.out[warp];
  float* diag = s.diag[pair];
  const uint32_t bar = 1 + pair;
  for (int hg = pair; hg < G; hg += 2) {
    if (hg >= 2) {
      named_sync(bar, 64);  // both warps are done with the last head
      if (!second) {
        fetch_decays(hg);
        scan(hg, hd);
      }
      named_sync(bar, 64);
      factors();
      named_sync(bar, 64);
    }
    uint8_t* out = ws + ((size_t)blk * a.Hv + hk * G + hg) * kBlock;
    // A's diagonal blocks, two per warp, and P's: e[y][2 x + z] is row g + 8 x, column 8 y + 2 t + z
#pragma unroll
    for (int x2 = 0; x2 < 2; ++x2) {
      const int ib = second * 2 + x2, b0 = ib * 16;
      float* d = diag + ib * kDiag;
      float e[2][4], p[2][4];
      float rhi[2], rlo[2], rk[2], rq[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = b0 + g + x * 8;
        rhi[x] = hd.ghi[r]; rlo[x] = hd.glo[r]; rk[x] = hd.beta[r] * s.ik[r]; rq[x] = s.iq[r];
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int c = y * 8 + t * 2;
        const float2 chi = *reinterpret_cast<const float2*>(&hd.ghi[b0 + c]);
        const float2 clo = *reinterpret_cast<const float2*>(&hd.glo[b0 + c]);
        const float2 ck = *reinterpret_cast<const float2*>(&s.ik[b0 + c]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = g + x * 8;
          const float2 kk = *reinterpret_cast<const float2*>(&s.kk[b0 + r][b0 + c]);
          const float2 qk = *reinterpret_cast<const float2*>(&s.qk[b0 + r][b0 + c]);
          const float w0 = ck.x * decay_factor(rhi[x], rlo[x], chi.x, clo.x);
          const float w1 = ck.y * decay_factor(rhi[x], rlo[x], chi.y, clo.y);
          e[y][2 * x] = c < r ? rk[x] * w0 * kk.x : 0.f;
          e[y][2 * x + 1] = c + 1 < r ? rk[x] * w1 * kk.y : 0.f;
          p[y][2 * x] = c <= r ? rq[x] * w0 * qk.x : 0.f;
          p[y][2 * x + 1] = c + 1 <= r ? rq[x] * w1 * qk.y : 0.f;
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          *reinterpret_cast<float2*>(&d[(g + x * 8) * kPitchD + y * 8 + t * 2]) = make_float2(e[y][2 * x], e[y][2 * x + 1]);
      uint32_t w[3][4];
      split_a(p[0], p[1], w);
      store_blocks<false>(out + kP, b0, b0, buf, lane, w);
    }
    // x_i = -sum_k A_ik x_k: a half warp per block, a lane per column
    {
      float* d = diag + (second * 2 + (lane >> 4)) * kDiag;
      const int c = lane & 15;
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = i == c ? 1.f : 0.f;
#pragma unroll
      for (int i = 1; i < 16; ++i) {
        float A[16];
#pragma unroll
        for (int k = 0; k < i; k += 4) {
          const float4 y = *reinterpret_cast<const float4*>(&d[i * kPitchD + k]);
          A[k] = y.x; A[k + 1] = y.y; A[k + 2] = y.z; A[k + 3] = y.w;
        }
        float even = 0.f, odd = 0.f;
#pragma unroll
        for (int k = 0; k < i; k += 2) {
          even = fmaf(A[k], v[k], even);
          if (k + 1 < i) odd = fmaf(A[k + 1], v[k + 1], odd);
        }
        v[i] -= even + odd;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) d[i * kPitchD + c] = v[i];
    }
    named_sync(bar, 64);
    if (!second) {
      invert_column<0, DK>(s, hd, diag, lane, buf, out);
      invert_column<3, DK>(s, hd, diag, lane, buf, out);
    } else {
      invert_column<1, DK>(s, hd, diag, lane, buf, out);
      invert_column<2, DK>(s, hd, diag, lane, buf, out);
    }
    // P below its diagonal blocks: row block 3, and 1 and 2 (what is above them is never read)
#pragma unroll 1
    for (int ib = second ? 1 : 3; ib < (second ? 3 : 4); ++ib) {
      float row[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = ib * 16 + x * 8 + g;
        row[x] = s.iq[r] * hd.e1[r];
      }
#pragma unroll 1
      for (int jb = 0; jb < ib; ++jb) {
        float c[2][4];  // tiles of columns
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int col = jb * 16 + y * 8 + t * 2;
          const float2 e2 = *reinterpret_cast<const float2*>(&hd.e2[e2_at(ib) + col]);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 qk = *reinterpret_cast<const float2*>(&s.qk[ib * 16 + x * 8 + g][col]);
            c[y][2 * x] = row[x] * (e2.x * qk.x);
            c[y][2 * x + 1] = row[x] * (e2.y * qk.y);
          }
        }
        uint32_t w[3][4];
        split_a(c[0], c[1], w);
        store_blocks<false>(out + kP, ib * 16, jb * 16, buf, lane, w);
      }
    }
    const int r = lane + second * 32;
    float* vec = reinterpret_cast<float*>(out + kVec);
    const float gh = hd.ghi[r], gl = hd.glo[r], e = expf(gh);
    const float Gh = hd.ghi[kC - 1], Gl = hd.glo[kC - 1];
    vec[r] = e * s.ik[r];
    vec[64 + r] = e * s.iq[r];
    vec[128 + r] = decay_factor(Gh, Gl, gh, gl) * s.ik[r];
    if (r == 0) vec[192] = expf(Gh);
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
// which an extra warp issues two chunks ahead.  Bound by mma.sync, a quarter of tcgen05's rate:
// 4096 tokens x 96 heads of 128 x 128 took 519 us so; it is kept for the heads that tcgen05's 128
// rows do not fit (per-chunk kernel included, 4096 tokens x 32 heads of 64 x 64: 436 us; 2000
// tokens in five sequences x 16 heads of 32 x 256: 104 us).
template <int DK, int W>
__global__ void __launch_bounds__(W * 32 + 32) gdr_chain_kernel(GdrArgs a, const uint8_t* ws) {
  using Smem = ChainSmem<DK, W>;
  extern __shared__ __align__(128) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = a.dv / Smem::kDv;
  const int unit = blockIdx.x;
  const int slice = unit % slices, h = unit / slices % a.Hv, n = longest_first(a, unit / slices / a.Hv);
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
      split_a(S[2 * x], S[2 * x + 1], f);
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
      split_a(X[2 * x], X[2 * x + 1], f);
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
      uint32_t f[3][4];
      split_a(U[2 * x], U[2 * x + 1], f);
#pragma unroll
      for (int p = x; p < 4; ++p) {
        const uint32_t at = sb + kP + tile_at(p * 16 + nb, x * 16 + kb * 8);
        const PlaceOfP third = third_of_p(p, x);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          uint32_t m[4];
          ldsm4(m, j < 2 ? at + j * kTile : sb + kP + third.tile * kTile +
                                                tile_at(third.row * 16 + nb, third.col * 16 + kb * 8));
#pragma unroll
          for (int i = 0; i < 3 - j; ++i) {
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
        split_a(U[2 * x], U[2 * x + 1], f);
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

template <int DK, int W>
cudaError_t launch_chain(const GdrArgs& a, const uint8_t* ws, cudaStream_t s) {
  const size_t bytes = sizeof(ChainSmem<DK, W>);
  const cudaError_t e = allow_smem<gdr_chain_kernel<DK, W>>(bytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)a.N * a.Hv * (a.dv / (16 * W));
  gdr_chain_kernel<DK, W><<<grid, W * 32 + 32, bytes, s>>>(a, ws);
  return cudaGetLastError();
}

template <int DK>
cudaError_t launch_dk(const GdrArgs& a, uint8_t* ws, cudaStream_t s) {
  const size_t bytes = sizeof(PrepSmem<DK>);
  cudaError_t e = allow_smem<gdr_prep_kernel<DK>>(bytes);
  if (e != cudaSuccess) return e;
  gdr_prep_kernel<DK><<<dim3(a.T_total / kC + a.N, a.Hk), kPrepThreads, bytes, s>>>(a, ws);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.dv % 128 == 0) {
    if constexpr (DK == 32) return launch_chain<DK, 8>(a, ws, s);
    else return launch_gdr_chain_tc(a, ws, s);
  }
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
