// gdr_recurrent.cu -- the gated delta rule token by token, on the CUDA cores:
// the decode step (a few tokens per sequence) and every prefill that is not
// taken in chunks (fp32 data, short sequences).
//
// Columns of the state (the d_v index) never meet: column j of S needs only k,
// q, the decay, beta and v_j.  So one warp owns 16 columns of one head's state
// from its load to its store, in registers, and no warp waits for another:
// lane = (row group rg of 8) x (4 columns of float4), d_k / 8 rows each.  Both
// reductions over d_k are taken on the state as it stands,
//     u = S^T k,  r = S^T q,   w = beta (v - e^g u),
//     S <- e^g S + k w^T,      o = e^g r + (k.q) w,
// in one pass over the registers, and finished over the eight row groups by
// seven shuffles: at each level a lane hands half of its sums to its partner and
// keeps the other half, so that of the eight sums (u and r of four columns) each
// row group ends up with one.
//
// One token per sequence (decode): bound by reading and writing the state: 64
// sequences x 96 heads of 128 x 128, 810 MB, take 120 us, 1.01 of the measured copy
// bandwidth (some of it stays in L2).  More tokens: four for 24 sequences x 32
// heads with the state after each, 304 MB, take 51.6 us (0.88); long sequences are
// bound by the latency of a token's chain of reductions, 0.49 us (fp32, 64 x 128).  So whatever does
// not hang on the state is taken off it: the rows of the next tokens are fetched
// into a ring in shared memory, the warp's own; decays and betas are taken 32 tokens
// at a time, a token per lane; norms and k.q four at a time, a token for each of the
// four lanes that hold the same rows.
#include "gdr.cuh"
#include "umma.cuh"

namespace kda {
namespace {

constexpr int kRecWarps = 4, kRing = 8;

// V consecutive elements (8 or 16 bytes) widened to fp32.
template <int V, typename T>
__device__ __forceinline__ void load_vec(float* x, const T* p) {
  uint32_t w[V * sizeof(T) / 4];
  if constexpr (V * sizeof(T) == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  }
#pragma unroll
  for (int i = 0; i < V * (int)sizeof(T) / 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// kMany: any number of tokens per sequence; else one.
template <int DK, typename T, bool kMany>
__global__ void __launch_bounds__(kRecWarps * 32, kMany ? 3 : 4) gdr_recurrent_kernel(GdrArgs a) {
  constexpr int R = DK / 8;  // rows of the state per lane, in vectors of V: row group rg has
  constexpr int V = R < 16 / (int)sizeof(T) ? R : 16 / (int)sizeof(T);  // every eighth vector
  // a token in the ring: k, q, this warp's 16 values
  constexpr int kTokenBytes = (2 * DK + 16) * (int)sizeof(T);
  extern __shared__ __align__(16) uint8_t ring_all[];
  uint8_t* ring = ring_all + (threadIdx.x >> 5) * kRing * kTokenBytes;

  const int lane = threadIdx.x & 31, rg = lane >> 2, c4 = lane & 3;
  const int slices = a.dv / 16;
  const long long unit = (long long)blockIdx.x * kRecWarps + (threadIdx.x >> 5);
  if (unit >= (long long)a.N * a.Hv * slices) return;
  const int slice = (int)(unit % slices);
  const long long nh = unit / slices;
  const int h = (int)(nh % a.Hv), n = (int)(nh / a.Hv);
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;
  const int hk = h / (a.Hv / a.Hk), col = slice * 16 + c4 * 4;
  // row i of this lane, behind its first one
  auto row_at = [](int i) { return i / V * 8 * V + i % V; };

  const size_t mat = ((size_t)slot * a.Hv + h) * DK * a.dv + (size_t)(rg * V) * a.dv + col;
  float4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    s[i] = a.S0 ? *reinterpret_cast<const float4*>(a.S0 + mat + (size_t)row_at(i) * a.dv)
                : make_float4(0.f, 0.f, 0.f, 0.f);

  const T* q = static_cast<const T*>(a.q) + (size_t)hk * DK;
  const T* k = static_cast<const T*>(a.k) + (size_t)hk * DK;
  const T* v = static_cast<const T*>(a.v) + (size_t)h * a.dv + slice * 16;
  const T* beta = static_cast<const T*>(a.beta) + h;
  T* o = static_cast<T*>(a.o) + (size_t)h * a.dv + col;

  // The rows of the next token on their way to the ring (one group of copies each, empty behind the
  // end).  A lane copies the same pieces of 16 bytes of every token.
  constexpr int kPieces = DK * (int)sizeof(T) / 16, kCopies = (2 * kPieces + 31) / 32;
  constexpr int kPiece = 16 / (int)sizeof(T);
  const T* from[kCopies];
  long long ahead[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int p = lane + i * 32;
    from[i] = p < kPieces ? k + (size_t)t0 * a.ldk + p * kPiece : q + (size_t)t0 * a.ldq + (p - kPieces) * kPiece;
    ahead[i] = p < kPieces ? a.ldk : a.ldq;
  }
  const T* from_v = v + (size_t)t0 * a.ldv + lane * kPiece;
  int left = t1 - t0;
  uint32_t to = 0;
  auto fetch = [&] {
    if (left > 0) {
      const uint32_t at = umma::smem_u32(ring) + to;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int p = lane + i * 32;
        if (p < 2 * kPieces) umma::cp_async16(at + p * 16, from[i], 16);
        from[i] += ahead[i];
      }
      if (lane < (int)sizeof(T)) umma::cp_async16(at + (2 * kPieces + lane) * 16, from_v, 16);
      from_v += a.ldv;
      to = to == (kRing - 1) * kTokenBytes ? 0 : to + kTokenBytes;
      --left;
    }
    umma::cp_async_commit();
  };
  if (kMany)
    for (int i = 0; i < kRing - 1; ++i) fetch();
  o += (size_t)t0 * a.Hv * a.dv;

  // 1 / |k|, q_scale / |q| and k.q of a token, summed over the row groups
  auto norms = [&](const float (&kx)[R], const float (&qx)[R], float& ik, float& iq, float& kq) {
    float kk = 0.f, qq = 0.f;
    kq = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      kk = fmaf(kx[i], kx[i], kk);
      qq = fmaf(qx[i], qx[i], qq);
      kq = fmaf(kx[i], qx[i], kq);
    }
#pragma unroll
    for (int m = 4; m < 32; m <<= 1) {
      kk += __shfl_xor_sync(0xffffffffu, kk, m);
      qq += __shfl_xor_sync(0xffffffffu, qq, m);
      kq += __shfl_xor_sync(0xffffffffu, kq, m);
    }
    ik = a.l2norm_qk ? gdr_inv_norm(kk, a.eps_l2) : 1.f;
    iq = a.q_scale * (a.l2norm_qk ? gdr_inv_norm(qq, a.eps_l2) : 1.f);
  };
  auto from_ring = [&](float (&kx)[R], float (&qx)[R], const T* at) {
#pragma unroll
    for (int i = 0; i < R; i += V) {
      load_vec<V>(&kx[i], at + rg * V + row_at(i));
      load_vec<V>(&qx[i], at + DK + rg * V + row_at(i));
    }
  };
  auto decay_and_beta = [&](float la, float be, float& al, float& b) {
    al = expf(gdr_log_decay(a, la, h));
    b = a.beta_is_logit ? sigmoidf_(be) : be;
  };

  float al32 = 0.f, b32 = 0.f;              // of the lane's token among 32
  float ik4 = 0.f, iq4 = 0.f, kq4 = 0.f;    // of token c4 among four
  for (int t = t0; t < (kMany ? t1 : t0 + 1); ++t) {
    struct {
      float k[R], q[R], v[4];
    } x;
    float al, b, ik, iq, kq;
    if (kMany) {
      const int i = t - t0;
      if (i % 32 == 0) {
        const size_t at = (size_t)min(t + lane, t1 - 1) * a.Hv;
        decay_and_beta(a.log_alpha[at + h], to_f32(beta[at]), al32, b32);
      }
      if (i % 4 == 0) {
        umma::cp_async_wait_group<kRing - 5>();  // tokens t to t + 3 are there
        __syncwarp();
        from_ring(x.k, x.q, reinterpret_cast<const T*>(ring + (i + c4) % kRing * kTokenBytes));
        norms(x.k, x.q, ik4, iq4, kq4);
      }
      al = __shfl_sync(0xffffffffu, al32, i % 32);
      b = __shfl_sync(0xffffffffu, b32, i % 32);
      ik = __shfl_sync(0xffffffffu, ik4, i % 4);
      iq = __shfl_sync(0xffffffffu, iq4, i % 4);
      kq = __shfl_sync(0xffffffffu, kq4, i % 4);
      const T* at = reinterpret_cast<const T*>(ring + i % kRing * kTokenBytes);
      from_ring(x.k, x.q, at);
      load_vec<4>(x.v, at + 2 * DK + c4 * 4);
      fetch();  // token t + kRing - 1, where t - 1 was: every lane has read that
    } else {
      const float la = a.log_alpha[(size_t)t * a.Hv + h], be = to_f32(beta[(size_t)t * a.Hv]);
#pragma unroll
      for (int i = 0; i < R; i += V) {
        load_vec<V>(&x.k[i], k + (size_t)t * a.ldk + rg * V + row_at(i));
        load_vec<V>(&x.q[i], q + (size_t)t * a.ldq + rg * V + row_at(i));
      }
      load_vec<4>(x.v, v + (size_t)t * a.ldv + c4 * 4);
      decay_and_beta(la, be, al, b);
      norms(x.k, x.q, ik, iq, kq);
    }

    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), r = u;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      u.x = fmaf(s[i].x, x.k[i], u.x); u.y = fmaf(s[i].y, x.k[i], u.y);
      u.z = fmaf(s[i].z, x.k[i], u.z); u.w = fmaf(s[i].w, x.k[i], u.w);
      r.x = fmaf(s[i].x, x.q[i], r.x); r.y = fmaf(s[i].y, x.q[i], r.y);
      r.z = fmaf(s[i].z, x.q[i], r.z); r.w = fmaf(s[i].w, x.q[i], r.w);
    }
    // row groups with bit 2 clear keep u, the others r; then columns (0, 1) or
    // (2, 3) by bit 1, then one column by bit 0
    const bool hi2 = rg & 4, hi1 = rg & 2, hi0 = rg & 1;
    float4 mine = hi2 ? r : u, give = hi2 ? u : r;
    mine.x += __shfl_xor_sync(0xffffffffu, give.x, 16);
    mine.y += __shfl_xor_sync(0xffffffffu, give.y, 16);
    mine.z += __shfl_xor_sync(0xffffffffu, give.z, 16);
    mine.w += __shfl_xor_sync(0xffffffffu, give.w, 16);
    float m0 = hi1 ? mine.z : mine.x, m1 = hi1 ? mine.w : mine.y;
    m0 += __shfl_xor_sync(0xffffffffu, hi1 ? mine.x : mine.z, 8);
    m1 += __shfl_xor_sync(0xffffffffu, hi1 ? mine.y : mine.w, 8);
    float sum = hi0 ? m1 : m0;
    sum += __shfl_xor_sync(0xffffffffu, hi0 ? m0 : m1, 4);
    // row group rg now holds column rg & 3 of u (rg < 4) or r (rg >= 4)
    const int j = rg & 3;
    const float vj = j == 0 ? x.v[0] : j == 1 ? x.v[1] : j == 2 ? x.v[2] : x.v[3];
    float wj = b * (vj - al * ik * sum);  // for rg < 4
    wj = __shfl_sync(0xffffffffu, wj, (j << 2) | c4);
    if (rg >= 4)
      o[j] = from_f32<T>(iq * (al * sum + kq * ik * wj));
    o += (size_t)a.Hv * a.dv;
    const float w0 = ik * __shfl_sync(0xffffffffu, wj, c4), w1 = ik * __shfl_sync(0xffffffffu, wj, 4 | c4),
                w2 = ik * __shfl_sync(0xffffffffu, wj, 8 | c4), w3 = ik * __shfl_sync(0xffffffffu, wj, 12 | c4);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[i].x = fmaf(x.k[i], w0, al * s[i].x); s[i].y = fmaf(x.k[i], w1, al * s[i].y);
      s[i].z = fmaf(x.k[i], w2, al * s[i].z); s[i].w = fmaf(x.k[i], w3, al * s[i].w);
    }
    if (a.snapshots) {  // [n][token of the sequence][h]: here sequences have equal lengths
      float* sp = a.snapshots + ((size_t)t * a.Hv + h) * DK * a.dv + (size_t)(rg * V) * a.dv + col;
#pragma unroll
      for (int i = 0; i < R; ++i) *reinterpret_cast<float4*>(sp + (size_t)row_at(i) * a.dv) = s[i];
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    *reinterpret_cast<float4*>(a.S_T + mat + (size_t)row_at(i) * a.dv) = s[i];
}

template <int DK, typename T>
void launch_dk(const GdrArgs& a, dim3 grid, dim3 block, cudaStream_t s) {
  // one token per sequence: equal lengths of one
  constexpr int ring = kRecWarps * kRing * (2 * DK + 16) * (int)sizeof(T);
  static_assert(ring <= 48 * 1024, "shared memory without asking");
  if (!a.cu_seqlens && a.T_total == a.N) gdr_recurrent_kernel<DK, T, false><<<grid, block, 0, s>>>(a);
  else gdr_recurrent_kernel<DK, T, true><<<grid, block, ring, s>>>(a);
}

template <typename T>
cudaError_t launch_t(const GdrArgs& a, cudaStream_t s) {
  const long long warps = (long long)a.N * a.Hv * (a.dv / 16);
  const long long blocks = (warps + kRecWarps - 1) / kRecWarps;
  const dim3 grid((unsigned)blocks), block(kRecWarps * 32);
  switch (a.dk) {
    case 32: launch_dk<32, T>(a, grid, block, s); break;
    case 64: launch_dk<64, T>(a, grid, block, s); break;
    case 128: launch_dk<128, T>(a, grid, block, s); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_recurrent(const GdrArgs& a, int dtype, cudaStream_t s) {
  return dtype == KDA_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace kda
