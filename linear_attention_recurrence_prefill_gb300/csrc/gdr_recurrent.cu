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
#include "gdr.cuh"

namespace kda {
namespace {

constexpr int kRecWarps = 4;

// R consecutive elements as they lie (R * sizeof(T) a multiple of 8 bytes, so aligned at least)
template <int R, typename T>
struct Row {
  uint2 raw[R * (int)sizeof(T) / 8];
  __device__ __forceinline__ void load(const T* p) {
    constexpr int n = R * (int)sizeof(T) / 16;
    if constexpr (n > 0) {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        raw[2 * i] = make_uint2(v.x, v.y);
        raw[2 * i + 1] = make_uint2(v.z, v.w);
      }
    } else {
      raw[0] = *reinterpret_cast<const uint2*>(p);
    }
  }
  __device__ __forceinline__ void widen(float (&x)[R]) const {
#pragma unroll
    for (int i = 0; i < R * (int)sizeof(T) / 4; ++i) {
      const uint32_t w = i & 1 ? raw[i / 2].y : raw[i / 2].x;
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w);
      } else {
        x[2 * i] = __uint_as_float(w << 16);
        x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  }
};

template <int R, typename T>
struct Token {
  Row<R, T> k, q;
  Row<4, T> v;
  float la, b;
};

// kMany: any number of tokens per sequence, the next one's rows fetched ahead; else one.
template <int DK, typename T, bool kMany>
__global__ void __launch_bounds__(kRecWarps * 32, kMany ? 3 : 4) gdr_recurrent_kernel(GdrArgs a) {
  constexpr int R = DK / 8;  // rows of the state per lane
  const int lane = threadIdx.x & 31, rg = lane >> 2, c4 = lane & 3;
  const int slices = a.dv / 16;
  const long long unit = (long long)blockIdx.x * kRecWarps + (threadIdx.x >> 5);
  if (unit >= (long long)a.N * a.Hv * slices) return;
  const int slice = (int)(unit % slices);
  const long long nh = unit / slices;
  const int h = (int)(nh % a.Hv), n = (int)(nh / a.Hv);
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;
  const int hk = h / (a.Hv / a.Hk), col = slice * 16 + c4 * 4, row = rg * R;

  const size_t mat = ((size_t)slot * a.Hv + h) * DK * a.dv + (size_t)row * a.dv + col;
  float4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    s[i] = a.S0 ? *reinterpret_cast<const float4*>(a.S0 + mat + (size_t)i * a.dv)
                : make_float4(0.f, 0.f, 0.f, 0.f);

  const T* q = static_cast<const T*>(a.q) + (size_t)hk * DK + row;
  const T* k = static_cast<const T*>(a.k) + (size_t)hk * DK + row;
  const T* v = static_cast<const T*>(a.v) + (size_t)h * a.dv + col;
  const T* beta = static_cast<const T*>(a.beta) + h;
  T* o = static_cast<T*>(a.o) + (size_t)h * a.dv + col;
  auto load = [&](Token<R, T>& x, int t) {
    x.k.load(k + (size_t)t * a.ldk);
    x.q.load(q + (size_t)t * a.ldq);
    x.v.load(v + (size_t)t * a.ldv);
    x.la = a.log_alpha[(size_t)t * a.Hv + h];
    x.b = to_f32(beta[(size_t)t * a.Hv]);
  };

  Token<R, T> next;
  if (t0 < t1) load(next, t0);
  for (int t = t0; t < (kMany ? t1 : t0 + 1); ++t) {
    struct {
      float k[R], q[R], v[4], la, b;
    } x;
    next.k.widen(x.k);
    next.q.widen(x.q);
    next.v.widen(x.v);
    x.la = next.la;
    x.b = next.b;
    if (kMany && t + 1 < t1) load(next, t + 1);
    // |k|^2, |q|^2, k.q over all rows
    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      kk = fmaf(x.k[i], x.k[i], kk);
      qq = fmaf(x.q[i], x.q[i], qq);
      kq = fmaf(x.k[i], x.q[i], kq);
    }
#pragma unroll
    for (int m = 4; m < 32; m <<= 1) {
      kk += __shfl_xor_sync(0xffffffffu, kk, m);
      qq += __shfl_xor_sync(0xffffffffu, qq, m);
      kq += __shfl_xor_sync(0xffffffffu, kq, m);
    }
    const float ik = a.l2norm_qk ? gdr_inv_norm(kk, a.eps_l2) : 1.f;
    const float iq = a.q_scale * (a.l2norm_qk ? gdr_inv_norm(qq, a.eps_l2) : 1.f);
    const float al = expf(gdr_log_decay(a, x.la, h));
    const float b = a.beta_is_logit ? sigmoidf_(x.b) : x.b;

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
      o[(size_t)t * a.Hv * a.dv + j] = from_f32<T>(iq * (al * sum + kq * ik * wj));
    const float w0 = ik * __shfl_sync(0xffffffffu, wj, c4), w1 = ik * __shfl_sync(0xffffffffu, wj, 4 | c4),
                w2 = ik * __shfl_sync(0xffffffffu, wj, 8 | c4), w3 = ik * __shfl_sync(0xffffffffu, wj, 12 | c4);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[i].x = fmaf(x.k[i], w0, al * s[i].x); s[i].y = fmaf(x.k[i], w1, al * s[i].y);
      s[i].z = fmaf(x.k[i], w2, al * s[i].z); s[i].w = fmaf(x.k[i], w3, al * s[i].w);
    }
    if (a.snapshots) {  // [n][token of the sequence][h]: here sequences have equal lengths
      float* sp = a.snapshots + ((size_t)t * a.Hv + h) * DK * a.dv + (size_t)row * a.dv + col;
#pragma unroll
      for (int i = 0; i < R; ++i) *reinterpret_cast<float4*>(sp + (size_t)i * a.dv) = s[i];
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    *reinterpret_cast<float4*>(a.S_T + mat + (size_t)i * a.dv) = s[i];
}

template <int DK, typename T>
void launch_dk(const GdrArgs& a, dim3 grid, dim3 block, cudaStream_t s) {
  // one token per sequence: equal lengths of one
  if (!a.cu_seqlens && a.T_total == a.N) gdr_recurrent_kernel<DK, T, false><<<grid, block, 0, s>>>(a);
  else gdr_recurrent_kernel<DK, T, true><<<grid, block, 0, s>>>(a);
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
