// glr_backward.cu -- the gradient of the gated linear recurrence.
//
//     G_t = dy_t + a_{t+1} G_{t+1}   (the last one with dh_T)
//     dx = G c s,   di = G c x s (1 - s)                      s = sigmoid(i)
//     dg = G (a h_{t-1} + c'(g) s x),   c'(g) = 0 | -a | -a^2 / c
//     dla = dg [la <= 0] | -A sigmoid(v) dg | -A sigmoid(v) (1 - sigmoid(v)) dg,   v = la + b
//     db = sum dla,   dA = -sum softplus(v) dg | -sum sigmoid(v) dg
//     dh_0 = a_1 G_1
//
// The states h_{t-1} are not read back from y, which is rounded, but scanned again inside each
// tile of 64 tokens from the states that the forward pass saved before each.
#include "glr.cuh"

namespace kda {
namespace {

using namespace umma;

// A running sum with what its additions lost.
struct Sum {
  float s, lost;
  __device__ __forceinline__ void add(float x) {
    const float y = x - lost, t = s + y;
    lost = (t - s) - y;
    s = t;
  }
  __device__ __forceinline__ double value() const { return (double)s - (double)lost; }
};

// As glr_scan_kernel, walking the rounds from the last to the first.
template <typename T, bool kPair>
__global__ void __launch_bounds__(kGlrTile / GlrLane<T>::kSeg * 32, 1024 / (kGlrTile / GlrLane<T>::kSeg * 64))
    glr_backward_kernel(GlrArgs a) {
  using G = GlrLane<T>;
  using Raw = typename G::Raw;
  constexpr int kSeg = G::kSeg, kWarps = kGlrTile / kSeg;
  constexpr bool kFast = G::kFast;
  __shared__ float4 seg[2][kWarps][32];        // a segment's decay (packed) and its state from zero
  __shared__ float2 seg_grad[2][kWarps][32];   // what it hands back from zero: a G of its first token
  __shared__ float2 seg_log[2][kWarps][32];    // its log decay
  __shared__ float4 tot[2][kGlrMaxRanks][32];  // decays and what is handed back, of a round's tiles
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = gridDim.z, rank = blockIdx.z;
  const int blocks = (a.D + 63) / 64;
  const int n = blockIdx.x / blocks, ch = (blockIdx.x % blocks * 32 + lane) * 2;
  const int in = max(0, min(2, a.D - ch));
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  int t0, t1, slot;
  double2* partial = a.partial ? a.partial + ((size_t)n * ranks + rank) * a.D + ch : nullptr;
  if (!gdr_sequence(a, n, t0, t1, slot)) {  // the whole cluster alike
    if (partial && warp == 0)
      for (int c = 0; c < in; ++c) partial[c] = make_double2(0., 0.);
    return;
  }
  const int L = t1 - t0;
  // what the tokens behind this round hand back
  float2 carry = load_states(a.dh_T ? a.dh_T + (size_t)n * a.D + ch : nullptr, in);
  const GlrChannels par = glr_channels(a, ch, in);
  const float2 minus_A = mul2(par.A, both(1.f / kLog2e));
  if (ranks > 1) cluster_sync();  // every CTA runs
  const T* x = static_cast<const T*>(a.x) + (size_t)t0 * a.ldx + ch;
  const T* la = static_cast<const T*>(a.la) + (size_t)t0 * a.ldla + ch;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + (size_t)t0 * a.ldg + ch : nullptr;
  const size_t out0 = (size_t)t0 * a.D + ch;
  const T* dy = a.dy ? static_cast<const T*>(a.dy) + out0 : nullptr;
  T* dx = static_cast<T*>(a.dx) + out0;
  T* dla = static_cast<T*>(a.dla) + out0;
  T* dgate = a.dgate ? static_cast<T*>(a.dgate) + out0 : nullptr;
  const size_t saved = glr_checkpoint_row(t0, n);
  const int tiles = (L + kGlrTile - 1) / kGlrTile, rounds = (tiles + ranks - 1) / ranks;
  const Raw zero = G::same(0.f), stay = G::same(glr_no_decay(a.decay_from));
  Sum dA[2] = {}, db[2] = {};

  for (int round = rounds - 1; round >= 0; --round) {
    const int tile = round * ranks + rank, p = round & 1;
    const int first = tile * kGlrTile + warp * kSeg;
    Raw rx[kSeg], rl[kSeg], rg[kSeg], rd[kSeg];
    {
      const T *px = x + (size_t)first * a.ldx, *pl = la + (size_t)first * a.ldla;
#pragma unroll
      for (int k = 0; k < kSeg; ++k) {
        const int m = first + k < L ? in : 0;
        rl[k] = G::template load<kPair>(pl + k * a.ldla, m, stay);
        rx[k] = G::template load<kPair>(px + k * a.ldx, m, zero);
        rg[k] = rd[k] = zero;
      }
      if (gate) {
        const T* pg = gate + (size_t)first * a.ldg;
#pragma unroll
        for (int k = 0; k < kSeg; ++k) rg[k] = G::template load<kPair>(pg + k * a.ldg, first + k < L ? in : 0, zero);
      }
      if (dy) {
        const T* pd = dy + (size_t)first * a.D;
#pragma unroll
        for (int k = 0; k < kSeg; ++k)
          rd[k] = G::template load<kPair>(pd + (size_t)k * a.D, first + k < L ? in : 0, zero);
      }
    }
    float2 h = load_states(a.checkpoints + (saved + tile) * a.D + ch, tile < tiles ? in : 0);

    Decay d[kSeg];
    float2 u[kSeg], lg = both(0.f);
    glr_decay_from(a.decay_from, [&](auto from) {
#pragma unroll
      for (int k = 0; k < kSeg; ++k) {
        const float2 g = glr_log_decay<from.value, kFast>(par, G::widen(rl[k]));
        lg = add2(lg, g);
        d[k] = decay_of<kFast>(g);
      }
    });
    if (a.input_scale == KDA_GLR_INPUT_NONE) {
#pragma unroll
      for (int k = 0; k < kSeg; ++k) u[k] = G::widen(rx[k]);
    } else if (a.input_scale == KDA_GLR_INPUT_COMPLEMENT) {
#pragma unroll
      for (int k = 0; k < kSeg; ++k)
        u[k] = mul2(input_factor<kFast>(KDA_GLR_INPUT_COMPLEMENT, d[k]), G::widen(rx[k]));
    } else {
#pragma unroll
      for (int k = 0; k < kSeg; ++k)
        u[k] = mul2(input_factor<kFast>(KDA_GLR_INPUT_NORMALIZED, d[k]), G::widen(rx[k]));
    }
    if (gate) {
#pragma unroll
      for (int k = 0; k < kSeg; ++k) u[k] = mul2(u[k], sigmoid2<kFast>(G::widen(rg[k])));
    }
    // this segment's states and gradients from zero
    float2 back = both(0.f), H = both(0.f);
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
      H = decay_apply(d[k], H, u[k]);
      back = decay_apply(d[kSeg - 1 - k], add2(back, G::widen(rd[kSeg - 1 - k])));
    }
    const float2 dt = decay_pack(decay_of<kFast>(lg));
    seg[p][warp][lane] = make_float4(dt.x, dt.y, H.x, H.y);
    seg_grad[p][warp][lane] = back;
    if (ranks > 1) seg_log[p][warp][lane] = lg;
    __syncthreads();
    if (ranks > 1) {
      if (warp < ranks) {
        float2 z = both(0.f), l = both(0.f);
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
          const float4 s = seg[p][w][lane];
          z = decay_apply(decay_unpack(make_float2(s.x, s.y)), z, seg_grad[p][w][lane]);
          l = add2(l, seg_log[p][w][lane]);
        }
        const float2 t = decay_pack(decay_of<kFast>(l));
        st_cluster_f32x4(map_to_rank(smem_u32(&tot[p][rank][lane]), warp), make_float4(t.x, t.y, z.x, z.y));
      }
      cluster_sync();
      back = carry;
      for (int r = ranks - 1; r >= 0; --r) {
        const float4 s = tot[p][r][lane];
        if (r == rank) back = carry;
        carry = decay_apply(decay_unpack(make_float2(s.x, s.y)), carry, make_float2(s.z, s.w));
      }
    } else {
      back = carry;
    }
    // the state before this segment, and what comes back from behind it
    float2 all = back;
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      const float4 s = seg[p][w][lane];
      if (w == warp) back = all;
      all = decay_apply(decay_unpack(make_float2(s.x, s.y)), all, seg_grad[p][w][lane]);
    }
    if (ranks == 1) carry = all;
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w) {
      const float4 s = seg[p][w][lane];
      if (w < warp) h = decay_apply(decay_unpack(make_float2(s.x, s.y)), h, make_float2(s.z, s.w));
    }
    // the faded state before each token, in the place of its input
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
      const float2 faded = decay_apply(d[k], h);
      h = add2(faded, u[k]);
      u[k] = faded;
    }
    float2 tA = both(0.f), tb = both(0.f);
    T *px = dx + (size_t)first * a.D, *pl = dla + (size_t)first * a.D;
    T* pg = dgate ? dgate + (size_t)first * a.D : nullptr;
    glr_decay_from(a.decay_from, [&](auto from) {
#pragma unroll
      for (int k = kSeg - 1; k >= 0; --k) {
        const float2 grad = add2(G::widen(rd[k]), back), xv = G::widen(rx[k]);
        back = decay_apply(d[k], grad);
        const int m = first + k < L ? in : 0;
        float2 sx = xv, inv = both(0.f);
        const float2 f = input_factor<kFast>(a.input_scale, d[k], &inv);
        float2 ox = mul2(grad, f);
        if (gate) {
          float2 rest;
          const float2 s = sigmoid2<kFast>(G::widen(rg[k]), rest);
          ox = mul2(ox, s);
          sx = mul2(s, xv);
          if (pg) G::template store<kPair>(pg + (size_t)k * a.D, mul2(mul2(ox, xv), rest), m);
        }
        G::template store<kPair>(px + (size_t)k * a.D, ox, m);
        float2 dg = u[k];
        if (a.input_scale != KDA_GLR_INPUT_NONE) {
          // the slope of c: -a or -a^2 / c
          const float2 av = decay_value(d[k]);
          float2 slope = mul2(av, both(-1.f));
          if (a.input_scale == KDA_GLR_INPUT_NORMALIZED) slope = mul2(mul2(slope, av), inv);
          dg = fma2(slope, sx, dg);
        }
        dg = mul2(dg, grad);
        const float2 lv = G::widen(rl[k]);
        float2 ol;
        if constexpr (from.value == KDA_GLR_LOG) {
          ol = make_float2(lv.x > 0.f ? 0.f : dg.x, lv.y > 0.f ? 0.f : dg.y);
        } else {
          const float2 v = add2(lv, par.b);
          float2 rest, val;
          const float2 sg = sigmoid2<kFast>(v, rest);
          if constexpr (from.value == KDA_GLR_SOFTPLUS) {
            val = softplus2<kFast>(v);
            ol = mul2(mul2(minus_A, sg), dg);
            // a decay of 0 has no gradient, however large its logarithm
            val = make_float2(dg.x == 0.f ? 0.f : val.x, dg.y == 0.f ? 0.f : val.y);
          } else {
            val = sg;
            ol = mul2(mul2(minus_A, mul2(sg, rest)), dg);
          }
          if (m) {
            tA = fma2(mul2(val, both(-1.f)), dg, tA);
            tb = add2(tb, ol);
          }
        }
        G::template store<kPair>(pl + (size_t)k * a.D, ol, m);
      }
    });
    dA[0].add(tA.x);
    dA[1].add(tA.y);
    db[0].add(tb.x);
    db[1].add(tb.y);
  }
  if (a.dh0 && rank == 0 && warp == 0) store_states(a.dh0 + (size_t)n * a.D + ch, carry, in);
  if (partial) {
    static_assert(sizeof(seg) >= kWarps * 2 * 32 * sizeof(double2), "the shares fit in its place");
    double2(*sums)[2][32] = reinterpret_cast<double2(*)[2][32]>(&seg[0][0][0]);
    __syncthreads();  // no warp reads segments any more
#pragma unroll
    for (int c = 0; c < 2; ++c) sums[warp][c][lane] = make_double2(dA[c].value(), db[c].value());
    __syncthreads();
    if (warp == 0)
      for (int c = 0; c < in; ++c) {
        double2 z = sums[0][c][lane];
        for (int w = 1; w < kWarps; ++w) {
          z.x += sums[w][c][lane].x;
          z.y += sums[w][c][lane].y;
        }
        partial[c] = z;
      }
  }
}

// dA and db: the shares of all CTAs, in their order.
__global__ void __launch_bounds__(256) glr_join_kernel(const double2* partial, long long rows, int D, float* dA,
                                                       float* db) {
  __shared__ double2 sums[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long ch = (long long)blockIdx.x * 32 + lane;
  grid_launch_dependents();
  grid_wait_prerequisites();
  double2 z = make_double2(0., 0.);
  if (ch < D)
    for (long long r = warp; r < rows; r += 8) {
      const double2 v = partial[r * D + ch];
      z.x += v.x;
      z.y += v.y;
    }
  sums[warp][lane] = z;
  __syncthreads();
  if (warp == 0 && ch < D) {
    for (int w = 1; w < 8; ++w) {
      z.x += sums[w][lane].x;
      z.y += sums[w][lane].y;
    }
    if (dA) dA[ch] = (float)z.x;
    if (db) db[ch] = (float)z.y;
  }
}

template <typename T, bool kPair>
cudaError_t launch(const GlrArgs& a, int ranks, cudaStream_t s) {
  const long long blocks = (a.D + 63LL) / 64 * a.N;
  return launch_early(glr_backward_kernel<T, kPair>, dim3((unsigned)blocks, 1, ranks),
                      kGlrTile / GlrLane<T>::kSeg * 32, 0, ranks, s, a);
}

}  // namespace

cudaError_t launch_glr_backward(const GlrArgs& a, int dtype, bool pair, int ranks, float* dA, float* db,
                                cudaStream_t s) {
  cudaError_t e = dtype == KDA_F32 ? (pair ? launch<float, true>(a, ranks, s) : launch<float, false>(a, ranks, s))
                  : pair           ? launch<__nv_bfloat16, true>(a, ranks, s)
                                   : launch<__nv_bfloat16, false>(a, ranks, s);
  if (e != cudaSuccess || !a.partial) return e;
  return launch_early(glr_join_kernel, dim3((unsigned)((a.D + 31LL) / 32)), 256, 0, 1, s, (const double2*)a.partial,
                      (long long)a.N * ranks, a.D, dA, db);
}

}  // namespace kda
