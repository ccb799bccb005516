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

// sigmoid(x) and 1 - sigmoid(x), neither by a difference
template <bool kFast>
__device__ __forceinline__ void sigmoids(float x, float& s, float& rest) {
  const float e = exp_of<kFast>(-fabsf(x)), r = quotient<kFast>(1.f, 1.f + e), er = e * r;
  s = x < 0.f ? er : r;
  rest = x < 0.f ? r : er;
}

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
__global__ void __launch_bounds__(kGlrWarps * 32, 2) glr_backward_kernel(GlrArgs a) {
  using G = GlrLane<T>;
  using Raw = typename G::Raw;
  constexpr int C = G::kCh, kMaxRanks = 16;
  constexpr bool kFast = G::kFast;
  __shared__ float2 seg[2][kGlrWarps][C][32];    // a segment's decay and its state from zero
  __shared__ float seg_grad[2][kGlrWarps][C][32];  // what it hands back from zero: a G of its first token
  __shared__ float seg_log[2][kGlrWarps][C][32];
  __shared__ float2 tot[2][kMaxRanks][C][32];    // decays and what is handed back, of a round's tiles
  __shared__ double2 sums[kGlrWarps][C][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = gridDim.z, rank = blockIdx.z;
  const int blocks = (a.D + 32 * C - 1) / (32 * C);
  const int n = blockIdx.x / blocks, ch = (blockIdx.x % blocks * 32 + lane) * C;
  const int in = max(0, min(C, a.D - ch));
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
  float carry[C];  // what the tokens behind this round hand back
  GlrChannel par[C];
  load_states<C>(carry, a.dh_T ? a.dh_T + (size_t)n * a.D + ch : nullptr, in);
#pragma unroll
  for (int c = 0; c < C; ++c) par[c] = glr_channel(a, ch + c, c < in);
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
  Sum dA[C], db[C];
#pragma unroll
  for (int c = 0; c < C; ++c) dA[c] = db[c] = Sum{0.f, 0.f};

  for (int round = rounds - 1; round >= 0; --round) {
    const int tile = round * ranks + rank, p = round & 1;
    const int first = tile * kGlrTile + warp * kGlrSeg;
    Raw rx[kGlrSeg], rl[kGlrSeg], rg[kGlrSeg], rd[kGlrSeg];
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) {
      const int m = first + k < L ? in : 0;
      rl[k] = G::template load<kPair>(la + (size_t)(first + k) * a.ldla, m);
      rx[k] = G::template load<kPair>(x + (size_t)(first + k) * a.ldx, m);
      rg[k] = gate ? G::template load<kPair>(gate + (size_t)(first + k) * a.ldg, m) : Raw(0);
      rd[k] = dy ? G::template load<kPair>(dy + (size_t)(first + k) * a.D, m) : Raw(0);
    }
    float h[C];
    load_states<C>(h, a.checkpoints + (saved + tile) * a.D + ch, tile < tiles ? in : 0);

    float d[kGlrSeg][C], u[kGlrSeg][C], lg[C];
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) G::widen(rl[k], d[k]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      lg[c] = 0.f;
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) {
        const float g = first + k < L ? glr_log_decay<kFast>(a.decay_from, par[c], d[k][c]) : 0.f;
        lg[c] += g;
        d[k][c] = decay_of(g);
      }
    }
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) {
      float v[C];
      G::widen(rx[k], u[k]);
      G::widen(rg[k], v);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        u[k][c] *= input_factor(a.input_scale, d[k][c]);
        if (gate) u[k][c] *= sigmoid_of<kFast>(v[c]);
      }
    }
    // this segment's states and gradients from zero
    float back[C];
#pragma unroll
    for (int c = 0; c < C; ++c) back[c] = 0.f;
#pragma unroll
    for (int k = kGlrSeg - 1; k >= 0; --k) {
      float v[C];
      G::widen(rd[k], v);
#pragma unroll
      for (int c = 0; c < C; ++c) back[c] = decay_apply(d[k][c], back[c] + v[c], 0.f);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float H = 0.f;
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) H = decay_apply(d[k][c], H, u[k][c]);
      seg[p][warp][c][lane] = make_float2(decay_of(lg[c]), H);
      seg_grad[p][warp][c][lane] = back[c];
      seg_log[p][warp][c][lane] = lg[c];
    }
    __syncthreads();
    if (ranks > 1) {
      if (warp < ranks) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float z = 0.f, l = 0.f;
#pragma unroll
          for (int w = kGlrWarps - 1; w >= 0; --w) {
            z = decay_apply(seg[p][w][c][lane].x, z, seg_grad[p][w][c][lane]);
            l += seg_log[p][w][c][lane];
          }
          const float t = decay_of(l);
          for (int r = warp; r < ranks; r += kGlrWarps)
            st_cluster_f32x2(map_to_rank(smem_u32(&tot[p][rank][c][lane]), r), t, z);
        }
      }
      cluster_sync();
#pragma unroll
      for (int c = 0; c < C; ++c) {
        back[c] = carry[c];
        for (int r = ranks - 1; r >= 0; --r) {
          const float2 s = tot[p][r][c][lane];
          if (r == rank) back[c] = carry[c];
          carry[c] = decay_apply(s.x, carry[c], s.y);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) back[c] = carry[c];
    }
    // the state before this segment, and what comes back from behind it
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int w = 0; w < kGlrWarps - 1; ++w) {
        const float2 s = seg[p][w][c][lane];
        if (w < warp) h[c] = decay_apply(s.x, h[c], s.y);
      }
      float all = back[c];
#pragma unroll
      for (int w = kGlrWarps - 1; w >= 0; --w) {
        if (w == warp) back[c] = all;
        all = decay_apply(seg[p][w][c][lane].x, all, seg_grad[p][w][c][lane]);
      }
      if (ranks == 1) carry[c] = all;
    }
    // the state before each token, in the place of its input
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float before = h[c];
        h[c] = decay_apply(d[k][c], h[c], u[k][c]);
        u[k][c] = before;
      }
    float tA[C], tb[C];
#pragma unroll
    for (int c = 0; c < C; ++c) tA[c] = tb[c] = 0.f;
#pragma unroll
    for (int k = kGlrSeg - 1; k >= 0; --k) {
      float xv[C], lv[C], gv[C], dv[C], ox[C], ol[C], og[C];
      G::widen(rx[k], xv);
      G::widen(rl[k], lv);
      G::widen(rg[k], gv);
      G::widen(rd[k], dv);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float grad = dv[c] + back[c], t = d[k][c];
        back[c] = decay_apply(t, grad, 0.f);
        const float f = input_factor(a.input_scale, t);
        float s = 1.f, rest = 0.f;
        if (gate) sigmoids<kFast>(gv[c], s, rest);
        ox[c] = grad * f * s;
        og[c] = ox[c] * xv[c] * rest;
        float dg = decay_apply(t, u[k][c], 0.f);
        if (a.input_scale != KDA_GLR_INPUT_NONE) {
          const float av = decay_value(t);
          // where the decay is 1 to the last bit its factor's slope is taken as 0
          const float slope = a.input_scale == KDA_GLR_INPUT_COMPLEMENT ? av
                              : f > 0.f ? quotient<kFast>(av * av, f) : f;
          dg = fmaf(-slope, s * xv[c], dg);
        }
        dg *= grad;
        if (a.decay_from == KDA_GLR_LOG) {
          ol[c] = lv[c] > 0.f ? 0.f : dg;
        } else {
          const float v = lv[c] + par[c].b;
          float sg, sr;
          sigmoids<kFast>(v, sg, sr);
          const bool soft = a.decay_from == KDA_GLR_SOFTPLUS;
          ol[c] = -par[c].A * (soft ? sg : sg * sr) * dg;
          if (partial && first + k < L) {
            // (a decay of 0 has no gradient, however large its logarithm)
            tA[c] -= dg == 0.f ? 0.f : (soft ? softplus_of<kFast>(v) : sg) * dg;
            tb[c] += ol[c];
          }
        }
      }
      const int m = first + k < L ? in : 0;
      const size_t at = (size_t)(first + k) * a.D;
      G::template store<kPair>(dx + at, G::narrow(ox), m);
      G::template store<kPair>(dla + at, G::narrow(ol), m);
      if (dgate) G::template store<kPair>(dgate + at, G::narrow(og), m);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      dA[c].add(tA[c]);
      db[c].add(tb[c]);
    }
  }
  if (a.dh0 && rank == 0 && warp == 0) store_states<C>(a.dh0 + (size_t)n * a.D + ch, carry, in);
  if (partial) {
#pragma unroll
    for (int c = 0; c < C; ++c) sums[warp][c][lane] = make_double2(dA[c].value(), db[c].value());
    __syncthreads();
    if (warp == 0)
      for (int c = 0; c < in; ++c) {
        double2 z = sums[0][c][lane];
        for (int w = 1; w < kGlrWarps; ++w) {
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
  constexpr int per = 32 * GlrLane<T>::kCh;
  const long long blocks = (a.D + (long long)per - 1) / per * a.N;
  return launch_early(glr_backward_kernel<T, kPair>, dim3((unsigned)blocks, 1, ranks), kGlrWarps * 32, 0, ranks, s, a);
}

}  // namespace

cudaError_t launch_glr_backward(const GlrArgs& a, int dtype, bool pair, int ranks, float* dA, float* db,
                                cudaStream_t s) {
  cudaError_t e = dtype == KDA_F32 ? launch<float, false>(a, ranks, s)
                  : pair           ? launch<__nv_bfloat16, true>(a, ranks, s)
                                   : launch<__nv_bfloat16, false>(a, ranks, s);
  if (e != cudaSuccess || !a.partial) return e;
  return launch_early(glr_join_kernel, dim3((unsigned)((a.D + 31LL) / 32)), 256, 0, 1, s, (const double2*)a.partial,
                      (long long)a.N * ranks, a.D, dA, db);
}

}  // namespace kda
