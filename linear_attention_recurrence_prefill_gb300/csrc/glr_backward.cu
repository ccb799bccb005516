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
//
// 8192 x 4096 in bf16 with an input gate: 186 us of 470 MB, 0.37 of the measured copy rate; the forward
// pass before it 83 us.  Both passes over 16,384 x 4096 in fp32: 1325 us (0.33).  Bound as glr_scan_kernel is,
// with 104 instructions an element.
#include "glr_maps.cuh"

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
template <typename T, int kBytes>
__global__ void __launch_bounds__(kGlrThreads, sizeof(T) == 2 ? 2 : 1) glr_backward_kernel(const __grid_constant__ GlrArgs a, const __grid_constant__ GlrMaps maps) {
  using G = GlrLane<T>;
  using Tile = GlrTile<T, kBytes>;
  constexpr bool kFast = G::kFast;
  extern __shared__ uint8_t smem[];
  uint8_t* stages = smem + ((128 - (smem_u32(smem) & 127)) & 127);  // two, of four arrays: log_alpha, x, dy, gate
  __shared__ float4 seg[2][kGlrWarps][32];           // a segment's decay (packed) and its state from zero
  __shared__ float2 seg_grad[2][kGlrWarps][32];      // what it hands back from zero: a G of its first token
  __shared__ float2 seg_log[2][32 * kGlrWarps];      // its log decay
  __shared__ float2 last[2][32];                     // what a round hands back, of a CTA alone
  __shared__ GlrExchange others;
  __shared__ uint64_t landed[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = gridDim.z, rank = blockIdx.z;
  const int blocks = (a.D + kGlrCols - 1) / kGlrCols;
  const int n = blockIdx.x / blocks, ch0 = blockIdx.x % blocks * kGlrCols, ch = ch0 + lane * 2;
  const int in = max(0, min(2, a.D - ch)), cols = min(kGlrCols, a.D - ch0);
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  int t0, t1, slot;
  // a sequence that is left out (by the whole cluster alike) has no tokens
  const bool live = gdr_sequence(a, n, t0, t1, slot);
  if (!live) t0 = t1 = 0;
  double2* partial = a.partial ? a.partial + ((size_t)n * ranks + rank) * a.D + ch : nullptr;
  const int L = t1 - t0;
  const int tiles = (L + kGlrTile - 1) / kGlrTile, rounds = (tiles + ranks - 1) / ranks;
  const bool gate = a.gate != nullptr, dy = a.dy != nullptr;
  const uint32_t stage = (gate ? 4 : 3) * Tile::kArray;
  const T none = from_f32<T>(glr_no_decay(a.decay_from));
  if (threadIdx.x == 0) {
    others.init();
    mbar_init(&landed[0], 1);
    mbar_init(&landed[1], 1);
    mbar_fence_init();
  }
  auto fetch = [&](int i) {  // the i-th round from the end
    const int first = ((rounds - 1 - i) * ranks + rank) * kGlrTile;
    uint8_t* to = stages + (i & 1) * stage;
    if constexpr (Tile::kTma) {
      if (threadIdx.x == kGlrThreads - 32) {  // (warp 0 has the tile's total to send)
        uint64_t* bar = &landed[i & 1];
        mbar_arrive_expect_tx(bar, dy ? stage : stage - Tile::kArray);
        tma_load_2d(to, &maps.la, ch0, t0 + first, bar);
        tma_load_2d(to + Tile::kArray, &maps.x, ch0, t0 + first, bar);
        if (dy) tma_load_2d(to + 2 * Tile::kArray, &maps.dy, ch0, t0 + first, bar);
        if (gate) tma_load_2d(to + 3 * Tile::kArray, &maps.gate, ch0, t0 + first, bar);
      }
    } else {
      const int rows = L - first;
      const size_t t = (size_t)t0 + first;
      const T zero = from_f32<T>(0.f);
      Tile::copy(to, static_cast<const T*>(a.la) + t * a.ldla + ch0, a.ldla, rows, cols, none);
      Tile::copy(to + Tile::kArray, static_cast<const T*>(a.x) + t * a.ldx + ch0, a.ldx, rows, cols, zero);
      if (dy) Tile::copy(to + 2 * Tile::kArray, static_cast<const T*>(a.dy) + t * a.D + ch0, a.D, rows, cols, zero);
      if (gate)
        Tile::copy(to + 3 * Tile::kArray, static_cast<const T*>(a.gate) + t * a.ldg + ch0, a.ldg, rows, cols, zero);
      cp_async_commit();
    }
  };
  if (!dy)  // zeros, once
    for (int i = 0; i < 2; ++i) Tile::clear(stages + i * stage + 2 * Tile::kArray, warp, lane, 0, from_f32<T>(0.f));
  __syncthreads();  // the barriers are there
  if (rounds > 0) fetch(0);
  // what the tokens behind this round hand back
  float2 carry = load_states(a.dh_T && live ? a.dh_T + (size_t)n * a.D + ch : nullptr, in);
  const GlrChannels par = glr_channels(a, ch, in);
  const float2 minus_A = mul2(par.A, both(1.f / kLog2e));
  if (ranks > 1) cluster_sync();  // every CTA runs, and has its barriers
  const size_t out0 = (size_t)t0 * a.D + ch;
  T* dx = static_cast<T*>(a.dx) + out0;
  T* dla = static_cast<T*>(a.dla) + out0;
  T* dgate = a.dgate ? static_cast<T*>(a.dgate) + out0 : nullptr;
  const size_t saved = glr_checkpoint_row(t0, n);
  Sum dA[2] = {}, db[2] = {};
  bool ok = true;  // of this thread, and of all behind the second barrier in the loop
  int i = 0;

  for (; i < rounds; ++i) {
    const int round = rounds - 1 - i, tile = round * ranks + rank, p = i & 1;
    const int first = tile * kGlrTile + warp * kGlrSeg;
    uint8_t* from = stages + p * stage;
    uint8_t *from_x = from + Tile::kArray, *from_dy = from + 2 * Tile::kArray, *from_gate = from + 3 * Tile::kArray;
    if (!Tile::kTma) cp_async_wait_all();
    __syncthreads();  // nobody reads the tile before any more (and this one is in shared memory)
    if (i + 1 < rounds) fetch(i + 1);
    if constexpr (Tile::kTma) {
      ok = ok && glr_wait<kGlrWaitTile>(&landed[p], (i >> 1) & 1);
      if (first + kGlrSeg > L) {
        Tile::clear(from, warp, lane, L - first, none);
        Tile::clear(from_x, warp, lane, L - first, from_f32<T>(0.f));
        Tile::clear(from_dy, warp, lane, L - first, from_f32<T>(0.f));
        if (gate) Tile::clear(from_gate, warp, lane, L - first, from_f32<T>(0.f));
        fence_proxy_async();  // the next copy to this place comes behind these writes
      }
    }
    float2 h = load_states(a.checkpoints + (saved + tile) * a.D + ch, tile < tiles ? in : 0);

    Decay d[kGlrSeg];
    float2 u[kGlrSeg], lg = both(0.f);
    glr_decay_from(a.decay_from, [&](auto form) {
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) {
        const float2 g = glr_log_decay<form.value, kFast>(par, Tile::get(from, warp, lane, k));
        lg = add2(lg, g);
        d[k] = decay_of<kFast>(g);
      }
    });
    // what segment w hands back of what comes from behind it
    auto before = [&](int w, float2 behind) {
      const float4 s = seg[p][w][lane];
      return decay_apply(decay_unpack(make_float2(s.x, s.y)), behind, seg_grad[p][w][lane]);
    };
    auto input = [&](auto scale) {
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) {
        u[k] = Tile::get(from_x, warp, lane, k);
        if (scale.value != KDA_GLR_INPUT_NONE) u[k] = mul2(input_factor<kFast>(scale.value, d[k]), u[k]);
      }
    };
    glr_input_scale(a.input_scale, input);
    if (gate) {
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) u[k] = mul2(u[k], sigmoid2<kFast>(Tile::get(from_gate, warp, lane, k)));
    }
    // this segment's states and gradients from zero
    float2 back = both(0.f), H = both(0.f);
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) {
      H = decay_apply(d[k], H, u[k]);
      back = decay_apply(d[kGlrSeg - 1 - k], add2(back, Tile::get(from_dy, warp, lane, kGlrSeg - 1 - k)));
    }
    const float2 ds = decay_pack(decay_of<kFast>(lg));
    seg[p][warp][lane] = make_float4(ds.x, ds.y, H.x, H.y);
    seg_grad[p][warp][lane] = back;
    if (ranks > 1) seg_log[p][threadIdx.x] = lg;
    ok = __syncthreads_and(ok);
    if (!ok) break;
    if (ranks > 1) {
      if (warp == 0) {
        float2 z = both(0.f), l = both(0.f);
#pragma unroll
        for (int w = kGlrWarps - 1; w >= 0; --w) {
          z = before(w, z);
          l = add2(l, seg_log[p][w * 32 + lane]);
        }
        const float2 t = decay_pack(decay_of<kFast>(l));
        others.send(p, rank, ranks, lane, make_float4(t.x, t.y, z.x, z.y));
      }
      ok = others.wait(p, i);
      back = carry;
      for (int r = ranks - 1; r >= 0; --r) {
        const float4 s = others.tot[p][r][lane];
        if (r == rank) back = carry;
        carry = decay_apply(decay_unpack(make_float2(s.x, s.y)), carry, make_float2(s.z, s.w));
      }
    } else {
      back = i > 0 ? last[1 - p][lane] : carry;
    }
    // the state before this segment, and what comes back from behind it
    for (int w = 0; w < warp; ++w) {
      const float4 s = seg[p][w][lane];
      h = decay_apply(decay_unpack(make_float2(s.x, s.y)), h, make_float2(s.z, s.w));
    }
    for (int w = kGlrWarps - 1; w > warp; --w) back = before(w, back);
    // the faded state before each token, in the place of its input
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) {
      const float2 faded = decay_apply(d[k], h);
      h = add2(faded, u[k]);
      u[k] = faded;
    }
    float2 tA = both(0.f), tb = both(0.f);
    const size_t at = (size_t)(first + kGlrSeg - 1) * a.D;
    T *px = dx + at, *pl = dla + at, *pg = dgate ? dgate + at : nullptr;
    const bool whole = first + kGlrSeg <= L;
    auto gradients = [&](auto form, auto scale) {
#pragma unroll
      for (int k = kGlrSeg - 1; k >= 0; --k) {
        const bool here = whole || first + k < L;
        const float2 grad = add2(Tile::get(from_dy, warp, lane, k), back), xv = Tile::get(from_x, warp, lane, k);
        back = decay_apply(d[k], grad);
        float2 sx = xv, inv = both(0.f), ox = grad;
        if constexpr (scale.value != KDA_GLR_INPUT_NONE)
          ox = mul2(grad, input_factor<kFast, scale.value == KDA_GLR_INPUT_NORMALIZED>(scale.value, d[k], &inv));
        if (gate) {
          float2 rest;
          const float2 s = sigmoid2<kFast>(Tile::get(from_gate, warp, lane, k), rest);
          ox = mul2(ox, s);
          sx = mul2(s, xv);
          if (dgate && here) G::template store<Tile::kPair>(pg, mul2(mul2(ox, xv), rest), in);
        }
        if (here) G::template store<Tile::kPair>(px, ox, in);
        float2 dg = u[k];
        if constexpr (scale.value != KDA_GLR_INPUT_NONE) {
          // the slope of c: -a or -a^2 / c
          const float2 av = decay_value(d[k]);
          float2 slope = mul2(av, both(-1.f));
          if constexpr (scale.value == KDA_GLR_INPUT_NORMALIZED) slope = mul2(mul2(slope, av), inv);
          dg = fma2(slope, sx, dg);
        }
        dg = mul2(dg, grad);
        const float2 lv = Tile::get(from, warp, lane, k);
        float2 ol;
        if constexpr (form.value == KDA_GLR_LOG) {
          ol = make_float2(lv.x > 0.f ? 0.f : dg.x, lv.y > 0.f ? 0.f : dg.y);
        } else {
          const float2 v = add2(lv, par.b);
          float2 rest, val;
          const float2 sg = sigmoid2<kFast>(v, rest);
          if constexpr (form.value == KDA_GLR_SOFTPLUS) {
            val = softplus2<kFast>(v);
            ol = mul2(mul2(minus_A, sg), dg);
            // a decay of 0 has no gradient, however large its logarithm
            val = make_float2(dg.x == 0.f ? 0.f : val.x, dg.y == 0.f ? 0.f : val.y);
          } else {
            val = sg;
            ol = mul2(mul2(minus_A, mul2(sg, rest)), dg);
          }
          if (here) {
            tA = fma2(mul2(val, both(-1.f)), dg, tA);
            tb = add2(tb, ol);
          }
        }
        if (here) G::template store<Tile::kPair>(pl, ol, in);
        px -= a.D;
        pl -= a.D;
        pg -= a.D;
      }
    };
    glr_decay_from(a.decay_from, [&](auto form) {
      glr_input_scale(a.input_scale, [&](auto scale) { gradients(form, scale); });
    });
    if (warp == 0) last[p][lane] = back;
    dA[0].add(tA.x);
    dA[1].add(tA.y);
    db[0].add(tb.x);
    db[1].add(tb.y);
  }
  ok = __syncthreads_and(ok);
  if (!ok) {
    if (threadIdx.x == 0) atomicExch(a.status, KDA_ERR_TIMEOUT);
    if (!Tile::kTma) cp_async_wait_all();
    glr_settle(landed, Tile::kTma ? min(i + 2, rounds) : 0, others.arrived, ranks > 1 ? i : 0);
  }
  if (ranks > 1) cluster_sync();  // no CTA leaves while another may write to it
  if (live && ok && a.dh0 && rank == 0 && warp == 0)
    store_states(a.dh0 + (size_t)n * a.D + ch, ranks > 1 || rounds == 0 ? carry : last[(rounds - 1) & 1][lane], in);
  if (partial) {
    static_assert(sizeof(seg) >= kGlrWarps * 2 * 32 * sizeof(double2), "the shares fit in its place");
    double2(*sums)[2][32] = reinterpret_cast<double2(*)[2][32]>(&seg[0][0][0]);
#pragma unroll
    for (int c = 0; c < 2; ++c) sums[warp][c][lane] = make_double2(dA[c].value(), db[c].value());
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

template <typename T, int kBytes>
cudaError_t launch(const GlrArgs& a, int ranks, cudaStream_t s) {
  constexpr auto kern = glr_backward_kernel<T, kBytes>;
  constexpr int kArray = GlrTile<T, kBytes>::kArray;
  const cudaError_t e = allow_smem<kern>(8 * kArray + 128);
  if (e != cudaSuccess) return e;
  GlrMaps maps;
  if (kBytes == 16 && !glr_maps<T>(maps, a)) return cudaErrorInvalidValue;
  const long long blocks = (a.D + kGlrCols - 1LL) / kGlrCols * a.N;
  return launch_early(kern, dim3((unsigned)blocks, 1, ranks), kGlrThreads, 2 * (a.gate ? 4 : 3) * kArray + 128, ranks, s, a,
                      maps);
}

}  // namespace

cudaError_t launch_glr_backward(const GlrArgs& a, int dtype, int bytes, int ranks, float* dA, float* db,
                                cudaStream_t s) {
  cudaError_t e;
  if (dtype == KDA_F32)
    e = bytes == 16 ? launch<float, 16>(a, ranks, s) : launch<float, 4>(a, ranks, s);
  else
    e = bytes == 16  ? launch<__nv_bfloat16, 16>(a, ranks, s)
        : bytes == 4 ? launch<__nv_bfloat16, 4>(a, ranks, s)
                     : launch<__nv_bfloat16, 2>(a, ranks, s);
  if (e != cudaSuccess || !a.partial) return e;
  return launch_early(glr_join_kernel, dim3((unsigned)((a.D + 31LL) / 32)), 256, 0, 1, s, (const double2*)a.partial,
                      (long long)a.N * ranks, a.D, dA, db);
}

}  // namespace kda
