// glr_scan.cu -- the gated linear recurrence forward: token by token for a few
// tokens per sequence, and as a scan over tiles for long sequences.
#include "glr.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kFewThreads = 128;

// A thread per channel (two in bf16) of a sequence walks its tokens.  Bound by the
// states and the token arrays where there are many sequences, by latency where not.
template <typename T, bool kPair>
__global__ void __launch_bounds__(kFewThreads) glr_few_kernel(GlrArgs a) {
  using G = GlrLane<T>;
  constexpr int C = G::kCh;
  const int blocks = (a.D + kFewThreads * C - 1) / (kFewThreads * C);
  const int n = blockIdx.x / blocks;
  const int ch = (blockIdx.x % blocks * kFewThreads + (int)threadIdx.x) * C;
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;
  const int in = min(C, a.D - ch);  // this thread's channels
  if (in <= 0) return;
  float h[C];
  GlrChannel par[C];
  load_states<C>(h, a.h0 ? a.h0 + (size_t)slot * a.D + ch : nullptr, in);
#pragma unroll
  for (int c = 0; c < C; ++c) par[c] = glr_channel(a, ch + c, c < in);
  const T* x = static_cast<const T*>(a.x) + (size_t)t0 * a.ldx + ch;
  const T* la = static_cast<const T*>(a.la) + (size_t)t0 * a.ldla + ch;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + (size_t)t0 * a.ldg + ch : nullptr;
  T* y = static_cast<T*>(a.y) + (size_t)t0 * a.D + ch;
  size_t saved = glr_checkpoint_row(t0, n);
  for (int t = 0; t < t1 - t0; ++t) {
    if (a.checkpoints && t % kGlrTile == 0) store_states<C>(a.checkpoints + saved++ * a.D + ch, h, in);
    float xv[C], lv[C], gv[C], out[C];
    G::widen(G::template load<kPair>(x, in), xv);
    G::widen(G::template load<kPair>(la, in), lv);
    if (gate) G::widen(G::template load<kPair>(gate, in), gv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float d = decay_of(glr_log_decay<G::kFast>(a.decay_from, par[c], lv[c]));
      float u = input_factor(a.input_scale, d) * xv[c];
      if (gate) u *= sigmoid_of<G::kFast>(gv[c]);
      out[c] = h[c] = decay_apply(d, h[c], u);
    }
    G::template store<kPair>(y, G::narrow(out), in);
    x += a.ldx;
    la += a.ldla;
    if (gate) gate += a.ldg;
    y += a.D;
  }
  store_states<C>(a.h_T + (size_t)slot * a.D + ch, h, in);
}

// One CTA, or a cluster of them, per sequence and 32 lanes of channels.  A tile of 64 tokens has
// eight tokens for each of the eight warps, a lane its channels of them in registers: decays and
// inputs, the segment's own scan from zero, then the states before it from the other segments
// of the tile (shared memory) and from the other CTAs' tiles of this round (distributed shared
// memory), and the scan once more from there.  All joins are taken in the order of the tokens, so
// that results repeat to the bit.
template <typename T, bool kPair>
__global__ void __launch_bounds__(kGlrWarps * 32, 2) glr_scan_kernel(GlrArgs a) {
  using G = GlrLane<T>;
  using Raw = typename G::Raw;
  constexpr int C = G::kCh, kMaxRanks = 16;
  __shared__ float2 seg[2][kGlrWarps][C][32];    // a segment's decay and its state from zero
  __shared__ float seg_log[2][kGlrWarps][C][32];  // and its log decay
  __shared__ float2 tot[2][kMaxRanks][C][32];    // the same of the tiles of a round
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = gridDim.z, rank = blockIdx.z;
  const int blocks = (a.D + 32 * C - 1) / (32 * C);
  const int n = blockIdx.x / blocks, ch = (blockIdx.x % blocks * 32 + lane) * C;
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;  // the whole cluster alike
  const int in = max(0, min(C, a.D - ch)), L = t1 - t0;
  float carry[C];  // the state before this round's first tile
  GlrChannel par[C];
  load_states<C>(carry, a.h0 ? a.h0 + (size_t)slot * a.D + ch : nullptr, in);
#pragma unroll
  for (int c = 0; c < C; ++c) par[c] = glr_channel(a, ch + c, c < in);
  if (ranks > 1) cluster_sync();  // every CTA runs, and has its first states
  const T* x = static_cast<const T*>(a.x) + (size_t)t0 * a.ldx + ch;
  const T* la = static_cast<const T*>(a.la) + (size_t)t0 * a.ldla + ch;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + (size_t)t0 * a.ldg + ch : nullptr;
  T* y = static_cast<T*>(a.y) + (size_t)t0 * a.D + ch;
  const size_t saved = glr_checkpoint_row(t0, n);
  const int tiles = (L + kGlrTile - 1) / kGlrTile, rounds = (tiles + ranks - 1) / ranks;

  Raw rx[kGlrSeg], rl[kGlrSeg], rg[kGlrSeg];
  auto fetch = [&](int round) {
    const int first = (round * ranks + rank) * kGlrTile + warp * kGlrSeg;
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) {
      const int m = first + k < L ? in : 0;
      rx[k] = G::template load<kPair>(x + (size_t)(first + k) * a.ldx, m);
      rl[k] = G::template load<kPair>(la + (size_t)(first + k) * a.ldla, m);
      rg[k] = gate ? G::template load<kPair>(gate + (size_t)(first + k) * a.ldg, m) : Raw(0);
    }
  };
  if (rounds > 0) fetch(0);
  for (int round = 0; round < rounds; ++round) {
    const int tile = round * ranks + rank, p = round & 1;
    const int first = tile * kGlrTile + warp * kGlrSeg;
    float d[kGlrSeg][C], u[kGlrSeg][C], lg[C], H[C];
    // log decays, then decays and inputs; tokens behind the end change nothing
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) G::widen(rl[k], d[k]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      lg[c] = 0.f;
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) {
        const float g = first + k < L ? glr_log_decay<G::kFast>(a.decay_from, par[c], d[k][c]) : 0.f;
        lg[c] += g;
        d[k][c] = decay_of(g);
      }
    }
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) {
      G::widen(rx[k], u[k]);
#pragma unroll
      for (int c = 0; c < C; ++c) u[k][c] *= input_factor(a.input_scale, d[k][c]);
    }
    if (gate) {
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) {
        float v[C];
        G::widen(rg[k], v);
#pragma unroll
        for (int c = 0; c < C; ++c) u[k][c] *= sigmoid_of<G::kFast>(v[c]);
      }
    }
    if (round + 1 < rounds) fetch(round + 1);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      H[c] = 0.f;
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) H[c] = decay_apply(d[k][c], H[c], u[k][c]);
      seg[p][warp][c][lane] = make_float2(decay_of(lg[c]), H[c]);
      seg_log[p][warp][c][lane] = lg[c];
    }
    __syncthreads();
    float h[C];
    if (ranks > 1) {
      // the tile's own decay and state from zero, to every CTA of the cluster
      if (warp < ranks) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float z = 0.f, l = 0.f;
#pragma unroll
          for (int w = 0; w < kGlrWarps; ++w) {
            const float2 s = seg[p][w][c][lane];
            z = decay_apply(s.x, z, s.y);
            l += seg_log[p][w][c][lane];
          }
          const float t = decay_of(l);
          for (int r = warp; r < ranks; r += kGlrWarps)
            st_cluster_f32x2(map_to_rank(smem_u32(&tot[p][rank][c][lane]), r), t, z);
        }
      }
      cluster_sync();
      // the state before this CTA's tile, and the one behind the round
#pragma unroll
      for (int c = 0; c < C; ++c) {
        h[c] = carry[c];
        for (int r = 0; r < ranks; ++r) {
          const float2 s = tot[p][r][c][lane];
          if (r == rank) h[c] = carry[c];
          carry[c] = decay_apply(s.x, carry[c], s.y);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) h[c] = carry[c];
    }
    if (a.checkpoints && warp == 0 && tile < tiles)
      store_states<C>(a.checkpoints + (saved + tile) * a.D + ch, h, in);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float all = h[c];
#pragma unroll
      for (int w = 0; w < kGlrWarps; ++w) {
        const float2 s = seg[p][w][c][lane];
        if (w == warp) h[c] = all;
        all = decay_apply(s.x, all, s.y);
      }
      if (ranks == 1) carry[c] = all;
    }
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) {
      float out[C];
#pragma unroll
      for (int c = 0; c < C; ++c) out[c] = h[c] = decay_apply(d[k][c], h[c], u[k][c]);
      G::template store<kPair>(y + (size_t)(first + k) * a.D, G::narrow(out), first + k < L ? in : 0);
    }
  }
  // (a state pool: every CTA has read its first states before the cluster's first barrier, and
  // every warp before the first of the CTA; without a tile this warp is the only one that read)
  if (rank == 0 && warp == 0) store_states<C>(a.h_T + (size_t)slot * a.D + ch, carry, in);
}

template <typename T, bool kPair>
cudaError_t launch_few(const GlrArgs& a, cudaStream_t s) {
  constexpr int per = kFewThreads * GlrLane<T>::kCh;
  const long long blocks = (a.D + (long long)per - 1) / per * a.N;
  return launch_early(glr_few_kernel<T, kPair>, dim3((unsigned)blocks), kFewThreads, 0, 1, s, a);
}
template <typename T, bool kPair>
cudaError_t launch_scan(const GlrArgs& a, int ranks, cudaStream_t s) {
  constexpr int per = 32 * GlrLane<T>::kCh;
  const long long blocks = (a.D + (long long)per - 1) / per * a.N;
  return launch_early(glr_scan_kernel<T, kPair>, dim3((unsigned)blocks, 1, ranks), kGlrWarps * 32, 0, ranks, s, a);
}

}  // namespace

cudaError_t launch_glr_few(const GlrArgs& a, int dtype, bool pair, cudaStream_t s) {
  if (dtype == KDA_F32) return launch_few<float, false>(a, s);
  return pair ? launch_few<__nv_bfloat16, true>(a, s) : launch_few<__nv_bfloat16, false>(a, s);
}
cudaError_t launch_glr_scan(const GlrArgs& a, int dtype, bool pair, int ranks, cudaStream_t s) {
  if (dtype == KDA_F32) return launch_scan<float, false>(a, ranks, s);
  return pair ? launch_scan<__nv_bfloat16, true>(a, ranks, s) : launch_scan<__nv_bfloat16, false>(a, ranks, s);
}

}  // namespace kda
