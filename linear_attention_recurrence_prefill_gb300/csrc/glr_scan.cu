// glr_scan.cu -- the gated linear recurrence forward: token by token for a few
// tokens per sequence, and as a scan over tiles for long sequences.
#include "glr.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kFewThreads = 128;

// A thread per two channels of a sequence walks its tokens.  Bound by the states and the token
// arrays where there are many sequences, by latency where not.
template <typename T, bool kPair>
__global__ void __launch_bounds__(kFewThreads) glr_few_kernel(GlrArgs a) {
  using G = GlrLane<T>;
  const int blocks = (a.D + 2 * kFewThreads - 1) / (2 * kFewThreads);
  const int n = blockIdx.x / blocks;
  const int ch = (blockIdx.x % blocks * kFewThreads + (int)threadIdx.x) * 2;
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;
  const int in = min(2, a.D - ch);  // this thread's channels
  if (in <= 0) return;
  float2 h = load_states(a.h0 ? a.h0 + (size_t)slot * a.D + ch : nullptr, in);
  const GlrChannels par = glr_channels(a, ch, in);
  const T* x = static_cast<const T*>(a.x) + (size_t)t0 * a.ldx + ch;
  const T* la = static_cast<const T*>(a.la) + (size_t)t0 * a.ldla + ch;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + (size_t)t0 * a.ldg + ch : nullptr;
  T* y = static_cast<T*>(a.y) + (size_t)t0 * a.D + ch;
  size_t saved = glr_checkpoint_row(t0, n);
  glr_decay_from(a.decay_from, [&](auto from) {
    for (int t = 0; t < t1 - t0; ++t) {
      if (a.checkpoints && t % kGlrTile == 0) store_states(a.checkpoints + saved++ * a.D + ch, h, in);
      const float2 xv = G::widen(G::template load<kPair>(x, in, G::same(0.f)));
      const float2 lv = G::widen(G::template load<kPair>(la, in, G::same(0.f)));
      const Decay d = decay_of<G::kFast>(glr_log_decay<from.value, G::kFast>(par, lv));
      float2 u = mul2(input_factor<G::kFast>(a.input_scale, d), xv);
      if (gate) u = mul2(u, sigmoid2<G::kFast>(G::widen(G::template load<kPair>(gate, in, G::same(0.f)))));
      h = decay_apply(d, h, u);
      G::template store<kPair>(y, h, in);
      x += a.ldx;
      la += a.ldla;
      if (gate) gate += a.ldg;
      y += a.D;
    }
  });
  store_states(a.h_T + (size_t)slot * a.D + ch, h, in);
}

// One CTA, or a cluster of them, per sequence and 64 channels.  A tile of 64 tokens has a segment
// of eight (four in fp32) tokens for each of the warps, a lane two channels of them in registers:
// decays and inputs, the segment's own scan from zero, then the states before it from the other
// segments of the tile (shared memory) and from the other CTAs' tiles of this round (distributed
// shared memory), and the scan once more from there.  All joins are taken in the order of the
// tokens, so that results repeat to the bit.
template <typename T, bool kPair>
__global__ void __launch_bounds__(kGlrTile / GlrLane<T>::kSeg * 32, 1024 / (kGlrTile / GlrLane<T>::kSeg * 64))
    glr_scan_kernel(GlrArgs a) {
  using G = GlrLane<T>;
  using Raw = typename G::Raw;
  constexpr int kSeg = G::kSeg, kWarps = kGlrTile / kSeg;
  constexpr bool kFast = G::kFast;
  __shared__ float4 seg[2][kWarps][32];        // a segment's decay (packed) and its state from zero
  __shared__ float2 seg_log[2][kWarps][32];    // and its log decay
  __shared__ float4 tot[2][kGlrMaxRanks][32];  // decays and states of the tiles of a round
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = gridDim.z, rank = blockIdx.z;
  const int blocks = (a.D + 63) / 64;
  const int n = blockIdx.x / blocks, ch = (blockIdx.x % blocks * 32 + lane) * 2;
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;  // the whole cluster alike
  const int in = max(0, min(2, a.D - ch)), L = t1 - t0;
  // the state before this round's first tile
  float2 carry = load_states(a.h0 ? a.h0 + (size_t)slot * a.D + ch : nullptr, in);
  const GlrChannels par = glr_channels(a, ch, in);
  if (ranks > 1) cluster_sync();  // every CTA runs, and has its first states
  const T* x = static_cast<const T*>(a.x) + (size_t)t0 * a.ldx + ch;
  const T* la = static_cast<const T*>(a.la) + (size_t)t0 * a.ldla + ch;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + (size_t)t0 * a.ldg + ch : nullptr;
  T* y = static_cast<T*>(a.y) + (size_t)t0 * a.D + ch;
  const size_t saved = glr_checkpoint_row(t0, n);
  const int tiles = (L + kGlrTile - 1) / kGlrTile, rounds = (tiles + ranks - 1) / ranks;
  const Raw zero = G::same(0.f), stay = G::same(glr_no_decay(a.decay_from));

  Raw rx[kSeg], rl[kSeg], rg[kSeg];
  auto fetch = [&](int round) {
    const int first = (round * ranks + rank) * kGlrTile + warp * kSeg;
    const T *px = x + (size_t)first * a.ldx, *pl = la + (size_t)first * a.ldla;
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
      const int m = first + k < L ? in : 0;
      rl[k] = G::template load<kPair>(pl + k * a.ldla, m, stay);
      rx[k] = G::template load<kPair>(px + k * a.ldx, m, zero);
    }
    if (gate) {
      const T* pg = gate + (size_t)first * a.ldg;
#pragma unroll
      for (int k = 0; k < kSeg; ++k) rg[k] = G::template load<kPair>(pg + k * a.ldg, first + k < L ? in : 0, zero);
    }
  };
  if (rounds > 0) fetch(0);
  for (int round = 0; round < rounds; ++round) {
    const int tile = round * ranks + rank, p = round & 1;
    const int first = tile * kGlrTile + warp * kSeg;
    Decay d[kSeg];
    float2 u[kSeg], lg = both(0.f);
    // decays and inputs; tokens behind the end have a decay of 1 and no input
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
    if (round + 1 < rounds) fetch(round + 1);
    float2 h = both(0.f);
#pragma unroll
    for (int k = 0; k < kSeg; ++k) h = decay_apply(d[k], h, u[k]);
    const float2 dt = decay_pack(decay_of<kFast>(lg));
    seg[p][warp][lane] = make_float4(dt.x, dt.y, h.x, h.y);
    if (ranks > 1) seg_log[p][warp][lane] = lg;
    __syncthreads();
    if (ranks > 1) {
      // the tile's own decay and state from zero, to every CTA of the cluster
      if (warp < ranks) {
        float2 z = both(0.f), l = both(0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 s = seg[p][w][lane];
          z = decay_apply(decay_unpack(make_float2(s.x, s.y)), z, make_float2(s.z, s.w));
          l = add2(l, seg_log[p][w][lane]);
        }
        const float2 t = decay_pack(decay_of<kFast>(l));
        st_cluster_f32x4(map_to_rank(smem_u32(&tot[p][rank][lane]), warp), make_float4(t.x, t.y, z.x, z.y));
      }
      cluster_sync();
      // the state before this CTA's tile, and the one behind the round
      h = carry;
      for (int r = 0; r < ranks; ++r) {
        const float4 s = tot[p][r][lane];
        if (r == rank) h = carry;
        carry = decay_apply(decay_unpack(make_float2(s.x, s.y)), carry, make_float2(s.z, s.w));
      }
    } else {
      h = carry;
    }
    if (a.checkpoints && warp == 0 && tile < tiles) store_states(a.checkpoints + (saved + tile) * a.D + ch, h, in);
    float2 all = h;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 s = seg[p][w][lane];
      if (w == warp) h = all;
      all = decay_apply(decay_unpack(make_float2(s.x, s.y)), all, make_float2(s.z, s.w));
    }
    if (ranks == 1) carry = all;
    T* py = y + (size_t)first * a.D;
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
      h = decay_apply(d[k], h, u[k]);
      G::template store<kPair>(py + (size_t)k * a.D, h, first + k < L ? in : 0);
    }
  }
  // (a state pool: every CTA has read its first states before the cluster's first barrier, and
  // every warp before the first of the CTA; without a tile this warp is the only one that read)
  if (rank == 0 && warp == 0) store_states(a.h_T + (size_t)slot * a.D + ch, carry, in);
}

template <typename T, bool kPair>
cudaError_t launch_few(const GlrArgs& a, cudaStream_t s) {
  const long long blocks = (a.D + 2LL * kFewThreads - 1) / (2 * kFewThreads) * a.N;
  return launch_early(glr_few_kernel<T, kPair>, dim3((unsigned)blocks), kFewThreads, 0, 1, s, a);
}
template <typename T, bool kPair>
cudaError_t launch_scan(const GlrArgs& a, int ranks, cudaStream_t s) {
  const long long blocks = (a.D + 63LL) / 64 * a.N;
  return launch_early(glr_scan_kernel<T, kPair>, dim3((unsigned)blocks, 1, ranks),
                      kGlrTile / GlrLane<T>::kSeg * 32, 0, ranks, s, a);
}

}  // namespace

cudaError_t launch_glr_few(const GlrArgs& a, int dtype, bool pair, cudaStream_t s) {
  if (dtype == KDA_F32) return pair ? launch_few<float, true>(a, s) : launch_few<float, false>(a, s);
  return pair ? launch_few<__nv_bfloat16, true>(a, s) : launch_few<__nv_bfloat16, false>(a, s);
}
cudaError_t launch_glr_scan(const GlrArgs& a, int dtype, bool pair, int ranks, cudaStream_t s) {
  if (dtype == KDA_F32) return pair ? launch_scan<float, true>(a, ranks, s) : launch_scan<float, false>(a, ranks, s);
  return pair ? launch_scan<__nv_bfloat16, true>(a, ranks, s) : launch_scan<__nv_bfloat16, false>(a, ranks, s);
}

}  // namespace kda
