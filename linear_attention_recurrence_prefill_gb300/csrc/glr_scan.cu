// glr_scan.cu -- the gated linear recurrence forward: token by token for a few
// tokens per sequence, and as a scan over tiles for long sequences.
#include "glr_maps.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kFewThreads = 128;

// kPairs pairs of neighbouring channels of a thread: 16 bytes of a token and of a state at once where
// there is more than one, else as in GlrLane.
template <typename T, int kPairs, bool kPair>
struct Wide {
  static __device__ __forceinline__ void load(float2 (&v)[kPairs], const T* p, int n) {
    if constexpr (kPairs == 1) {
      v[0] = GlrLane<T>::template load<kPair>(p, n);
    } else {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
      if constexpr (sizeof(T) == 2) {
        v[0] = GlrLane<T>::widen(q.x); v[1] = GlrLane<T>::widen(q.y);
        v[2] = GlrLane<T>::widen(q.z); v[3] = GlrLane<T>::widen(q.w);
      } else {
        v[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
        v[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, const float2 (&v)[kPairs], int n) {
    if constexpr (kPairs == 1) {
      GlrLane<T>::template store<kPair>(p, v[0], n);
    } else if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf162(v[0].x, v[0].y), pack_bf162(v[1].x, v[1].y),
                                                pack_bf162(v[2].x, v[2].y), pack_bf162(v[3].x, v[3].y));
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
  }
  static __device__ __forceinline__ void load_states(float2 (&v)[kPairs], const float* p, int n, float none) {
    if constexpr (kPairs == 1) {
      v[0] = p ? kda::load_states(p, n) : both(none);
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; i += 2) {
        const float4 q = p ? *reinterpret_cast<const float4*>(p + 2 * i) : make_float4(none, none, none, none);
        v[i] = make_float2(q.x, q.y);
        v[i + 1] = make_float2(q.z, q.w);
      }
    }
  }
  static __device__ __forceinline__ void store_states(float* p, const float2 (&v)[kPairs], int n) {
    if constexpr (kPairs == 1) {
      kda::store_states(p, v[0], n);
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; i += 2)
        *reinterpret_cast<float4*>(p + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
    }
  }
};

// A thread per one to four pairs of channels of a sequence walks its tokens.  Bound by the states and
// the token arrays where there are many sequences, by latency where not.
template <typename T, int kPairs, bool kPair>
__global__ void __launch_bounds__(kFewThreads) glr_few_kernel(GlrArgs a) {
  using W = Wide<T, kPairs, kPair>;
  constexpr bool kFast = GlrLane<T>::kFast;
  constexpr int kCh = 2 * kPairs;
  // unsigned: rounded up to a CTA's channels (1024 at most), the largest D is 2^31; a thread's first
  // channel is below that
  const unsigned blocks = ((unsigned)a.D + kFewThreads * kCh - 1) / (kFewThreads * kCh);
  const int n = blockIdx.x / blocks;
  const int ch = (blockIdx.x % blocks * kFewThreads + threadIdx.x) * kCh;
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  int t0, t1, slot;
  if (!gdr_sequence(a, n, t0, t1, slot)) return;
  const int in = min(kCh, a.D - ch);  // this thread's channels
  if (in <= 0) return;
  float2 h[kPairs], A[kPairs], b[kPairs];
  W::load_states(h, a.h0 ? a.h0 + (size_t)slot * a.D + ch : nullptr, in, 0.f);
  W::load_states(A, a.decay_scale ? a.decay_scale + ch : nullptr, in, 1.f);
  W::load_states(b, a.decay_bias ? a.decay_bias + ch : nullptr, in, 0.f);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) A[i] = mul2(A[i], both(-kLog2e));
  const T* x = static_cast<const T*>(a.x) + (size_t)t0 * a.ldx + ch;
  const T* la = static_cast<const T*>(a.la) + (size_t)t0 * a.ldla + ch;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + (size_t)t0 * a.ldg + ch : nullptr;
  T* y = static_cast<T*>(a.y) + (size_t)t0 * a.D + ch;
  size_t saved = glr_checkpoint_row(t0, n);
  glr_decay_from(a.decay_from, [&](auto from) {
    for (int t = 0; t < t1 - t0; ++t) {
      if (a.checkpoints && t % kGlrTile == 0) W::store_states(a.checkpoints + saved++ * a.D + ch, h, in);
      float2 xv[kPairs], lv[kPairs], gv[kPairs];
      W::load(xv, x, in);
      W::load(lv, la, in);
      if (gate) W::load(gv, gate, in);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const Decay d = decay_of<kFast>(glr_log_decay<from.value, kFast>(GlrChannels{A[i], b[i]}, lv[i]));
        float2 u = mul2(input_factor<kFast>(a.input_scale, d), xv[i]);
        if (gate) u = mul2(u, sigmoid2<kFast>(gv[i]));
        h[i] = decay_apply(d, h[i], u);
      }
      W::store(y, h, in);
      x += a.ldx;
      la += a.ldla;
      if (gate) gate += a.ldg;
      y += a.D;
    }
  });
  W::store_states(a.h_T + (size_t)slot * a.D + ch, h, in);
}

// One CTA, or a cluster of them, per sequence and 64 channels.  A tile of 64 tokens has a segment
// of eight for each of the eight warps, a lane two channels of them in registers: decays and
// inputs, the segment's own scan from zero, then the states before it from the other CTAs' tiles
// of this round (distributed shared memory) and from the tile's other segments (shared memory), and
// the scan once more from there.  All joins are taken in the order of the tokens, so that results
// repeat to the bit.  The next tile's arrays are copied to shared memory meanwhile.
//
// 32,768 x 4096 in bf16 (softplus): 290 us, 0.41 of the rate of its bytes; 12,000 tokens in nine
// prompts with an input gate 104 us (0.56); 16,384 x 4096 in fp32 338 us (0.35), with a gate 433 (0.37).
// Bound by the latency of a round, 2.3 us: two CTAs of 128
// registers a thread per SM, 3.3 warps per scheduler, which issue in half of the cycles, and 24 SMs
// without a CTA where 64 clusters of four fill 128.  Three CTAs of 80 registers took 419 us (they
// load their constants again and again), one per SM 405; the clusters' barrier instead of counted
// writes 367.
template <typename T, int kBytes>
__global__ void __launch_bounds__(kGlrThreads, 2)
    glr_scan_kernel(const __grid_constant__ GlrArgs a, const __grid_constant__ GlrMaps maps) {
  using G = GlrLane<T>;
  using Tile = GlrTile<T, kBytes>;
  constexpr bool kFast = G::kFast;
  extern __shared__ uint8_t smem[];
  uint8_t* stages = smem + ((128 - (smem_u32(smem) & 127)) & 127);  // two, of two or three arrays
  __shared__ float4 seg[2][kGlrWarps][32];           // a segment's decay (packed) and its state from zero
  __shared__ float2 seg_log[2][32 * kGlrWarps];      // and its log decay
  __shared__ float2 last[2][32];                     // the state behind a round, of a CTA alone
  __shared__ GlrExchange others;
  __shared__ uint64_t landed[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = gridDim.z, rank = blockIdx.z;
  const int blocks = (a.D + kGlrCols - 1) / kGlrCols;
  const int n = blockIdx.x / blocks, ch0 = blockIdx.x % blocks * kGlrCols, ch = ch0 + lane * 2;
  grid_launch_dependents();
  grid_wait_prerequisites();  // what ran before is complete
  // a sequence that is left out (by the whole cluster alike) has no tokens
  int t0 = 0, t1 = 0, slot = 0;
  const bool live = gdr_sequence(a, n, t0, t1, slot);
  if (!live) t0 = t1 = 0;
  const int in = max(0, min(2, a.D - ch)), cols = min(kGlrCols, a.D - ch0), L = t1 - t0;
  const int tiles = (L + kGlrTile - 1) / kGlrTile, rounds = (tiles + ranks - 1) / ranks;
  const bool gate = a.gate != nullptr;
  const uint32_t stage = (gate ? 3 : 2) * Tile::kArray;
  const T none = from_f32<T>(glr_no_decay(a.decay_from));
  if (threadIdx.x == 0) {
    others.init();
    mbar_init(&landed[0], 1);
    mbar_init(&landed[1], 1);
    mbar_fence_init();
  }
  auto fetch = [&](int round) {
    const int first = (round * ranks + rank) * kGlrTile;
    uint8_t* to = stages + (round & 1) * stage;
    if constexpr (Tile::kTma) {
      if (threadIdx.x == kGlrThreads - 32) {  // (warp 0 has the tile's total to send)
        uint64_t* bar = &landed[round & 1];
        mbar_arrive_expect_tx(bar, stage);
        tma_load_2d(to, &maps.la, ch0, t0 + first, bar);
        tma_load_2d(to + Tile::kArray, &maps.x, ch0, t0 + first, bar);
        if (gate) tma_load_2d(to + 2 * Tile::kArray, &maps.gate, ch0, t0 + first, bar);
      }
    } else {
      const int rows = L - first;
      const size_t t = (size_t)t0 + first;
      Tile::copy(to, static_cast<const T*>(a.la) + t * a.ldla + ch0, a.ldla, rows, cols, none);
      Tile::copy(to + Tile::kArray, static_cast<const T*>(a.x) + t * a.ldx + ch0, a.ldx, rows, cols, from_f32<T>(0.f));
      if (gate)
        Tile::copy(to + 2 * Tile::kArray, static_cast<const T*>(a.gate) + t * a.ldg + ch0, a.ldg, rows, cols,
                   from_f32<T>(0.f));
      cp_async_commit();
    }
  };
  __syncthreads();  // the barriers are there
  if (rounds > 0) fetch(0);
  if (rounds > 1) fetch(1);
  else if (!Tile::kTma) cp_async_commit();
  // the state before this round's first tile
  float2 carry = load_states(a.h0 && live ? a.h0 + (size_t)slot * a.D + ch : nullptr, in);
  const GlrChannels par = glr_channels(a, ch, in);
  if (!Tile::kTma) cp_async_wait_group<1>();
  if (ranks > 1) cluster_sync();  // every CTA runs, and has its first states and its barriers
  if (!Tile::kTma) __syncthreads();  // the first tile is in shared memory
  T* y = static_cast<T*>(a.y) + (size_t)t0 * a.D + ch;
  const size_t saved = glr_checkpoint_row(t0, n);
  bool ok = true;  // of this thread, and of all behind the barrier in the loop
  int round = 0;

  for (; round < rounds; ++round) {
    const int tile = round * ranks + rank, p = round & 1;
    const int first = tile * kGlrTile + warp * kGlrSeg;
    uint8_t* from = stages + p * stage;
    if constexpr (Tile::kTma) {
      ok = ok && glr_wait<kGlrWaitTile>(&landed[p], (round >> 1) & 1);
      if (first + kGlrSeg > L) {
        Tile::clear(from, warp, lane, L - first, none);
        Tile::clear(from + Tile::kArray, warp, lane, L - first, from_f32<T>(0.f));
        if (gate) Tile::clear(from + 2 * Tile::kArray, warp, lane, L - first, from_f32<T>(0.f));
      }
    }
    Decay d[kGlrSeg];
    float2 u[kGlrSeg], lg = both(0.f);
    // decays and inputs; tokens behind the end have a decay of 1 and no input
    glr_decay_from(a.decay_from, [&](auto form) {
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) {
        const float2 g = glr_log_decay<form.value, kFast>(par, Tile::get(from, warp, lane, k));
        lg = add2(lg, g);
        d[k] = decay_of<kFast>(g);
      }
    });
    auto input = [&](auto scale) {
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k) {
        u[k] = Tile::get(from + Tile::kArray, warp, lane, k);
        if (scale.value != KDA_GLR_INPUT_NONE) u[k] = mul2(input_factor<kFast>(scale.value, d[k]), u[k]);
      }
    };
    glr_input_scale(a.input_scale, input);
    if (gate) {
#pragma unroll
      for (int k = 0; k < kGlrSeg; ++k)
        u[k] = mul2(u[k], sigmoid2<kFast>(Tile::get(from + 2 * Tile::kArray, warp, lane, k)));
    }
    float2 h = both(0.f);
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) h = decay_apply(d[k], h, u[k]);
    const float2 dt = decay_pack(decay_of<kFast>(lg));
    seg[p][warp][lane] = make_float4(dt.x, dt.y, h.x, h.y);
    if (ranks > 1) seg_log[p][threadIdx.x] = lg;
    if (!Tile::kTma) cp_async_wait_all();  // the next tile
    ok = __syncthreads_and(ok);
    if (!ok) break;
    if (round + 2 < rounds) fetch(round + 2);  // where this tile was
    if (ranks > 1) {
      // the tile's own decay and state from zero, to every CTA of the cluster
      if (warp == 0) {
        float2 z = both(0.f), l = both(0.f);
#pragma unroll
        for (int w = 0; w < kGlrWarps; ++w) {
          const float4 s = seg[p][w][lane];
          z = decay_apply(decay_unpack(make_float2(s.x, s.y)), z, make_float2(s.z, s.w));
          l = add2(l, seg_log[p][w * 32 + lane]);
        }
        const float2 t = decay_pack(decay_of<kFast>(l));
        others.send(p, rank, ranks, lane, make_float4(t.x, t.y, z.x, z.y));
      }
      ok = others.wait(p, round);
      // the state before this CTA's tile, and the one behind the round
      h = carry;
      for (int r = 0; r < ranks; ++r) {
        const float4 s = others.tot[p][r][lane];
        if (r == rank) h = carry;
        carry = decay_apply(decay_unpack(make_float2(s.x, s.y)), carry, make_float2(s.z, s.w));
      }
    } else {
      h = round > 0 ? last[1 - p][lane] : carry;
    }
    if (a.checkpoints && warp == 0 && tile < tiles) store_states(a.checkpoints + (saved + tile) * a.D + ch, h, in);
    for (int w = 0; w < warp; ++w) {
      const float4 s = seg[p][w][lane];
      h = decay_apply(decay_unpack(make_float2(s.x, s.y)), h, make_float2(s.z, s.w));
    }
    T* py = y + (size_t)first * a.D;
#pragma unroll
    for (int k = 0; k < kGlrSeg; ++k) {
      h = decay_apply(d[k], h, u[k]);
      G::template store<Tile::kPair>(py, h, first + k < L ? in : 0);
      py += a.D;
    }
    if (warp == kGlrWarps - 1) last[p][lane] = h;
  }
  ok = __syncthreads_and(ok);
  if (!ok) {
    if (threadIdx.x == 0) atomicExch(a.status, KDA_ERR_TIMEOUT);
    glr_settle(landed, Tile::kTma ? min(round + 2, rounds) : 0, others.arrived, ranks > 1 ? round : 0);
  }
  if (ranks > 1) cluster_sync();  // no CTA leaves while another may write to it
  // (a state pool: every warp has read its first states by now)
  if (live && ok && rank == 0 && warp == 0)
    store_states(a.h_T + (size_t)slot * a.D + ch, ranks > 1 || rounds == 0 ? carry : last[(rounds - 1) & 1][lane], in);
}

template <typename T, int kPairs, bool kPair>
cudaError_t launch_few(const GlrArgs& a, cudaStream_t s) {
  constexpr int per = 2 * kPairs * kFewThreads;
  const long long blocks = (a.D + (long long)per - 1) / per * a.N;
  return launch_early(glr_few_kernel<T, kPairs, kPair>, dim3((unsigned)blocks), kFewThreads, 0, 1, s, a);
}
template <typename T, int kBytes>
cudaError_t launch_scan(const GlrArgs& a, int ranks, cudaStream_t s) {
  constexpr auto kern = glr_scan_kernel<T, kBytes>;
  constexpr int kArray = GlrTile<T, kBytes>::kArray;
  const cudaError_t e = allow_smem<kern>(6 * kArray + 128);
  if (e != cudaSuccess) return e;
  GlrMaps maps;
  if (kBytes == 16 && !glr_maps<T>(maps, a)) return cudaErrorInvalidValue;
  const long long blocks = (a.D + kGlrCols - 1LL) / kGlrCols * a.N;
  return launch_early(kern, dim3((unsigned)blocks, 1, ranks), kGlrThreads, 2 * (a.gate ? 3 : 2) * kArray + 128, ranks, s, a,
                      maps);
}

}  // namespace

cudaError_t launch_glr_few(const GlrArgs& a, int dtype, int bytes, cudaStream_t s) {
  // 16 bytes per thread where there are few tokens or threads enough all the same (32 sequences x 4096
  // channels, 1 and 16 tokens: 2.5 and 10.7 us so, 2.9 and 7.5 with 4 bytes; 256 sequences: 4.6 and 39.7, 7.0 and
  // 40.8)
  bool wide = bytes == 16 && (a.T_total <= 4LL * a.N || (long long)a.N * a.D >= 524288);
  for (const void* p : {(const void*)a.h0, (const void*)a.h_T, (const void*)a.decay_scale, (const void*)a.decay_bias,
                        (const void*)a.checkpoints})
    wide = wide && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
  if (dtype == KDA_F32) return wide ? launch_few<float, 2, true>(a, s) : launch_few<float, 1, false>(a, s);
  return wide         ? launch_few<__nv_bfloat16, 4, true>(a, s)
         : bytes >= 4 ? launch_few<__nv_bfloat16, 1, true>(a, s)
                      : launch_few<__nv_bfloat16, 1, false>(a, s);
}
cudaError_t launch_glr_scan(const GlrArgs& a, int dtype, int bytes, int ranks, cudaStream_t s) {
  if (dtype == KDA_F32)
    return bytes == 16 ? launch_scan<float, 16>(a, ranks, s) : launch_scan<float, 4>(a, ranks, s);
  return bytes == 16  ? launch_scan<__nv_bfloat16, 16>(a, ranks, s)
         : bytes == 4 ? launch_scan<__nv_bfloat16, 4>(a, ranks, s)
                      : launch_scan<__nv_bfloat16, 2>(a, ranks, s);
}

}  // namespace kda
