// gdr.cuh -- the gated delta rule: arguments and the per-token quantities that
// its recurrent and its chunked kernels share.
#pragma once

#include "kda_common.cuh"

namespace kda {

struct GdrArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* log_alpha;
  const void* beta;
  const float* S0;          // NULL: zeros
  float* S_T;
  void* o;
  const int32_t* cu_seqlens;  // NULL: N sequences of T_total / N tokens
  const int32_t* slots;       // NULL: state n belongs to sequence n
  const float* decay_scale;
  const float* decay_bias;
  float* snapshots;           // NULL, or the state after each token
  int* status;
  int N, T_total, Hk, Hv, dk, dv, n_slots;
  int l2norm_qk, beta_is_logit, decay_from_logit;
  float q_scale, eps_l2;
  long long ldq, ldk, ldv;    // elements between tokens
};

// The log decay of one token and head.  softplus(x) = max(x, 0) + log1p(e^-|x|).
// Everything below -200 acts as -200, so that sums of log decays stay finite:
// e^-200 is 0 in fp32 either way.
__device__ __forceinline__ float gdr_log_decay(const GdrArgs& a, float x, int h) {
  if (a.decay_from_logit) {
    const float A = a.decay_scale ? a.decay_scale[h] : 1.f;
    const float z = x + (a.decay_bias ? a.decay_bias[h] : 0.f);
    x = -A * (fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
  }
  return x > 0.f ? 0.f : x < -200.f ? -200.f : x;  // NaN stays
}

// 1 / sqrt(|x|^2 + eps) (0 for a zero row with eps = 0).
__device__ __forceinline__ float gdr_inv_norm(float sum_sq, float eps) {
  const float s = sum_sq + eps;
  return s > 0.f ? 1.0f / sqrtf(s) : 0.f;
}

// Offset i of the packed sequences (cu_seqlens, or equal lengths).
__device__ __forceinline__ int gdr_offset(const GdrArgs& a, int i) {
  return a.cu_seqlens ? a.cu_seqlens[i] : i * (a.T_total / a.N);
}

// The token range and the state matrix of sequence n, found by one whole warp
// (every lane gets the answer).  False: the sequence is left out, because its
// slot is negative, or (status word set) because its slot is out of range or
// taken by an earlier sequence, its tokens are out of range, or the offsets
// decrease at it or before it.  Up to 32 sequences take one round of loads, a
// sequence per lane.
__device__ __forceinline__ bool gdr_sequence(const GdrArgs& a, int n, int& t0, int& t1,
                                             int& slot) {
  const int lane = threadIdx.x & 31;
  bool bad;
  if (a.N <= 32) {
    const int i = lane < a.N ? lane : a.N - 1;
    const int off = gdr_offset(a, i), end = gdr_offset(a, i + 1), sl = a.slots ? a.slots[i] : i;
    t0 = __shfl_sync(0xffffffffu, off, n);
    t1 = __shfl_sync(0xffffffffu, end, n);
    slot = __shfl_sync(0xffffffffu, sl, n);
    if (slot < 0) return false;
    bad = t0 < 0 || t1 > a.T_total || (a.slots && slot >= a.n_slots) ||
          __any_sync(0xffffffffu, (lane <= n && off > end) || (lane < n && sl == slot));
  } else {
    seq_range(a.cu_seqlens, a.N, a.T_total, n, t0, t1);
    slot = a.slots ? a.slots[n] : n;
    if (slot < 0) return false;
    bad = t0 < 0 || t1 < t0 || t1 > a.T_total || (a.slots && slot >= a.n_slots);
    bool found = false;
    if (a.cu_seqlens)
      for (int i = lane; i < n; i += 32) found |= a.cu_seqlens[i] > a.cu_seqlens[i + 1];
    if (a.slots)
      for (int i = lane; i < n; i += 32) found |= a.slots[i] == slot;
    bad |= __any_sync(0xffffffffu, found);
  }
  if (bad && lane == 0) atomicExch(a.status, KDA_ERR_SHAPE);
  return !bad;
}

// Launchers; each returns the launch's cudaError_t.
cudaError_t launch_gdr_recurrent(const GdrArgs& a, int dtype, cudaStream_t s);
bool gdr_chunked_supported(int d_k, int d_v, int dtype);
size_t gdr_chunked_workspace_bytes(int T_total, int N, int Hv);
cudaError_t launch_gdr_chunked(const GdrArgs& a, void* workspace, cudaStream_t s);

}  // namespace kda
