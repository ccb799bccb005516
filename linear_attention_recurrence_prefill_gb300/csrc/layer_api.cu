// layer_api.cu -- the C ABI of the gated delta rule and of the projections and the
// norm around it: argument checks and path selection.  As in kda_api.cu, every check
// runs on the host before anything is enqueued; a rejected call launches nothing.
#include <string.h>

#include "checks.cuh"
#include "gdr.cuh"
#include "linear_i8.cuh"
#include "norm.cuh"

using namespace kda;

namespace {

bool gdr_dk(int d) { return d == 32 || d == 64 || d == 128; }
bool gdr_dv(int d) { return gdr_dk(d) || d == 256; }

// Checks that kda_gdr_prefill and kda_gdr_decode_step share.
int check_gdr_sizes(int N, int T_total, int H_k, int H_v, int d_k, int d_v, int dtype,
                    const kda_gdr_options* o) {
  if (N < 1 || T_total < 0 || T_total > kMaxSize || H_k < 1 || H_k > 65535 || H_v < 1 || H_v % H_k != 0)
    return KDA_ERR_SHAPE;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_DTYPE;
  if (!gdr_dk(d_k) || !gdr_dv(d_v)) return KDA_ERR_UNSUPPORTED;
  if (o->l2norm_qk != 0 && o->l2norm_qk != 1) return KDA_ERR_ARG;
  if (o->beta_is_logit != 0 && o->beta_is_logit != 1) return KDA_ERR_ARG;
  if (o->decay_from_logit != 0 && o->decay_from_logit != 1) return KDA_ERR_ARG;
  if (!(o->eps_l2 >= 0.0f) || o->q_scale != o->q_scale) return KDA_ERR_ARG;
  if (!aligned(o->decay_scale, 4) || !aligned(o->decay_bias, 4)) return KDA_ERR_ALIGN;
  if (o->slots && o->n_slots < 1) return KDA_ERR_SHAPE;
  if (!aligned(o->slots, 4)) return KDA_ERR_ALIGN;
  // token strides: at least a row, a multiple of 16 bytes
  const long long row[3] = {(long long)H_k * d_k, (long long)H_k * d_k, (long long)H_v * d_v};
  const long long ld[3] = {o->ldq, o->ldk, o->ldv};
  for (int i = 0; i < 3; ++i) {
    if (ld[i] == 0) continue;
    if (ld[i] < row[i]) return KDA_ERR_SHAPE;
    if (ld[i] % (long long)(16 / elem(dtype)) != 0) return KDA_ERR_ALIGN;
  }
  // grids: one warp per 16 columns of a state, one CTA per chunk and head
  if ((long long)N * H_v * (d_v / 16) > 0x7fffffffLL) return KDA_ERR_SHAPE;
  if (((long long)T_total / 64 + N) * H_v > 0x7fffffffLL) return KDA_ERR_SHAPE;
  return KDA_OK;
}

int check_gdr_arrays(const void* q, const void* k, const void* v, const float* log_alpha,
                     const void* beta, const float* S0, const void* o, const float* S_T,
                     int T_total, int dtype) {
  if (!S_T || (T_total > 0 && (!q || !k || !v || !log_alpha || !beta || !o))) return KDA_ERR_ARG;
  const void* p16[] = {q, k, v, S0, o, S_T};
  for (const void* p : p16)
    if (!aligned(p, 16)) return KDA_ERR_ALIGN;
  if (!aligned(log_alpha, 4) || !aligned(beta, elem(dtype))) return KDA_ERR_ALIGN;
  return KDA_OK;
}

GdrArgs gdr_args(const void* q, const void* k, const void* v, const float* log_alpha,
                 const void* beta, const float* S0, float* S_T, void* o, int N, int T_total,
                 int H_k, int H_v, int d_k, int d_v, const kda_gdr_options* op, int* status) {
  GdrArgs a;
  a.q = q; a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta;
  a.S0 = S0; a.S_T = S_T; a.o = o;
  a.cu_seqlens = nullptr; a.slots = op->slots; a.n_slots = op->n_slots;
  a.decay_scale = op->decay_scale; a.decay_bias = op->decay_bias;
  a.snapshots = nullptr; a.status = status;
  a.N = N; a.T_total = T_total; a.Hk = H_k; a.Hv = H_v; a.dk = d_k; a.dv = d_v;
  a.l2norm_qk = op->l2norm_qk; a.beta_is_logit = op->beta_is_logit;
  a.decay_from_logit = op->decay_from_logit;
  a.q_scale = op->q_scale; a.eps_l2 = op->eps_l2;
  // a single token's stride says nothing, and a tensor map takes none of 2^40 bytes
  const bool dense = T_total < 2;
  a.ldq = op->ldq && !dense ? op->ldq : (long long)H_k * d_k;
  a.ldk = op->ldk && !dense ? op->ldk : (long long)H_k * d_k;
  a.ldv = op->ldv && !dense ? op->ldv : (long long)H_v * d_v;
  return a;
}

}  // namespace

extern "C" {

void kda_gdr_options_init(kda_gdr_options* opt) {
  if (!opt) return;
  memset(opt, 0, sizeof(*opt));
  opt->l2norm_qk = 1;
  opt->q_scale = 1.0f;
  opt->eps_l2 = 1e-6f;
  opt->impl = KDA_IMPL_AUTO;
}

int kda_gdr_prefill_path(int T_total, int N, int H_k, int H_v, int d_k, int d_v, int dtype,
                         const kda_gdr_options* opt) {
  kda_gdr_options def;
  if (!opt) kda_gdr_options_init(&def);
  const kda_gdr_options* op = opt ? opt : &def;
  const int rc = check_gdr_sizes(N, T_total, H_k, H_v, d_k, d_v, dtype, op);
  if (rc != KDA_OK) return rc;
  if (op->max_seqlen < 0 || op->max_seqlen > T_total) return KDA_ERR_SHAPE;
  const bool tc = gdr_chunked_supported(d_k, d_v, dtype);
  switch (op->impl) {
    case KDA_IMPL_SIMT: return KDA_IMPL_SIMT;
    case KDA_IMPL_TC:  // without a token there is no chunk, only states to hand on
      if (!tc) return KDA_ERR_UNSUPPORTED;
      return T_total > 0 ? KDA_IMPL_TC : KDA_IMPL_SIMT;
    case KDA_IMPL_AUTO: {
      // Token by token where no sequence is longer than this.  32 heads of 128 x 128, 1, 16 and 256
      // sequences: 16 tokens took 14, 53 and 641 us that way and 21, 53 and 688 us in chunks, 24
      // tokens 19, 74 and 914 against 21, 56 and 697 us.  Heads of 64 x 64, 16 sequences: 48 tokens
      // 46 and 52 us, 64 tokens 59 and 60 us.
      const int longest = op->max_seqlen > 0 ? op->max_seqlen : T_total;
      return tc && longest > (d_k * d_v <= 64 * 64 ? 48 : 16) ? KDA_IMPL_TC : KDA_IMPL_SIMT;
    }
    default: return KDA_ERR_UNSUPPORTED;
  }
}

size_t kda_gdr_prefill_workspace_size(int T_total, int N, int H_k, int H_v, int d_k, int d_v,
                                      int dtype, const kda_gdr_options* opt) {
  const int path = kda_gdr_prefill_path(T_total, N, H_k, H_v, d_k, d_v, dtype, opt);
  return path == KDA_IMPL_TC ? gdr_chunked_workspace_bytes(T_total, N, H_v) : 0;
}

int kda_gdr_prefill(const void* q, const void* k, const void* v, const float* log_alpha,
                    const void* beta, const float* S0, const int32_t* cu_seqlens, int N, void* o,
                    float* S_T, int T_total, int H_k, int H_v, int d_k, int d_v, int dtype,
                    const kda_gdr_options* opt, kda_stream_t stream) {
  kda_gdr_options def;
  if (!opt) kda_gdr_options_init(&def);
  const kda_gdr_options* op = opt ? opt : &def;
  int rc = check_gdr_arrays(q, k, v, log_alpha, beta, S0, o, S_T, T_total, dtype);
  if (rc != KDA_OK) return rc;
  const int path = kda_gdr_prefill_path(T_total, N, H_k, H_v, d_k, d_v, dtype, op);
  if (path < 0) return path;
  if (!cu_seqlens && T_total % N != 0) return KDA_ERR_SHAPE;
  if (!aligned(cu_seqlens, 4)) return KDA_ERR_ALIGN;
  if (op->snapshots) return KDA_ERR_UNSUPPORTED;
  if (path == KDA_IMPL_TC) {
    if (!op->workspace || op->workspace_bytes < gdr_chunked_workspace_bytes(T_total, N, H_v))
      return KDA_ERR_WORKSPACE;
    if (!aligned(op->workspace, 16)) return KDA_ERR_ALIGN;
  }
  if (same(o, {q, k, v, log_alpha, beta, S0, S_T, op->workspace})) return KDA_ERR_ARG;
  if (same(S_T, {q, k, v, log_alpha, beta, op->workspace})) return KDA_ERR_ARG;
  for (const void* out : {(const void*)o, (const void*)S_T})
    if (same(out, {cu_seqlens, op->slots, op->decay_scale, op->decay_bias})) return KDA_ERR_ARG;
  int* status = status_word();
  if (!status) return KDA_ERR_CUDA;
  GdrArgs a = gdr_args(q, k, v, log_alpha, beta, S0, S_T, o, N, T_total, H_k, H_v, d_k, d_v, op,
                       status);
  a.cu_seqlens = cu_seqlens;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = path == KDA_IMPL_TC ? launch_gdr_chunked(a, op->workspace, s)
                                            : launch_gdr_recurrent(a, dtype, s);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_gdr_decode_step(const void* q, const void* k, const void* v, const float* log_alpha,
                        const void* beta, float* S, void* o, int N, int L, int H_k, int H_v,
                        int d_k, int d_v, int dtype, const kda_gdr_options* opt,
                        kda_stream_t stream) {
  kda_gdr_options def;
  if (!opt) kda_gdr_options_init(&def);
  const kda_gdr_options* op = opt ? opt : &def;
  if (N < 1 || L < 1 || (long long)N * L > 0x7fffffffLL) return KDA_ERR_SHAPE;
  const int T = N * L;
  int rc = check_gdr_arrays(q, k, v, log_alpha, beta, S, o, S, T, dtype);
  if (rc != KDA_OK) return rc;
  rc = check_gdr_sizes(N, T, H_k, H_v, d_k, d_v, dtype, op);
  if (rc != KDA_OK) return rc;
  if (!aligned(op->snapshots, 16)) return KDA_ERR_ALIGN;
  if (same(o, {q, k, v, log_alpha, beta, S, op->snapshots})) return KDA_ERR_ARG;
  if (same(S, {q, k, v, log_alpha, beta})) return KDA_ERR_ARG;
  if (same(op->snapshots, {q, k, v, log_alpha, beta, S})) return KDA_ERR_ARG;
  for (const void* out : {(const void*)o, (const void*)S, (const void*)op->snapshots})
    if (same(out, {op->slots, op->decay_scale, op->decay_bias})) return KDA_ERR_ARG;
  int* status = status_word();
  if (!status) return KDA_ERR_CUDA;
  GdrArgs a = gdr_args(q, k, v, log_alpha, beta, S, S, o, N, T, H_k, H_v, d_k, d_v, op, status);
  a.snapshots = op->snapshots;
  const cudaError_t e = launch_gdr_recurrent(a, dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_linear(const void* x, long long ldx, const void* w, long long ldw, const void* bias,
               const void* residual, long long ldr, void* y, long long ldy, int M, int N, int K,
               int act, int dtype, kda_stream_t stream) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxSize || N > kMaxSize || K > kMaxSize) return KDA_ERR_SHAPE;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_DTYPE;
  if (act < KDA_ACT_NONE || act > KDA_ACT_SIGMOID) return KDA_ERR_ARG;
  if (ldx == 0) ldx = K;
  if (ldw == 0) ldw = K;
  if (ldr == 0) ldr = N;
  if (ldy == 0) ldy = N;
  if (ldx < K || ldw < K || ldr < N || ldy < N) return KDA_ERR_SHAPE;
  if (M == 0 || N == 0) return KDA_OK;
  if (!y || (K > 0 && (!x || !w))) return KDA_ERR_ARG;
  const void* ptrs[] = {x, w, bias, residual, y};
  for (const void* p : ptrs)
    if (!aligned(p, elem(dtype))) return KDA_ERR_ALIGN;
  // in place only where every element is read and written by the same thread
  if (residual == y && ldr != ldy) return KDA_ERR_ARG;
  if (same(y, {bias}) || (K > 0 && same(y, {x, w}))) return KDA_ERR_ARG;
  LinearArgs a;
  a.x = x; a.w = w; a.bias = bias; a.residual = residual; a.y = y;
  a.ldx = ldx; a.ldw = ldw; a.ldr = ldr; a.ldy = ldy;
  a.M = M; a.N = N; a.K = K; a.act = act;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int sms = sm_count();
  cudaError_t e;
  if (linear_few_takes(a, dtype)) {
    e = launch_linear_few(a, dtype, sms, s);
  } else if (linear_tc_takes(a, dtype)) {
    int* status = status_word();
    if (!status) return KDA_ERR_CUDA;
    e = launch_linear_tc(a, sms, status, s);
  } else {
    e = launch_linear_simt(a, dtype, sms, s);
  }
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_linear_i8_workspace_size(int M, int N, int K) {
  if (M < 1 || N < 1 || K < 1 || M > kMaxSize || N > kMaxSize || K > kMaxSize) return 0;
  return linear_i8_workspace_bytes(M, N, K);
}

int kda_linear_i8(const int8_t* x, long long ldx, const float* x_scale, const int8_t* w,
                  long long ldw, const float* w_scale, const void* bias, const void* residual,
                  long long ldr, void* y, long long ldy, int M, int N, int K, int act, int dtype,
                  void* workspace, size_t workspace_bytes, kda_stream_t stream) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxSize || N > kMaxSize || K > kMaxSize) return KDA_ERR_SHAPE;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_DTYPE;
  if (act < KDA_ACT_NONE || act > KDA_ACT_SIGMOID) return KDA_ERR_ARG;
  if (ldx == 0) ldx = K;
  if (ldw == 0) ldw = K;
  if (ldr == 0) ldr = N;
  if (ldy == 0) ldy = N;
  if (ldx < K || ldw < K || ldr < N || ldy < N) return KDA_ERR_SHAPE;
  if (M == 0 || N == 0) return KDA_OK;
  if (!linear_i8_tc_takes(M, N)) return KDA_ERR_SHAPE;  // tiles in a grid
  if (!y || !x_scale || !w_scale || (K > 0 && (!x || !w))) return KDA_ERR_ARG;
  if (!aligned(x_scale, 4) || !aligned(w_scale, 4)) return KDA_ERR_ALIGN;
  for (const void* p : {bias, residual, (const void*)y})
    if (!aligned(p, elem(dtype))) return KDA_ERR_ALIGN;
  LinearI8Args a;
  a.l.x = x; a.l.w = w; a.l.bias = bias; a.l.residual = residual; a.l.y = y;
  a.l.ldx = ldx; a.l.ldw = ldw; a.l.ldr = ldr; a.l.ldy = ldy;
  a.l.M = M; a.l.N = N; a.l.K = K; a.l.act = act;
  a.x_scale = x_scale; a.w_scale = w_scale;
  const bool few = linear_i8_few_takes(a), needed = K > 0 && !few && linear_i8_tc_needs_workspace(a.l);
  if (needed) {
    if (!workspace || workspace_bytes < linear_i8_workspace_bytes(M, N, K)) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return KDA_ERR_ALIGN;
  }
  // in place only where every element is read and written by the same thread
  if (residual == y && ldr != ldy) return KDA_ERR_ARG;
  void* const ws = needed ? workspace : nullptr;
  if (same(y, {bias, x_scale, w_scale, ws}) || (K > 0 && same(y, {x, w}))) return KDA_ERR_ARG;
  if (same(ws, {x, w, x_scale, w_scale, bias, residual})) return KDA_ERR_ARG;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (K == 0) {
    e = launch_linear_i8_none(a, dtype, s);
  } else if (few) {
    e = launch_linear_i8_few(a, dtype, sm_count(), s);
  } else {
    int* status = status_word();
    if (!status) return KDA_ERR_CUDA;
    e = launch_linear_i8_tc(a, dtype, ws, sm_count(), status, s);
  }
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_rmsnorm(const void* x, long long ldx, const void* residual, long long ldr, const float* w,
                void* sum, long long lds, void* y, long long ldy, int8_t* q, long long ldq,
                float* scale, int M, int D, float eps, int dtype, kda_stream_t stream) {
  if (M < 0 || D < 1 || M > kMaxSize || D > kMaxSize) return KDA_ERR_SHAPE;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_DTYPE;
  if (!(eps >= 0.f)) return KDA_ERR_ARG;
  long long* const lds_of[] = {&ldx, &ldr, &lds, &ldy, &ldq};
  for (long long* ld : lds_of) {
    if (*ld == 0) *ld = D;
    if (*ld < D) return KDA_ERR_SHAPE;
  }
  if (M == 0) return KDA_OK;  // (arrays without an element have no address)
  if (!x || (q == nullptr) != (scale == nullptr) || (!y && !q)) return KDA_ERR_ARG;
  for (const void* p : {x, residual, (const void*)sum, (const void*)y})
    if (!aligned(p, elem(dtype))) return KDA_ERR_ALIGN;
  if (!aligned(w, 4) || !aligned(scale, 4)) return KDA_ERR_ALIGN;
  if (same(y, {x, residual, w, sum, q, scale}) || same(q, {x, residual, w, sum, scale})) return KDA_ERR_ARG;
  if (same(scale, {x, residual, w, sum}) || same(sum, {w})) return KDA_ERR_ARG;
  if ((sum == x && lds != ldx) || (sum && sum == residual && lds != ldr)) return KDA_ERR_ARG;
  NormArgs a;
  a.x = x; a.residual = residual; a.w = w; a.sum = sum; a.y = y; a.q = q; a.scale = scale;
  a.ldx = ldx; a.ldr = ldr; a.lds = lds; a.ldy = ldy; a.ldq = ldq;
  a.M = M; a.D = D; a.eps = eps; a.norm = true;
  const cudaError_t e = launch_norm(a, dtype, sm_count(), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_quantize_i8(const void* x, long long ldx, int8_t* q, long long ldq, float* scale, int M,
                    int D, int dtype, kda_stream_t stream) {
  if (M < 0 || D < 1 || M > kMaxSize || D > kMaxSize) return KDA_ERR_SHAPE;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_DTYPE;
  if (ldx == 0) ldx = D;
  if (ldq == 0) ldq = D;
  if (ldx < D || ldq < D) return KDA_ERR_SHAPE;
  if (M == 0) return KDA_OK;
  if (!x || !q || !scale) return KDA_ERR_ARG;
  if (!aligned(x, elem(dtype)) || !aligned(scale, 4)) return KDA_ERR_ALIGN;
  if (same(q, {x, scale}) || same(scale, {x})) return KDA_ERR_ARG;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.q = q; a.scale = scale;
  a.ldx = ldx; a.ldq = ldq;
  a.M = M; a.D = D; a.norm = false;
  const cudaError_t e = launch_norm(a, dtype, sm_count(), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
