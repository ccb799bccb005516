// layer_api.cu -- the C ABI of the gated delta rule and of the projections
// around it: argument checks and path selection.  As in kda_api.cu, every check
// runs on the host before anything is enqueued; a rejected call launches nothing.
#include <string.h>

#include <initializer_list>

#include "gdr.cuh"
#include "linear.cuh"

using namespace kda;

namespace {

// Sizes leave a tile's room below 2^31, so that the kernels round up in 32 bits.
constexpr int kMaxSize = 0x7fffffff - 256;

int sm_count() {  // of the current device
  static std::atomic<int> count[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  n = count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
    count[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool gdr_dk(int d) { return d == 32 || d == 64 || d == 128; }
bool gdr_dv(int d) { return gdr_dk(d) || d == 256; }
size_t elem(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }

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

// An output at the address of an input: other warps still read what one has written.
bool same(const void* out, std::initializer_list<const void*> in) {
  for (const void* p : in)
    if (out && out == p) return true;
  return false;
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

}  // extern "C"
