// glr_api.cu -- the C ABI of the gated linear recurrence: argument checks and
// path selection, on the host before anything is enqueued.
#include <string.h>

#include "checks.cuh"
#include "glr.cuh"

using namespace kda;

namespace {

// Tiles of tokens are counted in 32 bits, up to 16 CTAs of them beyond the end.
constexpr int kMaxTokens = 0x7fffffff - 2048;

int check_glr(int N, int T_total, int D, int dtype, const kda_glr_options* o) {
  if (N < 1 || T_total < 0 || T_total > kMaxTokens || D < 1 || D > kMaxSize) return KDA_ERR_SHAPE;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_DTYPE;
  if (o->decay_from < KDA_GLR_LOG || o->decay_from > KDA_GLR_SIGMOID) return KDA_ERR_ARG;
  if (o->input_scale < KDA_GLR_INPUT_NONE || o->input_scale > KDA_GLR_INPUT_NORMALIZED) return KDA_ERR_ARG;
  if (o->max_seqlen < 0 || o->max_seqlen > T_total) return KDA_ERR_SHAPE;
  for (long long ld : {o->ldx, o->ldla, o->ldg})
    if (ld != 0 && ld < D) return KDA_ERR_SHAPE;
  if (o->slots && o->n_slots < 1) return KDA_ERR_SHAPE;
  if (!aligned(o->slots, 4)) return KDA_ERR_ALIGN;
  for (const void* p : {(const void*)o->decay_scale, (const void*)o->decay_bias, (const void*)o->checkpoints})
    if (!aligned(p, 4)) return KDA_ERR_ALIGN;
  if (!aligned(o->input_gate, elem(dtype))) return KDA_ERR_ALIGN;
  if ((D + 63LL) / 64 * N > 0x7ffffffeLL) return KDA_ERR_SHAPE;  // the grid
  return KDA_OK;
}

GlrArgs glr_args(const void* x, const void* la, const int32_t* cu, int N, int T_total, int D,
                 const kda_glr_options* o, int* status) {
  GlrArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.la = la; a.gate = o->input_gate;
  a.cu_seqlens = cu; a.slots = o->slots; a.n_slots = o->n_slots;
  const bool log = o->decay_from == KDA_GLR_LOG;
  a.decay_scale = log ? nullptr : o->decay_scale;
  a.decay_bias = log ? nullptr : o->decay_bias;
  a.checkpoints = o->checkpoints; a.status = status;
  a.N = N; a.T_total = T_total; a.D = D;
  a.decay_from = o->decay_from; a.input_scale = o->input_scale;
  a.ldx = o->ldx ? o->ldx : D; a.ldla = o->ldla ? o->ldla : D; a.ldg = o->ldg ? o->ldg : D;
  return a;
}

// The bytes that rows, bases and D allow to move at once (GlrTile): 16 (which tensor maps take, up to
// 2^40 bytes from row to row), 4, or 2.
int piece(const GlrArgs& a, int dtype) {
  const int e = (int)elem(dtype);
  for (int bytes : {16, 4}) {
    const int n = bytes / e;
    bool fits = bytes < 16 || (a.ldx < (1LL << 37) && a.ldla < (1LL << 37) && a.ldg < (1LL << 37));
    fits = fits && a.D % n == 0 && a.ldx % n == 0 && a.ldla % n == 0 && (!a.gate || a.ldg % n == 0);
    for (const void* p : {a.x, a.la, a.gate, (const void*)a.y, a.dy, (const void*)a.dx, (const void*)a.dla,
                          (const void*)a.dgate})
      fits = fits && aligned(p, bytes);
    if (fits) return bytes;
  }
  return 2;
}

// CTAs that share a sequence's tokens, a power of two, by what they cost in tiles' times: a CTA has two
// more to begin and end, an SM two CTAs at a time (one in fp32, whose tiles take twice the shared
// memory), and a tile takes three tenths longer where its total goes to other CTAs.  Sequences of one length
// go in waves; of others the host knows the longest, which one row of CTAs walks, and all tokens together.
// Measured, bf16, us for 1, 2, 4, 8 CTAs: forward, 32,768 tokens x 4096 588, 464, 297, 344, nine prompts of
// 12,000 tokens in all 105, 113, 132, 183; with the gradient, one sequence of 4096 381, 254, 146, 159, four of
// 16,384 in all 939, 538, 499, 580, sixteen of 8000 in all x 2048 221, 176, 208, 317.
int glr_ranks(int T_total, int N, int D, int dtype, int max_seqlen) {
  const long long longest = max_seqlen > 0 ? max_seqlen : T_total;
  if (longest == 0) return 1;
  const long long tiles = (longest + kGlrTile - 1) / kGlrTile, blocks = (D + 63LL) / 64;
  const long long slots = (dtype == KDA_BF16 ? 2LL : 1LL) * sm_count();
  const bool alike = 5LL * T_total >= 4 * longest * N;
  int best = 1;
  double least = 0.;
  for (int ranks = 1; ranks <= kGlrMaxRanks && ranks <= tiles; ranks *= 2) {
    const double row = (double)((tiles + ranks - 1) / ranks) + 2.;
    const double all = alike ? (double)((N * blocks * ranks + slots - 1) / slots) * row
                             : ((double)T_total / kGlrTile + 2. * N * ranks) * blocks / slots;
    const double cost = (all > row ? all : row) * (ranks > 1 ? 1.3 : 1.);
    if (ranks == 1 || cost < least) {
      least = cost;
      best = ranks;
    }
  }
  return best;
}

// Whether the sequences are walked token by token, a thread per two channels: fastest where they
// are short and so many that they fill the GPU by themselves.  In units of 10 ns, fitted to what
// 4096 channels took: a token 0.25 us and the time of its share, a tile 3.5 us in waves as above.
// Measured this way and in tiles, bf16, us: 1 sequence of 4, 16, 64 tokens 2.9, 6.2, 19 and 3.7 each; 32
// of them 3.7, 7.5, 32 and 24 each; 256 of them 11, 41, 146 and 173, 188, 191, of 200 tokens 445
// and 491, of 1000 tokens 2196 and 1700.
bool glr_by_token(int T_total, int N, int D, int dtype, int max_seqlen) {
  const long long longest = max_seqlen > 0 ? max_seqlen : T_total;
  if (longest > 256) return false;
  const long long tiles = (longest + kGlrTile - 1) / kGlrTile, blocks = (D + 63LL) / 64;
  const long long slots = (dtype == KDA_BF16 ? 2LL : 1LL) * sm_count();
  const long long ranks = glr_ranks(T_total, N, D, dtype, max_seqlen);
  const double by_token = 200. + 25. * longest + (double)T_total * blocks / 60;
  const double all = ((double)T_total / kGlrTile + N / 2.) * blocks / slots, one = (double)(tiles + ranks - 1) / ranks;
  return by_token < 350. * (all > one ? all : one);
}

}  // namespace

extern "C" {

void kda_glr_options_init(kda_glr_options* opt) {
  if (!opt) return;
  memset(opt, 0, sizeof(*opt));
  opt->decay_from = KDA_GLR_LOG;
  opt->input_scale = KDA_GLR_INPUT_NONE;
}

int kda_glr_scan(const void* x, const void* log_alpha, const float* h0, const int32_t* cu_seqlens,
                 int N, void* y, float* h_T, int T_total, int D, int dtype,
                 const kda_glr_options* opt, kda_stream_t stream) {
  kda_glr_options def;
  if (!opt) kda_glr_options_init(&def);
  const kda_glr_options* o = opt ? opt : &def;
  const int rc = check_glr(N, T_total, D, dtype, o);
  if (rc != KDA_OK) return rc;
  if (!h_T || (T_total > 0 && (!x || !log_alpha || !y))) return KDA_ERR_ARG;
  for (const void* p : {x, log_alpha, (const void*)y})
    if (!aligned(p, elem(dtype))) return KDA_ERR_ALIGN;
  if (!aligned(h0, 4) || !aligned(h_T, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_ALIGN;
  if (!cu_seqlens && T_total % N != 0) return KDA_ERR_SHAPE;
  for (const void* out : {(const void*)y, (const void*)h_T, (const void*)o->checkpoints})
    if (same(out, {x, log_alpha, o->input_gate, o->decay_scale, o->decay_bias, cu_seqlens, o->slots})) return KDA_ERR_ARG;
  if (same(y, {h0, h_T, o->checkpoints}) || same(o->checkpoints, {h0, h_T})) return KDA_ERR_ARG;
  int* status = status_word();
  if (!status) return KDA_ERR_CUDA;
  GlrArgs a = glr_args(x, log_alpha, cu_seqlens, N, T_total, D, o, status);
  a.h0 = h0; a.h_T = h_T; a.y = y;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      glr_by_token(T_total, N, D, dtype, o->max_seqlen)
          ? launch_glr_few(a, dtype, piece(a, dtype), s)
          : launch_glr_scan(a, dtype, piece(a, dtype), glr_ranks(T_total, N, D, dtype, o->max_seqlen), s);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_glr_step(const void* x, const void* log_alpha, float* h, void* y, int N, int L, int D,
                 int dtype, const kda_glr_options* opt, kda_stream_t stream) {
  kda_glr_options def;
  if (!opt) kda_glr_options_init(&def);
  const kda_glr_options* o = opt ? opt : &def;
  if (N < 1 || L < 1 || (long long)N * L > kMaxTokens) return KDA_ERR_SHAPE;
  const int T = N * L;
  const int rc = check_glr(N, T, D, dtype, o);
  if (rc != KDA_OK) return rc;
  if (o->checkpoints) return KDA_ERR_UNSUPPORTED;
  if (!x || !log_alpha || !h || !y) return KDA_ERR_ARG;
  for (const void* p : {x, log_alpha, (const void*)y})
    if (!aligned(p, elem(dtype))) return KDA_ERR_ALIGN;
  if (!aligned(h, 4)) return KDA_ERR_ALIGN;
  for (const void* out : {(const void*)y, (const void*)h})
    if (same(out, {x, log_alpha, o->input_gate, o->decay_scale, o->decay_bias, o->slots})) return KDA_ERR_ARG;
  if (same(y, {h})) return KDA_ERR_ARG;
  int* status = status_word();
  if (!status) return KDA_ERR_CUDA;
  GlrArgs a = glr_args(x, log_alpha, nullptr, N, T, D, o, status);
  a.h0 = h; a.h_T = h; a.y = y;
  const cudaError_t e = launch_glr_few(a, dtype, piece(a, dtype), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_glr_backward_workspace_size(int T_total, int N, int D, int dtype,
                                       const kda_glr_options* opt) {
  kda_glr_options def;
  if (!opt) kda_glr_options_init(&def);
  const kda_glr_options* o = opt ? opt : &def;
  if (check_glr(N, T_total, D, dtype, o) != KDA_OK) return 0;
  return (size_t)N * glr_ranks(T_total, N, D, dtype, o->max_seqlen) * D * sizeof(double2);
}

int kda_glr_scan_backward(const void* dy, const float* dh_T, const void* x, const void* log_alpha,
                          const int32_t* cu_seqlens, int N, void* dx, void* dlog_alpha,
                          void* dinput_gate, float* dh0, float* ddecay_scale, float* ddecay_bias,
                          int T_total, int D, int dtype, const kda_glr_options* opt,
                          kda_stream_t stream) {
  kda_glr_options def;
  if (!opt) kda_glr_options_init(&def);
  const kda_glr_options* o = opt ? opt : &def;
  const int rc = check_glr(N, T_total, D, dtype, o);
  if (rc != KDA_OK) return rc;
  if (o->slots) return KDA_ERR_UNSUPPORTED;
  if (T_total > 0 && (!x || !log_alpha || !dx || !dlog_alpha || !o->checkpoints)) return KDA_ERR_ARG;
  if (dinput_gate && !o->input_gate) return KDA_ERR_ARG;
  const bool sums = ddecay_scale || ddecay_bias;
  if (sums && o->decay_from == KDA_GLR_LOG) return KDA_ERR_ARG;
  for (const void* p : {dy, x, log_alpha, (const void*)dx, (const void*)dlog_alpha, (const void*)dinput_gate})
    if (!aligned(p, elem(dtype))) return KDA_ERR_ALIGN;
  for (const void* p : {(const void*)dh_T, (const void*)dh0, (const void*)ddecay_scale, (const void*)ddecay_bias,
                        (const void*)cu_seqlens})
    if (!aligned(p, 4)) return KDA_ERR_ALIGN;
  if (!cu_seqlens && T_total % N != 0) return KDA_ERR_SHAPE;
  void* const ws = sums ? o->workspace : nullptr;
  if (sums) {
    if (!ws || o->workspace_bytes < kda_glr_backward_workspace_size(T_total, N, D, dtype, o)) return KDA_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return KDA_ERR_ALIGN;
  }
  const void* out[] = {dx, dlog_alpha, dinput_gate, dh0, ddecay_scale, ddecay_bias, ws};
  for (int i = 0; i < 7; ++i) {
    if (same(out[i], {dy, dh_T, x, log_alpha, o->input_gate, o->decay_scale, o->decay_bias, o->checkpoints, cu_seqlens}))
      return KDA_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (same(out[i], {out[j]})) return KDA_ERR_ARG;
  }
  int* status = status_word();
  if (!status) return KDA_ERR_CUDA;
  GlrArgs a = glr_args(x, log_alpha, cu_seqlens, N, T_total, D, o, status);
  a.dy = dy; a.dh_T = dh_T; a.dx = dx; a.dla = dlog_alpha; a.dgate = dinput_gate; a.dh0 = dh0;
  a.partial = static_cast<double2*>(ws);
  const cudaError_t e = launch_glr_backward(a, dtype, piece(a, dtype), glr_ranks(T_total, N, D, dtype, o->max_seqlen),
                                            ddecay_scale, ddecay_bias, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
