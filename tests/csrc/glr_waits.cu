// glr_waits.cu -- the kernels of the gated linear recurrence with waits that give up at once where the
// caller says so, driven by tests/test_glr_waits.py.  Nothing is made to hang, and what a kernel does
// then is the same as behind a wait that ran out.
__device__ int gives_up[2];
#define KDA_GLR_GIVES_UP(what) (gives_up[what] != 0)

#include "../../linear_attention_recurrence_prefill_gb300/csrc/glr_scan.cu"
#include "../../linear_attention_recurrence_prefill_gb300/csrc/glr_backward.cu"

namespace {

// One sequence of T tokens x D channels in bf16, log decays, no input gate.
kda::GlrArgs args(const void* x, const void* la, float* checkpoints, int* status, int T, int D) {
  kda::GlrArgs a = {};
  a.x = x; a.la = la; a.checkpoints = checkpoints; a.status = status;
  a.N = 1; a.T_total = T; a.D = D;
  a.decay_from = KDA_GLR_LOG; a.input_scale = KDA_GLR_INPUT_NONE;
  a.ldx = a.ldla = D;
  return a;
}

}  // namespace

extern "C" {

// Whether waits for a tile, and for the other CTAs' totals, give up.
int glr_waits_set(int tile, int totals) {
  const int v[2] = {tile, totals};
  return cudaMemcpyToSymbol(gives_up, v, sizeof(v));
}

// `bytes`: how tiles are fetched (16: TMA, 4: by the threads).  Returns the launch's cudaError_t, or
// the stream's behind it.
int glr_waits_scan(const void* x, const void* la, void* y, float* h_T, float* checkpoints, int* status, int T, int D,
                   int bytes, int ranks) {
  kda::GlrArgs a = args(x, la, checkpoints, status, T, D);
  a.y = y;
  a.h_T = h_T;
  const cudaError_t e = kda::launch_glr_scan(a, KDA_BF16, bytes, ranks, nullptr);
  return e != cudaSuccess ? e : cudaStreamSynchronize(nullptr);
}

int glr_waits_backward(const void* dy, const void* x, const void* la, float* checkpoints, void* dx, void* dla,
                       float* dh0, int* status, int T, int D, int bytes, int ranks) {
  kda::GlrArgs a = args(x, la, checkpoints, status, T, D);
  a.dy = dy;
  a.dx = dx;
  a.dla = dla;
  a.dh0 = dh0;
  const cudaError_t e = kda::launch_glr_backward(a, KDA_BF16, bytes, ranks, nullptr, nullptr, nullptr);
  return e != cudaSuccess ? e : cudaStreamSynchronize(nullptr);
}

}  // extern "C"
