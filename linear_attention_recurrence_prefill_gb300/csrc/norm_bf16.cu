// norm_bf16.cu -- the root-mean-square norm of bf16 data.
#include "norm_rows.cuh"

namespace kda {
cudaError_t launch_norm_bf16(const NormArgs& a, int sms, cudaStream_t s) { return launch_t<__nv_bfloat16>(a, sms, s); }
}  // namespace kda
