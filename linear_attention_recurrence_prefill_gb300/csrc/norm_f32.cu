// norm_f32.cu -- the root-mean-square norm of f32 data.
#include "norm_rows.cuh"

namespace kda {
cudaError_t launch_norm_f32(const NormArgs& a, int sms, cudaStream_t s) { return launch_t<float>(a, sms, s); }
}  // namespace kda
