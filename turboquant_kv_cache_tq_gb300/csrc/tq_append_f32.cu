// Append kernels for fp32 tokens (a translation unit of their own, so the
// library builds in parallel).
#include "tq_append.cuh"

namespace tq {
template cudaError_t launch_append<64, true>(const AppendParams&, cudaStream_t);
template cudaError_t launch_append<128, true>(const AppendParams&, cudaStream_t);
template cudaError_t launch_append<256, true>(const AppendParams&, cudaStream_t);
template cudaError_t launch_append<512, true>(const AppendParams&, cudaStream_t);
}  // namespace tq
