// The tree attention's kernels for fp32 outputs (a translation unit of their
// own, so the library builds in parallel).
#include "tq_tree_attention.cuh"

namespace tq {
template cudaError_t launch_tree_split<64, true>(const TreeParams&, cudaStream_t);
template cudaError_t launch_tree_split<128, true>(const TreeParams&, cudaStream_t);
template cudaError_t launch_tree_split<256, true>(const TreeParams&, cudaStream_t);
template cudaError_t launch_tree_split<512, true>(const TreeParams&, cudaStream_t);
}  // namespace tq
