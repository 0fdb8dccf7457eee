// Window and prefix attention by blocks of at most 16 query rows, head_dim 512 (one
// translation unit per head_dim and tile of rows, so the library builds in parallel).
#include "tq_span_few.cuh"

namespace tq {
template cudaError_t launch_span_few<512, 2>(SpanPass&, long long, bool, cudaStream_t);
}  // namespace tq
