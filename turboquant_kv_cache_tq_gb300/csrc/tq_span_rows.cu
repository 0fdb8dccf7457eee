// Window and prefix attention of many query rows, bf16 outputs (a translation
// unit of its own, so the library builds in parallel).
#include "tq_span_rows.cuh"

namespace tq {
template cudaError_t launch_span_rows<64, false>(const SpanPass&, cudaStream_t);
template cudaError_t launch_span_rows<128, false>(const SpanPass&, cudaStream_t);
template cudaError_t launch_span_rows<256, false>(const SpanPass&, cudaStream_t);
template cudaError_t launch_span_rows<512, false>(const SpanPass&, cudaStream_t);
}  // namespace tq
