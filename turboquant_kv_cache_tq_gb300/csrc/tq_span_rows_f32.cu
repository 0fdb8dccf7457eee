// Window and prefix attention of many query rows, fp32 outputs (a translation
// unit of its own, so the library builds in parallel).
#include "tq_span_rows.cuh"

namespace tq {
template cudaError_t launch_span_rows<64, true>(const SpanPass&, cudaStream_t);
template cudaError_t launch_span_rows<128, true>(const SpanPass&, cudaStream_t);
template cudaError_t launch_span_rows<256, true>(const SpanPass&, cudaStream_t);
template cudaError_t launch_span_rows<512, true>(const SpanPass&, cudaStream_t);
}  // namespace tq
