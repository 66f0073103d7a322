// The span attention's instances over 4-bit caches.
#include "span_attend.cuh"

namespace basiskv {

cudaError_t launch_span_q4(const SpanArgs& a, cudaStream_t st, bool pdl) {
  return launch_span_fmt<kSpanQ4>(a, st, pdl);
}

}  // namespace basiskv
