// The prompt attention's instances over 4-bit caches.
#include "span_tc.cuh"

namespace basiskv {

cudaError_t launch_span_tc_q4(const SpanArgs& a, cudaStream_t st, bool pdl) {
  return launch_span_tc_fmt<kSpanQ4>(a, st, pdl);
}

}  // namespace basiskv
