// The span attention's instances over bf16 caches.
#include "span_attend.cuh"

namespace basiskv {

cudaError_t launch_span_bf16(const SpanArgs& a, cudaStream_t st, bool pdl) {
  return launch_span_fmt<kSpanBf16>(a, st, pdl);
}

}  // namespace basiskv
