// The prompt attention's instances over bf16 caches.
#include "span_tc.cuh"

namespace basiskv {

cudaError_t launch_span_tc_bf16(const SpanArgs& a, cudaStream_t st, bool pdl) {
  return launch_span_tc_fmt<kSpanBf16>(a, st, pdl);
}

}  // namespace basiskv
