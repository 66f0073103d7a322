// The span attention's instances over 4-bit caches with pages of 32 tokens.
#include "span_attend.cuh"

namespace basiskv {

cudaError_t launch_span_q4_p32(const SpanArgs& a, cudaStream_t st, bool pdl) {
  return launch_span_fmt<kSpanQ4, true>(a, st, pdl);
}

}  // namespace basiskv
