// The span attention's instances over 4-bit caches with pages of 16 tokens.
#include "span_attend.cuh"

namespace basiskv {

cudaError_t launch_span_q4(const SpanArgs& a, cudaStream_t st, bool pdl) {
  return a.S == 32 ? launch_span_q4_p32(a, st, pdl) : launch_span_fmt<kSpanQ4>(a, st, pdl);
}

}  // namespace basiskv
