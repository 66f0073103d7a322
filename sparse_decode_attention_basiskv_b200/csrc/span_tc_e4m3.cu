// The prompt attention's instances over E4M3 caches.
#include "span_tc.cuh"

namespace basiskv {

cudaError_t launch_span_tc_e4m3(const SpanArgs& a, cudaStream_t st, bool pdl) {
  return launch_span_tc_fmt<kSpanE4m3>(a, st, pdl);
}

}  // namespace basiskv
