// The work of a ragged batch as one line: each sequence contributes count(b)
// units for each of its KV heads, in (sequence, KV head, unit) order, and a
// launch cuts the line into equal runs.
#pragma once

#include "common.cuh"

namespace basiskv {

constexpr int kLineMaxSeqs = 256;

// pre[b] = sum of count(b') over b' < b, pre[B] = the sum over all.  Called by
// all threads of a block of kLineMaxSeqs threads (B <= kLineMaxSeqs); ends
// with a barrier.
template <class Count>
__device__ __forceinline__ void line_scan(int B, long long* pre, Count count) {
  __shared__ long long wsum[kLineMaxSeqs / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long x = tid < B ? count(tid) : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += wsum[w];
  if (tid < B) pre[tid + 1] = x;
  if (tid == 0) pre[0] = 0;
  __syncthreads();
}

// The last b with heads * pre[b] <= x (x below heads * pre[B]).
__device__ __forceinline__ int line_find(int B, const long long* pre, int heads, long long x) {
  int b = 0, hi = B - 1;
  while (b < hi) {
    const int mid = (b + hi + 1) >> 1;
    if (pre[mid] * heads <= x)
      b = mid;
    else
      hi = mid - 1;
  }
  return b;
}

}  // namespace basiskv
