// fp4q_kv.hpp -- device pieces shared by the kernels that write and read the paged MXFP8 cache
// (fp4q_rotary.hip, fp4q_attn.hip).
//
// Lengths, starts and page ids are device data that the host never sees, so every kernel clamps or
// skips what lies outside the arrays instead of trusting it.
#pragma once
#include "fp4q_internal.hpp"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4q {
namespace {

// The last i in 0 .. n-1 for which holds(i), or -1: 64 places at a time by the whole wave (holds the same
// in all of its lanes), so one trip to memory for up to 64 sequences and two for 4096, where halving takes
// six and twelve.  It holds up to some place and not behind it; where that is not so, some place in range comes back.
template <typename F>
__device__ __forceinline__ int wave_last(int n, F holds) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  for (;;) {
    const int step = (n + 63) >> 6, at = lane * step;
    const bool below = at < n && holds(lo + min(at, n - 1));
    const int count = __popcll(__ballot(below));
    if (count == 0) return lo - 1;
    const int skip = min((count - 1) * step, n - 1);
    lo += skip;
    n = min(step, n - skip);
    if (step == 1) return lo;
  }
}

// The last i in 0 .. n-1 with starts[i] <= t, which do not fall, or -1, by one lane for its own t.
__device__ __forceinline__ int lane_find(const int32_t* __restrict__ starts, int n, int t) {
  int lo = -1, hi = n;   // starts[lo] <= t < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The sequence of token t (the same in the whole wave), or -1: t is behind the last or before the first.
__device__ __forceinline__ int wave_sequence(const int32_t* __restrict__ q_starts, int seqs, int t) {
  const int s = wave_last(seqs + 1, [&](int i) { return q_starts[i] <= t; });
  return s < seqs ? s : -1;
}

}  // namespace
}  // namespace fp4q
