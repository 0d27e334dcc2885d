// Row segments of the products grouped by expert, read from device memory.
#pragma once

#include "ql_common.cuh"

namespace ql {

// Segment e of a warp's 32 experts (e = first + lane): its offsets clipped to
// [0, T], and never below an earlier one, so that segments ascend and do not
// overlap whatever the array holds.  `carry` is the end of the segments
// before this warp's and becomes the end of this warp's.  Experts past E are
// empty segments at the end of the last one.
__device__ __forceinline__ void warp_segments(const int32_t* offsets, int E, int64_t T, int e, int64_t& carry,
                                              int64_t& lo, int64_t& hi) {
  auto clip = [&](int32_t v) { return min(max(static_cast<int64_t>(v), int64_t(0)), T); };
  lo = max(carry, clip(offsets[min(e, E)]));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, lo, o);
    if (static_cast<int>(lane_id()) >= o) lo = max(lo, v);
  }
  hi = max(lo, clip(offsets[min(e + 1, E)]));
  carry = __shfl_sync(0xffffffffu, hi, 31);
}

__device__ __forceinline__ int warp_inclusive_sum(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (static_cast<int>(lane_id()) >= o) v += u;
  }
  return v;
}

}  // namespace ql
