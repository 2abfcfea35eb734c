// packed.cuh -- device helpers shared by the kernels for packed sequences
// (fwd_packed.cu, bwd_packed.cu).
#pragma once

#include <cstdint>

namespace fattn {

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// The last s in [0, S) with first(s) <= v for a non-decreasing first(), or -1;
// by the whole warp, 32 candidates a round.
template <typename F>
__device__ __forceinline__ int warp_search(int S, int v, F first) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = S;
  while (true) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const uint32_t m = __ballot_sync(~0u, lane * step < n && first(i) <= v);
    if (m == 0) return -1;
    const int hit = 31 - __clz(m);
    if (step == 1) return lo + hit;
    lo += hit * step;
    n = min(step, n - hit * step);
  }
}

}  // namespace fattn
