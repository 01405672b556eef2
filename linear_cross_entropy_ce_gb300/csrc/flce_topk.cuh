// A warp's running list of the K <= 32 best (value, id) pairs, best first:
// larger values first, equal values by the lower id.  Lane j holds entry j;
// NaN is never taken.  The order of the offers does not change the result.
#pragma once

#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

namespace flce {

struct TopK {
  static constexpr int MAX = 32;
  static constexpr int NONE = INT_MAX;   // id of an entry not filled yet

  float v;
  int id;

  __device__ __forceinline__ void clear() {
    v = -INFINITY;
    id = NONE;
  }

  // Every lane offers one candidate (where ok).  Few pass the threshold once
  // the list has filled, so the loop over those that do is short.
  __device__ __forceinline__ void offer(float cv, int cid, bool ok, int k, int lane) {
    const float tv = __shfl_sync(0xffffffffu, v, k - 1);
    const int ti = __shfl_sync(0xffffffffu, id, k - 1);
    unsigned m = __ballot_sync(0xffffffffu, ok && (cv > tv || (cv == tv && cid < ti)));
    while (m) {   // uniform over the warp
      const int src = __ffs(m) - 1;
      m &= m - 1;
      const float nv = __shfl_sync(0xffffffffu, cv, src);
      const int ni = __shfl_sync(0xffffffffu, cid, src);
      const int pos = __popc(__ballot_sync(0xffffffffu, v > nv || (v == nv && id < ni)));   // entries before it
      const float uv = __shfl_up_sync(0xffffffffu, v, 1);
      const int ui = __shfl_up_sync(0xffffffffu, id, 1);
      if (lane > pos) { v = uv; id = ui; }
      if (lane == pos) { v = nv; id = ni; }
    }
  }

  // The lists of the block's WARPS warps become one, held by every warp.
  template <int WARPS>
  __device__ __forceinline__ void merge_block(float (*sv)[32], int (*si)[32], int k, int lane, int w) {
    __syncthreads();
    sv[w][lane] = v;
    si[w][lane] = id;
    __syncthreads();
#pragma unroll 1
    for (int o = 1; o < WARPS; ++o) {
      const int from = (w + o) % WARPS;
      offer(sv[from][lane], si[from][lane], lane < k && si[from][lane] != NONE, k, lane);
    }
  }
};

}  // namespace flce
