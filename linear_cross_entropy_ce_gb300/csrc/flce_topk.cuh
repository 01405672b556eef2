// A warp's running list of the K <= 32 best (value, id) pairs, best first:
// larger values first, equal values by the lower id.  Lane j holds entry j;
// NaN is never taken.  The order of the offers does not change the first K.
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

  static __device__ __forceinline__ bool better(float av, int ai, float bv, int bi) {
    return av > bv || (av == bv && ai < bi);
  }

  // One compare-exchange with the lane at distance o.
  static __device__ __forceinline__ void exchange(float& v, int& id, int o, bool keep_better) {
    const float pv = __shfl_xor_sync(0xffffffffu, v, o);
    const int pi = __shfl_xor_sync(0xffffffffu, id, o);
    if (better(pv, pi, v, id) == keep_better) { v = pv; id = pi; }
  }

  // The 32 best of this list and another sorted one (lane j holds its entry
  // j): the better of entry i and the other's entry 31 - i are those 32, in a
  // bitonic order that five exchanges sort.
  __device__ __forceinline__ void merge(float ov, int oi, int lane) {
    ov = __shfl_xor_sync(0xffffffffu, ov, 31);
    oi = __shfl_xor_sync(0xffffffffu, oi, 31);
    if (better(ov, oi, v, id)) { v = ov; id = oi; }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) exchange(v, id, o, (lane & o) == 0);
  }

  // Every lane offers one candidate (id NONE: none).  Few pass the threshold
  // once the list has filled: those are inserted one by one; more than a
  // handful are sorted and merged.
  __device__ __forceinline__ void offer(float cv, int cid, int k, int lane) {
    const float tv = __shfl_sync(0xffffffffu, v, k - 1);
    const int ti = __shfl_sync(0xffffffffu, id, k - 1);
    const bool pass = cid != NONE && better(cv, cid, tv, ti);
    unsigned m = __ballot_sync(0xffffffffu, pass);
    if (m == 0) return;                    // uniform over the warp, as all below
    if (__popc(m) > 4) {
      if (!pass) { cv = -INFINITY; cid = NONE; }
#pragma unroll
      for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size / 2; o > 0; o >>= 1) exchange(cv, cid, o, ((lane & o) == 0) == ((lane & size) == 0));
      merge(cv, cid, lane);
      return;
    }
    while (m) {
      const int src = __ffs(m) - 1;
      m &= m - 1;
      const float nv = __shfl_sync(0xffffffffu, cv, src);
      const int ni = __shfl_sync(0xffffffffu, cid, src);
      const int pos = __popc(__ballot_sync(0xffffffffu, better(v, id, nv, ni)));   // entries before it
      const float uv = __shfl_up_sync(0xffffffffu, v, 1);
      const int ui = __shfl_up_sync(0xffffffffu, id, 1);
      if (lane > pos) { v = uv; id = ui; }
      if (lane == pos) { v = nv; id = ni; }
    }
  }

  // Every lane offers B candidates.  Its best one goes first: with the lanes'
  // best in the list, few of the others pass.
  template <int B>
  __device__ __forceinline__ void offer_all(const float (&cv)[B], const int (&cid)[B], int k, int lane) {
    float bv = -INFINITY;
    int bi = NONE;
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (cid[b] != NONE && better(cv[b], cid[b], bv, bi)) { bv = cv[b]; bi = cid[b]; }
    const float tv = __shfl_sync(0xffffffffu, v, k - 1);
    const int ti = __shfl_sync(0xffffffffu, id, k - 1);
    if (!__any_sync(0xffffffffu, better(bv, bi, tv, ti))) return;
    offer(bv, bi, k, lane);
#pragma unroll 1
    for (;;) {   // the lanes' next best ones
      float nv = -INFINITY;
      int ni = NONE;
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (cid[b] != NONE && better(bv, bi, cv[b], cid[b]) && better(cv[b], cid[b], nv, ni)) { nv = cv[b]; ni = cid[b]; }
      const float wv = __shfl_sync(0xffffffffu, v, k - 1);
      const int wi = __shfl_sync(0xffffffffu, id, k - 1);
      if (!__any_sync(0xffffffffu, ni != NONE && better(nv, ni, wv, wi))) return;
      offer(nv, ni, k, lane);
      bv = nv;
      bi = ni;
    }
  }

  // The lists of the block's WARPS (a power of two) warps become one, held by
  // every warp: in each of log2(WARPS) rounds a warp merges its partner's list.
  template <int WARPS>
  __device__ __forceinline__ void merge_block(float (*sv)[32], int (*si)[32], int lane, int w) {
#pragma unroll 1
    for (int o = 1; o < WARPS; o <<= 1) {
      __syncthreads();
      sv[w][lane] = v;
      si[w][lane] = id;
      __syncthreads();
      merge(sv[w ^ o][lane], si[w ^ o][lane], lane);
    }
  }
};

}  // namespace flce
