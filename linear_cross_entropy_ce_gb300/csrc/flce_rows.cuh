// What the row kernels of a chunk share: the merge of the 128-column parts'
// statistics, and the best logits of the parts that may hold one.
#pragma once

#include "flce_internal.h"
#include "flce_softmax.cuh"
#include "flce_topk.cuh"

namespace flce {

__device__ __forceinline__ int chunk_rows(const int* hdr, long long c0, int C) {
  const long long rem = static_cast<long long>(hdr[HDR_NVALID]) - c0;
  return rem <= 0 ? 0 : (rem >= C ? C : static_cast<int>(rem));
}

constexpr int ROWS_WARPS = 32;
constexpr int ROWS_BATCH = 4;

// Lane = row (part-major statistics: coalesced), the parts dealt to the block's
// ROWS_WARPS warps and merged in a fixed order; part[0] holds the rows' results.
__device__ __forceinline__ void merge_parts(const float* stats, int nparts, int C, float c2, int r, bool valid, int lane,
                                            int w, Stat (*part)[32]) {
  Stat acc = {-INFINITY, 0.f, 0.f};
  if (valid) {
    const size_t np = static_cast<size_t>(nparts) * C;
    for (int p0 = w; p0 < nparts; p0 += ROWS_BATCH * ROWS_WARPS) {
      Stat q[ROWS_BATCH];
#pragma unroll
      for (int k = 0; k < ROWS_BATCH; ++k) {
        const int p = p0 + k * ROWS_WARPS;
        const float* f = stats + static_cast<size_t>(p) * C + r;
        q[k] = p < nparts ? Stat{f[0], f[np], f[2 * np]} : Stat{-INFINITY, 0.f, 0.f};
      }
      static_assert(ROWS_BATCH == 4, "pairwise");
      acc = merge(acc, merge(merge(q[0], q[1], c2), merge(q[2], q[3], c2), c2), c2);
    }
  }
  part[w][lane] = acc;
#pragma unroll
  for (int o = ROWS_WARPS / 2; o > 0; o >>= 1) {   // fixed order
    __syncthreads();
    if (w < o) part[w][lane] = merge(part[w][lane], part[w + o][lane], c2);
  }
}

// The same for 8 rows by a block's first 8 warps, of which warp w gets row w: for
// row kernels with work of their own, whose other warps do that meanwhile.  A
// warp reads four parts at a time, 32 bytes of each.  The order is that of
// merge_parts.
constexpr int ROWS8 = 8;
// WEIGHTED false: the statistics have no third value.
constexpr uint32_t ROWS8_BAR = 1, ROWS8_BAR_OTHERS = 2;   // named barriers of the 8 warps, and of the others
template <bool WEIGHTED>
__device__ __forceinline__ Stat merge_parts8(const float* stats, int nparts, int C, float c2, int r0, int Cl, int lane,
                                             int w, Stat (*part)[ROWS8]) {
  const int r = r0 + lane % ROWS8;
  Stat acc = {-INFINITY, 0.f, 0.f};
  if (r < Cl) {
    const size_t np = static_cast<size_t>(nparts) * C;
    for (int p0 = w * 4 + lane / ROWS8; p0 < nparts; p0 += 2 * ROWS_BATCH * 32) {
      Stat q[2 * ROWS_BATCH];   // in flight
#pragma unroll
      for (int k = 0; k < 2 * ROWS_BATCH; ++k) {
        const int p = p0 + k * 32;
        const float* f = stats + static_cast<size_t>(p) * C + r;
        q[k] = p < nparts ? Stat{f[0], f[np], WEIGHTED ? f[2 * np] : 0.f} : Stat{-INFINITY, 0.f, 0.f};
      }
      acc = merge(acc, merge(merge(q[0], q[1], c2), merge(q[2], q[3], c2), c2), c2);
      if (p0 + ROWS_BATCH * 32 < nparts) acc = merge(acc, merge(merge(q[4], q[5], c2), merge(q[6], q[7], c2), c2), c2);
    }
  }
  part[w * 4 + lane / ROWS8][lane % ROWS8] = acc;
  ptx::named_bar_sync(ROWS8_BAR, 32 * ROWS8);
  acc = part[lane][w];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    acc = merge(acc, Stat{__shfl_down_sync(0xffffffffu, acc.m, o), __shfl_down_sync(0xffffffffu, acc.s, o),
                          __shfl_down_sync(0xffffffffu, acc.d, o)}, c2);
  return acc;   // in lane 0
}

constexpr int TOP_WARPS = 4;
constexpr int TOP_BATCH = 8;

// The K best logits of row r, held by every one of the block's TOP_WARPS warps:
// of the K best parts by (max, position), by (value, id).  zr: the row's logits.
__device__ __forceinline__ TopK top_of_parts(const float* stats, const float* zr, int nparts, int C, int V, int K, int r,
                                             int lane, int w, float (*sv)[32], int (*si)[32]) {
  TopK best;
  best.clear();
  for (int p0 = w * 32; p0 < nparts; p0 += TOP_BATCH * TOP_WARPS * 32) {
    float x[TOP_BATCH];
    int id[TOP_BATCH];
#pragma unroll
    for (int k = 0; k < TOP_BATCH; ++k) {
      const int p = p0 + k * (TOP_WARPS * 32) + lane;
      x[k] = p < nparts ? stats[static_cast<size_t>(p) * C + r] : 0.f;
      id[k] = p < nparts ? p : TopK::NONE;
    }
    best.offer_all(x, id, K, lane);
  }
  best.merge_block<TOP_WARPS>(sv, si, lane, w);   // every warp holds the K best parts
  const int parts = best.id;
  // K parts hold a logit of at least the K-th part's max: a smaller one is not
  // among the K best (nothing is left out where fewer parts are numbers)
  const float least = __shfl_sync(0xffffffffu, best.v, K - 1);
  best.clear();
  for (int j = w; j < K; j += 2 * TOP_WARPS) {
    float x[TOP_BATCH];
    int id[TOP_BATCH];
#pragma unroll
    for (int k = 0; k < TOP_BATCH; ++k) {
      const int jj = j + (k / 4) * TOP_WARPS;
      const int p = __shfl_sync(0xffffffffu, parts, jj & 31);
      const long long at = static_cast<long long>(p) * PART_COLS + (k % 4) * 32 + lane;
      const bool in = jj < K && p != TopK::NONE && at < V;
      x[k] = in ? zr[at] : 0.f;
      id[k] = in && x[k] >= least ? static_cast<int>(at) : TopK::NONE;
    }
    best.offer_all(x, id, K, lane);
  }
  best.merge_block<TOP_WARPS>(sv, si, lane, w);
  return best;
}

}  // namespace flce
