// The chunked form (more than STREAM_MAX_TOKENS tokens) of the operators whose
// rows have lists: workspace and launch sequence.  Per chunk of valid tokens:
// rows gathered, lists made, the logits GEMM with the listed tokens or their
// parts left out (MODE_STATS, GemmArgs::listed), and the operator's own row
// kernels, which bring them back in.
#pragma once

#include <algorithm>
#include <cstring>

#include "flce.h"
#include "flce_internal.h"
#include "flce_topk.cuh"

namespace flce {

// flce_api.cu: the gradients of the log probabilities' call with a
// distillation's row constants, and dz in two parts.  Its workspace by default:
// `reserve` less than that call's where this is not one chunk of all rows.
size_t distill_grad_bytes(int64_t N, int64_t H, int64_t V, uint32_t flags, size_t reserve);
flce_status run_distill_grad(const DistillGrad& d, const void* hidden, const void* weight, int64_t N, int64_t H,
                             int64_t V, uint32_t flags, float temperature, void* grad_hidden, float* grad_weight,
                             void* workspace, size_t workspace_bytes, void* stream);

struct ListedSizes {
  long long N, H, V;
  int K;                 // top alternatives
  long long cap;         // entries of a row at most
  long long row_bytes;   // what the operator keeps per chunk row beside them
  int table;             // bytes of a row's place in the table by parts: 4 (where a part's entries begin), 2 (its slab)
  long long z;           // logits kept of a row
};

struct ListedPlan {
  long long C = 0, n_chunks = 0, ldz = 0;
  int nvt = 0, nparts = 0, group_stride = 0;
  size_t o_idx = 0, o_targets = 0, o_xc = 0, o_tc = 0, o_zt = 0, o_ml = 0, o_stats = 0, o_bound = 0,
         o_group = 0, o_zf = 0, o_start = 0, o_id = 0, o_z = 0, o_rows = 0, total = 0;
};

inline ListedPlan listed_layout(const ListedSizes& q, long long C) {
  ListedPlan p;
  p.C = C;
  p.n_chunks = cdiv(q.N, C);
  p.ldz = cdiv(q.V, 64) * 64;
  p.nvt = static_cast<int>(cdiv(q.V, BN));
  p.nparts = static_cast<int>(cdiv(q.V, PART_COLS));
  p.group_stride = (q.K + 3) / 4 * 4;
  size_t off = al256(HDR_WORDS * sizeof(int));
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += al256(bytes);
    return o;
  };
  p.o_idx = take(size_t(q.N) * 4);
  p.o_targets = take(size_t(q.N) * 4);
  p.o_xc = take(size_t(C) * q.H * 2);
  p.o_tc = take(size_t(C) * 4);
  // slabs leave max and sum of a part only, and pick no target
  const bool slabs = q.table == 2;
  p.o_zt = take(slabs ? 0 : size_t(C) * 4);
  p.o_ml = take(q.K > 0 ? size_t(C) * 8 : 0);
  p.o_stats = take(size_t(C) * p.nparts * (slabs ? 8 : 12));
  if (q.K > 0) {
    p.o_bound = take(size_t(C) * 4);
    p.o_group = take(size_t(C) * p.group_stride * 4);
    p.o_zf = take(size_t(C) * p.ldz * 4);
  }
  p.o_start = take(size_t(C) * (p.nparts + 1) * q.table);
  p.o_id = take(size_t(C) * q.cap * 4);
  p.o_z = take(size_t(C) * q.z * 4);
  p.o_rows = take(size_t(C) * q.row_bytes);
  p.total = off;
  return p;
}

// Largest chunk (a multiple of 128 rows) whose plan fits in `bytes`.
inline bool listed_plan(const ListedSizes& q, size_t bytes, ListedPlan* out) {
  long long lo = 1, hi = cdiv(q.N, BM);
  if (listed_layout(q, BM).total > bytes) return false;
  while (lo < hi) {
    const long long mid = (lo + hi + 1) / 2;
    if (listed_layout(q, mid * BM).total <= bytes) lo = mid;
    else hi = mid - 1;
  }
  *out = listed_layout(q, lo * BM);
  return true;
}

// As for the log probabilities without lists: 5% of the bf16 logits, or what a
// smaller problem needs for one chunk.
inline size_t listed_default_bytes(const ListedSizes& q) {
  const size_t budget = std::max(size_t(q.N) * size_t(q.V) * 2 / 20, size_t(q.K > 0 ? 2048 : 512) << 20);
  ListedPlan p;
  if (listed_plan(q, budget, &p)) return p.total;
  return listed_layout(q, BM).total;
}

struct ListedCall {
  ListedSizes q;
  const void *hidden, *weight;
  const int* targets;       // which rows count, and what is picked; null with listed_front(): all rows
  int ii;
  float temperature;
  int seg_kb;               // segment_blocks()
  bool by_token;            // the slabs' table has a column per token, not per row of the chunk
  const uint32_t* mask;     // or null
  long long mask_stride;
  float *logp, *entropy, *lse;   // what left-out rows get 0 (or NaN) in, in a call of one chunk
  int* top_ids;
  float* top_logp;
  void* ws;
  cudaStream_t st;
};

struct ListedChunk {
  long long c0;
  const GemmArgs* g;
};

// One kernel compacts the tokens and gathers their rows.
inline bool listed_front(const ListedPlan& p, long long N) { return p.n_chunks == 1 && N <= FRONT_MAX_TOKENS; }

// lists(chunk): launches what fills the lists of the chunk's rows; it waits for
// its predecessor.  rows(chunk): launches the row kernels.
template <class Lists, class Rows>
flce_status listed_chunks(const ListedPlan& p, const ListedCall& c, const DeviceState& dev, Lists&& lists, Rows&& rows) {
  void* ws = c.ws;
  const ListedSizes& q = c.q;
  GemmMaps m;
  std::memset(&m, 0, sizeof(m));
  const unsigned long long hb = static_cast<unsigned long long>(q.H) * 2;
  uint16_t* xc = at<uint16_t>(ws, p.o_xc);
  if (!make_map(&m.a0, xc, q.H, p.C, hb, BK, BM) || !make_map(&m.b0, c.weight, q.H, q.V, hb, BK, BN / 2))
    return FLCE_ECUDA;
  GemmArgs g;
  std::memset(&g, 0, sizeof(g));
  g.mode = MODE_STATS;
  g.hdr = at<int>(ws, 0);
  g.status = at<int>(ws, 0) + HDR_STATUS;
  g.C = static_cast<int>(p.C);
  g.H = static_cast<int>(q.H);
  g.V = static_cast<int>(q.V);
  g.ldz = p.ldz;
  g.nvt = p.nvt;
  g.nparts = p.nparts;
  g.timeout_ns = wait_timeout_ns();
  g.tc = at<int>(ws, p.o_tc);
  g.zt = q.table == 4 ? at<float>(ws, p.o_zt) : nullptr;
  g.idx = at<int>(ws, p.o_idx);
  g.stats = at<float>(ws, p.o_stats);
  g.K = q.K;
  g.zf = q.K > 0 ? at<float>(ws, p.o_zf) : nullptr;
  if (q.K > 0 && p.nparts >= 16 * q.K) {   // as for the log probabilities without lists
    g.bound = at<uint32_t>(ws, p.o_bound);
    g.group_max = at<uint32_t>(ws, p.o_group);
  }
  g.group_stride = p.group_stride;
  g.seg_kb = c.seg_kb;
  g.c2 = 1.4426950408889634f / c.temperature;
  g.listed = q.table == 4 ? LISTED_OUT : LISTED_SLABS;
  g.slab = at<short>(ws, p.o_start);
  g.slab_by_token = c.by_token;
  g.slabs_per_row = static_cast<int>(q.z / PART_COLS);
  g.lists.start = at<int>(ws, p.o_start);
  g.lists.id = at<int>(ws, p.o_id);
  g.lists.z = at<float>(ws, p.o_z);
  g.lists.cap = q.cap;
  g.lists.mask = c.mask;
  g.lists.mask_stride = c.mask_stride;

  const int grid = 2 * static_cast<int>(std::min<long long>(cdiv(p.C, PAIR_M) * p.nvt, dev.pairs));
  const bool front = listed_front(p, q.N);
  int* hdr = at<int>(ws, 0);
  int* idx = at<int>(ws, p.o_idx);
  if (front) {
    FrontArgs f;
    std::memset(&f, 0, sizeof(f));
    f.hidden = static_cast<const uint16_t*>(c.hidden);
    f.targets = c.targets;
    f.N = static_cast<int>(q.N); f.H = g.H; f.V = g.V; f.ii = c.ii; f.C = g.C; f.K = q.K;
    f.hdr = hdr; f.idx = idx; f.tc = at<int>(ws, p.o_tc); f.xc = xc;
    f.bound = g.bound; f.group_max = g.group_max; f.group_stride = g.group_stride;
    f.logp = c.logp; f.lse = c.lse; f.entropy = c.entropy; f.top_ids = c.top_ids; f.top_logp = c.top_logp;
    count_launches(1);
    if (launch_probs_front(f, c.st) != cudaSuccess) return FLCE_ECUDA;
  } else {
    count_launches(1 + p.n_chunks);
    if (launch_prep(c.targets, q.N, g.V, c.ii, hdr, idx, nullptr, nullptr, 0, c.st) != cudaSuccess) return FLCE_ECUDA;
  }
  for (long long i = 0; i < p.n_chunks; ++i) {
    const ListedChunk ch{i * p.C, &g};
    g.c0 = ch.c0;
    if (!front && launch_gather(static_cast<const uint16_t*>(c.hidden), c.targets, hdr, idx, g.c0, g.C, g.H, xc,
                                at<int>(ws, p.o_tc), 0, g.V, c.st) != cudaSuccess)
      return FLCE_ECUDA;
    if (!front && g.bound) {
      count_launches(1);
      if (launch_clear_bounds(g.bound, g.group_max, g.group_stride, q.K, g.C, c.st) != cudaSuccess) return FLCE_ECUDA;
    }
    if (lists(ch) != cudaSuccess) return FLCE_ECUDA;
    if (gemm_launch(g, m, grid, c.st, true) != cudaSuccess) return FLCE_ECUDA;
    if (rows(ch) != cudaSuccess) return FLCE_ECUDA;
  }
  return FLCE_OK;
}

}  // namespace flce
