// Distillation at the LM head from a teacher's top log probabilities, forward
// and backward.
//
// With q = softmax(X W^T / T) of the student, a row's teacher tokens I (each
// token once; tokens named twice add up) and their masses p:
//   with a tail      p_i = exp(t_i),  r = max(0, 1 - sum p),  s = sum_{v not in I} q_v
//     kl = sum_I p_i (log p_i - log q_i) + r (log r - log s)
//     dkl/dz_v = (A q_v - p_v - [v not in I] r q_v / s) / T,   A = sum p + r
//   without          p = softmax of t over I
//     kl = sum_I p_i (log p_i - log q_i),   dkl/dz_v = (q_v - p_v) / T
//
// The mass s behind the list is what is left of 1 and may be tiny, so it is not
// formed as a difference: the GEMM's epilogue leaves the 128-column parts that
// hold listed tokens out of the row's statistics and writes their logits side by
// side (K parts at most), and the row kernel goes through those.  (Taking the
// listed logits out one by one cost the epilogue more than the products: 4096
// tokens, 20 entries, at 512 x 16000 112 us a GEMM, so 57.)  All of a row's log
// probabilities are formed relative to its largest logit (an fp32 log-sum-exp of
// 20 is off by 1e-6, as much as kl is where student and teacher nearly agree),
// and r as (1 - p_max) - the others.
//
// Backward: behind the list dz_v = g (A s - r) / T * exp(z_v - lse_rest), one
// exponential per logit with constants of its row that neither overflow nor
// lose anything where s is small: the epilogue of the log probabilities'
// gradient (MODE_DZ) with another log-sum-exp and another upstream gradient.
// Between it and the two products a small kernel overwrites the listed places.
#include "flce_listed.cuh"
#include "flce_pair.cuh"
#include "flce_ptx.cuh"
#include "flce_rows.cuh"
#include "flce_softmax.cuh"
#include "flce_stream_range.cuh"

namespace flce {
namespace {

constexpr int MAX_TEACHER = 256;   // teacher tokens of a row at most
constexpr int NO_TOKEN = INT_MAX;

struct DistillOut {
  float *kl, *lse, *rest_logp, *student_logp;   // [N] x3, [N][K]
};

__device__ __forceinline__ void fill_row(const DistillOut& o, long long row, int K, float v, int lane) {
  if (lane == 0) {
    o.kl[row] = v;
    o.lse[row] = v;
    o.rest_logp[row] = v;
  }
  for (int j = lane; j < K; j += 32) o.student_logp[row * K + j] = v;
}

// A teacher row before anything else: the first token that it names, -1 where
// it names none, or one outside [0, V).  That is the row's target for the
// kernels that compact the rows.
__device__ __forceinline__ int row_target(const int* ids, int K, int V, int lane) {
  int t = -1;
  for (int j0 = 0; j0 < K; j0 += 32) {
    const int x = j0 + lane < K ? ids[j0 + lane] : -1;
    const unsigned bad = __ballot_sync(0xffffffffu, x >= V), some = __ballot_sync(0xffffffffu, x >= 0);
    if (bad) return __shfl_sync(0xffffffffu, x, __ffs(bad) - 1);
    if (t < 0 && some) t = __shfl_sync(0xffffffffu, x, __ffs(some) - 1);
  }
  return t;
}

// ---------------------------------------------------------------------------
// lists
// ---------------------------------------------------------------------------

// Shared scratch of one row's sort, by a warp.
struct SortRow {
  int* raw;      // [K rounded up to 32] as given (NO_TOKEN where there is none)
  int* id;       // [K] sorted, then each token once
  float* t;      // [K] their log masses
  short* at;     // [K] place of sorted entry i in the list of single tokens
};
__host__ __device__ __forceinline__ int sort_words(int K) { return ((K + 31) / 32 * 32 + 2 * K + (K + 1) / 2 + 3) / 4 * 4; }
__host__ __device__ __forceinline__ int list_words(int K) { return (sort_words(K) + (K + 1) / 2 + 3) / 4 * 4; }
__device__ __forceinline__ SortRow sort_scratch(int* p, int K) {
  const int padded = (K + 31) / 32 * 32;
  return SortRow{p, p + padded, reinterpret_cast<float*>(p + padded + K), reinterpret_cast<short*>(p + padded + 2 * K)};
}

// A row's teacher tokens in ascending order, each once, with their log masses,
// by a warp: s.id[0 .. n), s.t[0 .. n); slot[k]: the place of entry
// lane + 32 k, -1 where there is none.  Returns n.  An entry's rank is the
// number of smaller tokens and of equal ones before it: two instructions a
// pair, K^2 / 16 a lane (64 entries 256), which no order of the entries makes
// slower: lists and tables of 5735 rows of 32 over 2001 parts take 23 us, of 724
// of 100 17.
// Without a tail the log masses are made relative to the row's largest (exact, or
// rounded to 2^-24 of the difference), so that logits which all are large, or log
// probabilities of unlikely tokens alone, do not cost the masses' digits: sums of
// theirs, rounded, would be off by 2^-24 of what they share.
// SORT_GROUPS: 32s of entries, 1, 2, 4 or 8.
template <int SORT_GROUPS>
__device__ __forceinline__ int sort_row(const int* ids, const float* t, int K, bool tail, int lane, const SortRow& s,
                                        int (&slot)[SORT_GROUPS]) {
  const int groups = (K + 31) / 32;
  unsigned x[SORT_GROUPS];
  int rank[SORT_GROUPS];
#pragma unroll
  for (int e = 0; e < SORT_GROUPS; ++e) {
    const int j = e * 32 + lane;
    const int v = j < K ? ids[j] : -1;
    x[e] = v < 0 ? NO_TOKEN : v;
    rank[e] = 0;
    if (e < groups) s.raw[j] = static_cast<int>(x[e]);
  }
  __syncwarp();
  for (int g = 0; g < groups; ++g) {
    const uint4* from = reinterpret_cast<const uint4*>(s.raw + g * 32);
#pragma unroll
    for (int e = 0; e < SORT_GROUPS; ++e) {
      if (e >= groups) break;
      // equal tokens of groups before this one stand before it, of groups behind it do not
      const unsigned limit = x[e] + (g < e ? 1u : 0u);
      int r = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 b = from[i];
        if (g == e) {
          r += b.x < limit + (i * 4 < lane) ? 1 : 0;
          r += b.y < limit + (i * 4 + 1 < lane) ? 1 : 0;
          r += b.z < limit + (i * 4 + 2 < lane) ? 1 : 0;
          r += b.w < limit + (i * 4 + 3 < lane) ? 1 : 0;
        } else {
          r += b.x < limit ? 1 : 0;
          r += b.y < limit ? 1 : 0;
          r += b.z < limit ? 1 : 0;
          r += b.w < limit ? 1 : 0;
        }
      }
      rank[e] += r;
    }
  }
  float base = 0.f;
  if (!tail) {
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < SORT_GROUPS; ++e)
      if (e < groups && x[e] != NO_TOKEN) top = fmaxf(top, t[e * 32 + lane]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top > -INFINITY) base = top;
  }
  int n = 0;
#pragma unroll
  for (int e = 0; e < SORT_GROUPS; ++e) {
    const bool there = e < groups && x[e] != NO_TOKEN;
    if (there) {
      s.id[rank[e]] = static_cast<int>(x[e]);
      s.t[rank[e]] = t[e * 32 + lane] - base;
    }
    n += __popc(__ballot_sync(0xffffffffu, there));
  }
  __syncwarp();
  // each token once: its place is the number of different tokens before it
  int singles = 0;
  int id[SORT_GROUPS];
  float m[SORT_GROUPS];
  int place[SORT_GROUPS];
#pragma unroll
  for (int e = 0; e < SORT_GROUPS; ++e) {
    const int i = e * 32 + lane;
    place[e] = -1;
    if (e >= groups) continue;
    const bool there = i < n;
    id[e] = there ? s.id[i] : NO_TOKEN;
    m[e] = there ? s.t[i] : 0.f;
    const bool first = there && (i == 0 || s.id[i - 1] != id[e]);
    const unsigned f = __ballot_sync(0xffffffffu, first);
    const int u = singles + __popc(f & (0xffffffffu >> (31 - lane))) - 1;
    singles += __popc(f);
    if (there) s.at[i] = static_cast<short>(u);
    if (first) {
      place[e] = u;
      if (i + 1 < n && s.id[i + 1] == id[e]) {   // the token's masses add up
        float top = m[e];
        for (int k = i + 1; k < n && s.id[k] == id[e]; ++k) top = fmaxf(top, s.t[k]);
        if (top > -INFINITY) {
          float sum = 0.f;
          for (int k = i; k < n && s.id[k] == id[e]; ++k) sum += expf(s.t[k] - top);
          m[e] = top + logf(sum);
        }
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < SORT_GROUPS; ++e) {
    if (place[e] >= 0) {
      s.id[place[e]] = id[e];
      s.t[place[e]] = m[e];
    }
    slot[e] = e < groups && x[e] != NO_TOKEN ? s.at[rank[e]] : -1;
  }
  __syncwarp();
  return singles;
}

__device__ __forceinline__ int lower_bound(const int* id, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (id[mid] < x) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

struct ListArgs {
  const int* teacher_ids;     // [N][K]
  const float* teacher_logp;
  int K, V, tail;
  const int* hdr;             // chunked form
  const int* idx;             // null: lists of all N tokens, by token
  long long c0;
  int C, nparts, N;
  short* slab;                // [nparts][C] which of the row's slabs takes the part's logits, -1: none
  int* count;                 // [C] tokens of the row
  int ctas, max_tiles;        // streaming form
  int* start;
  int* id;                    // [rows][K]
  float* t;                   // [rows][K] log masses of the sorted tokens (without a tail, relative to the largest)
  short* slot;                // [rows][K] place of each given entry
};

template <int SORT_GROUPS>
__device__ __forceinline__ void store_row(const ListArgs& a, long long row, const SortRow& s, int n,
                                          const int (&slot)[SORT_GROUPS], int lane) {
  const long long to = row * a.K;
  for (int u = lane; u < n; u += 32) {
    a.id[to + u] = s.id[u];
    a.t[to + u] = s.t[u];
  }
#pragma unroll
  for (int e = 0; e < SORT_GROUPS; ++e)
    if (e * 32 + lane < a.K) a.slot[to + e * 32 + lane] = static_cast<short>(slot[e]);
}

// Chunked: 8 rows a block, each sorted by a warp; then a lane walks a run of
// one row's parts, four runs a warp.  By token (calls of one chunk), the kernel
// also does what distill_targets_kernel does, a launch less.
constexpr int LIST_WARPS = ROWS8;
template <int SORT_GROUPS>
__global__ void __launch_bounds__(32 * LIST_WARPS)
    distill_lists_kernel(const ListArgs a, int* targets, const DistillOut out) {
  extern __shared__ int smem[];   // per row: scratch of its sort, the slabs of its tokens
  __shared__ int count[ROWS8];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int words = list_words(a.K), slabs_at = sort_words(a.K);
  ptx::grid_dependency_wait();
  const int Cl = a.idx ? chunk_rows(a.hdr, a.c0, a.C) : a.N;
  const int r0 = blockIdx.x * ROWS8;
  if (r0 >= Cl) return;
  bool sort = r0 + w < Cl;
  if (!a.idx && sort) {
    const long long row = r0 + w;
    const int t = row_target(a.teacher_ids + row * a.K, a.K, a.V, lane);
    if (lane == 0) {
      targets[row] = t;
      count[w] = a.count[row] = 0;
    }
    sort = t >= 0 && t < a.V;
    if (!sort) fill_row(out, row, a.K, t < 0 ? 0.f : __int_as_float(0x7fc00000), lane);
  }
  if (sort) {
    const long long row = r0 + w, from = (a.idx ? a.idx[a.c0 + row] : row) * a.K;
    const SortRow s = sort_scratch(smem + w * words, a.K);
    int slot[SORT_GROUPS];
    const int n = sort_row(a.teacher_ids + from, a.teacher_logp + from, a.K, a.tail, lane, s, slot);
    store_row(a, row, s, n, slot, lane);
    short* slab = reinterpret_cast<short*>(smem + w * words + slabs_at);
    int q = -1;   // the last slab so far
    for (int u0 = 0; u0 < n; u0 += 32) {
      const int u = u0 + lane;
      const bool first = u < n && (u == 0 || s.id[u - 1] / PART_COLS != s.id[u] / PART_COLS);
      const unsigned f = __ballot_sync(0xffffffffu, first);
      if (u < n) slab[u] = static_cast<short>(q + __popc(f & (0xffffffffu >> (31 - lane))));
      q += __popc(f);
    }
    if (lane == 0) {
      count[w] = n;
      a.count[row] = n;
    }
  }
  __syncthreads();
  const int k = lane % ROWS8, r = r0 + k;
  if (r >= Cl) return;
  const int n = count[k];
  const int* id = sort_scratch(smem + k * words, a.K).id;
  const short* slab = reinterpret_cast<const short*>(smem + k * words + slabs_at);
  const int each = (a.nparts + 31) / 32;
  int p = (w * 4 + lane / ROWS8) * each;
  const int p1 = min(a.nparts, p + each);
  int e = p < p1 ? lower_bound(id, n, p * PART_COLS) : n;   // the next token
  int at = e < n ? id[e] / PART_COLS : a.nparts;            // its part
  for (; p < p1; ++p) {
    int q = -1;
    if (at == p) {
      q = slab[e];
      do ++e;
      while (e < n && id[e] / PART_COLS == p);
      at = e < n ? id[e] / PART_COLS : a.nparts;
    }
    a.slab[static_cast<long long>(p) * a.C + r] = static_cast<short>(q);
  }
}

// Streaming: a block per row; the weight streams meanwhile, on the same SMs
// (few threads, and less shared memory than the streaming kernel leaves).
constexpr int STREAM_LIST_THREADS = 128;
template <int SORT_GROUPS>
__global__ void __launch_bounds__(STREAM_LIST_THREADS) distill_stream_lists_kernel(const ListArgs a) {
  __shared__ __align__(16) int scratch[MAX_TEACHER + 2 * MAX_TEACHER + MAX_TEACHER / 2];
  __shared__ int count;
  ptx::grid_launch_dependents();
  const long long from = static_cast<long long>(blockIdx.x) * a.K;
  const SortRow s = sort_scratch(scratch, a.K);
  if (threadIdx.x < 32) {
    int slot[SORT_GROUPS];
    const int n = sort_row(a.teacher_ids + from, a.teacher_logp + from, a.K, a.tail, threadIdx.x, s, slot);
    store_row(a, blockIdx.x, s, n, slot, threadIdx.x);
    if (threadIdx.x == 0) count = n;
  }
  __syncthreads();
  const int tiles = a.ctas * a.max_tiles;
  int* start = a.start + static_cast<long long>(blockIdx.x) * (tiles + 1);
  for (int b = threadIdx.x; b <= tiles; b += STREAM_LIST_THREADS) {
    int x = a.V;
    if (b < tiles) {
      const Range r = range_of(a.V, a.ctas, b / a.max_tiles);
      x = b % a.max_tiles < r.tiles ? r.start(b % a.max_tiles) : r.u1 * UNIT_ROWS;
    }
    start[b] = lower_bound(s.id, count, min(x, a.V));
  }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------

// The masses of a row's teacher: given its largest log mass, p(t) of an entry.
struct Teacher {
  float top;     // largest log mass
  float shift;   // p = exp(t - shift)
  float rest;    // mass behind the list
};

// By a warp: t[0 .. n) the row's log masses, each token's once.
__device__ __forceinline__ Teacher teacher_of(const float* t, int n, bool tail, int lane) {
  float top = -INFINITY;
  bool nan = false;
  for (int u = lane; u < n; u += 32) {
    top = fmaxf(top, t[u]);
    nan = nan || t[u] != t[u];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (__any_sync(0xffffffffu, nan)) top = __int_as_float(0x7fc00000);
  Teacher q = {top, 0.f, 0.f};
  const float base = tail ? 0.f : top;
  float sum = 0.f;   // of all but one of the largest
  int tops = 0;
  for (int u = lane; u < n; u += 32) {
    if (t[u] == top) ++tops;
    else sum += expf(t[u] - base);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    tops += __shfl_xor_sync(0xffffffffu, tops, o);
  }
  if (tail) {
    // (1 - p_max) - the others: nothing is lost where p_max is nearly 1
    q.rest = fmaxf(0.f, -expm1f(top) - (sum + static_cast<float>(tops - 1) * expf(top)));
  } else if (top > -INFINITY) {
    q.shift = top + log1pf(sum + static_cast<float>(tops - 1));
  }
  if (top != top) q.shift = q.rest = top;
  return q;
}

// One row by a warp, from the statistics of the logits behind its list and the
// listed logits z[0 .. n), which may be shared memory.
//
// With x = (z - m) / T, m the largest logit, e the sum of exp(x) and b its part
// behind the list, and w = exp(t - base) with sum P (base 0 with a tail, else the
// largest log mass), r = 1 - P:
//   with a tail   kl = sum w (t - x) + P ln e + r (ln r + ln e - ln b)
//   without       kl = sum w (t - base - x) / P + ln e - ln P
// kl is what is left of terms that nearly cancel where student and teacher nearly
// agree, so whatever enters it to the first order there, w, r, e and the logarithms,
// is held to about 2^-28 (Pair).  Not so the logits: an error of theirs counts with
// the difference of the two distributions only.  (In fp32, with what the terms share
// kept apart, kl was off by 5.5e-8 however small it was: 5e-6 of divergences of 1e-2.
// In 64 bits, three logarithms a row, the row kernel took 120 us for 5735 rows, with
// fp32 97 then.)
__device__ __forceinline__ void finish_row(const DistillOut& o, long long row, int K, bool tail, float inv_t, Stat rest,
                                           const float* z, const float* t, const short* slot, int n,
                                           int lane) {
  float m = rest.m, top = -INFINITY;
  bool nan = false, t_nan = false;
  for (int u = lane; u < n; u += 32) {
    m = fmaxf(m, z[u]);
    top = fmaxf(top, t[u]);
    nan = nan || z[u] != z[u];
    t_nan = t_nan || t[u] != t[u];
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
  }
  if (__any_sync(0xffffffffu, nan)) m = __int_as_float(0x7fc00000);
  if (__any_sync(0xffffffffu, t_nan)) top = __int_as_float(0x7fc00000);
  const bool none = rest.m == -INFINITY && rest.s == 0.f;   // nothing behind the list
  const float base = tail || top == -INFINITY ? 0.f : top;
  PairSum e, others, terms;   // sum exp(x); sum w but for one of the largest; sum w (t - base - x)
  bool never = false;         // the student gives a token of some mass no chance
  int tops = 0;
  for (int u = lane; u < n; u += 32) {
    const float x = (z[u] - m) * inv_t, lp = t[u] - base;
    const Pair ex = exp_pair(x), w = exp_pair(lp);
    e.add(ex.hi, ex.lo);
    if (t[u] == top) ++tops;
    else others.add(w.hi, w.lo);
    if (w.hi == 0.f) continue;
    if (x == -INFINITY) { never = true; continue; }
    const float d = lp - x, b = d - lp, d_lo = (lp - (d - b)) - (x + b);   // two-sum of lp and -x
    const float q = w.hi * d;
    terms.add(q, fmaf(w.hi, d, -q) + fmaf(w.hi, d_lo, w.lo * d));
  }
  e.add_lanes();
  others.add_lanes();
  terms.add_lanes();
  tops = __reduce_add_sync(0xffffffffu, tops);
  const Pair w_top = exp_pair(top - base);
  const Pair but_one = others.value() + Pair{static_cast<float>(tops - 1), 0.f} * w_top, mass = w_top + but_one;
  Pair r = {0.f, 0.f};
  if (tail && !none) {   // (1 - the largest) - the others: nothing is lost where the largest is nearly 1
    r = (top > -0.0625f ? Pair{-expm1f(top), 0.f} : Pair{1.f, 0.f} - w_top) - but_one;
    if (r.hi <= 0.f) r = Pair{0.f, 0.f};
  }
  const float far = none ? -INFINITY : (rest.m - m) * inv_t;
  Pair all = e.value();
  if (!none) all = all + Pair{rest.s, 0.f} * exp_pair(far);
  // three logarithms, a lane each; what is not used may be no number
  const Pair mine = log_of(lane == 0 ? all : (lane == 1 ? (tail ? r : mass) : Pair{rest.s, 0.f}));
  auto of_lane = [&](int i) {
    return Pair{__shfl_sync(0xffffffffu, mine.hi, i), __shfl_sync(0xffffffffu, mine.lo, i)};
  };
  const Pair le = of_lane(0), lm = of_lane(1), lb = of_lane(2);
  for (int j = lane; j < K; j += 32) {
    const int u = slot[j];
    o.student_logp[row * K + j] = u < 0 || u >= n ? 0.f : fmaf(z[u] - m, inv_t, -le.hi) - le.lo;
  }
  never = __any_sync(0xffffffffu, never);
  if (lane == 0) {
    Pair kl = terms.value();
    const Pair behind = Pair{far, 0.f} - (le - lb);   // log s
    if (tail) {
      kl = kl + mass * le;
      // a teacher without any mass asks for nothing
      if (!(r.hi == 0.f)) kl = kl + r * (lm - behind);
    } else if (mass.hi > 0.f) {
      kl = kl / mass + (le - lm);
    }
    float k = kl.hi + kl.lo;
    if (never) k += INFINITY;
    if (top != top) k = top;
    o.kl[row] = k;
    o.lse[row] = fmaf(m, inv_t, le.hi);
    o.rest_logp[row] = none ? -INFINITY : behind.hi;
  }
}

constexpr int TARGET_WARPS = 8;
// The rows' targets, and the outputs of the rows without a teacher.
__global__ void __launch_bounds__(32 * TARGET_WARPS)
    distill_targets_kernel(const int* ids, long long N, int K, int V, int* targets, const DistillOut o) {
  const int lane = threadIdx.x % 32;
  const long long row = static_cast<long long>(blockIdx.x) * TARGET_WARPS + threadIdx.x / 32;
  if (row >= N) return;
  const int t = row_target(ids + row * K, K, V, lane);
  if (lane == 0) targets[row] = t;
  if (t < 0 || t >= V) fill_row(o, row, K, t < 0 ? 0.f : __int_as_float(0x7fc00000), lane);
}

struct RowsArgs {
  const int* hdr;
  const int* idx;
  long long c0;
  int C, nparts, V, K, tail, slabs;
  const float* stats;
  int by_token;               // lists, not slabs
  const int* count;
  const int* id;
  float* z;                   // [C][slabs][128] logits of the parts that hold listed tokens
  const float* t;
  const short* slot;
  float c2, inv_t;
  DistillOut out;
};

// 8 rows of a chunk.  Eight warps merge the statistics of the parts without listed
// tokens; SHARES warps a row go through the other parts' logits meanwhile: the
// listed ones aside, the others into statistics of their own.  Then a warp a row
// puts it all together.  All of it is loads (5735 rows of 32 entries over 2001
// parts: 230 MB, 57 us).  Three warps a row where the blocks are one wave and there
// is something to share, else one, and two blocks an SM: calls at H = 64 with one
// and three, 1152 rows at a vocabulary of 60000 with lists of 8, 32, 64, 200: 51, 57,
// 69, 127 and 51, 56, 64, 106 us; 1280 rows 52, 60, 71, 136 and 56, 63, 75, 142; 300
// rows at 16000 28, 34, 40, 69 and 28, 32, 36, 60; 2048 rows 38, 44, 54, 110 and 43,
// 48, 58, 118.
template <int SHARES>
__global__ void __launch_bounds__(32 * ROWS8 * (1 + SHARES)) distill_rows_kernel(const RowsArgs a) {
  __shared__ Stat part[32][ROWS8];
  __shared__ Stat share[1 + SHARES][ROWS8];
  __shared__ int slabs_used[ROWS8];
  extern __shared__ float4 smem4[];   // [8][slabs] which of a slab's columns are left out, [8][K] listed logits
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, k = w % ROWS8;
  ptx::grid_dependency_wait();
  const int Cl = chunk_rows(a.hdr, a.c0, a.C);
  const int r0 = blockIdx.x * ROWS8;
  if (r0 >= Cl) return;
  const long long r = r0 + k;
  const bool valid = r < Cl;
  float* mine = reinterpret_cast<float*>(smem4 + ROWS8 * a.slabs) + k * a.K;
  const long long row = valid ? a.idx[a.c0 + r] : 0, list = a.by_token ? row : r;
  const int n = valid ? min(a.K, a.count[list]) : 0;
  if (w < ROWS8) {
    const Stat s = merge_parts8<false>(a.stats, a.nparts, a.C, a.c2, r0, Cl, lane, w, part);
    if (lane == 0) share[0][w] = s;
  } else {
    uint32_t* out = reinterpret_cast<uint32_t*>(smem4 + k * a.slabs);   // [slabs][4] bits of the columns left out
    const float* slabs = a.z + r * a.slabs * PART_COLS;
    const int sub = w / ROWS8 - 1;
    if (sub == 0) {
      for (int q = lane; q < a.slabs * 4; q += 32) out[q] = 0u;
      __syncwarp();
      int used = 0;
      for (int u0 = 0; u0 < n; u0 += 32) {
        const int u = u0 + lane;
        const int id = u < n ? a.id[list * a.K + u] : 0, in = id / PART_COLS;
        const bool first = u < n && (u == 0 || a.id[list * a.K + u - 1] / PART_COLS != in);
        const unsigned f = __ballot_sync(0xffffffffu, first);
        if (u < n) {
          const int q = used + __popc(f & (0xffffffffu >> (31 - lane))) - 1, at = id % PART_COLS;
          mine[u] = slabs[q * PART_COLS + at];
          atomicOr(out + q * 4 + at / 32, 1u << (at % 32));
          const int left = a.V - in * PART_COLS;   // columns of the vocabulary
          if (first && left < PART_COLS)
            for (int j = 0; j < 4; ++j)
              if (left < (j + 1) * 32) atomicOr(out + q * 4 + j, 0xffffffffu << max(0, left - j * 32));
        }
        used += __popc(f);
      }
      if (lane == 0) slabs_used[k] = used;
    }
    ptx::named_bar_sync(ROWS8_BAR_OTHERS, 32 * ROWS8 * SHARES);
    const int used = slabs_used[k];
    const float4* slab = reinterpret_cast<const float4*>(slabs) + lane;
    Stat acc = {-INFINITY, 0.f, 0.f};
    for (int q = sub * 4; q < used; q += 4 * SHARES) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = q + i < used ? slab[(q + i) * (PART_COLS / 4)]
                                      : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = q + i < used ? out[(q + i) * 4 + lane / 8] >> (lane % 8 * 4) & 15u : 0u;
        if (b) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((b >> j) & 1u) v[4 * i + j] = -INFINITY;
        }
      }
      float m = fmaxf(acc.m, fmaxf(v[14], v[15]));
#pragma unroll
      for (int i = 0; i < 14; i += 2) m = ptx::max3(m, v[i], v[i + 1]);
      const float mb = m == -INFINITY ? 0.f : -m * a.c2;   // (nothing yet: every term is 0)
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) s += ptx::ex2(fmaf(v[i], a.c2, mb));
      // mb is rounded: every exponent is too large by rho (exact in the fused multiply-add)
      const float rho = m == -INFINITY ? 0.f : fmaf(m, a.c2, mb);
      acc = merge(acc, Stat{m, s * ptx::ex2(-rho), 0.f}, a.c2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {   // fixed order; lane 0 holds the result
      const Stat other = {__shfl_down_sync(0xffffffffu, acc.m, o), __shfl_down_sync(0xffffffffu, acc.s, o), 0.f};
      acc = merge(acc, other, a.c2);
    }
    if (lane == 0) share[1 + sub][k] = acc;
  }
  __syncthreads();
  if (w >= ROWS8 || !valid) return;
  if (a.hdr[HDR_STATUS] & STATUS_TIMEOUT) return fill_row(a.out, row, a.K, __int_as_float(0x7fc00000), lane);
  Stat rest = share[0][k];
#pragma unroll
  for (int i = 1; i <= SHARES; ++i) rest = merge(rest, share[i][k], a.c2);
  finish_row(a.out, row, a.K, a.tail, a.inv_t, rest, mine, a.t + list * a.K, a.slot + list * a.K, n, lane);
}

// After a call of several chunks: a pipeline that timed out in one of them
// leaves no row to be trusted.
__global__ void __launch_bounds__(256) distill_failed_kernel(const int* hdr, long long N, int K, const int* targets,
                                                             const DistillOut o) {
  ptx::grid_dependency_wait();
  if (!(hdr[HDR_STATUS] & STATUS_TIMEOUT)) return;
  for (long long row = blockIdx.x * 8ll + threadIdx.x / 32; row < N; row += gridDim.x * 8ll)
    if (targets[row] >= 0) fill_row(o, row, K, __int_as_float(0x7fc00000), threadIdx.x % 32);
}

struct StreamRowsArgs {
  int* hdr;
  const int* teacher_ids;
  int K, V, ctas, tail, tiles;
  const float4* stat;
  const int* fail;
  const int* start;
  const float *z, *t;
  const short* slot;
  float c2, inv_t;
  DistillOut out;
};

// One row per block of one warp, from the CTAs' statistics.
__global__ void __launch_bounds__(32) distill_stream_rows_kernel(const StreamRowsArgs a) {
  const int n0 = blockIdx.x, lane = threadIdx.x;
  const int target = row_target(a.teacher_ids + static_cast<long long>(n0) * a.K, a.K, a.V, lane);
  ptx::grid_dependency_wait();
  Stat acc = {-INFINITY, 0.f, 0.f};
  bool failed = false;
  for (int b = lane; b < a.ctas; b += 32) {
    failed = failed || a.fail[b];
    const float4 q = a.stat[static_cast<long long>(n0) * a.ctas + b];
    acc = merge(acc, Stat{q.x, q.y, q.z}, a.c2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {   // fixed order; lane 0 holds the result
    const Stat other = {__shfl_down_sync(0xffffffffu, acc.m, o), __shfl_down_sync(0xffffffffu, acc.s, o),
                        __shfl_down_sync(0xffffffffu, acc.d, o)};
    acc = merge(acc, other, a.c2);
  }
  acc.m = __shfl_sync(0xffffffffu, acc.m, 0);
  acc.s = __shfl_sync(0xffffffffu, acc.s, 0);
  failed = __any_sync(0xffffffffu, failed);
  const bool bad = target >= a.V;
  if (lane == 0 && (failed || bad))
    atomicOr(a.hdr + HDR_STATUS, (failed ? STATUS_TIMEOUT : 0) | (bad ? STATUS_BADTARGET : 0));
  if (target < 0) return fill_row(a.out, n0, a.K, 0.f, lane);
  if (failed || bad) return fill_row(a.out, n0, a.K, __int_as_float(0x7fc00000), lane);
  const long long at = static_cast<long long>(n0) * a.K;
  const int n = min(a.K, a.start[static_cast<long long>(n0) * (a.tiles + 1) + a.tiles]);
  finish_row(a.out, n0, a.K, a.tail, a.inv_t, acc, a.z + at, a.t + at, a.slot + at, n, lane);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// What the gradient needs of a row, by a warp: its target (for the kernels that
// compact the rows), the log-sum-exp and upstream gradient for MODE_DZ, which
// sets dz = -grad / T exp(z - lse), and dz at the listed tokens.
template <int SORT_GROUPS>
__global__ void __launch_bounds__(32 * TARGET_WARPS)
    distill_grad_rows_kernel(const int* ids, const float* logp, long long N, int K, int V, int tail, float temperature,
                             const float* lse, const float* rest_logp, const float* student_logp, const float* grad_kl,
                             int* targets, float* dz_lse, float* dz_grad, uint32_t* patch) {
  extern __shared__ int smem[];   // scratch of a sort per warp
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const long long row = static_cast<long long>(blockIdx.x) * TARGET_WARPS + w;
  if (row >= N) return;
  ids += row * K;
  const int target = row_target(ids, K, V, lane);
  if (lane == 0) targets[row] = target;
  if (target < 0 || target >= V) return;
  const SortRow s = sort_scratch(smem + w * sort_words(K), K);
  int slot[SORT_GROUPS];
  const int n = sort_row(ids, logp + row * K, K, tail, lane, s, slot);
  Teacher q = teacher_of(s.t, n, tail, lane);
  const float rl = rest_logp[row], g = grad_kl[row];
  const bool none = rl == -INFINITY;
  if (none) q.rest = 0.f;
  float mass = 0.f;
  for (int u = lane; u < n; u += 32) mass += expf(s.t[u] - q.shift);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  mass += q.rest;
  if (lane == 0) {
    dz_lse[row] = none ? lse[row] : lse[row] + rl;
    dz_grad[row] = none ? -g * mass : -g * (mass * expf(rl) - q.rest);
  }
  const float gt = g / temperature;
#pragma unroll
  for (int e = 0; e < SORT_GROUPS; ++e) {
    const int j = e * 32 + lane;
    if (j >= K) break;
    const float p = slot[e] >= 0 ? expf(s.t[slot[e]] - q.shift) : 0.f;
    const float dz = gt * (mass * expf(student_logp[row * K + j]) - p);
    // two bf16 parts, as MODE_DZ stores all of dz
    const uint32_t hi = ptx::pack_bf16x2(dz, 0.f) & 0xffffu;
    patch[row * K + j] = hi | ptx::pack_bf16x2(dz - __uint_as_float(hi << 16), 0.f) << 16;
  }
}

// dz of a chunk's listed tokens, both parts.  (Entries of the same token hold the same.)
__global__ void __launch_bounds__(256)
    distill_patch_kernel(const int* hdr, const int* idx, long long c0, int C, int K, int V, long long ldz, const int* ids,
                         const uint32_t* patch, uint16_t* z) {
  ptx::grid_dependency_wait();
  const long long total = static_cast<long long>(chunk_rows(hdr, c0, C)) * K;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long r = i / K, from = idx[c0 + r] * static_cast<long long>(K) + (i - r * K);
    const int x = ids[from];
    if (x < 0 || x >= V) continue;
    const uint32_t dz = patch[from];
    z[r * ldz + x] = static_cast<uint16_t>(dz & 0xffffu);
    z[(C + r) * ldz + x] = static_cast<uint16_t>(dz >> 16);
  }
}

size_t lists_smem(int K) { return size_t(ROWS8) * list_words(K) * 4; }
size_t rows_smem(int K, int slabs) { return size_t(ROWS8) * (size_t(slabs) * 16 + size_t(K) * 4); }
size_t grad_smem(int K) { return size_t(TARGET_WARPS) * sort_words(K) * 4; }
static_assert(ROWS8 * (MAX_TEACHER * 5 + 8) * 4 + 4096 <= 49152, "shared memory that needs no attribute");

// f(32s of entries of a sort, as a type)
template <int G>
struct Groups { static constexpr int value = G; };
template <class F>
cudaError_t by_groups(int K, F&& f) {
  if (K <= 32) return f(Groups<1>());
  if (K <= 64) return f(Groups<2>());
  if (K <= 128) return f(Groups<4>());
  return f(Groups<8>());
}

// K blocks of a segment of a logit's sum (see segment_blocks()).  A divergence of
// distributions that nearly agree keeps the logits' absolute errors, so its
// segments are shorter than those of the log probabilities: kl is off by about as
// much as with an fp32 product on the CUDA cores (2000 tokens at 1024, 2048, 4096 x
// 60000: 1.0e-6, 1.5e-6, 2.1e-6 of its norm and 1.1e-6, 1.7e-6, 2.7e-6; with the
// log probabilities' segments 1.5e-6, 2.1e-6, 3.0e-6 and 1 to 2% faster; 0.4 to 1.3
// times elsewhere, 1.5 for the one segment of 128).  Up to 64 tokens four blocks cost
// nothing, since the weight's bytes bound the kernel.
// Sums of 3 blocks and more are in two segments at least: in one, 600 tokens at 192
// and 248 x 2250 were off by 1.4 to 1.9 times what the fp32 product was, in two by 0.7
// to 0.9.  That costs short tiles much (8192 tokens at 256 x 128256 437 -> 713 us, 4096
// at 256 x 16000 64 -> 82, 300 at 16000 25 -> 29), as it does from five blocks on.
int distill_segment(long long N, long long H) {
  const int blocks = static_cast<int>(cdiv(H, BK));
  int most = N <= 64 ? 4 : std::max(4, static_cast<int>(1.75 * std::sqrt(static_cast<double>(blocks))));
  if (N <= STREAM_MAX_TOKENS) most = std::min(most, 8);
  most = std::min(most, std::max(2, (blocks + 1) / 2));
  return static_cast<int>(cdiv(blocks, cdiv(blocks, most)));   // of equal length
}

struct DistillStream {
  int ctas, max_tiles;
  size_t o_stat, o_start, o_id, o_z, o_t, o_slot, o_fail, total;
};

DistillStream distill_stream_plan(long long N, long long V, int K, int sms) {
  DistillStream p;
  p.ctas = stream_ctas(V, sms);
  p.max_tiles = stream_max_tiles(V, p.ctas);
  size_t off = al256(HDR_WORDS * sizeof(int));
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += al256(bytes);
    return o;
  };
  p.o_stat = take(size_t(N) * p.ctas * 16);
  p.o_start = take(size_t(N) * (p.ctas * p.max_tiles + 1) * 4);
  p.o_id = take(size_t(N) * K * 4);
  p.o_z = take(size_t(N) * K * 4);
  p.o_t = take(size_t(N) * K * 4);
  p.o_slot = take(size_t(N) * K * 2);
  p.o_fail = take(size_t(p.ctas) * 4);
  p.total = off;
  return p;
}

ListedSizes distill_sizes(long long N, long long H, long long V, int K) {
  // of a row: log masses and places of the entries, and the logits of the parts that hold any
  const long long slabs = std::min<long long>(K, cdiv(V, PART_COLS));
  return ListedSizes{N, H, V, 0, K, 6ll * K + 4, 2, slabs * PART_COLS};
}

// What the backward keeps of the call beside the workspace of the log
// probabilities' gradient, behind it.
struct GradExtra {
  size_t o_targets, o_lse, o_grad, o_patch, total;
};

GradExtra grad_extra(long long N, int K) {
  GradExtra x;
  x.o_targets = 0;
  x.o_lse = al256(size_t(N) * 4);
  x.o_grad = 2 * x.o_lse;
  x.o_patch = 3 * x.o_lse;
  x.total = x.o_patch + al256(size_t(N) * K * 4);
  return x;
}

bool sizes_bad(int64_t N, int64_t H, int64_t V) { return !sizes_ok(N, H, V) || V > PROBS_MAX_V; }

}  // namespace

cudaError_t launch_distill_grad_rows(const DistillGrad& d, long long N, int V, float temperature, cudaStream_t s) {
  return by_groups(d.K, [&](auto g) {
    distill_grad_rows_kernel<decltype(g)::value>
        <<<static_cast<unsigned>(cdiv(N, TARGET_WARPS)), 32 * TARGET_WARPS, grad_smem(d.K), s>>>(
            d.ids, d.logp, N, d.K, V, d.tail, temperature, d.lse_in, d.rest_logp, d.student_logp, d.grad_kl, d.targets,
            d.lse, d.grad, d.patch);
    return launch_result(cudaGetLastError());
  });
}

cudaError_t launch_distill_patch(const int* hdr, const int* idx, long long c0, int C, int K, int V, long long ldz,
                                 const int* ids, const uint32_t* patch, uint16_t* z, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(std::min<long long>(cdiv(static_cast<long long>(C) * K, 256), 152 * 8));
  return launch_dependent(distill_patch_kernel, blocks, 256, s, hdr, idx, c0, C, K, V, ldz, ids, patch, z);
}

}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_topk_distill_workspace_bytes(int64_t N, int64_t H, int64_t V, int32_t K) {
  if (sizes_bad(N, H, V) || K < 1 || K > MAX_TEACHER) return 0;
  if (N <= STREAM_MAX_TOKENS) return distill_stream_plan(N, V, K, device_sms()).total;
  return listed_default_bytes(distill_sizes(N, H, V, K));
}

flce_status flce_topk_distill(const void* hidden, const void* weight, const int32_t* teacher_ids,
                              const float* teacher_logp, int64_t N, int64_t H, int64_t V, int32_t K, float temperature,
                              int32_t tail, float* kl, float* lse, float* rest_logp, float* student_logp,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!hidden || !weight || !teacher_ids || !teacher_logp || !kl || !lse || !rest_logp || !student_logp || !workspace)
    return FLCE_EINVAL;
  if (N < 1 || H < 1 || V < 1 || K < 1 || (tail != 0 && tail != 1) || bad_temperature(temperature)) return FLCE_EINVAL;
  if (sizes_bad(N, H, V) || K > MAX_TEACHER) return FLCE_EUNSUPPORTED;
  if (!aligned16(hidden) || !aligned16(weight) || !aligned16(workspace) || !aligned4(teacher_ids) ||
      !aligned4(teacher_logp) || !aligned4(kl) || !aligned4(lse) || !aligned4(rest_logp) || !aligned4(student_logp))
    return FLCE_EUNSUPPORTED;
  // the logits of the chunked form are stored 32 bytes at a time
  if (N > STREAM_MAX_TOKENS && !aligned32(workspace)) return FLCE_EUNSUPPORTED;
  DeviceState dev;
  if (device_state(&dev) != cudaSuccess) { cudaGetLastError(); return FLCE_ECUDA; }
  if (dev.major < 10) return FLCE_EUNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto ok = [](cudaError_t e) { return e == cudaSuccess; };
  const DistillOut out{kl, lse, rest_logp, student_logp};
  ListArgs la;
  std::memset(&la, 0, sizeof(la));
  la.teacher_ids = teacher_ids; la.teacher_logp = teacher_logp; la.K = K; la.V = static_cast<int>(V); la.tail = tail;
  if (N <= STREAM_MAX_TOKENS) {
    const DistillStream p = distill_stream_plan(N, V, K, dev.sms);
    if (p.total > workspace_bytes) return FLCE_EWORKSPACE;
    StreamArgs a;
    StreamLists l;
    StreamMaps m;
    std::memset(&a, 0, sizeof(a));
    std::memset(&l, 0, sizeof(l));
    a.N = static_cast<int>(N); a.H = static_cast<int>(H); a.V = static_cast<int>(V);
    a.ctas = p.ctas; a.max_tiles = p.max_tiles;
    a.c2 = LOG2E / temperature;
    a.hdr = at<int>(workspace, 0);
    a.stat = at<float4>(workspace, p.o_stat);
    a.fail = at<int>(workspace, p.o_fail);
    l.lists.start = la.start = at<int>(workspace, p.o_start);
    l.lists.boundaries = p.ctas * p.max_tiles + 1;
    l.lists.id = la.id = at<int>(workspace, p.o_id);
    l.lists.z = at<float>(workspace, p.o_z);
    l.lists.cap = K;
    la.ctas = p.ctas; la.max_tiles = p.max_tiles;
    la.t = at<float>(workspace, p.o_t);
    la.slot = at<short>(workspace, p.o_slot);
    if (!stream_setup(&a, &m, hidden, weight, distill_segment(N, H))) return FLCE_ECUDA;
    count_launches(2);   // lists, rows
    if (!ok(by_groups(K, [&](auto g) {
          distill_stream_lists_kernel<decltype(g)::value><<<static_cast<unsigned>(N), STREAM_LIST_THREADS, 0, st>>>(la);
          return launch_result(cudaGetLastError());
        })))
      return FLCE_ECUDA;
    const ProfScope prof = prof_launch_begin(st);
    const cudaError_t e = launch_stream_taken(a, m, l, st);
    prof_launch_end(prof, MODE_STATS, st);
    if (!ok(e)) return FLCE_ECUDA;
    const StreamRowsArgs ra{a.hdr, teacher_ids, K, a.V, p.ctas, tail, p.ctas * p.max_tiles, a.stat, a.fail, la.start,
                            l.lists.z, la.t, la.slot, a.c2, 1.f / temperature, out};
    if (!ok(launch_dependent(distill_stream_rows_kernel, static_cast<unsigned>(N), 32, st, ra))) return FLCE_ECUDA;
    return FLCE_OK;
  }
  ListedPlan p;
  ListedCall c;
  std::memset(&c, 0, sizeof(c));
  c.q = distill_sizes(N, H, V, K);
  if (!listed_plan(c.q, workspace_bytes, &p)) return FLCE_EWORKSPACE;
  int* targets = at<int>(workspace, p.o_targets);
  const bool by_token = listed_front(p, N);
  la.N = static_cast<int>(N);
  auto launch_lists = [&](const int* idx) {
    la.idx = idx;
    count_launches(1);
    return by_groups(K, [&](auto g) {
      return launch_dependent_smem(distill_lists_kernel<decltype(g)::value>, static_cast<unsigned>(cdiv(idx ? la.C : N, ROWS8)),
                                   32 * LIST_WARPS, lists_smem(K), st, la, targets, out);
    });
  };
  if (!by_token) {
    count_launches(1);
    distill_targets_kernel<<<static_cast<unsigned>(cdiv(N, TARGET_WARPS)), 32 * TARGET_WARPS, 0, st>>>(
        teacher_ids, N, K, static_cast<int>(V), targets, out);
    if (!ok(launch_result(cudaGetLastError()))) return FLCE_ECUDA;
  }
  c.hidden = hidden; c.weight = weight; c.targets = targets; c.ii = -1; c.temperature = temperature;
  c.logp = kl; c.entropy = rest_logp; c.lse = lse;
  c.seg_kb = distill_segment(N, H);
  c.ws = workspace; c.st = st;
  la.t = at<float>(workspace, p.o_rows);
  la.count = reinterpret_cast<int*>(la.t + p.C * K);
  la.slot = reinterpret_cast<short*>(la.count + p.C);
  la.C = static_cast<int>(p.C);
  la.nparts = p.nparts;
  la.slab = at<short>(workspace, p.o_start);
  la.id = at<int>(workspace, p.o_id);
  c.by_token = by_token;
  if (by_token && !ok(launch_lists(nullptr))) return FLCE_ECUDA;
  flce_status s = listed_chunks(
      p, c, dev,
      [&](const ListedChunk& ch) {
        if (by_token) return cudaSuccess;
        la.hdr = ch.g->hdr; la.c0 = ch.c0;
        return launch_lists(ch.g->idx);
      },
      [&](const ListedChunk& ch) {
        const RowsArgs ra{ch.g->hdr, ch.g->idx, ch.c0, ch.g->C, ch.g->nparts, ch.g->V, K, tail, ch.g->slabs_per_row,
                          ch.g->stats, by_token, la.count, la.id, ch.g->lists.z, la.t, la.slot, ch.g->c2, 1.f / temperature, out};
        count_launches(1);
        const unsigned blocks = static_cast<unsigned>(cdiv(ch.g->C, ROWS8));
        const size_t smem = rows_smem(K, ch.g->slabs_per_row);
        return blocks > static_cast<unsigned>(dev.sms) || ch.g->slabs_per_row < 16
                   ? launch_dependent_smem(distill_rows_kernel<1>, blocks, 32 * ROWS8 * 2, smem, st, ra)
                   : launch_dependent_smem(distill_rows_kernel<3>, blocks, 32 * ROWS8 * 4, smem, st, ra);
      });
  if (s == FLCE_OK && p.n_chunks > 1) {
    count_launches(1);
    if (!ok(launch_dependent(distill_failed_kernel, 152, 256, st, at<int>(workspace, 0), N, K, targets, out)))
      return FLCE_ECUDA;
  }
  return s;
}

size_t flce_topk_distill_bwd_workspace_bytes(int64_t N, int64_t H, int64_t V, int32_t K, uint32_t flags) {
  if (sizes_bad(N, H, V) || K < 1 || K > MAX_TEACHER) return 0;
  const size_t extra = grad_extra(N, K).total, n = distill_grad_bytes(N, H, V, flags, al256(size_t(N) * K * 2));
  return n == 0 ? 0 : al256(n) + extra;
}

flce_status flce_topk_distill_bwd(const void* hidden, const void* weight, const int32_t* teacher_ids,
                                  const float* teacher_logp, int64_t N, int64_t H, int64_t V, int32_t K, uint32_t flags,
                                  float temperature, int32_t tail, const float* lse, const float* rest_logp,
                                  const float* student_logp, const float* grad_kl, void* grad_hidden,
                                  float* grad_weight, void* workspace, size_t workspace_bytes, void* stream) {
  if (!teacher_ids || !teacher_logp || !lse || !rest_logp || !student_logp || !grad_kl || !workspace) return FLCE_EINVAL;
  if (N < 1 || H < 1 || V < 1 || K < 1 || (tail != 0 && tail != 1)) return FLCE_EINVAL;
  if (sizes_bad(N, H, V) || K > MAX_TEACHER) return FLCE_EUNSUPPORTED;
  if (!aligned4(teacher_ids) || !aligned4(teacher_logp) || !aligned4(lse) || !aligned4(rest_logp) ||
      !aligned4(student_logp) || !aligned4(grad_kl) || !aligned16(workspace))
    return FLCE_EUNSUPPORTED;
  const GradExtra x = grad_extra(N, K);
  if (workspace_bytes < x.total + 256) return FLCE_EWORKSPACE;
  const size_t own = (workspace_bytes - x.total) & ~size_t(255);
  DistillGrad d;
  d.ids = teacher_ids;
  d.K = K;
  d.targets = at<int>(workspace, own + x.o_targets);
  d.lse = at<float>(workspace, own + x.o_lse);
  d.grad = at<float>(workspace, own + x.o_grad);
  d.patch = at<uint32_t>(workspace, own + x.o_patch);
  d.logp = teacher_logp; d.tail = tail; d.lse_in = lse; d.rest_logp = rest_logp; d.student_logp = student_logp;
  d.grad_kl = grad_kl;
  return run_distill_grad(d, hidden, weight, N, H, V, flags, temperature, grad_hidden, grad_weight, workspace, own,
                          stream);
}

}  // extern "C"
