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
// formed as a difference: the GEMM's epilogue takes the listed logits out of
// the row's statistics and writes them side by side, and the row kernel brings
// them back in.  All of a row's log probabilities are formed relative to its
// largest logit (an fp32 log-sum-exp of 20 is off by 1e-6, as much as kl is
// where student and teacher nearly agree), and r as (1 - p_max) - the others.
//
// Backward: behind the list dz_v = g (A s - r) / T * exp(z_v - lse_rest), one
// exponential per logit with constants of its row that neither overflow nor
// lose anything where s is small: the epilogue of the log probabilities'
// gradient (MODE_DZ) with another log-sum-exp and another upstream gradient.
// Between it and the two products a small kernel overwrites the listed places.
#include "flce_listed.cuh"
#include "flce_ptx.cuh"
#include "flce_rows.cuh"
#include "flce_softmax.cuh"
#include "flce_stream_range.cuh"

namespace flce {
namespace {

constexpr int MAX_TEACHER = 256;   // teacher tokens of a row at most
constexpr int NO_TOKEN = INT_MAX;

// ---------------------------------------------------------------------------
// lists
// ---------------------------------------------------------------------------

// A row's teacher tokens in ascending order, each once, by G threads (g: the
// thread's place among them).  id: shared copy of the sorted tokens; gid, gt:
// the same in memory with their log masses; slot[j]: the place of entry j, -1
// where there is none.  Returns their number.  K^2 comparisons: with 64 entries
// 128 a lane.
template <int G, class Sync>
__device__ __forceinline__ int sort_row(const int* ids, const float* t, int K, int g, int* all, int* first, int* id,
                                        int* gid, float* gt, short* slot, Sync sync) {
  for (int j = g; j < K; j += G) {
    const int x = ids[j];
    all[j] = x < 0 ? NO_TOKEN : x;
  }
  sync();
  for (int j = g; j < K; j += G) {
    const int x = all[j];
    bool f = true;
    for (int i = 0; i < j; ++i) f = f && all[i] != x;
    first[j] = f ? x : NO_TOKEN;
  }
  sync();
  int n = 0;
  for (int i = 0; i < K; ++i) n += first[i] != NO_TOKEN;
  for (int j = g; j < K; j += G) {
    const int x = all[j];
    if (x == NO_TOKEN) {
      slot[j] = -1;
      continue;
    }
    int u = 0, same = 0;
    for (int i = 0; i < K; ++i) {
      u += first[i] < x;
      same += all[i] == x;
    }
    slot[j] = static_cast<short>(u);
    if (first[j] != x) continue;
    float m = t[j];
    if (same > 1) {   // the token's masses add up
      for (int i = j + 1; i < K; ++i)
        if (all[i] == x) m = fmaxf(m, t[i]);
      if (m > -INFINITY) {
        float sum = 0.f;
        for (int i = j; i < K; ++i)
          if (all[i] == x) sum += expf(t[i] - m);
        m += logf(sum);
      }
    }
    id[u] = x;
    gid[u] = x;
    gt[u] = m;
  }
  sync();
  return n;
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
  int K, V;
  const int* hdr;             // chunked form
  const int* idx;
  long long c0;
  int C, nparts;
  int ctas, max_tiles;        // streaming form
  int* start;
  int* id;                    // [rows][K]
  float* t;                   // [rows][K] log masses of the sorted tokens
  short* slot;                // [rows][K] place of each given entry
};

// Chunked: 32 rows a block, a warp sorts four of them; then a lane walks a
// row's list along the parts, so that the boundaries are written 128 bytes at a
// time.
constexpr int LIST_ROWS = 32;
constexpr int LIST_WARPS = 8;
__global__ void __launch_bounds__(32 * LIST_WARPS) distill_lists_kernel(const ListArgs a) {
  extern __shared__ int smem[];   // [32][K | 1] sorted, [8][2 K] scratch
  __shared__ int count[LIST_ROWS];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int pitch = a.K | 1;      // odd: a column of the sorted lists is in 32 banks
  ptx::grid_dependency_wait();
  const int Cl = chunk_rows(a.hdr, a.c0, a.C);
  const int r0 = blockIdx.x * LIST_ROWS;
  if (r0 >= Cl) return;
  int* scratch = smem + LIST_ROWS * pitch + w * 2 * a.K;
  for (int k = w; k < LIST_ROWS && r0 + k < Cl; k += LIST_WARPS) {
    const long long row = r0 + k, from = static_cast<long long>(a.idx[a.c0 + row]) * a.K, to = row * a.K;
    const int n = sort_row<32>(a.teacher_ids + from, a.teacher_logp + from, a.K, lane, scratch, scratch + a.K,
                               smem + k * pitch, a.id + to, a.t + to, a.slot + to, [] { __syncwarp(); });
    if (lane == 0) count[k] = n;
  }
  __syncthreads();
  const int r = r0 + lane;
  if (r >= Cl) return;
  const int n = count[lane];
  const int* id = smem + lane * pitch;
  const int bounds = a.nparts + 1, each = (bounds + LIST_WARPS - 1) / LIST_WARPS;
  const int p1 = min(bounds, (w + 1) * each);
  int p = w * each;
  int e = lower_bound(id, n, p * PART_COLS);
  for (; p < p1; ++p) {
    while (e < n && id[e] < p * PART_COLS) ++e;
    a.start[static_cast<long long>(p) * a.C + r] = p == a.nparts ? n : e;
  }
}

// Streaming: a block per row; the weight streams meanwhile.
constexpr int STREAM_LIST_THREADS = 128;
__global__ void __launch_bounds__(STREAM_LIST_THREADS) distill_stream_lists_kernel(const ListArgs a) {
  __shared__ int all[MAX_TEACHER], first[MAX_TEACHER], id[MAX_TEACHER];
  ptx::grid_launch_dependents();
  const long long from = static_cast<long long>(blockIdx.x) * a.K;
  const int n = sort_row<STREAM_LIST_THREADS>(a.teacher_ids + from, a.teacher_logp + from, a.K, threadIdx.x, all, first,
                                              id, a.id + from, a.t + from, a.slot + from, [] { __syncthreads(); });
  const int tiles = a.ctas * a.max_tiles;
  int* start = a.start + static_cast<long long>(blockIdx.x) * (tiles + 1);
  for (int b = threadIdx.x; b <= tiles; b += STREAM_LIST_THREADS) {
    int x = a.V;
    if (b < tiles) {
      const Range r = range_of(a.V, a.ctas, b / a.max_tiles);
      x = b % a.max_tiles < r.tiles ? r.start(b % a.max_tiles) : r.u1 * UNIT_ROWS;
    }
    start[b] = lower_bound(id, n, min(x, a.V));
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

// One row by a warp, from the statistics of the logits behind its list and the
// listed logits z[0 .. n).
__device__ __forceinline__ void finish_row(const DistillOut& o, long long row, int K, bool tail, float c2, Stat rest,
                                           const float* z, const float* t, const short* slot, int n, int lane) {
  float m = rest.m;
  bool nan = false;
  for (int u = lane; u < n; u += 32) {
    m = fmaxf(m, z[u]);
    nan = nan || z[u] != z[u];
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  if (__any_sync(0xffffffffu, nan)) m = __int_as_float(0x7fc00000);
  float s = 0.f;
  for (int u = lane; u < n; u += 32) s += exp2f((z[u] - m) * c2);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  const bool none = rest.m == -INFINITY && rest.s == 0.f;   // nothing behind the list
  if (!none) s += rest.s * exp2f((rest.m - m) * c2);
  const float l2s = log2f(s);
  const float rest_logp = none ? -INFINITY : fmaf(rest.m - m, c2, log2f(rest.s) - l2s) * LN2;
  Teacher q = teacher_of(t, n, tail, lane);
  if (none) q.rest = 0.f;
  double kl = 0.0;   // of terms that nearly cancel
  for (int u = lane; u < n; u += 32) {
    const float lp = t[u] - q.shift, p = expf(lp), lq = fmaf(z[u] - m, c2, -l2s) * LN2;
    if (!(p == 0.f)) kl += static_cast<double>(p) * static_cast<double>(lp - lq);
  }
  for (int j = lane; j < K; j += 32) {
    const int u = slot[j];
    o.student_logp[row * K + j] = u < 0 || u >= n ? 0.f : fmaf(z[u] - m, c2, -l2s) * LN2;
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) kl += __shfl_xor_sync(0xffffffffu, kl, k);
  if (lane == 0) {
    if (!(q.rest == 0.f)) kl += static_cast<double>(q.rest) * static_cast<double>(logf(q.rest) - rest_logp);
    o.kl[row] = static_cast<float>(kl);
    o.lse[row] = fmaf(m, c2, l2s) * LN2;
    o.rest_logp[row] = rest_logp;
  }
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
  int C, nparts, K, tail;
  const float* stats;
  const int* start;
  const float *z, *t;
  const short* slot;
  float c2;
  DistillOut out;
};

// 32 rows of a chunk: the parts' statistics merged with a lane a row, then a
// warp a row.
__global__ void __launch_bounds__(32 * ROWS_WARPS) distill_rows_kernel(const RowsArgs a) {
  __shared__ Stat part[ROWS_WARPS][32];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  ptx::grid_dependency_wait();
  const int Cl = chunk_rows(a.hdr, a.c0, a.C);
  const int r0 = blockIdx.x * 32;
  if (r0 >= Cl) return;
  merge_parts(a.stats, a.nparts, a.C, a.c2, r0 + lane, r0 + lane < Cl, lane, w, part);
  __syncthreads();
  const long long r = r0 + w;
  if (r >= Cl) return;
  const long long row = a.idx[a.c0 + r];
  if (a.hdr[HDR_STATUS] & STATUS_TIMEOUT) return fill_row(a.out, row, a.K, __int_as_float(0x7fc00000), lane);
  const int n = min(a.K, a.start[static_cast<long long>(a.nparts) * a.C + r]);
  finish_row(a.out, row, a.K, a.tail, a.c2, part[0][w], a.z + r * a.K, a.t + r * a.K, a.slot + r * a.K, n, lane);
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
  float c2;
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
  finish_row(a.out, n0, a.K, a.tail, a.c2, acc, a.z + at, a.t + at, a.slot + at, n, lane);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// What the gradient needs of a row, by a warp: its target (for the kernels that
// compact the rows), the log-sum-exp and upstream gradient for MODE_DZ, which
// sets dz = -grad / T exp(z - lse), and dz at the listed tokens.
__global__ void __launch_bounds__(32 * TARGET_WARPS)
    distill_grad_rows_kernel(const int* ids, const float* logp, long long N, int K, int V, int tail, float temperature,
                             const float* lse, const float* rest_logp, const float* student_logp, const float* grad_kl,
                             int* targets, float* dz_lse, float* dz_grad, uint16_t* patch) {
  extern __shared__ float smem_t[];   // [warps][2 K]: log masses, each token's once, and ids
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const long long row = static_cast<long long>(blockIdx.x) * TARGET_WARPS + w;
  if (row >= N) return;
  ids += row * K;
  logp += row * K;
  const int target = row_target(ids, K, V, lane);
  if (lane == 0) targets[row] = target;
  if (target < 0 || target >= V) return;
  float* t = smem_t + w * 2 * K;
  int* all = reinterpret_cast<int*>(t + K);
  for (int j = lane; j < K; j += 32) all[j] = ids[j];
  __syncwarp();
  // each entry's token's mass in all; of a token named twice only the first entry has any in the row's sums
  for (int j = lane; j < K; j += 32) {
    const int x = all[j];
    float m = -INFINITY;
    if (x >= 0) {
      m = logp[j];
      bool first = true, again = false;
      for (int i = 0; i < K; ++i) {
        if (i != j && all[i] == x) {
          if (i < j) first = false;
          else again = true;
        }
      }
      if (!first) {
        m = -INFINITY;
      } else if (again) {
        for (int i = j + 1; i < K; ++i)
          if (all[i] == x) m = fmaxf(m, logp[i]);
        if (m > -INFINITY) {
          float sum = 0.f;
          for (int i = j; i < K; ++i)
            if (all[i] == x) sum += expf(logp[i] - m);
          m += logf(sum);
        }
      }
    }
    t[j] = m;
  }
  __syncwarp();
  Teacher q = teacher_of(t, K, tail, lane);
  const float rl = rest_logp[row], g = grad_kl[row];
  const bool none = rl == -INFINITY;
  if (none) q.rest = 0.f;
  float mass = 0.f;
  for (int j = lane; j < K; j += 32) mass += expf(t[j] - q.shift);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  mass += q.rest;
  if (q.top == -INFINITY && !tail) mass = 0.f;   // a teacher without any mass asks for nothing
  if (lane == 0) {
    dz_lse[row] = none ? lse[row] : lse[row] + rl;
    dz_grad[row] = none ? -g * mass : -g * (mass * expf(rl) - q.rest);
  }
  const float gt = g / temperature;
  for (int j = lane; j < K; j += 32) {
    const int x = all[j];
    float p = 0.f;
    if (x >= 0) {
      int i = 0;
      while (all[i] != x) ++i;   // the token's first entry; ends at j
      p = expf(t[i] - q.shift);
    }
    const float dz = gt * (mass * expf(student_logp[row * K + j]) - p);
    patch[row * K + j] = static_cast<uint16_t>(ptx::pack_bf16x2(dz, 0.f) & 0xffffu);
  }
}

// dz of a chunk's listed tokens.  (Entries of the same token hold the same.)
__global__ void __launch_bounds__(256)
    distill_patch_kernel(const int* hdr, const int* idx, long long c0, int C, int K, int V, long long ldz, const int* ids,
                         const uint16_t* patch, uint16_t* z) {
  ptx::grid_dependency_wait();
  const long long total = static_cast<long long>(chunk_rows(hdr, c0, C)) * K;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long r = i / K, from = idx[c0 + r] * static_cast<long long>(K) + (i - r * K);
    const int x = ids[from];
    if (x >= 0 && x < V) z[r * ldz + x] = patch[from];
  }
}

size_t lists_smem(int K) { return (size_t(LIST_ROWS) * (K | 1) + size_t(LIST_WARPS) * 2 * K) * 4; }

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
  return ListedSizes{N, H, V, 0, K, 6ll * K, 0};   // log masses and places
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
  x.total = x.o_patch + al256(size_t(N) * K * 2);
  return x;
}

bool sizes_bad(int64_t N, int64_t H, int64_t V) { return !sizes_ok(N, H, V) || V > PROBS_MAX_V; }

}  // namespace

cudaError_t distill_prepare() {
  return cudaFuncSetAttribute(distill_lists_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(lists_smem(MAX_TEACHER)));
}

cudaError_t launch_distill_grad_rows(const DistillGrad& d, long long N, int V, float temperature, cudaStream_t s) {
  distill_grad_rows_kernel<<<static_cast<unsigned>(cdiv(N, TARGET_WARPS)), 32 * TARGET_WARPS,
                             size_t(TARGET_WARPS) * 2 * d.K * 4, s>>>(
      d.ids, d.logp, N, d.K, V, d.tail, temperature, d.lse_in, d.rest_logp, d.student_logp, d.grad_kl, d.targets, d.lse,
      d.grad, d.patch);
  return launch_result(cudaGetLastError());
}

cudaError_t launch_distill_patch(const int* hdr, const int* idx, long long c0, int C, int K, int V, long long ldz,
                                 const int* ids, const uint16_t* patch, uint16_t* z, cudaStream_t s) {
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
  DeviceState dev;
  if (device_state(&dev) != cudaSuccess) { cudaGetLastError(); return FLCE_ECUDA; }
  if (dev.major < 10) return FLCE_EUNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto ok = [](cudaError_t e) { return e == cudaSuccess; };
  const DistillOut out{kl, lse, rest_logp, student_logp};
  ListArgs la;
  std::memset(&la, 0, sizeof(la));
  la.teacher_ids = teacher_ids; la.teacher_logp = teacher_logp; la.K = K; la.V = static_cast<int>(V);
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
    if (!stream_setup(&a, &m, hidden, weight)) return FLCE_ECUDA;
    count_launches(2);   // lists, rows
    distill_stream_lists_kernel<<<static_cast<unsigned>(N), STREAM_LIST_THREADS, 0, st>>>(la);
    if (!ok(launch_result(cudaGetLastError()))) return FLCE_ECUDA;
    const ProfScope prof = prof_launch_begin(st);
    const cudaError_t e = launch_stream_taken(a, m, l, st);
    prof_launch_end(prof, MODE_STATS, st);
    if (!ok(e)) return FLCE_ECUDA;
    const StreamRowsArgs ra{a.hdr, teacher_ids, K, a.V, p.ctas, tail, p.ctas * p.max_tiles, a.stat, a.fail, la.start,
                            l.lists.z, la.t, la.slot, a.c2, out};
    if (!ok(launch_dependent(distill_stream_rows_kernel, static_cast<unsigned>(N), 32, st, ra))) return FLCE_ECUDA;
    return FLCE_OK;
  }
  ListedPlan p;
  ListedCall c;
  std::memset(&c, 0, sizeof(c));
  c.q = distill_sizes(N, H, V, K);
  if (!listed_plan(c.q, workspace_bytes, &p)) return FLCE_EWORKSPACE;
  int* targets = at<int>(workspace, p.o_targets);
  count_launches(1);
  distill_targets_kernel<<<static_cast<unsigned>(cdiv(N, TARGET_WARPS)), 32 * TARGET_WARPS, 0, st>>>(
      teacher_ids, N, K, static_cast<int>(V), targets, out);
  if (!ok(launch_result(cudaGetLastError()))) return FLCE_ECUDA;
  c.hidden = hidden; c.weight = weight; c.targets = targets; c.ii = -1; c.temperature = temperature;
  c.logp = kl; c.entropy = rest_logp; c.lse = lse;
  c.ws = workspace; c.st = st;
  la.t = at<float>(workspace, p.o_rows);
  la.slot = reinterpret_cast<short*>(la.t + p.C * K);
  flce_status s = listed_chunks(
      p, c, dev,
      [&](const ListedChunk& ch) {
        la.hdr = ch.g->hdr; la.idx = ch.g->idx; la.c0 = ch.c0; la.C = ch.g->C; la.nparts = ch.g->nparts;
        la.start = const_cast<int*>(ch.g->lists.start);
        la.id = const_cast<int*>(ch.g->lists.id);
        count_launches(1);
        return launch_dependent_smem(distill_lists_kernel, static_cast<unsigned>(cdiv(la.C, LIST_ROWS)), 32 * LIST_WARPS,
                                     lists_smem(K), st, la);
      },
      [&](const ListedChunk& ch) {
        const RowsArgs ra{ch.g->hdr, ch.g->idx, ch.c0, ch.g->C, ch.g->nparts, K, tail, ch.g->stats, ch.g->lists.start,
                          ch.g->lists.z, la.t, la.slot, ch.g->c2, out};
        count_launches(1);
        return launch_dependent(distill_rows_kernel, static_cast<unsigned>(cdiv(ch.g->C, 32)), 32 * ROWS_WARPS, st, ra);
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
  const size_t n = flce_logprobs_bwd_workspace_bytes(N, H, V, flags);
  return n == 0 ? 0 : al256(n) + grad_extra(N, K).total;
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
  d.patch = at<uint16_t>(workspace, own + x.o_patch);
  d.logp = teacher_logp; d.tail = tail; d.lse_in = lse; d.rest_logp = rest_logp; d.student_logp = student_logp;
  d.grad_kl = grad_kl;
  return run_distill_grad(d, hidden, weight, N, H, V, flags, temperature, grad_hidden, grad_weight, workspace, own,
                          stream);
}

}  // extern "C"
