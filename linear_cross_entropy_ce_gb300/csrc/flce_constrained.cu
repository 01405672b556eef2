// Log probabilities of the next token under constraints, for serving: penalties
// for repeated tokens, biases and a grammar's mask are applied to the logits
// before the softmax, which then knows nothing of them.
//
//   z = X W^T;  a token that the row's history holds: z <- z > 0 ? z / r : z r,
//   one that its output holds c > 0 times: z <- z - f c - p;  a biased token:
//   z <- z + b;  a forbidden one: z <- -inf;  then lse, entropy, log
//   probabilities and top alternatives of z / T.
//
// Histories and biases change few of a row's logits, the mask takes many but
// needs a bit each.  One kernel makes each row's list of changed tokens from a
// bitmap of the vocabulary in shared memory: bits set by the ids in any order,
// forbidden tokens cleared, and the rank of a token (the set bits before it) is
// its place in the ascending list, so equal ids meet without a sort and counts
// are added by integer atomics, whose order changes nothing.
// Up to 128 tokens the streaming kernel changes the logits of a tile in place
// (flce_stream.cuh) while it is bound by the weight's bytes anyway; beyond, the
// GEMM's epilogue takes them out of the statistics (flce_gemm.cu) and the row
// kernels here bring them back under their rules.
#include "flce_listed.cuh"
#include "flce_ptx.cuh"
#include "flce_rows.cuh"
#include "flce_softmax.cuh"
#include "flce_stream_range.cuh"

namespace flce {
namespace {

// Few rows: all of a block's latency counts, so it is wide; many rows: several
// blocks an SM, and narrow ones where there is little to do (a call of 4096 rows of
// 200 ids at a vocabulary of 4000 74 us with 128 threads a list, 110 with 512; 1307
// of 1359 ids at 753 103 and 133; but 2000 of 6000 ids at 16000 384 and 374).  A
// thread keeps HELD ids and HELD words of the mask and bitmap in registers, all
// loads at once.
constexpr int HELD = 8;
constexpr int STREAM_THREADS = 1024, CHUNK_THREADS = 512, SMALL_THREADS = 128;
constexpr int SMALL_VOCABULARY = 8192, SMALL_HISTORY = 4096;

__host__ __device__ __forceinline__ int pad_words(int words) { return (words + HELD - 1) / HELD * HELD; }

struct RuleArgs {
  int V;
  const int* history;          // [N][L] by stride
  long long L, history_stride;
  const int *history_lens, *prompt_lens;   // or null: L, 0
  const int* bias_ids;         // [N][B] by stride
  const float* bias;
  int B;
  long long bias_ids_stride, bias_stride;
  const uint32_t* mask;
  long long mask_stride;
  const int* hdr;              // chunked form
  const int* idx;
  long long c0;
  int C, nparts;
  int ctas, max_tiles;         // streaming form
  uint32_t* group_max;         // or null: cleared
  int* start;
  int* id;                     // [rows][cap]
  int* seen;
  int* bias_at;                // the last entry that names the token + 1, then its bias (as a float), or null
  long long cap;
  int counts;                  // tokens of a window whose times are counted in shared memory
};

// A block per row, in windows of 32 HELD THREADS tokens (262144 for few rows: one
// window covers most vocabularies).  61 rows of 1500 ids at a vocabulary of
// 256007 with masks 12 us, 2048 rows of up to 2947 ids at 128256 55.  (The bitmap in
// memory, so that the blocks fit beside the streaming kernel's, took 53 us for the
// former, longer than the first tile.)
template <bool STREAM, int THREADS, bool COUNTED>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) constrained_lists_kernel(const RuleArgs a) {
  constexpr int WARPS = THREADS / 32;
  constexpr int WINDOW = HELD * THREADS;   // words
  // [words of a window] the marked tokens, and the marked ones before each word; [counts] times of its first tokens
  extern __shared__ __align__(16) uint32_t bits[];
  __shared__ int sums[WARPS];
  const int tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  long long r = blockIdx.x, n = blockIdx.x;
  if constexpr (STREAM) {
    ptx::grid_launch_dependents();
    if (a.group_max && tid < TopK::MAX) a.group_max[n * TopK::MAX + tid] = 0u;
  } else {
    ptx::grid_dependency_wait();
    if (r >= chunk_rows(a.hdr, a.c0, a.C)) return;
    n = a.idx[a.c0 + r];
  }
  const int V = a.V, words = (V + 31) / 32, window = min(words, WINDOW);
  const int padded = pad_words(window);
  uint32_t* rank = bits + padded;
  int* times = reinterpret_cast<int*>(rank + padded);
  const int* history = a.history + n * a.history_stride;
  const int* bias_ids = a.bias_ids + n * a.bias_ids_stride;
  const uint32_t* mask = a.mask ? a.mask + n * a.mask_stride : nullptr;
  int len = static_cast<int>(a.L), prompt = 0;
  if (a.history_lens) len = max(0, min(len, a.history_lens[n]));
  if (a.prompt_lens) prompt = a.prompt_lens[n];
  int* id = a.id + r * a.cap;
  int* seen = a.seen + r * a.cap;
  int* bias_at = a.bias_at ? a.bias_at + r * a.cap : nullptr;
  const int tiles = STREAM ? a.ctas * a.max_tiles : 0;
  int held[HELD];
#pragma unroll
  for (int k = 0; k < HELD; ++k) held[k] = k * THREADS + tid < len ? history[k * THREADS + tid] : -1;
  int base = 0;   // listed tokens before this window
  for (int w0 = 0; w0 < words; w0 += window) {
    const int nw = min(window, words - w0);
    uint32_t allowed[HELD];
#pragma unroll
    for (int k = 0; k < HELD; ++k)
      allowed[k] = mask && k * THREADS + tid < nw ? mask[w0 + k * THREADS + tid] : 0xffffffffu;
    for (int i = tid; i < padded / 4; i += THREADS) reinterpret_cast<uint4*>(bits)[i] = make_uint4(0u, 0u, 0u, 0u);
    const int base0 = base;
    if constexpr (COUNTED)
      for (int i = tid; i < a.counts; i += THREADS) times[i] = 0;
    __syncthreads();
    const unsigned t0 = static_cast<unsigned>(w0) * 32u, span = min(static_cast<unsigned>(V) - t0, nw * 32u);
    auto mark = [&](int x) {   // (negative ids are far above the span)
      const unsigned at = static_cast<unsigned>(x) - t0;
      if (at < span) atomicOr(bits + at / 32, 1u << (at % 32));
    };
#pragma unroll
    for (int k = 0; k < HELD; ++k) mark(held[k]);
#pragma unroll 4
    for (int i = HELD * THREADS + tid; i < len; i += THREADS) mark(history[i]);
    for (int i = tid; i < a.B; i += THREADS) mark(bias_ids[i]);
    __syncthreads();
    if (mask) {   // forbidden tokens leave
#pragma unroll
      for (int k = 0; k < HELD; ++k) {
        const int i = k * THREADS + tid;
        if (i >= nw) break;
        const uint32_t b = bits[i];
        if (b & ~allowed[k]) bits[i] = b & allowed[k];
      }
      __syncthreads();
    }
    // the words' ranks: a thread has a run of 4 or HELD words
    const int run = nw <= 4 * THREADS ? 4 : HELD, i0 = tid * run;
    uint32_t word[HELD];
    int count_here = 0;
#pragma unroll
    for (int k = 0; k < HELD; k += 4) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (k < run && i0 + k < nw) x = *reinterpret_cast<const uint4*>(bits + i0 + k);
      word[k] = x.x; word[k + 1] = x.y; word[k + 2] = x.z; word[k + 3] = x.w;
      count_here += __popc(x.x) + __popc(x.y) + __popc(x.z) + __popc(x.w);
    }
    int incl = count_here;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sums[w] = incl;
    __syncthreads();
    const int of_warp = lane < WARPS ? sums[lane] : 0;
    int at = base + __reduce_add_sync(0xffffffffu, lane < w ? of_warp : 0) + incl - count_here;
    base += __reduce_add_sync(0xffffffffu, of_warp);
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      if (k >= run || i0 + k >= nw) break;
      rank[i0 + k] = static_cast<uint32_t>(at);
      for (uint32_t b = word[k]; b; b &= b - 1, ++at) {
        if (at >= a.cap) break;
        id[at] = static_cast<int>(t0) + (i0 + k) * 32 + __ffs(b) - 1;
        if (!COUNTED || at - base0 >= a.counts) seen[at] = 0;
        if (bias_at) bias_at[at] = 0;
      }
    }
    __syncthreads();
    // the place of a listed token of this window, or -1
    auto place = [&](int x) {
      const unsigned at = static_cast<unsigned>(x) - t0;
      if (at >= span) return -1;
      const uint32_t b = bits[at / 32];
      const int p = static_cast<int>(rank[at / 32]) + __popc(b & ((1u << (at % 32)) - 1u));
      return (b >> (at % 32)) & 1u && p < a.cap ? p : -1;
    };
    auto count = [&](int i, int x) {
      const int at = place(x);
      if (at < 0) return;
      int* to = COUNTED && at - base0 < a.counts ? times + (at - base0) : seen + at;
      if (i < prompt) atomicOr(to, static_cast<int>(0x80000000u));
      else atomicAdd(to, 1);
    };
#pragma unroll
    for (int k = 0; k < HELD; ++k) count(k * THREADS + tid, held[k]);
#pragma unroll 4
    for (int i = HELD * THREADS + tid; i < len; i += THREADS) count(i, history[i]);
    for (int i = tid; i < a.B; i += THREADS) {
      const int at = place(bias_ids[i]);
      if (at >= 0) atomicMax(bias_at + at, i + 1);
    }
    if constexpr (COUNTED) {
      __syncthreads();
      for (int i = tid; i < min(a.counts, base - base0); i += THREADS)
        if (base0 + i < a.cap) seen[base0 + i] = times[i];
    }
    // where tiles or parts begin
    if constexpr (STREAM) {
      for (int b = tid; b < tiles; b += THREADS) {
        const Range g = range_of(V, a.ctas, b / a.max_tiles);
        const unsigned x = b % a.max_tiles < g.tiles ? g.start(b % a.max_tiles) : g.u1 * UNIT_ROWS;
        const unsigned at = x - t0;
        if (at < span)
          a.start[r * (tiles + 1) + b] = static_cast<int>(rank[at / 32]) + __popc(bits[at / 32] & ((1u << (at % 32)) - 1u));
      }
    } else {
      for (int i = tid * (PART_COLS / 32); i < nw; i += THREADS * (PART_COLS / 32))
        a.start[static_cast<long long>((w0 + i) / (PART_COLS / 32)) * a.C + r] = static_cast<int>(rank[i]);
    }
    if (w0 + window < words) __syncthreads();
  }
  base = static_cast<int>(min(static_cast<long long>(base), a.cap));
  if constexpr (STREAM) {   // boundaries at the end of the vocabulary
    for (int b = tid; b <= tiles; b += THREADS) {
      int x = V;
      if (b < tiles) {
        const Range g = range_of(V, a.ctas, b / a.max_tiles);
        x = b % a.max_tiles < g.tiles ? g.start(b % a.max_tiles) : g.u1 * UNIT_ROWS;
      }
      if (x >= V) a.start[r * (tiles + 1) + b] = base;
    }
  } else if (tid == 0) {
    a.start[static_cast<long long>(a.nparts) * a.C + r] = base;
  }
  if (bias_at) {
    __syncthreads();
    const float* bias = a.bias + n * a.bias_stride;
    for (int i = tid; i < base; i += THREADS) {
      const int at = __ldcg(bias_at + i);
      reinterpret_cast<float*>(bias_at)[i] = at > 0 ? bias[at - 1] : 0.f;
    }
  }
}

struct RowsArgs {
  const int* hdr;
  const int* idx;
  const int* targets;
  long long c0;
  int C, nparts, K;
  const float* stats;
  const float* zt;
  float c2;
  ListView lists;
  RuleView rules;
  float *logp, *entropy, *lse;   // logp: or null
  float2* ml;
};

// 8 rows of a chunk.  Eight warps merge the parts' statistics; three warps a row
// meanwhile bring its listed logits under their rules, where they stay for the
// alternatives, and into statistics of their own.  (2048 rows of 1900 entries
// over 1002 parts 32 us, by a warp a row 62.)
constexpr int ROW_SHARES = 3;
constexpr int ROW_WARPS = ROWS8 * (1 + ROW_SHARES);
__global__ void __launch_bounds__(32 * ROW_WARPS) constrained_rows_kernel(const RowsArgs a) {
  __shared__ Stat part[32][ROWS8];
  __shared__ Stat share[1 + ROW_SHARES][ROWS8];
  __shared__ int hits[ROW_SHARES][ROWS8];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, k = w % ROWS8;
  ptx::grid_dependency_wait();
  const int Cl = chunk_rows(a.hdr, a.c0, a.C);
  const int r0 = blockIdx.x * ROWS8;
  if (r0 >= Cl) return;
  const long long r = r0 + k, at = r * a.lists.cap;
  const bool valid = r < Cl;
  const long long row = valid ? a.idx[a.c0 + r] : 0;
  const int t = a.targets ? a.targets[row] : 0;
  if (w < ROWS8) {
    const Stat s = merge_parts8<true>(a.stats, a.nparts, a.C, a.c2, r0, Cl, lane, w, part);
    if (lane == 0) share[0][w] = s;
  } else {
    const int sub = w / ROWS8 - 1;
    const RowRules rules = row_rules(a.rules, row);
    const int n = valid ? static_cast<int>(min(
        a.lists.cap, static_cast<long long>(a.lists.start[static_cast<long long>(a.nparts) * a.C + r]))) : 0;
    float m = -INFINITY;
    int hit = -1;
#pragma unroll 4
    for (int e = sub * 32 + lane; e < n; e += 32 * ROW_SHARES) {
      const float z = ruled(a.lists.z[at + e], a.rules.seen[at + e], a.rules.bias ? a.rules.bias[at + e] : 0.f, rules);
      a.lists.z[at + e] = z;
      if (a.lists.id[at + e] == t) hit = e;
      m = fmaxf(m, z);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    hit = __reduce_max_sync(0xffffffffu, hit);
    Stat mine = {m, 0.f, 0.f};
#pragma unroll 4
    for (int e = sub * 32 + lane; e < n; e += 32 * ROW_SHARES) {   // what this lane has written
      const float z = a.lists.z[at + e], y = (z - m) * a.c2;
      const float x = z == -INFINITY ? 0.f : ptx::ex2(y);          // (where all are -inf, y is not a number)
      mine.s += x;
      mine.d = fmaf(fmaxf(y, -1e30f), x, mine.d);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {   // fixed order
      mine.s += __shfl_xor_sync(0xffffffffu, mine.s, o);
      mine.d += __shfl_xor_sync(0xffffffffu, mine.d, o);
    }
    if (lane == 0) {
      share[1 + sub][k] = mine;
      hits[sub][k] = hit;
    }
  }
  __syncthreads();
  if (w >= ROWS8 || !valid || lane != 0) return;
  float zt = a.zt[r];
  if (a.lists.mask && !((a.lists.mask[row * a.lists.mask_stride + t / 32] >> (t % 32)) & 1u)) zt = -INFINITY;
  Stat acc = share[0][k];
#pragma unroll
  for (int i = 0; i < ROW_SHARES; ++i) {
    acc = merge(acc, share[1 + i][k], a.c2);
    if (hits[i][k] >= 0) zt = a.lists.z[at + hits[i][k]];
  }
  if (a.hdr[HDR_STATUS] & STATUS_TIMEOUT) acc.m = acc.s = __int_as_float(0x7fc00000);
  const float l2s = log2f(acc.s);
  const bool nan = acc.s != acc.s, nothing = acc.m == -INFINITY && acc.s == 0.f;
  if (a.logp) a.logp[row] = zt == -INFINITY && !nan ? -INFINITY : fmaf(zt - acc.m, a.c2, -l2s) * LN2;
  a.lse[row] = nothing ? -INFINITY : fmaf(acc.m, a.c2, l2s) * LN2;
  if (a.entropy) a.entropy[row] = nothing ? 0.f : fmaf(0.f, acc.m, l2s - acc.d / acc.s) * LN2;
  if (a.K > 0) a.ml[r] = make_float2(acc.m, l2s);
}

struct TopArgs {
  const int* hdr;
  const int* idx;
  long long c0;
  int C, V, nparts, K;
  long long ldz;
  const float *stats, *zf;
  const float2* ml;
  float c2;
  ListView lists;
  int* top_ids;
  float* top_logp;
};

// Top alternatives of one row per block: the best of the logits behind the
// list, then the listed ones are offered too.
__global__ void __launch_bounds__(32 * TOP_WARPS) constrained_top_kernel(const TopArgs a) {
  __shared__ float sv[TOP_WARPS][32];
  __shared__ int si[TOP_WARPS][32];
  const int r = blockIdx.x;
  ptx::grid_dependency_wait();
  if (r >= chunk_rows(a.hdr, a.c0, a.C)) return;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const long long row = a.idx[a.c0 + r];
  if (a.hdr[HDR_STATUS] & STATUS_TIMEOUT) {   // uniform over the grid
    if (static_cast<int>(threadIdx.x) < a.K) {
      a.top_ids[row * a.K + threadIdx.x] = -1;
      a.top_logp[row * a.K + threadIdx.x] = __int_as_float(0x7fc00000);
    }
    return;
  }
  TopK best = top_of_parts(a.stats, a.zf + static_cast<size_t>(r) * a.ldz, a.nparts, a.C, a.V, a.K, r, lane, w, sv, si);
  const int n = static_cast<int>(min(a.lists.cap, static_cast<long long>(a.lists.start[static_cast<long long>(a.nparts) * a.C + r])));
  const long long at = r * a.lists.cap;
  // Each warp's own share of the list (from empty, since the best so far are in every warp); what is below the K-th of
  // those is not among the K best.
  const float least = __shfl_sync(0xffffffffu, best.v, a.K - 1);
  TopK mine;
  mine.clear();
  for (int e0 = w * 32; e0 < n; e0 += TOP_BATCH * TOP_WARPS * 32) {
    float x[TOP_BATCH];
    int id[TOP_BATCH];
#pragma unroll
    for (int k = 0; k < TOP_BATCH; ++k) {
      const int e = e0 + k * (TOP_WARPS * 32) + lane;
      x[k] = e < n ? a.lists.z[at + e] : 0.f;
      id[k] = e < n && x[k] >= least ? a.lists.id[at + e] : TopK::NONE;
    }
    mine.offer_all(x, id, a.K, lane);
  }
  mine.merge_block<TOP_WARPS>(sv, si, lane, w);
  best.merge(mine.v, mine.id, lane);
  if (w == 0 && lane < a.K) {
    const bool some = best.id != TopK::NONE && best.v > -INFINITY;   // forbidden tokens are no alternatives
    const float2 ml = a.ml[r];
    a.top_ids[row * a.K + lane] = some ? best.id : -1;
    a.top_logp[row * a.K + lane] =
        some ? fmaf(best.v - ml.x, a.c2, -ml.y) * LN2 : (ml.y == ml.y ? -INFINITY : __int_as_float(0x7fc00000));
  }
}

// Calls of several chunks: the rows left out, and after a time-out in any chunk
// every row.
__global__ void __launch_bounds__(256)
    constrained_left_kernel(const int* hdr, long long N, int K, const int* targets, int ii, int V, float* logp,
                            float* entropy, float* lse, int* top_ids, float* top_logp) {
  ptx::grid_dependency_wait();
  const bool failed = hdr[HDR_STATUS] & STATUS_TIMEOUT;
  for (long long row = blockIdx.x * 256ll + threadIdx.x; row < N; row += gridDim.x * 256ll) {
    const int t = targets[row];
    const bool left = t == ii;
    if (!left && !failed && t >= 0 && t < V) continue;
    const float v = left ? 0.f : __int_as_float(0x7fc00000);
    if (logp) logp[row] = v;
    lse[row] = v;
    if (entropy) entropy[row] = v;
    for (int k = 0; k < K; ++k) {
      top_ids[row * K + k] = -1;
      top_logp[row * K + k] = v;
    }
  }
}

__global__ void __launch_bounds__(256) all_rows_kernel(int* targets, long long N) {
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < N; i += gridDim.x * 256ll) targets[i] = 0;
}

// Histories of LONG_HISTORY ids and more have their times counted in shared
// memory, for the first MAX_COUNTS listed tokens of a window; the others' go to L2.
// Calls at H = 64, ids of a Zipf distribution, in L2 and in shared memory, us:
//   rows x vocabulary   300 ids       1280          4000          16000
//   1 x 4000            21.6   18.6   22.7   19.6   25.1   23.7   36.0   33.9
//   1 x 128256          25.7   25.7   25.7   25.7   27.7   27.7   42.1   35.9
//   128 x 128256        72.8   72.8   81.0   83.0   87.2   85.1   108.6  96.4
//   300 x 16000         32.9   33.9   41.1   41.1   58.5   52.3   121.9  93.3
//   2048 x 4000         48.2   48.3   74.8   66.7   146.7  111.7  287.9  194.7
//   2048 x 16000        87.1   91.2   111.8  113.8  181.4  156.8  318.6  222.3
//   2048 x 128256       260.2  263.3  320.6  323.7  418.9  400.5  539.7  443.5
// Around the border both are within 3% of each other but for few rows at a very small
// vocabulary (1 x 753: 25.7 and 27.8 at 1280, 37.0 and 36.0 at 16000).  Two kernels,
// as one with the choice at run time costs short histories as much.
constexpr int MAX_COUNTS = 8192, LONG_HISTORY = 1280;
// Ids (of history and biases) times windows up to which the streaming kernel comes
// up while the lists are made: its waits, which are limited, then last as long as
// that takes, 0.8 to 1.2 ns an id and window (1.2 ms here).  Side by side saves 4 to
// 16 us: 64 ids at 512 x 600000 128 us, one after the other 144; 2^18 ids 781 and
// 785, 2^20 2422 and 2426.
constexpr long long LISTS_BESIDE = 1ll << 20;
size_t rule_smem(long long V, int threads, int counts) {
  return size_t(pad_words(static_cast<int>(std::min<long long>(cdiv(V, 32), HELD * threads)))) * 8 + size_t(counts) * 4;
}

// Entries of a row at most.
long long list_cap(long long V, long long L, long long B) { return std::max(1ll, std::min(V, L + B)); }

struct ConstrainedStream {
  int ctas, max_tiles;
  long long ldz;
  size_t o_zt, o_stat, o_max, o_group, o_zf, o_start, o_id, o_seen, o_bias, o_fail, total;
};

ConstrainedStream constrained_stream_plan(long long N, long long V, int K, long long L, long long B, int sms) {
  ConstrainedStream p;
  p.ctas = stream_ctas(V, sms);
  p.max_tiles = stream_max_tiles(V, p.ctas);
  p.ldz = cdiv(V, 32) * 32;
  size_t off = al256(HDR_WORDS * sizeof(int));
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += al256(bytes);
    return o;
  };
  const size_t cap = static_cast<size_t>(list_cap(V, L, B));
  p.o_zt = take(size_t(N) * 4);
  p.o_stat = take(size_t(N) * p.ctas * 16);
  p.o_max = take(K > 0 ? size_t(N) * p.ctas * p.max_tiles * 4 : 0);
  p.o_group = take(K > 0 ? size_t(N) * TopK::MAX * 4 : 0);
  p.o_zf = take(K > 0 ? size_t(N) * p.ldz * 4 : 0);
  p.o_start = take(size_t(N) * (p.ctas * p.max_tiles + 1) * 4);
  p.o_id = take(size_t(N) * cap * 4);
  p.o_seen = take(size_t(N) * cap * 4);
  p.o_bias = take(B > 0 ? size_t(N) * cap * 4 : 0);
  p.o_fail = take(size_t(p.ctas) * 4);
  p.total = off;
  return p;
}

ListedSizes constrained_sizes(long long N, long long H, long long V, int K, long long L, long long B) {
  const long long cap = list_cap(V, L, B);
  return ListedSizes{N, H, V, K, cap, cap * (B > 0 ? 8 : 4), 4, cap};   // seen, biases
}

bool sizes_bad(int64_t N, int64_t H, int64_t V) { return !sizes_ok(N, H, V) || V > PROBS_MAX_V; }

// An index and a block's stride stay in 32 bits.
constexpr long long MAX_HISTORY = 1ll << 30, MAX_BIASES = 1ll << 20;

}  // namespace

cudaError_t constrained_prepare() {
  cudaError_t e = cudaSuccess;
  auto allow = [&](auto* kernel, size_t bytes) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  };
  allow(constrained_lists_kernel<true, STREAM_THREADS, false>, HELD * STREAM_THREADS * 8);
  allow(constrained_lists_kernel<true, STREAM_THREADS, true>, HELD * STREAM_THREADS * 8 + MAX_COUNTS * 4);
  allow(constrained_lists_kernel<false, CHUNK_THREADS, true>, HELD * CHUNK_THREADS * 8 + MAX_COUNTS * 4);
  return e;
}

}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_constrained_workspace_bytes(int64_t N, int64_t H, int64_t V, int32_t top_k, int64_t history, int64_t biases) {
  if (sizes_bad(N, H, V) || top_k < 0 || top_k > TopK::MAX || top_k > V || history < 0 || history > MAX_HISTORY ||
      biases < 0 || biases > MAX_BIASES)
    return 0;
  if (N <= STREAM_MAX_TOKENS) return constrained_stream_plan(N, V, top_k, history, biases, device_sms()).total;
  return listed_default_bytes(constrained_sizes(N, H, V, top_k, history, biases));
}

flce_status flce_constrained_logprobs(const void* hidden, const void* weight, const int32_t* targets, int64_t N,
                                      int64_t H, int64_t V, int32_t ignore_index, float temperature, int32_t top_k,
                                      const flce_constraints* rules, float* logp, float* entropy, float* lse,
                                      int32_t* top_ids, float* top_logp, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (!hidden || !weight || !rules || !lse || !workspace || (targets && !logp)) return FLCE_EINVAL;
  const flce_constraints& c = *rules;
  if (N < 1 || H < 1 || V < 1 || top_k < 0 || top_k > V || bad_temperature(temperature)) return FLCE_EINVAL;
  if (top_k > 0 && (!top_ids || !top_logp)) return FLCE_EINVAL;
  if (c.history_len < 0 || (c.history_len > 0 && !c.history) || c.history_stride < 0 || c.n_bias < 0 ||
      (c.n_bias > 0 && (!c.bias_ids || !c.bias)) || c.bias_ids_stride < 0 || c.bias_stride < 0 || c.mask_stride < 0)
    return FLCE_EINVAL;
  if (sizes_bad(N, H, V) || top_k > TopK::MAX || c.history_len > MAX_HISTORY || c.n_bias > MAX_BIASES) return FLCE_EUNSUPPORTED;
  if (!aligned16(hidden) || !aligned16(weight) || !aligned16(workspace) || !aligned4(targets) || !aligned4(logp) ||
      !aligned4(entropy) || !aligned4(lse) || !aligned4(top_ids) || !aligned4(top_logp) || !aligned4(c.history) ||
      !aligned4(c.history_lens) || !aligned4(c.prompt_lens) || !aligned4(c.repetition_penalty) ||
      !aligned4(c.frequency_penalty) || !aligned4(c.presence_penalty) || !aligned4(c.bias_ids) || !aligned4(c.bias) ||
      !aligned4(c.mask))
    return FLCE_EUNSUPPORTED;
  if (top_k > 0 && N > STREAM_MAX_TOKENS && !aligned32(workspace)) return FLCE_EUNSUPPORTED;
  DeviceState dev;
  if (device_state(&dev) != cudaSuccess) { cudaGetLastError(); return FLCE_ECUDA; }
  if (dev.major < 10) return FLCE_EUNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto ok = [](cudaError_t e) { return e == cudaSuccess; };
  if (!targets) logp = nullptr;
  const long long L = c.history_len, B = c.n_bias;
  RuleArgs la;
  std::memset(&la, 0, sizeof(la));
  la.V = static_cast<int>(V);
  la.history = c.history; la.L = L; la.history_stride = c.history_stride;
  la.history_lens = c.history_lens; la.prompt_lens = c.prompt_lens;
  la.bias_ids = c.bias_ids; la.bias = c.bias; la.B = static_cast<int>(B);
  la.bias_ids_stride = c.bias_ids_stride; la.bias_stride = c.bias_stride;
  la.mask = reinterpret_cast<const uint32_t*>(c.mask); la.mask_stride = c.mask_stride;
  la.cap = list_cap(V, L, B);
  la.counts = static_cast<int>(std::min<long long>(L >= LONG_HISTORY ? la.cap : 0, MAX_COUNTS));
  RuleView rv;
  rv.repetition = c.repetition_penalty; rv.frequency = c.frequency_penalty; rv.presence = c.presence_penalty;
  if (N <= STREAM_MAX_TOKENS) {
    const ConstrainedStream p = constrained_stream_plan(N, V, top_k, L, B, dev.sms);
    if (p.total > workspace_bytes) return FLCE_EWORKSPACE;
    StreamArgs a;
    StreamLists l;
    StreamMaps m;
    std::memset(&a, 0, sizeof(a));
    std::memset(&l, 0, sizeof(l));
    a.N = static_cast<int>(N); a.H = static_cast<int>(H); a.V = static_cast<int>(V); a.K = top_k;
    a.ctas = p.ctas; a.max_tiles = p.max_tiles;
    a.c2 = LOG2E / temperature;
    a.ii = ignore_index;
    a.targets = targets;
    a.hdr = at<int>(workspace, 0);
    a.zt = at<float>(workspace, p.o_zt);
    a.stat = at<float4>(workspace, p.o_stat);
    a.zf = at<float>(workspace, p.o_zf);
    a.ldz = p.ldz;
    a.tile_max = at<float>(workspace, p.o_max);
    a.group_max = top_k > 0 && p.max_tiles > 1 ? at<uint32_t>(workspace, p.o_group) : nullptr;
    a.fail = at<int>(workspace, p.o_fail);
    a.logp = logp; a.entropy = entropy; a.lse = lse; a.top_ids = top_ids; a.top_logp = top_logp;
    la.ctas = p.ctas; la.max_tiles = p.max_tiles; la.group_max = a.group_max;
    l.lists.start = la.start = at<int>(workspace, p.o_start);
    l.lists.boundaries = p.ctas * p.max_tiles + 1;
    l.lists.id = la.id = at<int>(workspace, p.o_id);
    l.lists.cap = la.cap;
    l.lists.mask = la.mask; l.lists.mask_stride = la.mask_stride;
    rv.seen = la.seen = at<int>(workspace, p.o_seen);
    la.bias_at = B > 0 ? at<int>(workspace, p.o_bias) : nullptr;
    rv.bias = reinterpret_cast<const float*>(la.bias_at);
    l.rules = rv;
    if (!stream_setup(&a, &m, hidden, weight, segment_blocks(H))) return FLCE_ECUDA;
    count_launches(2);   // lists, the merge
    auto* const lists =
        la.counts > 0 ? constrained_lists_kernel<true, STREAM_THREADS, true> : constrained_lists_kernel<true, STREAM_THREADS, false>;
    lists<<<static_cast<unsigned>(N), STREAM_THREADS, rule_smem(V, STREAM_THREADS, la.counts), st>>>(la);
    if (!ok(launch_result(cudaGetLastError()))) return FLCE_ECUDA;
    const ProfScope prof = prof_launch_begin(st);
    const long long windows = cdiv(cdiv(V, 32), HELD * STREAM_THREADS);
    const cudaError_t e = launch_stream_ruled(a, m, l, (L + B) * windows <= LISTS_BESIDE, st);
    prof_launch_end(prof, MODE_STATS, st);
    return ok(e) ? FLCE_OK : FLCE_ECUDA;
  }
  ListedPlan p;
  ListedCall k;
  std::memset(&k, 0, sizeof(k));
  k.q = constrained_sizes(N, H, V, top_k, L, B);
  if (!listed_plan(k.q, workspace_bytes, &p)) return FLCE_EWORKSPACE;
  if (!targets) ignore_index = -1;
  if (!targets && !listed_front(p, N)) {   // the loss's compaction reads targets
    int* all = at<int>(workspace, p.o_targets);
    count_launches(1);
    all_rows_kernel<<<static_cast<unsigned>(std::min<long long>(cdiv(N, 256), 152)), 256, 0, st>>>(all, N);
    if (!ok(launch_result(cudaGetLastError()))) return FLCE_ECUDA;
    targets = all;
  }
  k.hidden = hidden; k.weight = weight; k.targets = targets; k.ii = ignore_index; k.temperature = temperature;
  k.mask = la.mask; k.mask_stride = la.mask_stride;
  k.logp = logp ? logp : lse; k.entropy = entropy; k.lse = lse; k.top_ids = top_ids; k.top_logp = top_logp;
  k.seg_kb = segment_blocks(H);
  k.ws = workspace; k.st = st;
  rv.seen = la.seen = at<int>(workspace, p.o_rows);
  la.bias_at = B > 0 ? la.seen + p.C * la.cap : nullptr;
  rv.bias = reinterpret_cast<const float*>(la.bias_at);
  const flce_status s = listed_chunks(
      p, k, dev,
      [&](const ListedChunk& ch) {
        la.hdr = ch.g->hdr; la.idx = ch.g->idx; la.c0 = ch.c0; la.C = ch.g->C; la.nparts = ch.g->nparts;
        la.start = const_cast<int*>(ch.g->lists.start);
        la.id = const_cast<int*>(ch.g->lists.id);
        count_launches(1);
        const bool small = V <= SMALL_VOCABULARY && L + B <= SMALL_HISTORY, counted = la.counts > 0;
        const unsigned threads = small ? SMALL_THREADS : CHUNK_THREADS;
        auto* const lists = small ? counted ? constrained_lists_kernel<false, SMALL_THREADS, true>
                                            : constrained_lists_kernel<false, SMALL_THREADS, false>
                                  : counted ? constrained_lists_kernel<false, CHUNK_THREADS, true>
                                            : constrained_lists_kernel<false, CHUNK_THREADS, false>;
        return launch_dependent_smem(lists, static_cast<unsigned>(la.C), threads, rule_smem(V, static_cast<int>(threads), la.counts),
                                     st, la);
      },
      [&](const ListedChunk& ch) {
        float2* ml = at<float2>(workspace, p.o_ml);
        const RowsArgs ra{ch.g->hdr, ch.g->idx, targets, ch.c0, ch.g->C, ch.g->nparts, top_k, ch.g->stats, ch.g->zt,
                          ch.g->c2, ch.g->lists, rv, logp, entropy, lse, ml};
        count_launches(top_k > 0 ? 2 : 1);
        const cudaError_t e = launch_dependent(constrained_rows_kernel, static_cast<unsigned>(cdiv(ch.g->C, ROWS8)),
                                               32 * ROW_WARPS, st, ra);
        if (e != cudaSuccess || top_k == 0) return e;
        const TopArgs ta{ch.g->hdr, ch.g->idx, ch.c0, ch.g->C, ch.g->V, ch.g->nparts, top_k, p.ldz, ch.g->stats,
                         ch.g->zf, ml, ch.g->c2, ch.g->lists, top_ids, top_logp};
        return launch_dependent(constrained_top_kernel, static_cast<unsigned>(ch.g->C), 32 * TOP_WARPS, st, ta);
      });
  if (s == FLCE_OK && (p.n_chunks > 1 || N > FRONT_MAX_TOKENS)) {
    count_launches(1);
    if (!ok(launch_dependent(constrained_left_kernel, 152, 256, st, at<int>(workspace, 0), N, top_k, targets, ignore_index,
                             static_cast<int>(V), logp, entropy, lse, top_ids, top_logp)))
      return FLCE_ECUDA;
  }
  return s;
}

}  // extern "C"
