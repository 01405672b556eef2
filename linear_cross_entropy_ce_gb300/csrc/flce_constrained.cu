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

constexpr int RULE_THREADS = 512;
constexpr int RULE_WARPS = RULE_THREADS / 32;
constexpr int WINDOW_WORDS = 24576;   // of the vocabulary at a time: 786432 tokens, 192 KB with the words' ranks
static_assert(WINDOW_WORDS * 32 % PART_COLS == 0, "windows end between parts");

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
};

// A block per row.  (57 ids at a vocabulary of 128256: see the streaming kernel,
// which runs meanwhile.)
template <bool STREAM>
__global__ void __launch_bounds__(RULE_THREADS) constrained_lists_kernel(const RuleArgs a) {
  extern __shared__ uint32_t bits[];   // [window words] and their ranks
  __shared__ int warp_sum[RULE_WARPS];
  const int tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  const int words = (a.V + 31) / 32, window = min(words, WINDOW_WORDS);
  uint32_t* rank = bits + window;
  long long r = blockIdx.x, n = blockIdx.x;
  if constexpr (STREAM) {
    ptx::grid_launch_dependents();
    if (a.group_max && tid < TopK::MAX) a.group_max[n * TopK::MAX + tid] = 0u;
  } else {
    ptx::grid_dependency_wait();
    if (r >= chunk_rows(a.hdr, a.c0, a.C)) return;
    n = a.idx[a.c0 + r];
  }
  const int* history = a.history + n * a.history_stride;
  long long len = a.L, prompt = 0;
  if (a.history_lens) len = max(0ll, min(a.L, static_cast<long long>(a.history_lens[n])));
  if (a.prompt_lens) prompt = a.prompt_lens[n];
  const int* bias_ids = a.bias_ids + n * a.bias_ids_stride;
  int* id = a.id + r * a.cap;
  int* seen = a.seen + r * a.cap;
  int* bias_at = a.bias_at ? a.bias_at + r * a.cap : nullptr;
  const int tiles = STREAM ? a.ctas * a.max_tiles : 0;
  int base = 0;   // listed tokens before this window
  for (int w0 = 0; w0 < words; w0 += window) {
    const int nw = min(window, words - w0);
    const long long t0 = static_cast<long long>(w0) * 32, t1 = min(static_cast<long long>(a.V), t0 + nw * 32ll);
    for (int i = tid; i < nw; i += RULE_THREADS) bits[i] = 0u;
    __syncthreads();
    auto mark = [&](int x) {
      if (x >= t0 && x < t1) atomicOr(bits + (x - t0) / 32, 1u << (x % 32));
    };
#pragma unroll 4
    for (long long i = tid; i < len; i += RULE_THREADS) mark(history[i]);
    for (int i = tid; i < a.B; i += RULE_THREADS) mark(bias_ids[i]);
    __syncthreads();
    // forbidden tokens leave; the words' ranks, a run of words per thread
    const int each = (nw + RULE_THREADS - 1) / RULE_THREADS;
    const int i0 = min(nw, tid * each), i1 = min(nw, i0 + each);
    int sum = 0;
    for (int i = i0; i < i1; ++i) {
      uint32_t b = bits[i];
      if (b != 0u && a.mask) bits[i] = b &= a.mask[n * a.mask_stride + w0 + i];
      sum += __popc(b);
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[w] = incl;
    __syncthreads();
    int before = base + incl - sum, total = 0;
#pragma unroll
    for (int k = 0; k < RULE_WARPS; ++k) {
      if (k < w) before += warp_sum[k];
      total += warp_sum[k];
    }
    for (int i = i0; i < i1; ++i) {
      rank[i] = static_cast<uint32_t>(before);
      uint32_t b = bits[i];
      while (b) {
        const int k = __ffs(b) - 1;
        b &= b - 1;
        if (before < a.cap) {
          id[before] = static_cast<int>(t0) + i * 32 + k;
          seen[before] = 0;
          if (bias_at) bias_at[before] = 0;
        }
        ++before;
      }
    }
    __syncthreads();
    // the place of a listed token, or -1
    auto place = [&](int x) {
      if (x < t0 || x >= t1) return -1;
      const int i = static_cast<int>(x - t0) / 32;
      const uint32_t b = bits[i], below = (1u << (x % 32)) - 1u;
      const int at = static_cast<int>(rank[i]) + __popc(b & below);
      return (b >> (x % 32)) & 1u && at < a.cap ? at : -1;
    };
#pragma unroll 4
    for (long long i = tid; i < len; i += RULE_THREADS) {
      const int at = place(history[i]);
      if (at < 0) continue;
      if (i < prompt) atomicOr(seen + at, static_cast<int>(0x80000000u));
      else atomicAdd(seen + at, 1);
    }
    for (int i = tid; i < a.B; i += RULE_THREADS) {
      const int at = place(bias_ids[i]);
      if (at >= 0) atomicMax(bias_at + at, i + 1);
    }
    // where tiles or parts begin
    if constexpr (STREAM) {
      for (int b = tid; b < tiles; b += RULE_THREADS) {
        const Range g = range_of(a.V, a.ctas, b / a.max_tiles);
        const int x = b % a.max_tiles < g.tiles ? g.start(b % a.max_tiles) : g.u1 * UNIT_ROWS;
        if (x >= t0 && x < t1) {
          const int i = static_cast<int>(x - t0) / 32;
          a.start[r * (tiles + 1) + b] = static_cast<int>(rank[i]) + __popc(bits[i] & ((1u << (x % 32)) - 1u));
        }
      }
    } else {
      for (int p = w0 / (PART_COLS / 32) + tid; p < a.nparts && p * static_cast<long long>(PART_COLS) < t1; p += RULE_THREADS)
        a.start[static_cast<long long>(p) * a.C + r] = static_cast<int>(rank[p * (PART_COLS / 32) - w0]);
    }
    base += total;
    __syncthreads();
  }
  base = static_cast<int>(min(static_cast<long long>(base), a.cap));
  if constexpr (STREAM) {
    for (int b = tid; b <= tiles; b += RULE_THREADS) {
      int x = a.V;
      if (b < tiles) {
        const Range g = range_of(a.V, a.ctas, b / a.max_tiles);
        x = b % a.max_tiles < g.tiles ? g.start(b % a.max_tiles) : g.u1 * UNIT_ROWS;
      }
      if (x >= a.V) a.start[r * (tiles + 1) + b] = base;
    }
  } else if (tid == 0) {
    a.start[static_cast<long long>(a.nparts) * a.C + r] = base;
  }
  if (bias_at) {
    const float* bias = a.bias + n * a.bias_stride;
    for (int i = tid; i < base; i += RULE_THREADS) {
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

// 32 rows of a chunk: the parts' statistics merged with a lane a row, then a
// warp a row brings the listed logits in, under their rules, and leaves them so
// for the alternatives.
__global__ void __launch_bounds__(32 * ROWS_WARPS) constrained_rows_kernel(const RowsArgs a) {
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
  const int t = a.targets[row];
  const RowRules rules = row_rules(a.rules, row);
  const int n = static_cast<int>(min(a.lists.cap, static_cast<long long>(a.lists.start[static_cast<long long>(a.nparts) * a.C + r])));
  float zt = a.zt[r];
  if (a.lists.mask && !((a.lists.mask[row * a.lists.mask_stride + t / 32] >> (t % 32)) & 1u)) zt = -INFINITY;
  Stat mine = {-INFINITY, 0.f, 0.f};
  const long long at = r * a.lists.cap;
  for (int e0 = 0; e0 < n; e0 += 32) {
    const int e = e0 + lane;
    float z = -INFINITY;
    bool hit = false;
    if (e < n) {
      z = ruled(a.lists.z[at + e], a.rules.seen[at + e], a.rules.bias ? a.rules.bias[at + e] : 0.f, rules);
      a.lists.z[at + e] = z;
      hit = a.lists.id[at + e] == t;
      mine = merge(mine, Stat{z, z != z ? z : (z > -INFINITY ? 1.f : 0.f), 0.f}, a.c2);
    }
    const unsigned found = __ballot_sync(0xffffffffu, hit);
    if (found) zt = __shfl_sync(0xffffffffu, z, __ffs(found) - 1);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {   // fixed order; lane 0 holds the result
    const Stat other = {__shfl_down_sync(0xffffffffu, mine.m, o), __shfl_down_sync(0xffffffffu, mine.s, o),
                        __shfl_down_sync(0xffffffffu, mine.d, o)};
    mine = merge(mine, other, a.c2);
  }
  if (lane != 0) return;
  Stat acc = merge(part[0][w], mine, a.c2);
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
  // Each warp's own share of the list (from empty, since the list before is in every warp)
  TopK mine;
  mine.clear();
  for (int e0 = w * 32; e0 < n; e0 += TOP_BATCH * TOP_WARPS * 32) {
    float x[TOP_BATCH];
    int id[TOP_BATCH];
#pragma unroll
    for (int k = 0; k < TOP_BATCH; ++k) {
      const int e = e0 + k * (TOP_WARPS * 32) + lane;
      x[k] = e < n ? a.lists.z[at + e] : 0.f;
      id[k] = e < n ? a.lists.id[at + e] : TopK::NONE;
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

size_t rule_smem(long long V) { return size_t(std::min<long long>(cdiv(V, 32), WINDOW_WORDS)) * 8; }

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
  return ListedSizes{N, H, V, K, cap, cap * (B > 0 ? 8 : 4), 0};   // seen, biases
}

bool sizes_bad(int64_t N, int64_t H, int64_t V) { return !sizes_ok(N, H, V) || V > PROBS_MAX_V; }

constexpr long long MAX_LIST = (1ll << 31) - 1;

}  // namespace

cudaError_t constrained_prepare() {
  const int most = WINDOW_WORDS * 8;
  cudaError_t e = cudaFuncSetAttribute(constrained_lists_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(constrained_lists_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_constrained_workspace_bytes(int64_t N, int64_t H, int64_t V, int32_t top_k, int64_t history, int64_t biases) {
  if (sizes_bad(N, H, V) || top_k < 0 || top_k > TopK::MAX || top_k > V || history < 0 || history > MAX_LIST ||
      biases < 0 || biases > MAX_LIST)
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
  if (sizes_bad(N, H, V) || top_k > TopK::MAX || c.history_len > MAX_LIST || c.n_bias > MAX_LIST) return FLCE_EUNSUPPORTED;
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
    if (!stream_setup(&a, &m, hidden, weight)) return FLCE_ECUDA;
    count_launches(2);   // lists, the merge
    constrained_lists_kernel<true><<<static_cast<unsigned>(N), RULE_THREADS, rule_smem(V), st>>>(la);
    if (!ok(launch_result(cudaGetLastError()))) return FLCE_ECUDA;
    const ProfScope prof = prof_launch_begin(st);
    const cudaError_t e = launch_stream_ruled(a, m, l, st);
    prof_launch_end(prof, MODE_STATS, st);
    return ok(e) ? FLCE_OK : FLCE_ECUDA;
  }
  ListedPlan p;
  ListedCall k;
  std::memset(&k, 0, sizeof(k));
  k.q = constrained_sizes(N, H, V, top_k, L, B);
  if (!listed_plan(k.q, workspace_bytes, &p)) return FLCE_EWORKSPACE;
  if (!targets) {
    int* all = at<int>(workspace, p.o_targets);
    count_launches(1);
    all_rows_kernel<<<static_cast<unsigned>(std::min<long long>(cdiv(N, 256), 152)), 256, 0, st>>>(all, N);
    if (!ok(launch_result(cudaGetLastError()))) return FLCE_ECUDA;
    targets = all;
    ignore_index = -1;
  }
  k.hidden = hidden; k.weight = weight; k.targets = targets; k.ii = ignore_index; k.temperature = temperature;
  k.mask = la.mask; k.mask_stride = la.mask_stride;
  k.logp = logp ? logp : lse; k.entropy = entropy; k.lse = lse; k.top_ids = top_ids; k.top_logp = top_logp;
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
        return launch_dependent_smem(constrained_lists_kernel<false>, static_cast<unsigned>(la.C), RULE_THREADS,
                                     rule_smem(V), st, la);
      },
      [&](const ListedChunk& ch) {
        float2* ml = at<float2>(workspace, p.o_ml);
        const RowsArgs ra{ch.g->hdr, ch.g->idx, targets, ch.c0, ch.g->C, ch.g->nparts, top_k, ch.g->stats, ch.g->zt,
                          ch.g->c2, ch.g->lists, rv, logp, entropy, lse, ml};
        count_launches(top_k > 0 ? 2 : 1);
        const cudaError_t e = launch_dependent(constrained_rows_kernel, static_cast<unsigned>(cdiv(ch.g->C, 32)),
                                               32 * ROWS_WARPS, st, ra);
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
