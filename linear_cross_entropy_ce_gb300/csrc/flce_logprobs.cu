// Token log probabilities at the LM head, with entropy and top alternatives, in
// chunks of tokens: of a chunk's logits only statistics are kept, and with top
// alternatives those that may be among them (in fp32, in room for all: a chunk's
// logits fit in the workspace, and so do all of a small problem's).
//
//   z = X W^T / T,   lse_n = log sum_v exp z_nv,   logp_n = z_{n,t_n} - lse_n,
//   H_n = -sum_v p_nv log p_nv = lse_n - sum_v p_nv z_nv,   p = exp(z - lse),
//   and the K largest z_nv with their ids (equal values: the lowest id first).
//
// The tcgen05 GEMM (MODE_STATS) leaves per row and 128-column part the max m,
// S = sum 2^d and D = sum d 2^d of d = (z - m) c2, c2 = log2(e)/T.  Two parts
// merge at the larger max M with f = 2^((m - M) c2):
//   S <- f S,   D <- f (D + (m - M) c2 S)      (d grows by (m - M) c2)
// so that log2 sum = M c2 + log2 S and H = ln 2 (log2 S - D / S).
//
// Top alternatives: every one of a row's K best logits lies in one of its K
// best parts (parts ordered by their max, equal ones by position: K better
// parts each hold a better logit, an equal one having a lower id), so of the
// fp32 logits of a chunk only K parts of 128 columns are read back per row.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "flce.h"
#include "flce_internal.h"
#include "flce_ptx.cuh"
#include "flce_softmax.cuh"
#include "flce_topk.cuh"

namespace flce {
namespace {

__device__ __forceinline__ int chunk_rows(const int* hdr, long long c0, int C) {
  const long long rem = static_cast<long long>(hdr[HDR_NVALID]) - c0;
  return rem <= 0 ? 0 : (rem >= C ? C : static_cast<int>(rem));
}

// The constants of MODE_DZ of token n (see DzRow).
__device__ __forceinline__ DzRow dz_row(float temperature, float lse, const float* entropy, const float* grad_logp,
                                        const float* grad_entropy, long long n) {
  const float it = 1.f / temperature;
  const float g = grad_logp ? grad_logp[n] : 0.f;
  const float e = grad_entropy ? grad_entropy[n] : 0.f;
  return DzRow{lse * LOG2E, -it * (grad_entropy ? fmaf(e, entropy[n], g) : g), -it * LN2 * e, it * g};
}

// (Calls of several chunks.)  Chunk rows and their targets in a dense [C, H] tile source (rows up to the
// next multiple of 128 are zero), with the constants of MODE_DZ:
//   dz = (g ([v = t] - p) - e p (log p + H)) / T.
__global__ void __launch_bounds__(128)
    gather_dz_kernel(const uint16_t* __restrict__ X, const int* __restrict__ t, const int* hdr,
                     const int* __restrict__ idx, long long c0, int C, int H, float temperature,
                     const float* __restrict__ lse, const float* __restrict__ entropy,
                     const float* __restrict__ grad_logp, const float* __restrict__ grad_entropy,
                     uint16_t* __restrict__ xc, int* __restrict__ tc, DzRow* __restrict__ rowc) {
  const int r = blockIdx.x;
  const int Cl = chunk_rows(hdr, c0, C);
  if (r >= min(C, (Cl + BM - 1) / BM * BM)) return;
  uint4* dst = reinterpret_cast<uint4*>(xc + static_cast<size_t>(r) * H);
  const int n16 = H / 8;
  if (r >= Cl) {
    for (int c = threadIdx.x; c < n16; c += blockDim.x) dst[c] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0) {
      tc[r] = -1;
      rowc[r] = DzRow{0.f, 0.f, 0.f, 0.f};
    }
    return;
  }
  const long long row = idx[c0 + r];
  const uint4* src = reinterpret_cast<const uint4*>(X + row * H);
  for (int c = threadIdx.x; c < n16; c += blockDim.x) dst[c] = src[c];
  if (threadIdx.x == 0) {
    tc[r] = t[row];
    rowc[r] = dz_row(temperature, lse[row], entropy, grad_logp, grad_entropy, row);
  }
}

// Bounds of the top alternatives before the first logit; the groups behind the
// K-th (up to the stride) never bind.
__device__ __forceinline__ void clear_bounds(uint32_t* bound, uint32_t* group_max, int stride, int K, int C, int first,
                                             int step) {
  if (!bound) return;
  for (int i = first; i < C; i += step) bound[i] = 0u;
  for (long long i = first; i < static_cast<long long>(C) * stride; i += step)
    group_max[i] = static_cast<int>(i % stride) < K ? 0u : 0xffffffffu;
}

__global__ void clear_bounds_kernel(uint32_t* bound, uint32_t* group_max, int stride, int K, int C) {
  clear_bounds(bound, group_max, stride, K, C, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
}

// Everything before the first GEMM of a call of one chunk, in one launch: the
// valid tokens' rows gathered into the tile source in order, their targets (and
// for the backward the constants of MODE_DZ), the outputs of the tokens left
// out, the header and the backward GEMM's counter and flags.  Every block counts the valid
// targets before its own tokens itself (16384 targets are 64 KB from L2), which
// costs less than a launch of its own for the scan: 4096 tokens of 512 take 5.7
// us, against 16 us for the three launches it replaces.
constexpr int FRONT_THREADS = 256;
constexpr int FRONT_WARPS = FRONT_THREADS / 32;
constexpr int FRONT_TOKENS = FRONT_WARPS;   // per block: one per warp

__global__ void __launch_bounds__(FRONT_THREADS) probs_front_kernel(const FrontArgs a) {
  __shared__ int red[2][FRONT_WARPS];
  __shared__ int dst[FRONT_TOKENS];
  const int tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  ptx::grid_launch_dependents();
  const int n0 = blockIdx.x * FRONT_TOKENS;
  int before = 0, total = 0, bad = 0;
#pragma unroll 8
  for (int i = tid; i < a.N; i += FRONT_THREADS) {
    const int x = a.targets[i];
    const bool in = x >= 0 && x < a.V;
    const bool valid = in && x != a.ii;
    total += valid;
    before += valid && i < n0;
    bad |= !in && x != a.ii;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) { red[0][w] = before; red[1][w] = total; }
  bad = __syncthreads_or(bad);
  before = total = 0;
#pragma unroll
  for (int k = 0; k < FRONT_WARPS; ++k) { before += red[0][k]; total += red[1][k]; }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (tid == 0) {
      a.hdr[HDR_STATUS] = bad ? STATUS_BADTARGET : 0;
      a.hdr[HDR_NVALID] = total;
      a.hdr[HDR_STALL] = a.hdr[HDR_STALL_COUNT] = 0;
    }
    for (int i = tid; i < a.n_counters; i += FRONT_THREADS) a.counters[i] = 0;
  }
  if (w == 0) {   // the place of each token of this block, or -1
    const int n = n0 + lane;
    const int x = lane < FRONT_TOKENS && n < a.N ? a.targets[n] : -1;
    const bool valid = x >= 0 && x < a.V && x != a.ii && lane < FRONT_TOKENS && n < a.N;
    const unsigned m = __ballot_sync(0xffffffffu, valid);
    if (lane < FRONT_TOKENS) dst[lane] = valid ? before + __popc(m & ((1u << lane) - 1u)) : -1;
  }
  __syncthreads();
  // the columns this block moves (16-byte units)
  const int n16 = a.H / 8, each = (n16 + gridDim.y - 1) / gridDim.y;
  const int lo = static_cast<int>(blockIdx.y) * each, hi = min(n16, lo + each);
  const bool first = blockIdx.y == 0;
  for (int k = w; k < FRONT_TOKENS; k += FRONT_WARPS) {   // a warp per token
    const long long n = n0 + k;
    if (n >= a.N) break;
    const int r = dst[k];
    if (r >= 0) {
      const uint4* from = reinterpret_cast<const uint4*>(a.hidden + n * a.H);
      uint4* to = reinterpret_cast<uint4*>(a.xc + static_cast<size_t>(r) * a.H);
#pragma unroll 8
      for (int c = lo + lane; c < hi; c += 32) to[c] = from[c];
      if (first && lane == 0) {
        a.tc[r] = a.targets[n];
        a.idx[r] = static_cast<int>(n);
        if (a.rowc) a.rowc[r] = dz_row(a.temperature, a.lse_in[n], a.entropy_in, a.grad_logp, a.grad_entropy, n);
      }
    } else if (a.rowc) {   // backward: no gradient
      if (a.grad_hidden) {
        uint4* to = reinterpret_cast<uint4*>(a.grad_hidden + n * a.H);
        for (int c = lo + lane; c < hi; c += 32) to[c] = make_uint4(0u, 0u, 0u, 0u);
      }
    } else if (first) {    // forward: 0 for an ignored token, NaN for a target outside [0, V)
      const float v = a.targets[n] == a.ii ? 0.f : __int_as_float(0x7fc00000);
      if (lane == 0) {
        a.logp[n] = v;
        a.lse[n] = v;
        if (a.entropy) a.entropy[n] = v;
      }
      if (lane < a.K) {
        a.top_ids[n * a.K + lane] = -1;
        a.top_logp[n * a.K + lane] = v;
      }
    }
  }
  if (first)
    clear_bounds(a.bound, a.group_max, a.group_stride, a.K, a.C, blockIdx.x * FRONT_THREADS + tid,
                 gridDim.x * FRONT_THREADS);
  // padding rows up to the next multiple of 128
  const int end = min(a.C, (total + BM - 1) / BM * BM);
  for (int r = total + static_cast<int>(blockIdx.x) * FRONT_WARPS + w; r < end; r += gridDim.x * FRONT_WARPS) {
    uint4* to = reinterpret_cast<uint4*>(a.xc + static_cast<size_t>(r) * a.H);
    for (int c = lo + lane; c < hi; c += 32) to[c] = make_uint4(0u, 0u, 0u, 0u);
    if (first && lane == 0) {
      a.tc[r] = -1;
      if (a.rowc) a.rowc[r] = DzRow{0.f, 0.f, 0.f, 0.f};
    }
  }
}

// One chunk's rows: lane = row (part-major statistics: coalesced), the parts
// dealt to the block's warps and merged in a fixed order.  Reads 12 bytes per
// row and part; 32 warps with four parts in flight each, since a block waits
// for nothing but these loads (1002 parts of 723 rows: 11 us; 58 us with 8
// warps and one part at a time).  Blocks past the chunk's (last chunk only) write the rows left out:
// 0 for an ignored token, NaN for a target outside [0, V); and after a pipeline
// time-out NaN for every other row, those of finished chunks too.
constexpr int ROWS_WARPS = 32;
constexpr int ROWS_BATCH = 4;

struct RowArgs {
  const int* hdr;
  const int* idx;
  const int* targets;
  long long c0, N;
  int C, nparts, ii, K, row_blocks;
  const float* stats;
  const float* zt;
  float c2;
  float *logp, *entropy, *lse;
  float2* ml;
  int* top_ids;
  float* top_logp;
};

__global__ void __launch_bounds__(32 * ROWS_WARPS) logprob_rows_kernel(const RowArgs a) {
  __shared__ Stat part[ROWS_WARPS][32];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  // no early trigger: the waiting blocks of the top kernel would take the SMs
  // this one's blocks need (1033 tokens at 4096 x 128256: 17 us)
  ptx::grid_dependency_wait();
  if (static_cast<int>(blockIdx.x) >= a.row_blocks) {
    const long long step = static_cast<long long>(gridDim.x - a.row_blocks) * blockDim.x;
    const long long from = (a.hdr[HDR_STATUS] & STATUS_TIMEOUT) ? 0 : a.hdr[HDR_NVALID];
    for (long long i = from + static_cast<long long>(blockIdx.x - a.row_blocks) * blockDim.x + threadIdx.x;
         i < a.N; i += step) {
      const long long row = a.idx[i];   // the scored rows come first
      const float v = a.targets[row] == a.ii ? 0.f : __int_as_float(0x7fc00000);
      a.logp[row] = v;
      a.lse[row] = v;
      if (a.entropy) a.entropy[row] = v;
      for (int k = 0; k < a.K; ++k) {
        a.top_ids[row * a.K + k] = -1;
        a.top_logp[row * a.K + k] = v;
      }
    }
    return;
  }
  const int Cl = chunk_rows(a.hdr, a.c0, a.C);
  const int r = blockIdx.x * 32 + lane;
  if (static_cast<int>(blockIdx.x) * 32 >= Cl) return;
  Stat acc = {-INFINITY, 0.f, 0.f};
  if (r < Cl) {
    const size_t np = static_cast<size_t>(a.nparts) * a.C;
    for (int p0 = w; p0 < a.nparts; p0 += ROWS_BATCH * ROWS_WARPS) {
      Stat q[ROWS_BATCH];
#pragma unroll
      for (int k = 0; k < ROWS_BATCH; ++k) {
        const int p = p0 + k * ROWS_WARPS;
        const float* f = a.stats + static_cast<size_t>(p) * a.C + r;
        q[k] = p < a.nparts ? Stat{f[0], f[np], f[2 * np]} : Stat{-INFINITY, 0.f, 0.f};
      }
      static_assert(ROWS_BATCH == 4, "pairwise");
      acc = merge(acc, merge(merge(q[0], q[1], a.c2), merge(q[2], q[3], a.c2), a.c2), a.c2);
    }
  }
  part[w][lane] = acc;
#pragma unroll
  for (int o = ROWS_WARPS / 2; o > 0; o >>= 1) {   // fixed order
    __syncthreads();
    if (w < o) part[w][lane] = merge(part[w][lane], part[w + o][lane], a.c2);
  }
  if (w != 0 || r >= Cl) return;
  acc = part[0][lane];
  // after a pipeline time-out the statistics are not to be trusted
  if (a.hdr[HDR_STATUS] & STATUS_TIMEOUT) acc.m = __int_as_float(0x7fc00000);
  const float l2s = log2f(acc.s);
  const long long row = a.idx[a.c0 + r];
  a.logp[row] = fmaf(a.zt[r] - acc.m, a.c2, -l2s) * LN2;
  a.lse[row] = fmaf(acc.m, a.c2, l2s) * LN2;
  if (a.entropy) a.entropy[row] = fmaf(0.f, acc.m, l2s - acc.d / acc.s) * LN2;   // NaN where the max is not finite
  if (a.K > 0) a.ml[r] = make_float2(acc.m, l2s);
}

// Top alternatives of one row per block: the K best parts by (max, position),
// then the K best of their logits by (value, id).  The loads of eight groups
// (one or two parts) are in flight at a time.  Latency: 20 alternatives of 723
// rows over 1002 parts take 20 us.
constexpr int TOP_WARPS = 4;
constexpr int TOP_BATCH = 8;
__global__ void __launch_bounds__(32 * TOP_WARPS)
    logprob_top_kernel(const int* hdr, const int* idx, long long c0, int C, int V, long long ldz, int nparts, int K,
                       const float* stats, const float* zf, const float2* ml, float c2, int* top_ids,
                       float* top_logp) {
  __shared__ float sv[TOP_WARPS][32];
  __shared__ int si[TOP_WARPS][32];
  const int r = blockIdx.x;
  ptx::grid_dependency_wait();
  if (r >= chunk_rows(hdr, c0, C)) return;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  if (hdr[HDR_STATUS] & STATUS_TIMEOUT) {   // uniform over the grid
    if (static_cast<int>(threadIdx.x) < K) {
      const long long at = static_cast<long long>(idx[c0 + r]) * K + threadIdx.x;
      top_ids[at] = -1;
      top_logp[at] = __int_as_float(0x7fc00000);
    }
    return;
  }
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
  const float* zr = zf + static_cast<size_t>(r) * ldz;
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
  if (w == 0 && lane < K) {
    const long long row = idx[c0 + r];
    const bool some = best.id != TopK::NONE;   // false only where fewer than K logits are numbers
    top_ids[row * K + lane] = some ? best.id : -1;
    top_logp[row * K + lane] = some ? fmaf(best.v - ml[r].x, c2, -ml[r].y) * LN2 : __int_as_float(0x7fc00000);
  }
}

// grad_hidden rows of a chunk from the fp32 parts of its vocabulary splits,
// added in order and rounded once.  Reads what L2 still holds: S C H 4 bytes.
constexpr int DXR_THREADS = 256;
constexpr int DXR_BATCH = 8;   // parts in flight
__global__ void __launch_bounds__(DXR_THREADS)
    dx_reduce_kernel(const int* hdr, const int* idx, long long c0, int C, int H, int splits, const float* parts,
                     uint16_t* grad_hidden) {
  ptx::grid_dependency_wait();
  const int Cl = chunk_rows(hdr, c0, C);
  const int n8 = H / 8;
  const long long total = static_cast<long long>(Cl) * n8, slab = static_cast<long long>(C) * H;
  for (long long i = static_cast<long long>(blockIdx.x) * DXR_THREADS + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * DXR_THREADS) {
    const int r = static_cast<int>(i / n8), c = static_cast<int>(i - static_cast<long long>(r) * n8);
    const float* p = parts + static_cast<long long>(r) * H + c * 8;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < splits; k0 += DXR_BATCH) {
      float4 x[DXR_BATCH][2];
#pragma unroll
      for (int k = 0; k < DXR_BATCH; ++k)
        if (k0 + k < splits) {
          const float4* q = reinterpret_cast<const float4*>(p + (k0 + k) * slab);
          x[k][0] = q[0];
          x[k][1] = q[1];
        }
#pragma unroll
      for (int k = 0; k < DXR_BATCH; ++k)
        if (k0 + k < splits) {
          s[0] += x[k][0].x; s[1] += x[k][0].y; s[2] += x[k][0].z; s[3] += x[k][0].w;
          s[4] += x[k][1].x; s[5] += x[k][1].y; s[6] += x[k][1].z; s[7] += x[k][1].w;
        }
    }
    const long long tok = idx[c0 + r];
    reinterpret_cast<uint4*>(grad_hidden + tok * H)[c] =
        make_uint4(ptx::pack_bf16x2(s[0], s[1]), ptx::pack_bf16x2(s[2], s[3]), ptx::pack_bf16x2(s[4], s[5]),
                   ptx::pack_bf16x2(s[6], s[7]));
  }
}

// The gradients of a call whose pipeline timed out begin with a NaN, so that a
// caller who never reads the status still sees that they are not to be trusted.
__global__ void mark_failed_kernel(const int* hdr, uint16_t* grad_hidden, float* grad_weight, int gw_bf16) {
  ptx::grid_dependency_wait();
  if (!(hdr[HDR_STATUS] & STATUS_TIMEOUT)) return;
  if (grad_hidden) grad_hidden[0] = 0x7fc0;
  if (grad_weight && gw_bf16) reinterpret_cast<uint16_t*>(grad_weight)[0] = 0x7fc0;
  else if (grad_weight) grad_weight[0] = __int_as_float(0x7fc00000);
}

// ---------------------------------------------------------------------------
// workspace of the forward
// ---------------------------------------------------------------------------
struct LpPlan {
  long long C = 0, n_chunks = 0, ldz = 0;
  int nvt = 0, nparts = 0;
  size_t o_idx = 0, o_xc = 0, o_tc = 0, o_zt = 0, o_ml = 0, o_stats = 0, o_bound = 0, o_group = 0,
         o_zf = 0, total = 0;
  int group_stride = 0;
};

LpPlan lp_layout(long long N, long long H, long long V, long long C, int K) {
  LpPlan p;
  p.C = C;
  p.n_chunks = cdiv(N, C);
  p.ldz = cdiv(V, 64) * 64;
  p.nvt = static_cast<int>(cdiv(V, BN));
  p.nparts = static_cast<int>(cdiv(V, PART_COLS));
  size_t off = al256(HDR_WORDS * sizeof(int));
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += al256(bytes);
    return o;
  };
  p.o_idx = take(size_t(N) * 4);
  p.o_xc = take(size_t(C) * H * 2);
  p.o_tc = take(size_t(C) * 4);
  p.o_zt = take(size_t(C) * 4);
  p.o_ml = take(size_t(C) * 8);
  p.o_stats = take(size_t(C) * p.nparts * 12);
  p.group_stride = (K + 3) / 4 * 4;
  if (K > 0) {
    p.o_bound = take(size_t(C) * 4);
    p.o_group = take(size_t(C) * p.group_stride * 4);
    p.o_zf = take(size_t(C) * p.ldz * 4);
  }
  p.total = off;
  return p;
}

// Largest chunk (a multiple of 128 rows) whose plan fits in `bytes`.
bool lp_plan(long long N, long long H, long long V, int K, size_t bytes, LpPlan* out) {
  long long lo = 1, hi = cdiv(N, BM);
  if (lp_layout(N, H, V, BM, K).total > bytes) return false;
  while (lo < hi) {
    const long long mid = (lo + hi + 1) / 2;
    if (lp_layout(N, H, V, mid * BM, K).total <= bytes) lo = mid;
    else hi = mid - 1;
  }
  *out = lp_layout(N, H, V, lo * BM, K);
  return true;
}

// Default workspace: 5% of the bf16 logits as for the loss, but no less than
// what lets problems of up to 16384 tokens run in one chunk (512 MiB, 0.2% of
// the memory; 2 GiB with the fp32 logits of top alternatives): every chunk reads
// the weight and rounds its rows up to the tiles' 256.
size_t lp_default_bytes(long long N, long long H, long long V, int K) {
  const size_t budget = std::max(size_t(N) * size_t(V) * 2 / 20, size_t(K > 0 ? 2048 : 512) << 20);
  LpPlan p;
  if (lp_plan(N, H, V, K, budget, &p)) return p.total;
  return lp_layout(N, H, V, BM, K).total;
}

}  // namespace

namespace {

// Workspace of the streaming form (N <= STREAM_MAX_TOKENS).
struct StreamPlan {
  int ctas = 0;
  int max_tiles = 0;
  long long ldz = 0;
  size_t o_zt = 0, o_stat = 0, o_max = 0, o_group = 0, o_zf = 0, o_fail = 0, total = 0;
};

StreamPlan stream_plan(long long N, long long V, int K, int sms) {
  StreamPlan p;
  p.ctas = stream_ctas(V, sms);
  size_t off = al256(HDR_WORDS * sizeof(int));
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += al256(bytes);
    return o;
  };
  p.o_zt = take(size_t(N) * 4);
  p.o_stat = take(size_t(N) * p.ctas * 16);
  p.max_tiles = stream_max_tiles(V, p.ctas);
  p.ldz = cdiv(V, 32) * 32;
  if (K > 0) {
    p.o_max = take(size_t(N) * p.ctas * p.max_tiles * 4);
    p.o_group = take(size_t(N) * TopK::MAX * 4);
    p.o_zf = take(size_t(N) * p.ldz * 4);
  }
  p.o_fail = take(size_t(p.ctas) * 4);
  p.total = off;
  return p;
}

}  // namespace

bool bad_temperature(float t) { return !(t > 0.f) || !std::isfinite(t) || !std::isfinite(LOG2E / t); }

cudaError_t launch_dx_reduce(const int* hdr, const int* idx, long long c0, int C, int H, int splits, const float* parts,
                             uint16_t* grad_hidden, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(std::min<long long>(cdiv(static_cast<long long>(C) * (H / 8), DXR_THREADS), 152 * 8));
  return launch_dependent(dx_reduce_kernel, blocks, DXR_THREADS, s, hdr, idx, c0, C, H, splits, parts, grad_hidden);
}

cudaError_t launch_mark_failed(const int* hdr, uint16_t* grad_hidden, float* grad_weight, int gw_bf16,
                               cudaStream_t s) {
  return launch_dependent(mark_failed_kernel, 1, 1, s, hdr, grad_hidden, grad_weight, gw_bf16);
}

cudaError_t launch_probs_front(const FrontArgs& a, cudaStream_t s) {
  // few tokens: several blocks share a row, 1024 columns each
  const unsigned slices = a.N <= 2048 ? static_cast<unsigned>(std::min<long long>(cdiv(a.H, 1024), 64)) : 1;
  probs_front_kernel<<<dim3(static_cast<unsigned>(cdiv(a.N, FRONT_TOKENS)), slices), FRONT_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_gather_dz(const uint16_t* hidden, const int* targets, const int* hdr, const int* idx, long long c0,
                             int C, int H, float temperature, const float* lse, const float* entropy,
                             const float* grad_logp, const float* grad_entropy, uint16_t* xc, int* tc, DzRow* rowc,
                             cudaStream_t s) {
  gather_dz_kernel<<<C, 128, 0, s>>>(hidden, targets, hdr, idx, c0, C, H, temperature, lse, entropy, grad_logp,
                                     grad_entropy, xc, tc, rowc);
  return cudaGetLastError();
}

}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_logprobs_workspace_bytes(int64_t N, int64_t H, int64_t V, int32_t top_k) {
  if (!sizes_ok(N, H, V) || V > PROBS_MAX_V || top_k < 0 || top_k > TopK::MAX || top_k > V) return 0;
  if (N <= STREAM_MAX_TOKENS) return stream_plan(N, V, top_k, device_sms()).total;
  return lp_default_bytes(N, H, V, top_k);
}

flce_status flce_logprobs(const void* hidden, const void* weight, const int32_t* targets, int64_t N, int64_t H,
                          int64_t V, int32_t ignore_index, float temperature, int32_t top_k, float* logp,
                          float* entropy, float* lse, int32_t* top_ids, float* top_logp, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!hidden || !weight || !targets || !logp || !lse || !workspace) return FLCE_EINVAL;
  if (N < 1 || H < 1 || V < 1 || top_k < 0 || top_k > V || bad_temperature(temperature)) return FLCE_EINVAL;
  if (top_k > 0 && (!top_ids || !top_logp)) return FLCE_EINVAL;
  if (!sizes_ok(N, H, V) || V > PROBS_MAX_V || top_k > TopK::MAX) return FLCE_EUNSUPPORTED;
  if (!aligned16(hidden) || !aligned16(weight) || !aligned16(workspace) || !aligned4(targets) || !aligned4(logp) ||
      !aligned4(entropy) || !aligned4(lse) || !aligned4(top_ids) || !aligned4(top_logp))
    return FLCE_EUNSUPPORTED;
  // the logits of the chunked form are stored 32 bytes at a time
  if (top_k > 0 && N > STREAM_MAX_TOKENS && !aligned32(workspace)) return FLCE_EUNSUPPORTED;
  DeviceState dev;
  if (device_state(&dev) != cudaSuccess) { cudaGetLastError(); return FLCE_ECUDA; }
  if (dev.major < 10) return FLCE_EUNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* hdr = at<int>(workspace, 0);
  if (N <= STREAM_MAX_TOKENS) {
    const StreamPlan p = stream_plan(N, V, top_k, dev.sms);
    if (p.total > workspace_bytes) return FLCE_EWORKSPACE;
    StreamArgs a;
    std::memset(&a, 0, sizeof(a));
    a.N = static_cast<int>(N); a.H = static_cast<int>(H); a.V = static_cast<int>(V); a.K = top_k;
    a.seg_kb = segment_blocks(H);
    a.ctas = p.ctas;
    a.c2 = LOG2E / temperature;
    a.ii = ignore_index;
    a.timeout_ns = wait_timeout_ns();
    if (const unsigned long long t = take_armed_stall()) {
      a.debug_stall = 1;
      a.timeout_ns = t;
    }
    a.targets = targets;
    a.hdr = hdr;
    a.zt = at<float>(workspace, p.o_zt);
    a.stat = at<float4>(workspace, p.o_stat);
    a.zf = at<float>(workspace, p.o_zf);
    a.ldz = p.ldz;
    a.tile_max = at<float>(workspace, p.o_max);
    a.max_tiles = p.max_tiles;
    // With one tile a CTA, all of them finish at once and no bound is known in
    // time: every logit is kept, and nothing needs clearing.
    a.group_max = top_k > 0 && p.max_tiles > 1 ? at<uint32_t>(workspace, p.o_group) : nullptr;
    a.fail = at<int>(workspace, p.o_fail);
    a.logp = logp; a.entropy = entropy; a.lse = lse; a.top_ids = top_ids; a.top_logp = top_logp;
    StreamMaps m;
    const unsigned long long hb = static_cast<unsigned long long>(H) * 2;
    bool ok = make_map(&m.x, hidden, H, N, hb, BK, stream_tokens(a.N));
    for (int k = 0; k < 4; ++k) ok = ok && make_map(&m.w[k], weight, H, V, hb, BK, 128u >> k);
    if (!ok) return FLCE_ECUDA;
    const ProfScope prof = prof_launch_begin(st);
    const cudaError_t e = launch_stream(a, m, st);
    prof_launch_end(prof, MODE_STATS, st);
    count_launches(a.group_max ? 2 : 1);   // the merge, the clearing
    return e == cudaSuccess ? FLCE_OK : FLCE_ECUDA;
  }
  LpPlan p;
  if (!lp_plan(N, H, V, top_k, workspace_bytes, &p)) return FLCE_EWORKSPACE;

  int* idx = at<int>(workspace, p.o_idx);
  uint16_t* xc = at<uint16_t>(workspace, p.o_xc);
  int* tc = at<int>(workspace, p.o_tc);
  float* zt = at<float>(workspace, p.o_zt);
  float2* ml = at<float2>(workspace, p.o_ml);
  float* stats = at<float>(workspace, p.o_stats);
  float* zf = top_k > 0 ? at<float>(workspace, p.o_zf) : nullptr;

  GemmMaps m;
  std::memset(&m, 0, sizeof(m));
  const unsigned long long hb = static_cast<unsigned long long>(H) * 2;
  if (!make_map(&m.a0, xc, H, p.C, hb, BK, BM) || !make_map(&m.b0, weight, H, V, hb, BK, BN / 2)) return FLCE_ECUDA;

  GemmArgs g;
  std::memset(&g, 0, sizeof(g));
  g.mode = MODE_STATS;
  g.hdr = hdr;
  g.status = hdr + HDR_STATUS;
  g.C = static_cast<int>(p.C);
  g.H = static_cast<int>(H);
  g.V = static_cast<int>(V);
  g.ldz = p.ldz;
  g.nvt = p.nvt;
  g.nparts = p.nparts;
  g.timeout_ns = wait_timeout_ns();
  g.tc = tc;
  g.zt = zt;
  g.stats = stats;
  g.K = top_k;
  g.zf = zf;
  // The bound pays once each of its K groups has several parts (by 16 parts a
  // group: 1024 tokens x 8 at 2048 x 256000, 2000 parts, GEMM 20% faster; x 32
  // at 512 x 16000, 125 parts, 15% slower).
  if (top_k > 0 && p.nparts >= 16 * top_k) {
    g.bound = at<uint32_t>(workspace, p.o_bound);
    g.group_max = at<uint32_t>(workspace, p.o_group);
  }
  g.group_stride = p.group_stride;
  g.seg_kb = segment_blocks(H);
  g.c2 = LOG2E / temperature;

  const int grid = 2 * static_cast<int>(std::min<long long>(cdiv(p.C, PAIR_M) * p.nvt, dev.pairs));
  auto chk = [](cudaError_t e) { return e == cudaSuccess; };
  const bool front = p.n_chunks == 1 && N <= FRONT_MAX_TOKENS;
  count_launches(front ? (top_k > 0 ? 3 : 2) : 1 + p.n_chunks * (top_k > 0 ? 4 : 2));
  RowArgs ra;
  ra.hdr = hdr; ra.idx = idx; ra.targets = targets;
  ra.N = N; ra.C = g.C; ra.nparts = p.nparts; ra.ii = ignore_index; ra.K = top_k;
  ra.row_blocks = static_cast<int>(cdiv(p.C, 32));
  ra.stats = stats; ra.zt = zt; ra.c2 = g.c2;
  ra.logp = logp; ra.entropy = entropy; ra.lse = lse; ra.ml = ml; ra.top_ids = top_ids; ra.top_logp = top_logp;
  const int left_blocks = static_cast<int>(std::min<long long>(cdiv(N, 32 * ROWS_WARPS), 152));
  if (front) {
    FrontArgs f;
    std::memset(&f, 0, sizeof(f));
    f.hidden = static_cast<const uint16_t*>(hidden);
    f.targets = targets;
    f.N = static_cast<int>(N); f.H = g.H; f.V = g.V; f.ii = ignore_index; f.C = g.C; f.K = top_k;
    f.hdr = hdr; f.idx = idx; f.tc = tc; f.xc = xc;
    f.bound = g.bound; f.group_max = g.group_max; f.group_stride = g.group_stride;
    f.logp = logp; f.lse = lse; f.entropy = entropy; f.top_ids = top_ids; f.top_logp = top_logp;
    if (!chk(launch_probs_front(f, st))) return FLCE_ECUDA;
  } else if (!chk(launch_prep(targets, N, static_cast<int>(V), ignore_index, hdr, idx, nullptr, nullptr, 0, st))) {
    return FLCE_ECUDA;
  }
  for (long long c = 0; c < p.n_chunks; ++c) {
    g.c0 = c * p.C;
    if (!front && !chk(launch_gather(static_cast<const uint16_t*>(hidden), targets, hdr, idx, g.c0, g.C, g.H, xc, tc, 0,
                                     g.V, st)))
      return FLCE_ECUDA;
    if (!front && g.bound) {
      clear_bounds_kernel<<<152, 256, 0, st>>>(g.bound, g.group_max, g.group_stride, top_k, g.C);
      if (!chk(cudaGetLastError())) return FLCE_ECUDA;
    }
    if (!chk(gemm_launch(g, m, grid, st, front))) return FLCE_ECUDA;
    ra.c0 = g.c0;
    if (!chk(launch_dependent(logprob_rows_kernel, ra.row_blocks + (!front && c == p.n_chunks - 1 ? left_blocks : 0),
                              32 * ROWS_WARPS, st, ra)))
      return FLCE_ECUDA;
    if (top_k > 0 && !chk(launch_dependent(logprob_top_kernel, g.C, 32 * TOP_WARPS, st, hdr, idx, g.c0, g.C, g.V, p.ldz,
                                           p.nparts, top_k, stats, zf, ml, g.c2, top_ids, top_logp)))
      return FLCE_ECUDA;
  }
  return FLCE_OK;
}

}  // extern "C"
