// Token log probabilities of few tokens (N <= 128: decode steps, short
// completions): the weight is read once and everything else hides behind it.
//
//   z^T = W X^T tile by tile: 256 rows of W are the M side of two
//   tcgen05.mma (M = 128), the tokens (padded to 16, 32, 64 or 128) the N side,
//   so no tensor work or shared memory is spent on absent tokens.
//
// One persistent CTA per SM owns a contiguous range of the vocabulary, cut in
// units of 16 rows so that the ranges differ by 16 rows at most, and walks it
// in tiles of up to 256 rows.  Warp 0 streams W (and, from L2, X) through a
// TMA ring of 64-column K blocks, warp 1 issues the MMAs into one of two TMEM
// accumulators, and eight epilogue warps turn a finished 256 x 32 slice of
// logits around in shared memory, where each warp takes whole tokens: the
// running softmax statistics and the target's logit.  Every CTA leaves its
// statistics per token; the second kernel, a block per token, merges them.
// For top alternatives a tile's max and, where it matters, its logits are
// stored, and the second kernel reads back the K best tiles only.  It does not
// matter where K other tiles are known to have a larger max: the tiles are
// dealt to K groups, and the least of the groups' maxima (kept in global
// memory, read once a tile) bounds the K-th best logit from below.  After the
// first tile of each CTA few pass.  (Storing every logit: 64 tokens, 8
// alternatives at 2048 x 256000 184 us, with none stored 164; a sorted list per
// CTA and token: 175, with 32 alternatives 212.)
//
// Long sums over H are taken in segments (segment_blocks()), each in an
// accumulator of its own, which the epilogue warps add up in registers (1 to 64
// tokens no slower; 128 tokens at 1024 x 128256 80 us, 76 in one piece, at 4096
// 181 and 180).
//
// Bound by the weight's bytes: 2 H V at the HBM rate (4096 x 128256: 158 us for
// 1 token, 6.66 TB/s; 164 for 64, 172 for 128).  Every wait is bounded:
// on time-out the CTA lets its copies in flight land, waits for its MMAs, frees
// TMEM and returns, and the call's rows become NaN (status FLCE_ETIMEOUT).
#include "flce_internal.h"
#include "flce_ptx.cuh"
#include "flce_softmax.cuh"
#include "flce_topk.cuh"

namespace flce {
namespace {

constexpr int TILE_ROWS = 256;
constexpr int UNIT_ROWS = 16;
constexpr int W_BYTES = TILE_ROWS * BK * 2;
constexpr int EPI_WARPS = 8;
constexpr int EPI_THREADS = 32 * EPI_WARPS;
constexpr int THREADS = 64 + EPI_THREADS;
constexpr uint32_t EPI_BAR = 1;

// The ring takes what the slice buffer leaves of 227 KB.
constexpr int MAX_STAGES = 6;
template <int NT>
struct Cfg {
  static constexpr int STAGES = NT == 16 ? 6 : (NT == 128 ? 4 : 5);
  static constexpr int SLICE = NT == 32 ? 32 : 16;                // tokens turned around at once
  static constexpr int X_BYTES = NT * BK * 2;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int TURN_BYTES = SLICE * TILE_ROWS * 4;
  static constexpr int TMEM_COLS = 4 * NT;                        // two accumulators of two halves
  static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + TURN_BYTES + NT * 20 + 256;
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct Ctl {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t tfull[2], tempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Ctl) <= 256, "control block");

// Wait sites recorded in the workspace header (numbers as in flce_query_stall).
enum Site : int { S_STAGE_EMPTY = 3, S_DRAIN = 4, S_TMEM_EMPTY = 6, S_STAGE_FULL = 7, S_MMA_DONE = 8, S_TMEM_FULL = 10 };

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Ctl* ctl, uint64_t timeout_ns, bool honor_abort,
                                       int* hdr, int site) {
  const uint64_t t0 = ptx::global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (ptx::mbar_test(bar, parity)) return true;
    if ((i & 31u) == 0) {
      if (honor_abort && *reinterpret_cast<volatile int*>(&ctl->abort)) return false;
      if (ptx::global_timer_ns() - t0 > timeout_ns) {
        *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
        atomicCAS(hdr + HDR_STALL, 0, site | (static_cast<int>(blockIdx.x) << 12));
        atomicAdd(hdr + HDR_STALL_COUNT, 1);
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctl* ctl, uint64_t timeout_ns, int* hdr, int site,
                                     bool honor_abort = true) {
  return ptx::mbar_test(bar, parity) || wait_slow(bar, parity, ctl, timeout_ns, honor_abort, hdr, site);
}

// This CTA's tiles: units [u0, u1) of 16 rows, spread evenly over its tiles (a
// short last tile would fill the ring's stages with few bytes: one token at
// 4096 x 128256 177 us against 166).
struct Range {
  int u0, u1, tiles;
  __device__ __forceinline__ int start(int i) const {   // first row of tile i (also: the end of tile i - 1)
    return (u0 + static_cast<int>(static_cast<long long>(u1 - u0) * i / tiles)) * UNIT_ROWS;
  }
};

__device__ __forceinline__ Range range_of(const StreamArgs& a, int cta) {
  const long long units = (static_cast<long long>(a.V) + UNIT_ROWS - 1) / UNIT_ROWS;
  Range r;
  r.u0 = static_cast<int>(units * cta / a.ctas);
  r.u1 = static_cast<int>(units * (cta + 1) / a.ctas);
  r.tiles = (r.u1 - r.u0 + TILE_ROWS / UNIT_ROWS - 1) / (TILE_ROWS / UNIT_ROWS);
  return r;
}

// SEG: the sum over H in segments (segment_blocks()), added up in registers.
template <int NT, bool SEG>
__global__ void __launch_bounds__(THREADS, 1)
    logprob_stream_kernel(const __grid_constant__ StreamMaps maps, const StreamArgs a) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* turn = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE_BYTES);          // [SLICE][TILE_ROWS]
  float4* stat = reinterpret_cast<float4*>(turn + C::SLICE * TILE_ROWS);              // [NT]
  uint32_t* bound = reinterpret_cast<uint32_t*>(stat + NT);                           // [NT]
  Ctl* ctl = reinterpret_cast<Ctl*>(bound + NT);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint64_t to = a.timeout_ns;
  const Range range = range_of(a, static_cast<int>(blockIdx.x));
  const int kbt = (a.H + BK - 1) / BK;

  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.hdr[HDR_STATUS] = 0;
    a.hdr[HDR_STALL] = 0;
    a.hdr[HDR_STALL_COUNT] = 0;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      ptx::mbar_init(&ctl->full[i], 1);
      ptx::mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl->tfull[i], 1);
      ptx::mbar_init(&ctl->tempty[i], EPI_WARPS);
    }
    ptx::mbar_init(&ctl->mma_done, 1);
    ctl->abort = 0;
    ptx::mbar_fence_init();
    ptx::tma_prefetch_desc(&maps.x);
    for (int k = 0; k < 4; ++k) ptx::tma_prefetch_desc(&maps.w[k]);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl->tmem_base, C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  ptx::grid_launch_dependents();   // the merge kernel's blocks may come up; they wait for this grid's end

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer ----------------
    const uint64_t once = ptx::policy_evict_first(), keep = ptx::policy_evict_last();
    uint32_t stage = 0, phase = 0, issued_mask = 0, issued_parity = 0;
    bool ok = true;
    for (int i = 0; ok && i < range.tiles; ++i) {
      const int r0 = range.start(i), rows = range.start(i + 1) - r0;   // rows: a multiple of 16
      for (int kb = 0; kb < kbt; ++kb) {
        if (!wait(&ctl->empty[stage], phase ^ 1u, ctl, to, a.hdr, S_STAGE_EMPTY)) { ok = false; break; }
        uint8_t* sw = smem + stage * C::STAGE_BYTES;
        uint64_t* bar = &ctl->full[stage];
        ptx::mbar_arrive_expect_tx(bar, rows * (BK * 2) + C::X_BYTES);
        int done = 0;
        if (rows >= 256) {
          ptx::tma_load_2d(sw, &maps.w[0], bar, kb * BK, r0, once);
          done = 128;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (rows - done >= (128 >> k)) {
            ptx::tma_load_2d(sw + done * (BK * 2), &maps.w[k], bar, kb * BK, r0 + done, once);
            done += 128 >> k;
          }
        }
        ptx::tma_load_2d(sw + W_BYTES, &maps.x, bar, kb * BK, 0, keep);
        issued_mask |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    // Let the copies in flight land before the CTA exits.  Without a time-out
    // the MMAs have waited for all of them; with one, also where this thread
    // had issued its last copy before another role gave up.
    for (int i = 0; i < C::STAGES; ++i)
      if (issued_mask & (1u << i)) wait(&ctl->full[i], (issued_parity >> i) & 1u, ctl, to, a.hdr, S_DRAIN, false);
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMA issuer ----------------
    constexpr uint32_t idesc = ptx::idesc_bf16_f32(128, NT, 0, 0);
    uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
    bool withhold = a.debug_stall != 0, ok = true;
    for (int i = 0; ok && i < range.tiles; ++i) {
      const bool two = range.start(i + 1) - range.start(i) > 128;
      int kb = 0;
      do {   // one accumulator: the whole sum, or a segment of it
        const int kb0 = kb, kb1 = SEG ? min(kbt, kb0 + a.seg_kb) : kbt;
        if (!wait(&ctl->tempty[acc], acc_phase ^ 1u, ctl, to, a.hdr, S_TMEM_EMPTY)) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t d = tmem + acc * 2 * NT;
        for (; kb < kb1; ++kb) {
          if (!wait(&ctl->full[stage], phase, ctl, to, a.hdr, S_STAGE_FULL)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t sw = ptx::smem_u32(smem + stage * C::STAGE_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint32_t go = (kb > kb0 || kk > 0) ? 1u : 0u;
            const uint64_t wd = ptx::smem_desc_sw128(0, 16, 1024) | ((sw >> 4) + kk * 2);
            const uint64_t xd = wd + W_BYTES / 16;
            ptx::umma_bf16(d, wd, xd, idesc, go);
            if (two) ptx::umma_bf16(d + NT, wd + 128 * BK * 2 / 16, xd, idesc, go);
          }
          ptx::umma_commit(&ctl->empty[stage]);
          if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (!withhold) ptx::umma_commit(&ctl->tfull[acc]);
        withhold = false;
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      } while (SEG && kb < kbt);
    }
    ptx::umma_commit(&ctl->mma_done);
    wait(&ctl->mma_done, 0, ctl, to, a.hdr, S_MMA_DONE, false);
  } else if (warp >= 2) {
    // ---------------- epilogue ----------------
    const int w = warp - 2;
    const int q = warp & 3;            // TMEM lane quarter this warp may access
    const int half = w / 4;            // the 128 rows of the tile it reads
    for (int tk = w; tk < a.N; tk += EPI_WARPS)
      if (lane == 0) stat[tk] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    __syncwarp();
    if (a.group_max) ptx::grid_dependency_wait();   // the groups' maxima have been cleared
    uint32_t acc = 0, acc_phase = 0;
    for (int i = 0; i < range.tiles; ++i) {
      if (a.group_max) {   // the bounds of this warp's tokens
        for (int t0 = w; t0 < a.N; t0 += 4 * EPI_WARPS) {
          uint32_t g[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int tk = t0 + u * EPI_WARPS;
            g[u] = tk < a.N && lane < a.K ? ptx::ld_relaxed_gpu(a.group_max + tk * TopK::MAX + lane) : 0xffffffffu;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t least = __reduce_min_sync(0xffffffffu, g[u]);
            if (lane == 0 && t0 + u * EPI_WARPS < a.N) bound[t0 + u * EPI_WARPS] = least;
          }
        }
        __syncwarp();
      }
      const int r0 = range.start(i), rows = min(range.start(i + 1), a.V) - r0;
      const uint32_t tb0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * NT;
      float sum[SEG ? NT : 1];   // SEG: this row's logits so far
      bool ok;
      if constexpr (SEG) {
        ok = true;
#pragma unroll
        for (int k = 0; k < NT; ++k) sum[k] = 0.f;
#pragma unroll 1
        for (int kb = 0; kb < kbt; kb += a.seg_kb) {
          ok = __all_sync(0xffffffffu, wait(&ctl->tfull[acc], acc_phase, ctl, to, a.hdr, S_TMEM_FULL));
          if (!ok) break;   // uniform over the warp; the others give up at their own wait
          ptx::tc_fence_after();
          if (half * 128 < rows) {
#pragma unroll
            for (int j = 0; j < NT; j += C::SLICE) {
              if (j >= a.N) break;
              float v[C::SLICE];
              if constexpr (C::SLICE == 32) ptx::tmem_ld32(tb0 + acc * 2 * NT + j, v);
              else ptx::tmem_ld16(tb0 + acc * 2 * NT + j, v);
#pragma unroll
              for (int k = 0; k < C::SLICE; ++k) sum[j + k] += v[k];
            }
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&ctl->tempty[acc]);
          acc ^= 1u;
          if (acc == 0) acc_phase ^= 1u;
        }
      } else {
        ok = wait(&ctl->tfull[acc], acc_phase, ctl, to, a.hdr, S_TMEM_FULL);
      }
      if (!ptx::named_bar_and(EPI_BAR, EPI_THREADS, ok)) break;   // all epilogue threads leave together
      ptx::tc_fence_after();
      const uint32_t tb = tb0 + acc * 2 * NT;
      constexpr int UNROLL = SEG ? NT / C::SLICE : 1;   // registers have no index
#pragma unroll UNROLL
      for (int n0 = 0; n0 < NT; n0 += C::SLICE) {
        if (n0 >= a.N) break;
        if (half * 128 < rows) {
          float v[C::SLICE];
          if constexpr (SEG) {
#pragma unroll
            for (int k = 0; k < C::SLICE; ++k) v[k] = sum[n0 + k];
          } else if constexpr (C::SLICE == 32) {
            ptx::tmem_ld32(tb + n0, v);
          } else {
            ptx::tmem_ld16(tb + n0, v);
          }
          float* p = turn + half * 128 + q * 32 + lane;
#pragma unroll
          for (int k = 0; k < C::SLICE; ++k) p[k * TILE_ROWS] = v[k];
        }
        if (!SEG && n0 + C::SLICE >= a.N) {   // this warp has read its part of the accumulator
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&ctl->tempty[acc]);
        }
        ptx::named_bar_sync(EPI_BAR, EPI_THREADS);
#pragma unroll 1
        for (int k = w; k < C::SLICE; k += EPI_WARPS) {
          const int tk = n0 + k;
          if (tk >= a.N) break;
          const float* z = turn + k * TILE_ROWS;
          float x[8], mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = j * 32 + lane < rows ? z[j * 32 + lane] : -INFINITY;
            mx = fmaxf(mx, x[j]);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float mb = mx == -INFINITY ? 0.f : -mx * a.c2;
          float s = 0.f, d = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = fmaf(x[j], a.c2, mb);
            const float e = ptx::ex2(y);
            s += e;
            d = fmaf(fmaxf(y, -1e30f), e, d);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            d += __shfl_xor_sync(0xffffffffu, d, o);
          }
          if (lane == 0) {
            // mb is rounded: every y is too large by rho (exact in the fused multiply-add)
            const float rho = mx == -INFINITY ? 0.f : fmaf(mx, a.c2, mb);
            const float back = ptx::ex2(-rho);
            const float4 old = stat[tk];
            const Stat t = merge(Stat{old.x, old.y, old.z}, Stat{mx, back * s, back * fmaf(-rho, s, d)}, a.c2);
            stat[tk] = make_float4(t.m, t.s, t.d, 0.f);
            const unsigned at = static_cast<unsigned>(a.targets[tk]) - static_cast<unsigned>(r0);
            if (at < static_cast<unsigned>(rows)) a.zt[tk] = z[at];
          }
          if (a.K > 0) {
            if (!a.group_max || order_key(mx) >= bound[tk]) {
              float* zf = a.zf + static_cast<size_t>(tk) * a.ldz + r0 + lane;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (j * 32 + lane < rows) zf[j * 32] = x[j];
              if (a.group_max && lane == 0) atomicMax(a.group_max + tk * TopK::MAX + (blockIdx.x + i) % a.K, order_key(mx));
            }
            if (lane == 0)
              a.tile_max[static_cast<size_t>(tk) * a.ctas * a.max_tiles + blockIdx.x * a.max_tiles + i] = mx;
          }
        }
        ptx::named_bar_sync(EPI_BAR, EPI_THREADS);   // the slice buffer is free again
      }
      if (!SEG) {
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
    for (int tk = w; tk < a.N; tk += EPI_WARPS) {
      __syncwarp();
      if (lane == 0) {
        const size_t o = static_cast<size_t>(tk) * a.ctas + blockIdx.x;
        a.stat[o] = stat[tk];
        // the last entry of a CTA of fewer tiles than others: NaN is never taken
        if (a.K > 0 && range.tiles < a.max_tiles)
          a.tile_max[o * a.max_tiles + a.max_tiles - 1] = __int_as_float(0x7fc00000);
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (threadIdx.x == 0) a.fail[blockIdx.x] = *reinterpret_cast<volatile int*>(&ctl->abort);
}

// One token per block: its row from the CTAs' statistics, and its top
// alternatives from the K best tiles (an alternative lies in one of them, as in
// the chunked form).  Launched while the first kernel drains; what it reads is
// loaded in batches, since the latency of a few dependent loads is all there is
// to it.
constexpr int MERGE_WARPS = 8;
constexpr int MERGE_THREADS = 32 * MERGE_WARPS;
constexpr int MERGE_BATCH = 4;   // tile maxima per thread in flight
__global__ void __launch_bounds__(MERGE_THREADS) logprob_stream_merge_kernel(const StreamArgs a) {
  __shared__ Stat part[MERGE_WARPS];
  __shared__ float sv[MERGE_WARPS][32];
  __shared__ int si[MERGE_WARPS][32];
  const int n = blockIdx.x, tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  const int t = a.targets[n];
  const bool bad = t != a.ii && (t < 0 || t >= a.V);
  ptx::grid_dependency_wait();
  const float zt = bad || t == a.ii ? 0.f : a.zt[n];
  const int tiles = a.K > 0 ? a.ctas * a.max_tiles : 0;
  const float* tile_max = a.tile_max + static_cast<size_t>(n) * tiles;
  float cv[MERGE_BATCH];
  int ci[MERGE_BATCH];
  auto fetch = [&](int e0) {
#pragma unroll
    for (int k = 0; k < MERGE_BATCH; ++k) {
      const int e = e0 + k * MERGE_THREADS + tid;
      ci[k] = e < tiles ? e : TopK::NONE;
      cv[k] = e < tiles ? tile_max[e] : 0.f;
    }
  };
  fetch(0);
  int failed = 0;
  Stat acc = {-INFINITY, 0.f, 0.f};
  for (int b = tid; b < a.ctas; b += MERGE_THREADS) {
    failed |= a.fail[b];
    const float4 q = a.stat[static_cast<size_t>(n) * a.ctas + b];
    acc = merge(acc, Stat{q.x, q.y, q.z}, a.c2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {   // fixed order; lane 0 holds the result
    const Stat other = {__shfl_down_sync(0xffffffffu, acc.m, o), __shfl_down_sync(0xffffffffu, acc.s, o),
                        __shfl_down_sync(0xffffffffu, acc.d, o)};
    acc = merge(acc, other, a.c2);
  }
  if (lane == 0) part[w] = acc;
  failed = __syncthreads_or(failed);
  if (tid == 0 && (failed || bad))
    atomicOr(a.hdr + HDR_STATUS, (failed ? STATUS_TIMEOUT : 0) | (bad ? STATUS_BADTARGET : 0));
  if (failed || bad || t == a.ii) {
    const float v = t == a.ii ? 0.f : __int_as_float(0x7fc00000);
    if (tid == 0) {
      a.logp[n] = v;
      a.lse[n] = v;
      if (a.entropy) a.entropy[n] = v;
    }
    if (tid < a.K) {
      a.top_ids[static_cast<size_t>(n) * a.K + tid] = -1;
      a.top_logp[static_cast<size_t>(n) * a.K + tid] = v;
    }
    return;
  }
  acc = part[0];
#pragma unroll
  for (int k = 1; k < MERGE_WARPS; ++k) acc = merge(acc, part[k], a.c2);
  const float l2s = log2f(acc.s);
  if (tid == 0) {
    a.logp[n] = fmaf(zt - acc.m, a.c2, -l2s) * LN2;
    a.lse[n] = fmaf(acc.m, a.c2, l2s) * LN2;
    if (a.entropy) a.entropy[n] = fmaf(0.f, acc.m, l2s - acc.d / acc.s) * LN2;
  }
  if (a.K == 0) return;
  TopK best;
  best.clear();
  for (int e0 = 0;;) {
    best.offer_all(cv, ci, a.K, lane);
    e0 += MERGE_BATCH * MERGE_THREADS;
    if (e0 >= tiles) break;
    fetch(e0);
  }
  best.merge_block<MERGE_WARPS>(sv, si, lane, w);   // every warp holds the K best tiles
  const int top = best.id;
  const float least = __shfl_sync(0xffffffffu, best.v, a.K - 1);   // of K logits at least
  best.clear();
  const float* z = a.zf + static_cast<size_t>(n) * a.ldz;
  for (int j = w; j < a.K; j += 2 * MERGE_WARPS) {   // two tiles in flight
    float x[16];
    int id[16];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int jj = j + u * MERGE_WARPS;
      const int e = __shfl_sync(0xffffffffu, top, jj & 31);
      int r0 = 0, rows = 0;
      if (jj < a.K && e != TopK::NONE) {
        const Range r = range_of(a, e / a.max_tiles);
        r0 = r.start(e % a.max_tiles);
        rows = min(r.start(e % a.max_tiles + 1), a.V) - r0;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = k * 32 + lane;
        x[u * 8 + k] = at < rows ? z[r0 + at] : 0.f;
        id[u * 8 + k] = at < rows ? r0 + at : TopK::NONE;
      }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (!(x[k] >= least)) id[k] = TopK::NONE;
    best.offer_all(x, id, a.K, lane);
  }
  best.merge_block<MERGE_WARPS>(sv, si, lane, w);
  if (w == 0 && lane < a.K) {
    const bool some = best.id != TopK::NONE;   // false only where fewer than K logits are numbers
    a.top_ids[static_cast<size_t>(n) * a.K + lane] = some ? best.id : -1;
    a.top_logp[static_cast<size_t>(n) * a.K + lane] =
        some ? fmaf(best.v - acc.m, a.c2, -l2s) * LN2 : __int_as_float(0x7fc00000);
  }
}

__global__ void clear_groups_kernel(uint32_t* group_max, int n) {
  ptx::grid_launch_dependents();
  for (int i = threadIdx.x; i < n; i += blockDim.x) group_max[i] = 0u;
}

template <int NT>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(logprob_stream_kernel<NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<NT>::SMEM);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(logprob_stream_kernel<NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NT>::SMEM);
}

template <int NT, bool SEG>
cudaError_t launch_form(const StreamArgs& a, const StreamMaps& m, cudaStream_t s) {
  if (!a.group_max) {
    logprob_stream_kernel<NT, SEG><<<a.ctas, THREADS, Cfg<NT>::SMEM, s>>>(m, a);
    return cudaGetLastError();
  }
  // the weight streams while the groups' maxima are cleared
  clear_groups_kernel<<<1, 512, 0, s>>>(a.group_max, a.N * TopK::MAX);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent_smem(logprob_stream_kernel<NT, SEG>, a.ctas, THREADS, Cfg<NT>::SMEM, s, m, a);
}

template <int NT>
cudaError_t launch(const StreamArgs& a, const StreamMaps& m, cudaStream_t s) {
  return a.seg_kb * BK < a.H ? launch_form<NT, true>(a, m, s) : launch_form<NT, false>(a, m, s);
}

}  // namespace

int stream_max_tiles(long long V, int ctas) {
  return static_cast<int>(cdiv(cdiv(cdiv(V, UNIT_ROWS), ctas), TILE_ROWS / UNIT_ROWS));
}

int stream_ctas(long long V, int sms) {
  const long long units = cdiv(V, UNIT_ROWS);
  return static_cast<int>(units < sms ? units : sms);
}

cudaError_t stream_prepare() {
  cudaError_t e = prepare<16>();
  if (e == cudaSuccess) e = prepare<32>();
  if (e == cudaSuccess) e = prepare<64>();
  if (e == cudaSuccess) e = prepare<128>();
  return e;
}

int stream_tokens(int N) { return N <= 16 ? 16 : (N <= 32 ? 32 : (N <= 64 ? 64 : 128)); }

cudaError_t launch_stream(const StreamArgs& a, const StreamMaps& m, cudaStream_t s) {
  cudaError_t e;
  switch (stream_tokens(a.N)) {
    case 16: e = launch<16>(a, m, s); break;
    case 32: e = launch<32>(a, m, s); break;
    case 64: e = launch<64>(a, m, s); break;
    default: e = launch<128>(a, m, s); break;
  }
  if (e != cudaSuccess) return e;
  return launch_dependent(logprob_stream_merge_kernel, a.N, MERGE_THREADS, s, a);
}

}  // namespace flce
