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
// logits around in shared memory, where each warp takes whole tokens, two at a
// time: the running softmax statistics and the target's logit.  Every CTA leaves its
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
//
// With lists (ListView; the streaming kernel waits for them before its first
// finished tile, the weight streams meanwhile) a warp that has turned a token's
// tile around first treats the token's listed logits of that tile: under rules
// (LISTS_RULED) they are changed in place, and forbidden tokens count as -inf; a
// teacher's tokens (LISTS_TAKEN) are written out and leave the statistics.  Where
// the tile's entries begin and the words of its mask are fetched while the tile
// is being computed, a token's entries while the two before it are worked on.
// (128 tokens with 4001 ids of history, masks and 20 alternatives at 4096 x
// 128256, a call: fetched when needed 253 us, ahead 224, and with two tokens at a
// time 218; without lists 197 and 194.)
#pragma once

#include "flce_internal.h"
#include "flce_lists.cuh"
#include "flce_ptx.cuh"
#include "flce_softmax.cuh"
#include "flce_stream_range.cuh"
#include "flce_topk.cuh"

namespace flce {
namespace {

constexpr int W_BYTES = TILE_ROWS * BK * 2;
constexpr int EPI_WARPS = 8;
constexpr int EPI_THREADS = 32 * EPI_WARPS;
constexpr int THREADS = 64 + EPI_THREADS;
constexpr uint32_t EPI_BAR = 1;

// The ring takes what the slice buffer leaves of 227 KB.
constexpr int MAX_STAGES = 6;
enum Lists : int { LISTS_NONE = 0, LISTS_RULED = 1, LISTS_TAKEN = 2 };
constexpr int AHEAD = 12;   // words per token fetched ahead: first and last entry of the tile, nine words of its mask

template <int NT, int LISTS>
struct Cfg {
  static constexpr int STAGES = NT == 16 ? 6 : (NT == 128 ? 4 : 5);
  static constexpr int SLICE = NT == 32 ? 32 : 16;                // tokens turned around at once
  static constexpr int X_BYTES = NT * BK * 2;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int TURN_BYTES = SLICE * TILE_ROWS * 4;
  static constexpr int TMEM_COLS = 4 * NT;                        // two accumulators of two halves
  static constexpr int AHEAD_BYTES = LISTS == LISTS_NONE ? 0 : NT * AHEAD * 4;
  static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + TURN_BYTES + NT * 20 + AHEAD_BYTES + 256;
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

// One of a token's entries in a tile, per lane: fetched while the two tokens
// before it are worked on (the loads of one entry after the other cost the epilogue 1.5
// us a token and tile).
struct Entry {
  int id, seen;
  float bias;
};

template <int LISTS>
__device__ __forceinline__ Entry fetch_entry(const StreamLists& l, int tk, int e, int e1) {
  Entry x = {-1, 0, 0.f};
  if (e < e1) {
    const long long at = tk * l.lists.cap + e;
    x.id = l.lists.id[at];
    if (LISTS == LISTS_RULED) {
      x.seen = l.rules.seen[at];
      if (l.rules.bias) x.bias = l.rules.bias[at];
    }
  }
  return x;
}

// One token's listed logits of a tile, [r0, r0 + rows) of the vocabulary, in its
// slice z of shared memory, by the warp that goes on with it.  x: each lane's
// first entry.
template <int LISTS>
__device__ __forceinline__ void treat_listed(const StreamLists& l, int tk, int e0, int e1, Entry x, const RowRules& rules,
                                             int r0, int rows, float* z, int lane) {
  if (e0 >= e1) return;   // uniform
  for (int e = e0 + lane;;) {
    const int at = x.id - r0;
    if (x.id >= 0 && static_cast<unsigned>(at) < static_cast<unsigned>(rows)) {
      if (LISTS == LISTS_RULED) {
        z[at] = ruled(z[at], x.seen, x.bias, rules);
      } else {
        l.lists.z[tk * l.lists.cap + e] = z[at];
        z[at] = -INFINITY;
      }
    }
    e += 32;
    if (e >= e1) break;
    x = fetch_entry<LISTS>(l, tk, e, e1);
  }
  __syncwarp();
}

// SEG: the sum over H in segments (segment_blocks()), added up in registers.
template <int NT, bool SEG, int LISTS>
__global__ void __launch_bounds__(THREADS, 1)
    logprob_stream_kernel(const __grid_constant__ StreamMaps maps, const StreamArgs a, const StreamLists l) {
  using C = Cfg<NT, LISTS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* turn = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE_BYTES);          // [SLICE][TILE_ROWS]
  float4* stat = reinterpret_cast<float4*>(turn + C::SLICE * TILE_ROWS);              // [NT]
  uint32_t* bound = reinterpret_cast<uint32_t*>(stat + NT);                           // [NT]
  int* ahead = reinterpret_cast<int*>(bound + NT);                                   // [NT][AHEAD] with lists
  Ctl* ctl = reinterpret_cast<Ctl*>(ahead + C::AHEAD_BYTES / 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint64_t to = a.timeout_ns;
  const Range range = range_of(a.V, a.ctas, static_cast<int>(blockIdx.x));
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
    // the groups' maxima have been cleared, the lists have been made
    if (LISTS != LISTS_NONE || a.group_max) ptx::grid_dependency_wait();
    RowRules rules = {1.f, 0.f, 0.f};   // lane j: of this warp's j-th token
    static_assert(NT / EPI_WARPS <= 32, "a lane per token");
    if (LISTS == LISTS_RULED && lane < NT / EPI_WARPS && w + lane * EPI_WARPS < a.N)
      rules = row_rules(l.rules, w + lane * EPI_WARPS);
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
      if constexpr (LISTS != LISTS_NONE) {   // of this warp's tokens
        const int b = static_cast<int>(blockIdx.x) * a.max_tiles + i;
        const int words = (a.V + 31) / 32;
        for (int e = lane; e < NT / EPI_WARPS * AHEAD; e += 32) {
          const int tk = w + e / AHEAD * EPI_WARPS, c = e % AHEAD;
          if (tk >= a.N) break;
          int x = -1;
          if (c < 2) x = l.lists.start[static_cast<long long>(tk) * l.lists.boundaries + b + c];
          else if (l.lists.mask && c < 11 && r0 / 32 + c - 2 < words)
            x = static_cast<int>(l.lists.mask[tk * l.lists.mask_stride + r0 / 32 + c - 2]);
          ahead[tk * AHEAD + c] = x;
        }
        __syncwarp();
      }
      Entry entry[2];   // of the next two tokens
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        entry[k] = Entry{-1, 0, 0.f};
        const int tk = w + k * EPI_WARPS;
        if (LISTS != LISTS_NONE && tk < a.N)
          entry[k] = fetch_entry<LISTS>(l, tk, ahead[tk * AHEAD] + lane, ahead[tk * AHEAD + 1]);
      }
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
        // two tokens at a time, whose chains of latencies overlap
        static_assert(C::SLICE % (2 * EPI_WARPS) == 0, "pairs of a warp's tokens");
#pragma unroll 1
        for (int k = w; k < C::SLICE; k += 2 * EPI_WARPS) {
          const int tk = n0 + k;
          if (tk >= a.N) break;
          const bool two = tk + EPI_WARPS < a.N;   // else the second is the first again, and writes nothing
          const int other = two ? EPI_WARPS : 0;
          float* z[2] = {turn + k * TILE_ROWS, turn + (k + other) * TILE_ROWS};
          if constexpr (LISTS != LISTS_NONE) {
            const Entry now[2] = {entry[0], entry[1]};
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const int next = tk + (2 + p) * EPI_WARPS;
              if (next < a.N)
                entry[p] = fetch_entry<LISTS>(l, next, ahead[next * AHEAD] + lane, ahead[next * AHEAD + 1]);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              if (p == 1 && !two) break;
              const int t = tk + p * EPI_WARPS, j = t / EPI_WARPS;
              const RowRules mine = {__shfl_sync(0xffffffffu, rules.repetition, j),
                                     __shfl_sync(0xffffffffu, rules.frequency, j),
                                     __shfl_sync(0xffffffffu, rules.presence, j)};
              treat_listed<LISTS>(l, t, ahead[t * AHEAD], ahead[t * AHEAD + 1], now[p], mine, r0, rows, z[p], lane);
            }
          }
          float x[2][8], mx[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            mx[p] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              x[p][j] = j * 32 + lane < rows ? z[p][j * 32 + lane] : -INFINITY;
              if (LISTS == LISTS_RULED && l.lists.mask) {
                const int bit = r0 % 32 + lane;   // r0: a multiple of 16
                if (!((ahead[(tk + p * other) * AHEAD + 2 + j + bit / 32] >> (bit % 32)) & 1)) x[p][j] = -INFINITY;
              }
              mx[p] = fmaxf(mx[p], x[p][j]);
            }
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int p = 0; p < 2; ++p) mx[p] = fmaxf(mx[p], __shfl_xor_sync(0xffffffffu, mx[p], o));
          float mb[2], s[2], d[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            mb[p] = mx[p] == -INFINITY ? 0.f : -mx[p] * a.c2;
            s[p] = d[p] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float y = fmaf(x[p][j], a.c2, mb[p]);
              const float e = ptx::ex2(y);
              s[p] += e;
              d[p] = fmaf(fmaxf(y, -1e30f), e, d[p]);
            }
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              s[p] += __shfl_xor_sync(0xffffffffu, s[p], o);
              d[p] += __shfl_xor_sync(0xffffffffu, d[p], o);
            }
          if (lane < (two ? 2 : 1)) {   // a lane per token
            const bool q = lane == 1;
            const int t = tk + lane * EPI_WARPS;
            const float m = q ? mx[1] : mx[0], b = q ? mb[1] : mb[0], sum = q ? s[1] : s[0], wsum = q ? d[1] : d[0];
            // mb is rounded: every y is too large by rho (exact in the fused multiply-add)
            const float rho = m == -INFINITY ? 0.f : fmaf(m, a.c2, b);
            const float back = ptx::ex2(-rho);
            const float4 old = stat[t];
            const Stat r = merge(Stat{old.x, old.y, old.z}, Stat{m, back * sum, back * fmaf(-rho, sum, wsum)}, a.c2);
            stat[t] = make_float4(r.m, r.s, r.d, 0.f);
            if (LISTS == LISTS_NONE || a.targets) {
              const unsigned at = static_cast<unsigned>(a.targets[t]) - static_cast<unsigned>(r0);
              if (at < static_cast<unsigned>(rows)) a.zt[t] = (q ? z[1] : z[0])[at];
            }
            if (a.K > 0) {
              a.tile_max[static_cast<size_t>(t) * a.ctas * a.max_tiles + blockIdx.x * a.max_tiles + i] = m;
              if (a.group_max && order_key(m) >= bound[t])
                atomicMax(a.group_max + t * TopK::MAX + (blockIdx.x + i) % a.K, order_key(m));
            }
          }
          if (a.K > 0) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              if (p == 1 && !two) break;
              const int t = tk + p * EPI_WARPS;
              if (!a.group_max || order_key(mx[p]) >= bound[t]) {
                float* zf = a.zf + static_cast<size_t>(t) * a.ldz + r0 + lane;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (j * 32 + lane < rows) zf[j * 32] = x[p][j];
              }
            }
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

// RULED: forbidden tokens have logits of -inf.  They are no alternatives, a
// forbidden target has a log probability of -inf, and a row with nothing left a
// log-sum-exp of -inf and no entropy; without targets all rows count.
template <bool RULED>
__global__ void __launch_bounds__(MERGE_THREADS) logprob_stream_merge_kernel(const StreamArgs a, const ListView v) {
  __shared__ Stat part[MERGE_WARPS];
  __shared__ float sv[MERGE_WARPS][32];
  __shared__ int si[MERGE_WARPS][32];
  const int n = blockIdx.x, tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  const bool scored = !RULED || a.targets != nullptr;
  const int t = scored ? a.targets[n] : 0;
  const bool left = scored && t == a.ii;
  const bool bad = scored && !left && (t < 0 || t >= a.V);
  ptx::grid_dependency_wait();
  float zt = bad || left || !scored ? 0.f : a.zt[n];
  if (RULED && scored && !left && !bad && v.mask && !((v.mask[n * v.mask_stride + t / 32] >> (t % 32)) & 1u)) zt = -INFINITY;
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
  if (failed || bad || left) {
    const float v = left ? 0.f : __int_as_float(0x7fc00000);
    if (tid == 0) {
      if (!RULED || a.logp) a.logp[n] = v;
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
    const bool nothing = RULED && acc.m == -INFINITY && acc.s == 0.f;
    if (!RULED || a.logp)
      a.logp[n] = RULED && zt == -INFINITY && !(acc.s != acc.s) ? -INFINITY : fmaf(zt - acc.m, a.c2, -l2s) * LN2;
    a.lse[n] = nothing ? -INFINITY : fmaf(acc.m, a.c2, l2s) * LN2;
    if (a.entropy) a.entropy[n] = nothing ? 0.f : fmaf(0.f, acc.m, l2s - acc.d / acc.s) * LN2;
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
        const Range r = range_of(a.V, a.ctas, e / a.max_tiles);
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
    const bool some = best.id != TopK::NONE &&   // false only where fewer than K logits are numbers
                      !(RULED && best.v == -INFINITY);
    a.top_ids[static_cast<size_t>(n) * a.K + lane] = some ? best.id : -1;
    a.top_logp[static_cast<size_t>(n) * a.K + lane] =
        some ? fmaf(best.v - acc.m, a.c2, -l2s) * LN2
             : (RULED && acc.s == acc.s ? -INFINITY : __int_as_float(0x7fc00000));
  }
}

template <int NT, int LISTS>
cudaError_t prepare() {
  constexpr int SMEM = Cfg<NT, LISTS>::SMEM;
  cudaError_t e = cudaFuncSetAttribute(logprob_stream_kernel<NT, false, LISTS>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(logprob_stream_kernel<NT, true, LISTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
}

template <int LISTS>
cudaError_t prepare_all() {
  cudaError_t e = prepare<16, LISTS>();
  if (e == cudaSuccess) e = prepare<32, LISTS>();
  if (e == cudaSuccess) e = prepare<64, LISTS>();
  if (e == cudaSuccess) e = prepare<128, LISTS>();
  return e;
}

// The streaming kernel; `dependent`: the weight streams while the previous
// kernel of the stream (the groups' maxima cleared, the lists made) runs.
template <int NT, int LISTS>
cudaError_t launch_tokens(const StreamArgs& a, const StreamMaps& m, const StreamLists& l, bool dependent, cudaStream_t s) {
  const auto kernel = a.seg_kb * BK < a.H ? logprob_stream_kernel<NT, true, LISTS> : logprob_stream_kernel<NT, false, LISTS>;
  if (dependent) return launch_dependent_smem(kernel, a.ctas, THREADS, Cfg<NT, LISTS>::SMEM, s, m, a, l);
  kernel<<<a.ctas, THREADS, Cfg<NT, LISTS>::SMEM, s>>>(m, a, l);
  return launch_result(cudaGetLastError());
}

template <int LISTS>
cudaError_t launch_all(const StreamArgs& a, const StreamMaps& m, const StreamLists& l, bool dependent, cudaStream_t s) {
  switch (stream_tokens(a.N)) {
    case 16: return launch_tokens<16, LISTS>(a, m, l, dependent, s);
    case 32: return launch_tokens<32, LISTS>(a, m, l, dependent, s);
    case 64: return launch_tokens<64, LISTS>(a, m, l, dependent, s);
    default: return launch_tokens<128, LISTS>(a, m, l, dependent, s);
  }
}

}  // namespace
}  // namespace flce
