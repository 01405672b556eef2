// Scaled embedding lookup and its gradient.
//
//   out[n] = round(scale W[ids[n]])
//   grad_weight[v] (+)= scale sum_{n : ids[n] = v} grad_out[n]
//
// Both move bytes and compute next to nothing; the lookup reads the rows it
// needs and writes N rows.  The gradient must add the rows of equal ids, in a
// fixed order and without atomics, however often an id occurs (a frequent
// token takes a tenth of a batch).  So the tokens are sorted by id (a stable
// radix sort: equal ids stay in token order), and the sorted list is cut into
// chunks of equal length, whatever ids they hold:
//   segments  one warp per chunk and column slice adds up each run of equal
//             ids in fp32 registers.  A run inside the chunk is finished; one
//             that crosses a chunk's edge leaves a partial sum per chunk.
//   join      the partial sums of each crossing run, in chunk order.
// In the same launch as the segments, the rows of ids that do not occur are
// set to zero, so the dense gradient is written exactly once; these blocks
// need the ids only, not their order, and run while the sort does.
#include <algorithm>
#include <cuda_fp16.h>

#include "flce.h"
#include "flce_internal.h"
#include "flce_ptx.cuh"

namespace flce {
namespace {

// ---------------------------------------------------------------------------
// element types: 8 elements <-> 8 floats
// ---------------------------------------------------------------------------
struct Bf16 {
  static constexpr int SIZE = 2;
  using Raw = uint4;
  static __device__ __forceinline__ void unpack(const Raw& w, float (&f)[8]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(q[k] << 16);
      f[2 * k + 1] = __uint_as_float(q[k] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
    *static_cast<uint4*>(p) = make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]),
                                         ptx::pack_bf16x2(f[4], f[5]), ptx::pack_bf16x2(f[6], f[7]));
  }
};

struct F16 {
  static constexpr int SIZE = 2;
  using Raw = uint4;
  static __device__ __forceinline__ void unpack(const Raw& w, float (&f)[8]) {
    const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = __half22float2(h[k]);
      f[2 * k] = x.x;
      f[2 * k + 1] = x.y;
    }
  }
  static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
    uint4 w;
    __half2* h = reinterpret_cast<__half2*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
    *static_cast<uint4*>(p) = w;
  }
};

struct F32 {
  static constexpr int SIZE = 4;
  struct Raw {
    float4 a, b;
  };
  static __device__ __forceinline__ void unpack(const Raw& w, float (&f)[8]) {
    const float4 a = w.a, b = w.b;
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
    static_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    static_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <typename T>
__device__ __forceinline__ void load8(const void* p, float (&f)[8]) {
  T::unpack(*static_cast<const typename T::Raw*>(p), f);
}

constexpr int COLS = 32 * 8;   // columns a warp moves at once: 8 per lane

// ---------------------------------------------------------------------------
// lookup: a warp moves ROWS rows of one slice of 256 columns, all of them in
// flight at once (the latency of id, row and store is what a warp waits for).
// Bound by HBM: 65536 rows of 512 16.4 us with the launch (one 16-byte item per
// thread: 28.0), 65536 of 2048 72.6 us, 6.2 TB/s.
// ---------------------------------------------------------------------------
constexpr int LOOKUP_WARPS = 8;

template <typename T, int ROWS>
__global__ void __launch_bounds__(32 * LOOKUP_WARPS)
    embedding_kernel(const unsigned char* __restrict__ W, const int* __restrict__ ids, int N, int H, int V, int slices,
                     float scale, unsigned char* __restrict__ out) {
  const long long warp = static_cast<long long>(blockIdx.x) * LOOKUP_WARPS + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const long long n0 = warp / slices * ROWS;
  const int h = static_cast<int>(warp % slices) * COLS + lane * 8;
  if (n0 >= N || h >= H) return;
  int v[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) v[k] = n0 + k < N ? ids[n0 + k] : -1;
  typename T::Raw x[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
    if (static_cast<unsigned>(v[k]) < static_cast<unsigned>(V))
      x[k] = *reinterpret_cast<const typename T::Raw*>(W + (static_cast<long long>(v[k]) * H + h) * T::SIZE);
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    if (n0 + k >= N) break;
    float f[8];
    if (static_cast<unsigned>(v[k]) < static_cast<unsigned>(V)) {
      T::unpack(x[k], f);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] *= scale;
    } else {   // an id outside the table: a row of NaN
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = __int_as_float(0x7fc00000);
    }
    T::store(out + ((n0 + k) * H + h) * T::SIZE, f);
  }
}

template <typename T>
void launch_lookup(const void* W, const int* ids, long long N, int H, int V, float scale, void* out, cudaStream_t st) {
  const int slices = static_cast<int>(cdiv(H, COLS));
  const unsigned char* w = static_cast<const unsigned char*>(W);
  unsigned char* o = static_cast<unsigned char*>(out);
  // four rows a warp once that still fills the GPU (152 SMs x 16 warps)
  if (N * slices >= 4 * 16 * 152) {
    const unsigned grid = static_cast<unsigned>(cdiv(cdiv(N, 4) * slices, LOOKUP_WARPS));
    embedding_kernel<T, 4><<<grid, 32 * LOOKUP_WARPS, 0, st>>>(w, ids, static_cast<int>(N), H, V, slices, scale, o);
  } else {
    const unsigned grid = static_cast<unsigned>(cdiv(N * slices, LOOKUP_WARPS));
    embedding_kernel<T, 1><<<grid, 32 * LOOKUP_WARPS, 0, st>>>(w, ids, static_cast<int>(N), H, V, slices, scale, o);
  }
}

// ---------------------------------------------------------------------------
// stable radix sort of (id, token); ids left out (padding, out of range) are
// replaced by V and end up behind all others
// ---------------------------------------------------------------------------
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_MAX_BITS = 9;
constexpr int SORT_BINS = 1 << SORT_MAX_BITS;
static_assert(SORT_BINS == SORT_THREADS, "one thread per bin");
// Items per thread: small tiles keep the few thousand tokens of a step on many
// SMs; past 2^17 tokens larger ones bound the counts each tile has to add up.
constexpr int SORT_ITEMS_SMALL = 4;
constexpr int SORT_ITEMS_LARGE = 16;
constexpr long long SORT_LARGE = 1ll << 17;

__device__ __forceinline__ int sort_key(const int* ids, long long i, int V, int padding) {
  const int v = ids[i];
  return v < 0 || v >= V || v == padding ? V : v;
}

// Every kernel but the first is launched while its predecessor drains and waits
// for its end.  What a predecessor wrote is therefore read through plain
// pointers only: loads through const __restrict__ ones may be taken for
// invariant and moved ahead of the wait.  All positions, tokens and ids read
// back from the workspace are checked against their arrays before use.

// Lanes of the warp with the same digit (of `bits` bits) as this one, among
// those with ok; one ballot per bit.
__device__ __forceinline__ unsigned same_digit(int d, int bits, bool ok) {
  unsigned m = __ballot_sync(0xffffffffu, ok);
  for (int b = 0; b < bits; ++b) {
    const bool on = (d >> b) & 1;
    const unsigned y = __ballot_sync(0xffffffffu, on);
    m &= on ? y : ~y;
  }
  return m;
}

// Counts of one digit, per tile.  FIRST: the keys come from the ids, and ids
// outside the table are flagged per tile.
template <bool FIRST, int ITEMS>
__global__ void __launch_bounds__(SORT_THREADS)
    sort_count_kernel(const int* ids, const int2* items, int N, int V, int padding, int* bad, int shift, int bits,
                      int* counts) {
  __shared__ int bin[SORT_BINS];
  ptx::grid_launch_dependents();
  bin[threadIdx.x] = 0;
  __syncthreads();
  if (!FIRST) ptx::grid_dependency_wait();
  const int mask = (1 << bits) - 1;
  const long long base = static_cast<long long>(blockIdx.x) * (SORT_THREADS * ITEMS);
  int outside = 0;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const long long i = base + k * SORT_THREADS + threadIdx.x;
    if (i < N) {
      const int key = FIRST ? sort_key(ids, i, V, padding) : items[i].x;
      if (FIRST && key == V) outside |= ids[i] < 0 || ids[i] >= V;
      atomicAdd(&bin[(key >> shift) & mask], 1);
    }
  }
  outside = __syncthreads_or(outside);
  counts[blockIdx.x * SORT_BINS + threadIdx.x] = bin[threadIdx.x];
  if (FIRST && threadIdx.x == 0) bad[blockIdx.x] = outside;
}

template <int WARPS>
__device__ __forceinline__ int block_exclusive_scan(int x, int* scratch) {
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) scratch[w] = inc;
  __syncthreads();
  if (w == 0) {
    const int t = lane < WARPS ? scratch[lane] : 0;
    int ti = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) ti += y;
    }
    if (lane < WARPS) scratch[lane] = ti - t;
  }
  __syncthreads();
  return scratch[w] + inc - x;
}

// Counts of many tiles: block r turns the counts of a range of tiles into the
// sums over the range's tiles before each, and leaves the range's total.  A
// scatter block then reads one row per range, not one per tile, which would
// make the reads grow with the square of the tokens.  One more launch per digit
// for that (gradient at H = 8, V = 1000, without and with it: 2^19 tokens 103
// and 108 us, 2^20, 128 tiles, 155 and 156, 2^22 605 and 542, 2^26 25.3 and 9.3 ms).
constexpr int SCAN_TILES = 128;    // more tiles than this
constexpr int SCAN_RANGES = 64;    // their ranges
constexpr int SCAN_BATCH = 16;     // rows in flight
__global__ void __launch_bounds__(SORT_THREADS) sort_ranges_kernel(int* counts, int tiles, int each, int* range_sums) {
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int t0 = blockIdx.x * each, t1 = min(tiles, t0 + each);
  int sum = 0;
  for (int t = t0; t < t1; t += SCAN_BATCH) {
    int c[SCAN_BATCH];
#pragma unroll
    for (int k = 0; k < SCAN_BATCH; ++k) c[k] = t + k < t1 ? counts[(t + k) * SORT_BINS + threadIdx.x] : 0;
#pragma unroll
    for (int k = 0; k < SCAN_BATCH; ++k) {
      if (t + k < t1) counts[(t + k) * SORT_BINS + threadIdx.x] = sum;
      sum += c[k];
    }
  }
  range_sums[blockIdx.x * SORT_BINS + threadIdx.x] = sum;
}

// Every item moves to (items of smaller digits) + (items of its digit in
// earlier tiles) + (its rank among the tile's items of its digit).  A warp
// ranks its 32 x ITEMS consecutive items in order, so the sort is stable.
template <bool FIRST, int ITEMS>
__global__ void __launch_bounds__(SORT_THREADS)
    sort_scatter_kernel(const int* ids, const int2* items, int N, int V, int padding, int shift, int bits,
                        const int* counts, int tiles, const int* range_sums, int each, int2* out) {
  __shared__ int cnt[SORT_WARPS][SORT_BINS];
  __shared__ int scratch[32];
  const int tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  ptx::grid_launch_dependents();
  for (int k = 0; k < SORT_WARPS; ++k) cnt[k][tid] = 0;
  __syncthreads();
  const int mask = (1 << bits) - 1;
  int2 it[ITEMS];
  int rank[ITEMS];
  const long long base = static_cast<long long>(blockIdx.x) * (SORT_THREADS * ITEMS) + w * (32 * ITEMS);
  ptx::grid_dependency_wait();
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const long long i = base + k * 32 + lane;
    it[k] = make_int2(-1, 0);
    if (i < N) it[k] = FIRST ? make_int2(sort_key(ids, i, V, padding), static_cast<int>(i)) : items[i];
  }
  // thread d: total of digit d and its items in earlier tiles
  int total = 0, earlier = 0;
  const int* rows = each ? range_sums : counts;
  const int n_rows = each ? (tiles + each - 1) / each : tiles;
  const int my_row = each ? static_cast<int>(blockIdx.x) / each : static_cast<int>(blockIdx.x);
#pragma unroll 16
  for (int b = 0; b < n_rows; ++b) {
    const int c = rows[b * SORT_BINS + tid];
    total += c;
    earlier += b < my_row ? c : 0;
  }
  if (each) earlier += counts[blockIdx.x * SORT_BINS + tid];   // of the tiles before this one in its range
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const bool ok = base + k * 32 + lane < N;
    const int d = (it[k].x >> shift) & mask;
    const unsigned same = same_digit(d, bits, ok);
    int before = 0;
    if (ok) before = cnt[w][d];
    __syncwarp();
    if (ok && lane == __ffs(same) - 1) cnt[w][d] = before + __popc(same);
    __syncwarp();
    rank[k] = before + __popc(same & ((1u << lane) - 1u));
  }
  __syncthreads();
  int off = block_exclusive_scan<SORT_WARPS>(total, scratch) + earlier;   // then the warps' offsets
  for (int k = 0; k < SORT_WARPS; ++k) {
    const int c = cnt[k][tid];
    cnt[k][tid] = off;
    off += c;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if (base + k * 32 + lane < N) {
      const int pos = cnt[w][(it[k].x >> shift) & mask] + rank[k];
      if (static_cast<unsigned>(pos) < static_cast<unsigned>(N)) out[pos] = it[k];
    }
  }
}

// (15 us cold for 16384 tokens.)  The whole sort of up to 16384 tokens in one launch: a cluster of eight blocks
// holds the items in registers, adds up its digit counts through distributed
// shared memory and moves the items through L2 between passes.  (Past that the
// scattered stores of eight SMs take longer than three more launches.)
constexpr int CS_BLOCKS = 8;
constexpr int CS_THREADS = 1024;
constexpr int CS_WARPS = CS_THREADS / 32;
constexpr int CS_MAX_ITEMS = 2;
constexpr long long CS_MAX = static_cast<long long>(CS_BLOCKS) * CS_THREADS * CS_MAX_ITEMS;
constexpr int CS_SMEM = (CS_WARPS + 1) * SORT_BINS * 4;

struct ClusterSort {
  const int* ids;
  int N, V, padding, passes, bits;
  int* bad;
  int2 *items0, *items1;   // even passes write 0
};

template <int ITEMS>
__global__ void __cluster_dims__(CS_BLOCKS, 1, 1) __launch_bounds__(CS_THREADS)
    sort_cluster_kernel(const ClusterSort a) {
  extern __shared__ int sort_smem[];
  int(*cnt)[SORT_BINS] = reinterpret_cast<int(*)[SORT_BINS]>(sort_smem);   // [CS_WARPS][SORT_BINS]
  int* hist = sort_smem + CS_WARPS * SORT_BINS;                            // this block's counts, read by the others
  __shared__ int scratch[32];
  const int tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  const int rank_ = static_cast<int>(ptx::cluster_ctarank());
  const int base = (rank_ * CS_THREADS + w * 32) * ITEMS;
  const int mask = (1 << a.bits) - 1;
  ptx::grid_launch_dependents();
  int2 it[ITEMS];
  int rank[ITEMS];
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const int2* in = pass & 1 ? a.items0 : a.items1;
    int2* out = pass & 1 ? a.items1 : a.items0;
    int outside = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int i = base + k * 32 + lane;
      it[k] = make_int2(-1, i);
      if (i < a.N) {
        if (pass == 0) {
          const int v = a.ids[i];
          const bool bad = v < 0 || v >= a.V;
          outside |= bad;
          it[k].x = bad || v == a.padding ? a.V : v;
        } else {
          it[k] = __ldcg(in + i);
        }
      }
    }
    for (int k = 0; k < CS_WARPS * SORT_BINS / CS_THREADS; ++k) sort_smem[k * CS_THREADS + tid] = 0;
    outside = __syncthreads_or(outside);
    if (pass == 0 && tid == 0) a.bad[rank_] = outside;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const bool ok = base + k * 32 + lane < a.N;
      const int d = (it[k].x >> shift) & mask;
      const unsigned same = same_digit(d, a.bits, ok);
      int before = 0;
      if (ok) before = cnt[w][d];
      __syncwarp();
      if (ok && lane == __ffs(same) - 1) cnt[w][d] = before + __popc(same);
      __syncwarp();
      rank[k] = before + __popc(same & ((1u << lane) - 1u));
    }
    __syncthreads();
    if (tid < SORT_BINS) {
      int t = 0;
#pragma unroll
      for (int k = 0; k < CS_WARPS; ++k) t += cnt[k][tid];
      hist[tid] = t;
    }
    ptx::cluster_sync();
    int total = 0, earlier = 0;
    if (tid < SORT_BINS) {
#pragma unroll
      for (int b = 0; b < CS_BLOCKS; ++b) {
        const int c = ptx::ld_shared_cluster(ptx::map_to_rank(hist + tid, b));
        total += c;
        earlier += b < rank_ ? c : 0;
      }
    }
    int off = block_exclusive_scan<CS_WARPS>(total, scratch) + earlier;
    if (tid < SORT_BINS) {
#pragma unroll
      for (int k = 0; k < CS_WARPS; ++k) {
        const int c = cnt[k][tid];
        cnt[k][tid] = off;
        off += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      if (base + k * 32 + lane < a.N) {
        const int pos = cnt[w][(it[k].x >> shift) & mask] + rank[k];
        if (static_cast<unsigned>(pos) < static_cast<unsigned>(a.N)) out[pos] = it[k];
      }
    }
    ptx::cluster_sync();   // the items have moved, and no block reads this one's counts any more
  }
}

// ---------------------------------------------------------------------------
// sums over runs of equal ids
// ---------------------------------------------------------------------------
constexpr int SEG_WARPS = 8;
constexpr int CHUNK = 64;              // sorted entries per chunk (32 to 128 tried), fewer where that leaves
constexpr int MIN_CHUNK = 8;           // less than eight warps an SM, and
constexpr int MAX_CHUNKS = 4096;       // at most this many chunks (two partial sums of H floats each)
constexpr int ZERO_ROWS = 32;          // grad_weight rows a warp looks up at once
constexpr int ZERO_MAX_ROWS = 8192;    // rows a block marks at most (1 KB of bits)
constexpr long long ZERO_BYTES = 768 << 10;

struct SegArgs {
  const int2* items;     // (id, token) sorted by id, [N]
  const unsigned char* dout;
  int N, H, V;
  int chunk;             // entries per chunk
  int n_chunks, slices;
  float scale;
  int accumulate;
  unsigned char* gw;
  float* part;           // [n_chunks][2][H]: 0 = sum of the run that came in, 1 = of the run that goes out
  int* hdr;
  const int* bad;        // [tiles] whether a tile of the first sort pass held an id outside the table
  int tiles;
  const int* ids;        // the unsorted ids, and
  int padding;
  int scan;              // whether the zeroing blocks go by them
  int seg_blocks;        // blocks that add up runs, and
  int zero_blocks;       // blocks that set rows to zero
  int zero_rows;         // rows per such block
};

template <typename O>
__device__ __forceinline__ void write_row(const SegArgs& a, int v, int h, const float (&s)[8]) {
  unsigned char* p = a.gw + (static_cast<long long>(v) * a.H + h) * O::SIZE;
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = s[k] * a.scale;
  if (a.accumulate) {
    float g[8];
    load8<O>(p, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] += g[k];
  }
  O::store(p, f);
}

template <typename T, typename O>
__device__ __forceinline__ void segments(const SegArgs& a, long long warp, int lane) {
  constexpr int SEG_ROWS = 16 / T::SIZE;   // rows a warp has in flight: 128 bytes a lane
  const int c = static_cast<int>(warp / a.slices), slice = static_cast<int>(warp % a.slices);
  const int h = slice * COLS + lane * 8;
  const bool live = h < a.H;
  const int i0 = c * a.chunk, i1 = min(a.N, i0 + a.chunk);
  const int before = i0 > 0 ? a.items[i0 - 1].x : -1;
  const int after = i1 < a.N ? a.items[i1].x : a.V;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const unsigned nv = static_cast<unsigned>(a.V), nn = static_cast<unsigned>(a.N);
  auto group = [&](int g0) { return g0 + lane < i1 ? a.items[g0 + lane] : make_int2(a.V, 0); };
  typename T::Raw x[SEG_ROWS];   // a rolling window: a row's place is refilled as soon as it has been added
  auto fetch = [&](const int2& from, int j, typename T::Raw& to) {
    const unsigned key = __shfl_sync(0xffffffffu, from.x, j), tok = __shfl_sync(0xffffffffu, from.y, j);
    if (live && key < nv && tok < nn)
      to = *reinterpret_cast<const typename T::Raw*>(a.dout + (static_cast<long long>(tok) * a.H + h) * T::SIZE);
  };
  int2 my = group(i0);
  int cur = __shfl_sync(0xffffffffu, my.x, 0);
  bool came_in = cur == before;
#pragma unroll
  for (int q = 0; q < SEG_ROWS; ++q) fetch(my, q, x[q]);
  for (int g0 = i0; g0 < i1; g0 += 32) {
    const int2 next = group(g0 + 32);
    const int m = min(32, i1 - g0);
#pragma unroll 1
    for (int j0 = 0; j0 < m; j0 += SEG_ROWS) {
      const int2 from = j0 + SEG_ROWS < 32 ? my : next;
#pragma unroll
      for (int q = 0; q < SEG_ROWS; ++q) {
        const int key = __shfl_sync(0xffffffffu, my.x, j0 + q);   // the table's size behind the last entry
        if (key != cur) {   // uniform over the warp: the run ends inside the chunk
          if (live && static_cast<unsigned>(cur) < nv && j0 + q < m) {
            if (came_in) F32::store(a.part + (2ll * c) * a.H + h, s);
            else write_row<O>(a, cur, h, s);
          }
          if (j0 + q < m) {
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = 0.f;
            cur = key;
            came_in = false;
          }
        }
        if (live && static_cast<unsigned>(key) < nv) {
          float f[8];
          T::unpack(x[q], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) s[k] += f[k];
        }
        fetch(from, (j0 + SEG_ROWS + q) & 31, x[q]);
      }
    }
    my = next;
  }
  if (!live || static_cast<unsigned>(cur) >= nv) return;
  if (came_in) F32::store(a.part + (2ll * c) * a.H + h, s);
  else if (cur == after) F32::store(a.part + (2ll * c + 1) * a.H + h, s);
  else write_row<O>(a, cur, h, s);
}

// First position whose key is >= v.
__device__ __forceinline__ int lower_bound(const int2* items, int n, int v) {
  int lo = 0, len = n;
  while (len > 0) {
    const int half = len / 2;
    if (items[lo + half].x < v) {
      lo += half + 1;
      len -= half + 1;
    } else {
      len = half;
    }
  }
  return lo;
}

// The rows of one block whose id does not occur.  With `scan`, the block reads
// all the ids (from L2) and marks those of its rows, so it need not wait for
// the sort; else its warps look up 32 rows each in the sorted ids (262144 tokens
// at 64 x 128256: 91 us for the gradient, 111 with one search after another).
template <typename O>
__device__ __forceinline__ void zero_absent(const SegArgs& a, int block, unsigned* seen) {
  constexpr int THREADS = 32 * SEG_WARPS;
  const long long r0 = static_cast<long long>(block) * a.zero_rows;
  const long long r1 = min(r0 + a.zero_rows, static_cast<long long>(a.V));
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  if (a.scan) {
    for (int i = threadIdx.x; i < ZERO_MAX_ROWS / 32; i += THREADS) seen[i] = 0;
    __syncthreads();
#pragma unroll 8
    for (int i = threadIdx.x; i < a.N; i += THREADS) {
      const int v = a.ids[i];
      if (v >= r0 && v < r1 && v != a.padding) {
        const int k = static_cast<int>(v - r0);
        atomicOr(&seen[k / 32], 1u << (k % 32));
      }
    }
  } else {   // 32 rows a warp; every search is some 20 dependent loads
    for (long long q = r0 + w * 32; q < r1; q += SEG_WARPS * 32) {
      bool found = false;
      if (q + lane < r1) {
        const int v = static_cast<int>(q + lane);
        const int at = lower_bound(a.items, a.N, v);
        found = at < a.N && a.items[at].x == v;
      }
      const unsigned m = __ballot_sync(0xffffffffu, found);
      if (lane == 0) seen[(q - r0) / 32] = m;
    }
  }
  __syncthreads();
  const long long row_bytes = static_cast<long long>(a.H) * O::SIZE;
  for (long long q0 = r0; q0 < r1; q0 += ZERO_ROWS) {
    unsigned m = ~seen[(q0 - r0) / 32];   // rows q0 + k that do not occur
    if (r1 - q0 < 32) m &= (1u << (r1 - q0)) - 1u;
    // a long row by the whole block, others dealt to the warps: fewer places
    // are written at once
    const bool whole = row_bytes >= THREADS * 16;
    for (int n = 0; m; ++n) {
      const int k = __ffs(m) - 1;
      m &= m - 1;
      if (!whole && n % SEG_WARPS != w) continue;
      uint4* p = reinterpret_cast<uint4*>(a.gw + (q0 + k) * row_bytes);
      for (int i = whole ? static_cast<int>(threadIdx.x) : lane; i < row_bytes / 16; i += whole ? THREADS : 32)
        p[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

template <typename T, typename O>
__global__ void __launch_bounds__(32 * SEG_WARPS, 2) embedding_segments_kernel(const SegArgs a) {
  __shared__ unsigned seen[ZERO_MAX_ROWS / 32];
  ptx::grid_launch_dependents();
  // zeroing blocks that need not wait come first, others last
  const int first = a.scan ? 0 : a.seg_blocks;
  const int block = static_cast<int>(blockIdx.x);
  if (block >= first && block < first + a.zero_blocks) {
    // the sort's first kernel starts behind everything before the call, so
    // grad_weight may be written from here on
    if (!a.scan) ptx::grid_dependency_wait();
    zero_absent<O>(a, block - first, seen);
    return;
  }
  ptx::grid_dependency_wait();
  const long long warp = static_cast<long long>(block - (a.scan ? a.zero_blocks : 0)) * SEG_WARPS + threadIdx.x / 32;
  if (warp < static_cast<long long>(a.n_chunks) * a.slices) segments<T, O>(a, warp, threadIdx.x % 32);
}

// A run that goes out of chunk c and comes into c + 1, c + 2, ...: its partial
// sums.  A block looks at 16 chunks (of one column slice), one per warp.  A
// short chain is added up by its warp; a long one (a token that makes a tenth
// of 65536 has 100 links) by the whole block, cut in as many equal parts as
// there are warps, whose sums are added in order.  Latency: 8 us at 65536 x 512
// (151 us with one warp per chain).  All tokens alike at 262144 x 64: 130 us for
// the gradient with 16 warps a block, 147 with eight, 128 with 32, which are up
// to 17% slower where chains are short.
constexpr int JOIN_WARPS = 16;
constexpr int JOIN_LINKS = 8;          // partial sums a warp has in flight
constexpr int JOIN_SHORT = JOIN_LINKS;

__device__ __forceinline__ void add_links(const SegArgs& a, int k0, int k1, int h, float (&s)[8]) {
  for (int k = k0; k < k1; k += JOIN_LINKS) {
    F32::Raw x[JOIN_LINKS];
#pragma unroll
    for (int q = 0; q < JOIN_LINKS; ++q)
      if (k + q < k1) x[q] = *reinterpret_cast<const F32::Raw*>(a.part + (2ll * (k + q)) * a.H + h);
#pragma unroll
    for (int q = 0; q < JOIN_LINKS; ++q) {
      if (k + q >= k1) break;
      float f[8];
      F32::unpack(x[q], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += f[j];
    }
  }
}

template <typename O>
__global__ void __launch_bounds__(32 * JOIN_WARPS) embedding_join_kernel(const SegArgs a) {
  __shared__ __align__(16) float sums[JOIN_WARPS][COLS];
  __shared__ int links[JOIN_WARPS];   // of the long chains, else 0
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int c0 = static_cast<int>(blockIdx.x / a.slices) * JOIN_WARPS;
  const int h = static_cast<int>(blockIdx.x % a.slices) * COLS + lane * 8;
  ptx::grid_dependency_wait();
  if (blockIdx.x == 0) {   // the status word of the call
    int outside = 0;
    for (int t = threadIdx.x; t < a.tiles; t += 32 * JOIN_WARPS) outside |= a.bad[t];
    outside = __syncthreads_or(outside);
    if (threadIdx.x == 0) {
      a.hdr[HDR_STATUS] = outside ? STATUS_BADTARGET : 0;
      a.hdr[HDR_STALL] = a.hdr[HDR_STALL_COUNT] = 0;
    }
  }
  // this warp's chunk: does a run begin in it and go out, and how many chunks
  // does it come into?
  const int c = c0 + w;
  int n = 0;
  const long long i0 = static_cast<long long>(c) * a.chunk, i1 = i0 + a.chunk;
  if (i1 < a.N) {
    const int v = a.items[i1 - 1].x;
    const bool from_before = i0 > 0 && a.items[i0 - 1].x == v;
    if (static_cast<unsigned>(v) < static_cast<unsigned>(a.V) && !from_before) {
      for (bool more = true; more;) {   // 128 chunks at a time; uniform over the warp
        int key[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // first entries of later chunks
          const long long at = (static_cast<long long>(c) + 1 + n + q * 32 + lane) * a.chunk;
          key[q] = at < a.N ? a.items[at].x : -1;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (!more) continue;
          const unsigned in = __ballot_sync(0xffffffffu, key[q] == v);
          more = in == 0xffffffffu;
          n += more ? 32 : __ffs(~in) - 1;
        }
      }
    }
    if (n > 0 && n <= JOIN_SHORT && h < a.H) {
      float s[8];
      load8<F32>(a.part + (2ll * c + 1) * a.H + h, s);
      add_links(a, c + 1, c + 1 + n, h, s);
      write_row<O>(a, v, h, s);
    }
  }
  if (lane == 0) links[w] = n > JOIN_SHORT ? n : 0;
  __syncthreads();
  for (int j = 0; j < JOIN_WARPS; ++j) {
    const int m = links[j];
    if (m == 0) continue;   // uniform over the block
    const int first = c0 + j + 1;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (h < a.H) {
      if (w == 0) load8<F32>(a.part + (2ll * first - 1) * a.H + h, s);   // the first chunk's outgoing sum
      add_links(a, first + static_cast<int>(static_cast<long long>(m) * w / JOIN_WARPS),
                first + static_cast<int>(static_cast<long long>(m) * (w + 1) / JOIN_WARPS), h, s);
    }
    F32::store(&sums[w][lane * 8], s);
    __syncthreads();
    if (w == 0 && h < a.H) {
#pragma unroll
      for (int k = 1; k < JOIN_WARPS; ++k) {
        float f[8];
        load8<F32>(&sums[k][lane * 8], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) s[q] += f[q];
      }
      write_row<O>(a, a.items[static_cast<long long>(first) * a.chunk - 1].x, h, s);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
struct EmbPlan {
  int tiles = 0, passes = 0, bits = 0, chunk = 0, n_chunks = 0;
  int range_tiles = 0;   // tiles of a range of counts (0: the counts are few)
  size_t o_items[2] = {0, 0}, o_cnt = 0, o_range = 0, o_bad = 0, o_part = 0, total = 0;
};

EmbPlan emb_plan(long long N, long long H, long long V) {
  EmbPlan p;
  int key_bits = 1;
  while ((V >> key_bits) != 0) ++key_bits;   // keys 0 .. V
  p.passes = static_cast<int>(cdiv(key_bits, SORT_MAX_BITS));
  p.bits = static_cast<int>(cdiv(key_bits, p.passes));
  p.tiles = N <= CS_MAX ? CS_BLOCKS : static_cast<int>(cdiv(N, SORT_THREADS * (N <= SORT_LARGE ? SORT_ITEMS_SMALL : SORT_ITEMS_LARGE)));
  if (p.tiles > SCAN_TILES) p.range_tiles = static_cast<int>(cdiv(p.tiles, SCAN_RANGES));
  p.chunk = static_cast<int>(cdiv(std::max<long long>(CHUNK, cdiv(N, MAX_CHUNKS)), 32) * 32);
  while (p.chunk > MIN_CHUNK && cdiv(N, p.chunk) * cdiv(H, COLS) < 8 * 152) p.chunk /= 2;
  p.n_chunks = static_cast<int>(cdiv(N, p.chunk));
  size_t off = al256(HDR_WORDS * sizeof(int));
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += al256(bytes);
    return o;
  };
  for (int k = 0; k < 2; ++k) p.o_items[k] = take(size_t(N) * sizeof(int2));
  p.o_cnt = take(size_t(p.tiles) * SORT_BINS * 4);
  if (p.range_tiles) p.o_range = take(size_t(SCAN_RANGES) * SORT_BINS * 4);
  p.o_bad = take(size_t(p.tiles) * 4);
  p.o_part = take(size_t(p.n_chunks) * 2 * H * 4);
  p.total = off;
  return p;
}

bool emb_sizes_ok(long long N, long long H, long long V) { return sizes_ok(N, H, V) && N <= (1ll << 30); }

struct SortPass {
  const int* ids;
  const int2* items;
  int N, V, padding, shift, bits, tiles, range_tiles;
  int *bad, *counts, *range_sums;
  int2* out;
};

template <bool FIRST, int ITEMS>
cudaError_t sort_pass(const SortPass& s, cudaStream_t st) {
  cudaError_t e;
  if (FIRST) {   // behind everything before the call
    sort_count_kernel<FIRST, ITEMS><<<s.tiles, SORT_THREADS, 0, st>>>(s.ids, s.items, s.N, s.V, s.padding,
                                                                      s.bad, s.shift, s.bits, s.counts);
    e = cudaGetLastError();
  } else {
    e = launch_dependent(sort_count_kernel<FIRST, ITEMS>, s.tiles, SORT_THREADS, st, s.ids, s.items, s.N, s.V,
                         s.padding, s.bad, s.shift, s.bits, s.counts);
  }
  if (e != cudaSuccess) return e;
  if (s.range_tiles) {
    e = launch_dependent(sort_ranges_kernel, static_cast<unsigned>(cdiv(s.tiles, s.range_tiles)), SORT_THREADS, st,
                         s.counts, s.tiles, s.range_tiles, s.range_sums);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(sort_scatter_kernel<FIRST, ITEMS>, s.tiles, SORT_THREADS, st, s.ids, s.items, s.N, s.V,
                          s.padding, s.shift, s.bits, s.counts, s.tiles, s.range_sums, s.range_tiles, s.out);
}

template <int ITEMS>
cudaError_t sort_cluster(const ClusterSort& s, cudaStream_t st) {
  sort_cluster_kernel<ITEMS><<<CS_BLOCKS, CS_THREADS, CS_SMEM, st>>>(s);
  return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t sums(const SegArgs& a, long long blocks, cudaStream_t st) {
  const cudaError_t e =
      launch_dependent(embedding_segments_kernel<T, O>, static_cast<unsigned>(blocks), 32 * SEG_WARPS, st, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(embedding_join_kernel<O>, static_cast<unsigned>(cdiv(a.n_chunks, JOIN_WARPS) * a.slices),
                          32 * JOIN_WARPS, st, a);
}

template <typename T>
cudaError_t sums(const SegArgs& a, int out_dtype, long long blocks, cudaStream_t st) {
  if (out_dtype == FLCE_BF16) return sums<T, Bf16>(a, blocks, st);
  if (out_dtype == FLCE_F16) return sums<T, F16>(a, blocks, st);
  return sums<T, F32>(a, blocks, st);
}

bool known_dtype(int d) { return d == FLCE_BF16 || d == FLCE_F16 || d == FLCE_F32; }

}  // namespace

cudaError_t embedding_prepare() {
  cudaError_t e = cudaFuncSetAttribute(sort_cluster_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, CS_SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(sort_cluster_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, CS_SMEM);
  return e;
}

}  // namespace flce

using namespace flce;

extern "C" {

flce_status flce_embedding(const void* weight, const int32_t* ids, int64_t N, int64_t H, int64_t V, int32_t dtype,
                           float scale, void* out, void* stream) {
  if (!weight || !ids || !out || N < 1 || H < 1 || V < 1 || !known_dtype(dtype)) return FLCE_EINVAL;
  if (!sizes_ok(N, H, V) || !aligned16(weight) || !aligned16(out) || !aligned4(ids)) return FLCE_EUNSUPPORTED;
  DeviceState dev;
  if (device_state(&dev) != cudaSuccess) { cudaGetLastError(); return FLCE_ECUDA; }
  if (dev.major < 10) return FLCE_EUNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int h = static_cast<int>(H), v = static_cast<int>(V);
  count_launches(1);
  if (dtype == FLCE_BF16) launch_lookup<Bf16>(weight, ids, N, h, v, scale, out, st);
  else if (dtype == FLCE_F16) launch_lookup<F16>(weight, ids, N, h, v, scale, out, st);
  else launch_lookup<F32>(weight, ids, N, h, v, scale, out, st);
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ECUDA;
}

size_t flce_embedding_bwd_workspace_bytes(int64_t N, int64_t H, int64_t V) {
  return emb_sizes_ok(N, H, V) ? emb_plan(N, H, V).total : 0;
}

flce_status flce_embedding_bwd(const void* grad_out, const int32_t* ids, int64_t N, int64_t H, int64_t V,
                               int32_t dtype, float scale, int32_t padding_idx, uint32_t flags, void* grad_weight,
                               int32_t grad_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!grad_out || !ids || !grad_weight || !workspace || N < 1 || H < 1 || V < 1) return FLCE_EINVAL;
  if (!known_dtype(dtype) || !known_dtype(grad_dtype) || (flags & ~FLCE_ACCUMULATE)) return FLCE_EINVAL;
  if ((flags & FLCE_ACCUMULATE) && grad_dtype != FLCE_F32) return FLCE_EINVAL;
  if (padding_idx >= V) return FLCE_EINVAL;
  if (!emb_sizes_ok(N, H, V) || !aligned16(grad_out) || !aligned16(grad_weight) || !aligned16(workspace) ||
      !aligned4(ids))
    return FLCE_EUNSUPPORTED;
  DeviceState dev;
  if (device_state(&dev) != cudaSuccess) { cudaGetLastError(); return FLCE_ECUDA; }
  if (dev.major < 10) return FLCE_EUNSUPPORTED;
  const EmbPlan p = emb_plan(N, H, V);
  if (p.total > workspace_bytes) return FLCE_EWORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* hdr = at<int>(workspace, 0);
  int2* items[2] = {at<int2>(workspace, p.o_items[0]), at<int2>(workspace, p.o_items[1])};
  int* cnt = at<int>(workspace, p.o_cnt);
  int* ranges = at<int>(workspace, p.o_range);
  const int n = static_cast<int>(N), v = static_cast<int>(V);

  int* bad = at<int>(workspace, p.o_bad);

  count_launches(2 + (N <= CS_MAX ? 1 : (p.range_tiles ? 3 : 2) * p.passes));
  if (N <= CS_MAX) {
    const ClusterSort s = {ids, n, v, padding_idx, p.passes, p.bits, bad, items[0], items[1]};
    const long long each = CS_BLOCKS * CS_THREADS;
    const cudaError_t e = N <= each ? sort_cluster<1>(s, st) : sort_cluster<2>(s, st);
    if (e != cudaSuccess) return FLCE_ECUDA;
  }
  for (int k = 0; N > CS_MAX && k < p.passes; ++k) {
    const SortPass s = {ids, items[(k + 1) & 1], n, v, padding_idx, k * p.bits, p.bits, p.tiles, p.range_tiles, bad,
                        cnt, ranges, items[k & 1]};
    const bool large = N > SORT_LARGE;
    const cudaError_t e =
        k == 0 ? (large ? sort_pass<true, SORT_ITEMS_LARGE>(s, st) : sort_pass<true, SORT_ITEMS_SMALL>(s, st))
               : (large ? sort_pass<false, SORT_ITEMS_LARGE>(s, st) : sort_pass<false, SORT_ITEMS_SMALL>(s, st));
    if (e != cudaSuccess) return FLCE_ECUDA;
  }
  SegArgs a;
  a.items = items[(p.passes - 1) & 1];
  a.dout = static_cast<const unsigned char*>(grad_out);
  a.N = n; a.H = static_cast<int>(H); a.V = v;
  a.chunk = p.chunk; a.n_chunks = p.n_chunks;
  a.slices = static_cast<int>(cdiv(H, COLS));
  a.scale = scale;
  a.accumulate = (flags & FLCE_ACCUMULATE) ? 1 : 0;
  a.gw = static_cast<unsigned char*>(grad_weight);
  a.part = at<float>(workspace, p.o_part);
  a.hdr = hdr;
  a.bad = bad;
  a.tiles = p.tiles;
  a.ids = ids;
  a.padding = padding_idx;
  const long long seg_blocks = cdiv(static_cast<long long>(a.n_chunks) * a.slices, SEG_WARPS);
  // zeroing: at least four blocks per SM, of whole groups of 32 rows and of no
  // more than about 1 MB: larger ones leave a second wave that few SMs share
  // (16384 tokens at 4096 x 128256: 410 us with 3.6 MB a block, 332 with 1 MB)
  const long long row_bytes = H * (grad_dtype == FLCE_F32 ? 4 : 2);
  const long long zero_rows = std::min(cdiv(V, 4 * 152), ZERO_BYTES / row_bytes);
  a.zero_rows = static_cast<int>(std::min<long long>(std::max(1ll, cdiv(zero_rows, ZERO_ROWS)) * ZERO_ROWS, ZERO_MAX_ROWS));
  const long long zero_blocks = a.accumulate ? 0 : cdiv(V, a.zero_rows);
  // reading all ids is worth it where it is little next to the rows written, and
  // for no more tokens than that (65536 at 4096 x 128256: 507 us with it, 423 without)
  a.scan = N <= CS_MAX && 16 * N <= a.zero_rows * row_bytes ? 1 : 0;
  a.zero_blocks = static_cast<int>(zero_blocks);
  a.seg_blocks = static_cast<int>(seg_blocks);
  const long long blocks = seg_blocks + zero_blocks;
  if (blocks >= (1ll << 31)) return FLCE_EUNSUPPORTED;
  const cudaError_t e = dtype == FLCE_BF16  ? sums<Bf16>(a, grad_dtype, blocks, st)
                        : dtype == FLCE_F16 ? sums<F16>(a, grad_dtype, blocks, st)
                                            : sums<F32>(a, grad_dtype, blocks, st);
  return e == cudaSuccess ? FLCE_OK : FLCE_ECUDA;
}

}  // extern "C"
