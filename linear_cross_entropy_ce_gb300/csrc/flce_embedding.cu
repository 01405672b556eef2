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
// set to zero (found by binary search in the sorted ids), so the dense
// gradient is written exactly once.
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
  static __device__ __forceinline__ void load(const void* p, float (&f)[8]) {
    const uint4 w = *static_cast<const uint4*>(p);
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
  static __device__ __forceinline__ void load(const void* p, float (&f)[8]) {
    const uint4 w = *static_cast<const uint4*>(p);
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
  static __device__ __forceinline__ void load(const void* p, float (&f)[8]) {
    const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
    static_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    static_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// ---------------------------------------------------------------------------
// lookup: one thread per 8 columns of a row, grid-stride
// ---------------------------------------------------------------------------
constexpr int LOOKUP_THREADS = 256;

template <typename T>
__global__ void __launch_bounds__(LOOKUP_THREADS)
    embedding_kernel(const unsigned char* __restrict__ W, const int* __restrict__ ids, long long N, int H8, int V,
                     float scale, unsigned char* __restrict__ out) {
  const long long total = N * H8;
  for (long long i = static_cast<long long>(blockIdx.x) * LOOKUP_THREADS + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * LOOKUP_THREADS) {
    const long long n = i / H8;
    const int c = static_cast<int>(i - n * H8);
    const int v = ids[n];
    float f[8];
    if (v >= 0 && v < V) {
      T::load(W + (static_cast<long long>(v) * H8 + c) * (8 * T::SIZE), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= scale;
    } else {   // an id outside the table: a row of NaN
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = __int_as_float(0x7fc00000);
    }
    T::store(out + i * (8 * T::SIZE), f);
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
constexpr int SORT_ITEMS = 8;                           // per thread
constexpr int SORT_TILE = SORT_THREADS * SORT_ITEMS;

__device__ __forceinline__ int sort_key(const int* ids, long long i, int V, int padding, int* hdr) {
  const int v = ids[i];
  if (v < 0 || v >= V) {
    atomicOr(hdr + HDR_STATUS, STATUS_BADTARGET);
    return V;
  }
  return v == padding ? V : v;
}

// Counts of one digit, per tile.  first: keys come from ids.
template <bool FIRST>
__global__ void __launch_bounds__(SORT_THREADS)
    sort_count_kernel(const int* __restrict__ keys, int N, int V, int padding, int* hdr, int shift, int bits,
                      int* __restrict__ counts) {
  __shared__ int bin[SORT_BINS];
  bin[threadIdx.x] = 0;
  __syncthreads();
  const int mask = (1 << bits) - 1;
  const long long base = static_cast<long long>(blockIdx.x) * SORT_TILE;
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) {
    const long long i = base + k * SORT_THREADS + threadIdx.x;
    if (i < N) {
      const int key = FIRST ? sort_key(keys, i, V, padding, hdr) : keys[i];
      atomicAdd(&bin[(key >> shift) & mask], 1);
    }
  }
  __syncthreads();
  counts[blockIdx.x * SORT_BINS + threadIdx.x] = bin[threadIdx.x];
}

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
    const int t = lane < SORT_WARPS ? scratch[lane] : 0;
    int ti = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) ti += y;
    }
    if (lane < SORT_WARPS) scratch[lane] = ti - t;
  }
  __syncthreads();
  return scratch[w] + inc - x;
}

// Every item moves to (items of smaller digits) + (items of its digit in
// earlier tiles) + (its rank among the tile's items of its digit).  A warp
// ranks its 32 x ITEMS consecutive items in order, so the sort is stable.
template <bool FIRST>
__global__ void __launch_bounds__(SORT_THREADS)
    sort_scatter_kernel(const int* __restrict__ keys, const int* __restrict__ toks, int N, int V, int padding,
                        int* hdr, int shift, int bits, const int* __restrict__ counts, int tiles,
                        int* __restrict__ out_keys, int* __restrict__ out_toks) {
  __shared__ int cnt[SORT_WARPS][SORT_BINS];
  __shared__ int scratch[32];
  const int tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  for (int k = 0; k < SORT_WARPS; ++k) cnt[k][tid] = 0;
  __syncthreads();
  const int mask = (1 << bits) - 1;
  int key[SORT_ITEMS], rank[SORT_ITEMS];
  const long long base = static_cast<long long>(blockIdx.x) * SORT_TILE + w * (32 * SORT_ITEMS);
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) {
    const long long i = base + k * 32 + lane;
    const bool ok = i < N;
    key[k] = ok ? (FIRST ? sort_key(keys, i, V, padding, hdr) : keys[i]) : -1;
    const int d = ok ? (key[k] >> shift) & mask : SORT_BINS;   // past the end: a group of their own
    const unsigned same = __match_any_sync(0xffffffffu, d);
    int before = 0;
    if (ok) before = cnt[w][d];
    __syncwarp();
    if (ok && lane == __ffs(same) - 1) cnt[w][d] = before + __popc(same);
    __syncwarp();
    rank[k] = before + __popc(same & ((1u << lane) - 1u));
  }
  __syncthreads();
  // thread d: total of digit d, its items in earlier tiles, then the warps' offsets
  int total = 0, earlier = 0;
#pragma unroll 8
  for (int b = 0; b < tiles; ++b) {
    const int c = counts[b * SORT_BINS + tid];
    total += c;
    earlier += b < static_cast<int>(blockIdx.x) ? c : 0;
  }
  int off = block_exclusive_scan(total, scratch) + earlier;
  for (int k = 0; k < SORT_WARPS; ++k) {
    const int c = cnt[k][tid];
    cnt[k][tid] = off;
    off += c;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) {
    const long long i = base + k * 32 + lane;
    if (i < N) {
      const int pos = cnt[w][(key[k] >> shift) & mask] + rank[k];
      out_keys[pos] = key[k];
      out_toks[pos] = FIRST ? static_cast<int>(i) : toks[i];
    }
  }
}

// ---------------------------------------------------------------------------
// sums over runs of equal ids
// ---------------------------------------------------------------------------
constexpr int SEG_WARPS = 8;
constexpr int SEG_COLS = 32 * 8;       // columns of a warp's slice
constexpr int ZERO_ROWS = 32;          // grad_weight rows a warp looks up at once

struct SegArgs {
  const int* keys;       // sorted ids, [N]
  const int* toks;
  const unsigned char* dout;
  int N, H, V;
  int chunk;             // entries per chunk
  int n_chunks, slices;
  float scale;
  int accumulate;
  unsigned char* gw;
  float* part;           // [n_chunks][2][H]: 0 = sum of the run that came in, 1 = of the run that goes out
  long long seg_warps;   // warps of the first kind; the others set rows to zero
};

template <typename O>
__device__ __forceinline__ void write_row(const SegArgs& a, int v, int h, const float (&s)[8]) {
  unsigned char* p = a.gw + (static_cast<long long>(v) * a.H + h) * O::SIZE;
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = s[k] * a.scale;
  if (a.accumulate) {
    float g[8];
    O::load(p, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] += g[k];
  }
  O::store(p, f);
}

template <typename T, typename O>
__device__ __forceinline__ void segments(const SegArgs& a, long long warp, int lane) {
  const int c = static_cast<int>(warp / a.slices), slice = static_cast<int>(warp % a.slices);
  const int h = slice * SEG_COLS + lane * 8;
  const bool live = h < a.H;
  const int i0 = c * a.chunk, i1 = min(a.N, i0 + a.chunk);
  const int before = i0 > 0 ? a.keys[i0 - 1] : -1;
  const int after = i1 < a.N ? a.keys[i1] : a.V;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int cur = a.keys[i0];
  bool came_in = cur == before;
  for (int g0 = i0; g0 < i1; g0 += 32) {
    const int m = min(32, i1 - g0);
    const int my_key = lane < m ? a.keys[g0 + lane] : a.V;
    const int my_tok = lane < m ? a.toks[g0 + lane] : 0;
    for (int j0 = 0; j0 < m; j0 += 4) {
      float x[4][8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int key = __shfl_sync(0xffffffffu, my_key, j0 + q);
        const long long tok = __shfl_sync(0xffffffffu, my_tok, j0 + q);
        if (live && key < a.V) T::load(a.dout + (tok * a.H + h) * T::SIZE, x[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (j0 + q >= m) break;
        const int key = __shfl_sync(0xffffffffu, my_key, j0 + q);
        if (key != cur) {   // uniform over the warp: the run ends inside the chunk
          if (live && cur < a.V) {
            if (came_in) F32::store(a.part + (2ll * c) * a.H + h, s);
            else write_row<O>(a, cur, h, s);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) s[k] = 0.f;
          cur = key;
          came_in = false;
        }
        if (live && key < a.V) {
#pragma unroll
          for (int k = 0; k < 8; ++k) s[k] += x[q][k];
        }
      }
    }
  }
  if (!live || cur >= a.V) return;
  if (came_in) F32::store(a.part + (2ll * c) * a.H + h, s);
  else if (cur == after) F32::store(a.part + (2ll * c + 1) * a.H + h, s);
  else write_row<O>(a, cur, h, s);
}

// First position whose key is >= v.
__device__ __forceinline__ int lower_bound(const int* __restrict__ keys, int n, int v) {
  int lo = 0, len = n;
  while (len > 0) {
    const int half = len / 2;
    if (keys[lo + half] < v) {
      lo += half + 1;
      len -= half + 1;
    } else {
      len = half;
    }
  }
  return lo;
}

template <typename T, typename O>
__global__ void __launch_bounds__(32 * SEG_WARPS) embedding_segments_kernel(const SegArgs a) {
  const long long warp = static_cast<long long>(blockIdx.x) * SEG_WARPS + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (warp < a.seg_warps) {
    if (warp < static_cast<long long>(a.n_chunks) * a.slices) segments<T, O>(a, warp, lane);
    return;
  }
  // rows whose id does not occur
  const long long r0 = (warp - a.seg_warps) * ZERO_ROWS;
  if (r0 >= a.V) return;
  const int v = static_cast<int>(r0) + lane;
  bool absent = false;
  if (v < a.V) {
    const int at = lower_bound(a.keys, a.N, v);
    absent = at >= a.N || a.keys[at] != v;
  }
  unsigned m = __ballot_sync(0xffffffffu, absent);
  const int row_bytes = a.H * O::SIZE;
  while (m) {
    const int k = __ffs(m) - 1;
    m &= m - 1;
    uint4* p = reinterpret_cast<uint4*>(a.gw + (r0 + k) * row_bytes);
    for (int i = lane; i < row_bytes / 16; i += 32) p[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// A run that goes out of chunk c and comes into c + 1, c + 2, ...: its partial
// sums in chunk order.  One warp per chunk and column slice.
template <typename O>
__global__ void __launch_bounds__(32 * SEG_WARPS) embedding_join_kernel(const SegArgs a) {
  const long long warp = static_cast<long long>(blockIdx.x) * SEG_WARPS + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (warp >= static_cast<long long>(a.n_chunks) * a.slices) return;
  const int c = static_cast<int>(warp / a.slices), slice = static_cast<int>(warp % a.slices);
  const int h = slice * SEG_COLS + lane * 8;
  const int i0 = c * a.chunk, i1 = min(a.N, i0 + a.chunk);
  if (i1 >= a.N) return;
  const int v = a.keys[i1 - 1];
  if (v >= a.V || a.keys[i1] != v) return;
  if (i0 > 0 && a.keys[i0] == v && a.keys[i0 - 1] == v) return;   // the run began in an earlier chunk
  if (h >= a.H) return;
  float s[8];
  F32::load(a.part + (2ll * c + 1) * a.H + h, s);
  const int end = lower_bound(a.keys, a.N, v + 1);   // past the run
  const int last = (end - 1) / a.chunk;
#pragma unroll 4
  for (int k = c + 1; k <= last; ++k) {
    float x[8];
    F32::load(a.part + (2ll * k) * a.H + h, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) s[q] += x[q];
  }
  write_row<O>(a, v, h, s);
}

__global__ void clear_header_kernel(int* hdr) {
  if (threadIdx.x < HDR_WORDS) hdr[threadIdx.x] = 0;
}

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
struct EmbPlan {
  int tiles = 0, passes = 0, bits = 0, chunk = 0, n_chunks = 0;
  size_t o_keys[2] = {0, 0}, o_toks[2] = {0, 0}, o_cnt = 0, o_part = 0, total = 0;
};

EmbPlan emb_plan(long long N, long long H, long long V) {
  EmbPlan p;
  int key_bits = 1;
  while ((V >> key_bits) != 0) ++key_bits;   // keys 0 .. V
  p.passes = static_cast<int>(cdiv(key_bits, SORT_MAX_BITS));
  p.bits = static_cast<int>(cdiv(key_bits, p.passes));
  p.tiles = static_cast<int>(cdiv(N, SORT_TILE));
  p.chunk = 32;
  p.n_chunks = static_cast<int>(cdiv(N, p.chunk));
  size_t off = al256(HDR_WORDS * sizeof(int));
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += al256(bytes);
    return o;
  };
  for (int k = 0; k < 2; ++k) {
    p.o_keys[k] = take(size_t(N) * 4);
    p.o_toks[k] = take(size_t(N) * 4);
  }
  p.o_cnt = take(size_t(p.tiles) * SORT_BINS * 4);
  p.o_part = take(size_t(p.n_chunks) * 2 * H * 4);
  p.total = off;
  return p;
}

bool emb_sizes_ok(long long N, long long H, long long V) { return sizes_ok(N, H, V) && N <= (1ll << 30); }

template <typename T, typename O>
void launch_segments(const SegArgs& a, long long blocks, cudaStream_t st) {
  embedding_segments_kernel<T, O><<<static_cast<unsigned>(blocks), 32 * SEG_WARPS, 0, st>>>(a);
}

template <typename T>
void launch_segments(const SegArgs& a, int out_dtype, long long blocks, cudaStream_t st) {
  if (out_dtype == FLCE_BF16) launch_segments<T, Bf16>(a, blocks, st);
  else if (out_dtype == FLCE_F16) launch_segments<T, F16>(a, blocks, st);
  else launch_segments<T, F32>(a, blocks, st);
}

bool known_dtype(int d) { return d == FLCE_BF16 || d == FLCE_F16 || d == FLCE_F32; }

}  // namespace
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
  const int H8 = static_cast<int>(H / 8);
  const unsigned grid = static_cast<unsigned>(std::min<long long>(cdiv(N * H8, LOOKUP_THREADS), 1 << 20));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned char* w = static_cast<const unsigned char*>(weight);
  unsigned char* o = static_cast<unsigned char*>(out);
  count_launches(1);
  if (dtype == FLCE_BF16) embedding_kernel<Bf16><<<grid, LOOKUP_THREADS, 0, st>>>(w, ids, N, H8, static_cast<int>(V), scale, o);
  else if (dtype == FLCE_F16) embedding_kernel<F16><<<grid, LOOKUP_THREADS, 0, st>>>(w, ids, N, H8, static_cast<int>(V), scale, o);
  else embedding_kernel<F32><<<grid, LOOKUP_THREADS, 0, st>>>(w, ids, N, H8, static_cast<int>(V), scale, o);
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
  int* keys[2] = {at<int>(workspace, p.o_keys[0]), at<int>(workspace, p.o_keys[1])};
  int* toks[2] = {at<int>(workspace, p.o_toks[0]), at<int>(workspace, p.o_toks[1])};
  int* cnt = at<int>(workspace, p.o_cnt);
  const int n = static_cast<int>(N), v = static_cast<int>(V);

  count_launches(3 + 2 * p.passes);
  clear_header_kernel<<<1, HDR_WORDS, 0, st>>>(hdr);
  if (cudaGetLastError() != cudaSuccess) return FLCE_ECUDA;
  for (int k = 0; k < p.passes; ++k) {
    const int shift = k * p.bits;
    const int *ki = keys[(k + 1) & 1], *ti = toks[(k + 1) & 1];
    int *ko = keys[k & 1], *to = toks[k & 1];
    if (k == 0) {
      sort_count_kernel<true><<<p.tiles, SORT_THREADS, 0, st>>>(ids, n, v, padding_idx, hdr, shift, p.bits, cnt);
      sort_scatter_kernel<true><<<p.tiles, SORT_THREADS, 0, st>>>(ids, nullptr, n, v, padding_idx, hdr, shift, p.bits,
                                                                  cnt, p.tiles, ko, to);
    } else {
      sort_count_kernel<false><<<p.tiles, SORT_THREADS, 0, st>>>(ki, n, v, padding_idx, hdr, shift, p.bits, cnt);
      sort_scatter_kernel<false><<<p.tiles, SORT_THREADS, 0, st>>>(ki, ti, n, v, padding_idx, hdr, shift, p.bits, cnt,
                                                                   p.tiles, ko, to);
    }
    if (cudaGetLastError() != cudaSuccess) return FLCE_ECUDA;
  }
  SegArgs a;
  a.keys = keys[(p.passes - 1) & 1];
  a.toks = toks[(p.passes - 1) & 1];
  a.dout = static_cast<const unsigned char*>(grad_out);
  a.N = n; a.H = static_cast<int>(H); a.V = v;
  a.chunk = p.chunk; a.n_chunks = p.n_chunks;
  a.slices = static_cast<int>(cdiv(H, SEG_COLS));
  a.scale = scale;
  a.accumulate = (flags & FLCE_ACCUMULATE) ? 1 : 0;
  a.gw = static_cast<unsigned char*>(grad_weight);
  a.part = at<float>(workspace, p.o_part);
  const long long seg_blocks = cdiv(static_cast<long long>(a.n_chunks) * a.slices, SEG_WARPS);
  const long long zero_blocks = a.accumulate ? 0 : cdiv(cdiv(V, ZERO_ROWS), SEG_WARPS);
  if (seg_blocks + zero_blocks >= (1ll << 31)) return FLCE_EUNSUPPORTED;
  a.seg_warps = seg_blocks * SEG_WARPS;
  if (dtype == FLCE_BF16) launch_segments<Bf16>(a, grad_dtype, seg_blocks + zero_blocks, st);
  else if (dtype == FLCE_F16) launch_segments<F16>(a, grad_dtype, seg_blocks + zero_blocks, st);
  else launch_segments<F32>(a, grad_dtype, seg_blocks + zero_blocks, st);
  if (cudaGetLastError() != cudaSuccess) return FLCE_ECUDA;
  const unsigned join_blocks = static_cast<unsigned>(seg_blocks);
  if (grad_dtype == FLCE_BF16) embedding_join_kernel<Bf16><<<join_blocks, 32 * SEG_WARPS, 0, st>>>(a);
  else if (grad_dtype == FLCE_F16) embedding_join_kernel<F16><<<join_blocks, 32 * SEG_WARPS, 0, st>>>(a);
  else embedding_join_kernel<F32><<<join_blocks, 32 * SEG_WARPS, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ECUDA;
}

}  // extern "C"
