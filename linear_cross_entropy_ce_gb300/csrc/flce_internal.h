// Internal declarations shared by the CUDA translation units of libflce.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "flce_lists.cuh"

namespace flce {

// Device status word bits (workspace header word 0).
constexpr int STATUS_BADTARGET = 1;
constexpr int STATUS_TIMEOUT = 2;

// Workspace header words.
constexpr int HDR_STATUS = 0;
constexpr int HDR_NVALID = 1;
constexpr int HDR_STALL = 2;   // first pipeline wait that timed out: site | rank << 8 | block << 12
constexpr int HDR_STALL_COUNT = 3;   // number of timed-out waits
constexpr int HDR_STALL_LOG = 8;     // up to 8 records (code, detail) of timed-out waits
constexpr int STALL_LOG_MAX = 8;
constexpr int HDR_WORDS = 64;

// GEMM tile shape: a CTA pair (cluster of 2, tcgen05 cta_group::2) owns a
// 256 x 256 fp32 accumulator, 128 rows in each CTA's TMEM, and streams K in
// blocks of 64 bf16 (one 128-byte swizzle row).  BM is the rows per CTA.
constexpr int BM = 128;
constexpr int PAIR_M = 2 * BM;
constexpr int BN = 256;
constexpr int BK = 64;
// The logits epilogue keeps one (max, sum exp) pair per row and 128-column
// vocabulary part (each epilogue warpgroup owns half of a 256-column tile).
constexpr int PART_COLS = 128;

enum GemmMode : int {
  MODE_LOGITS = 0,  // z = Xc W^T, epilogue: per 128-column part (max, sum exp), z_t, shifted bf16 logits
  MODE_BWD = 1,     // one launch holding both consumers of dz:
                    //   grad_hidden rows = dz W          (units [0, n_dx))
                    //   grad_weight (+)= dz^T Xc         (units [n_dx, n_dx + n_dw))
  MODE_STATS = 2,   // z = Xc W^T, epilogue: per 128-column part the max, sum exp and sum of (log weight x exp),
                    // z_t, and the fp32 logits themselves where top alternatives are asked for
  MODE_DZ = 3,      // z = Xc W^T again, epilogue: dz of the token log probabilities and entropies, from the
                    // rows' log-sum-exp, entropy and upstream gradients, as bf16
};

// Tokens of a row that MODE_STATS treats apart (GemmArgs::listed).
constexpr int LISTED_OUT = 1;     // taken out one by one, forbidden ones left out; their logits in lists.z [C][cap]
constexpr int LISTED_SLABS = 2;   // a part that holds any is left out whole, its logits in lists.z [C][slabs_per_row][128]

// Unit kinds a MODE_BWD launch leaves out (GemmArgs::skip).
constexpr int SKIP_DX = 1;
constexpr int SKIP_DW = 2;

// Per-row constants of MODE_DZ, with l2 = z c - lse2 (the base-2 log probability):
// dz = 2^l2 (a + b l2) + [v = t] g.
struct DzRow {
  float lse2, a, b, g;
};

struct GemmArgs {
  int mode;
  const int* hdr;       // workspace header (n_valid lives in HDR_NVALID)
  int* status;          // workspace header word HDR_STATUS
  int* counter;         // LOGITS, BWD: dynamic tile counter of this launch (zero before it)
  long long c0;         // first compacted row of this chunk
  int C;                // chunk capacity (rows)
  int H, V;
  long long ldz;        // row stride (elements) of the chunk logits buffer
  int nvt;              // vocabulary tiles: ceil(V / BN)
  int nparts;           // vocabulary parts: ceil(V / PART_COLS)
  int store_z;          // LOGITS: write the shifted bf16 logits
  int accumulate;       // BWD: add into grad_weight (chunks after the first)
  int first_chunk;      // BWD: chunk 0 (writes zeros when it is empty)
  int splits;           // BWD: vocabulary splits of the grad_hidden GEMM
  int kb_per_split;     // BWD: K blocks per split
  int interleave;       // BWD: spread the dX units through the dW units (else dX units first)
  int pf_threads;       // BWD, accumulating: the epilogue threads prefetch the grad_weight tile into L2
                        // (else one TMA prefetch when the tile's main loop starts)
  int* flags;           // BWD, splits > 1: per (tile, CTA, warpgroup) count of finished splits (zero before)
  unsigned long long timeout_ns;
  int debug_stall;      // test hook: the MMA issuer withholds the accumulator-ready signal of each
                        // pair's first unit, so that the epilogue's bounded wait runs out
  // epilogue operands
  uint16_t* z;          // [C][ldz] bf16
  float2* part;         // [C][nparts] (part max, part sum of exp)
  float* zt;            // [C] target logit
  const int* tc;        // [C] chunk targets (-1 for padding rows)
  const int* idx;       // [N] compacted row -> token row
  uint16_t* grad_hidden;// [N][H] bf16
  float* grad_hidden_f32; // [N][H] fp32 instead of grad_hidden when not null (vocabulary shards)
  float* grad_weight;   // [V][H] fp32 (zero fill of an empty first chunk)
  const float* dxacc;   // [C][H] fp32 sum of the grad_hidden splits (splits > 1)
  // MODE_STATS, MODE_DZ
  int skip;             // BWD: SKIP_DX, SKIP_DW
  int slabs;            // BWD, splits > 1: each split stores its fp32 part to dxacc + split C H
                        // (dx_reduce adds them) instead of adding onto the previous one
  int two;              // DZ, BWD: dz in two bf16 parts, the second C rows behind the first
  int gw_bf16;          // BWD of a call with one chunk: grad_weight tiles are rounded and stored as bf16
  float c2;             // log2(e) / temperature: z c2 is the scaled logit in base-2 units
  float* stats;         // STATS: [3][nparts][C] part max (raw z), sum of 2^d, sum of d 2^d, d = (z - max) c2
  int seg_kb;           // STATS, DZ: K blocks of a segment of a logit's sum (segment_blocks)
  int K;                // STATS: top alternatives, and for K > 0
  float* zf;            //   [C][ldz] fp32 logits of the parts that may hold one
  uint32_t* bound;      //   [C] ordered integer that a part's max has to reach, or null: every part is kept
  uint32_t* group_max;  //   [C][group_stride] largest part max of each of K groups of parts
  int group_stride;     //   K rounded up to 4
  const DzRow* rowc;    // DZ: [C] (rows past the valid ones hold zeros)
  int listed;           // STATS: LISTED_*
  ListView lists;       // LISTED_OUT: the tokens taken out; z of both
  const short* slab;    // LISTED_SLABS: [nparts][C] the row's slab of the part, or -1
  int slab_by_token;    //   by token, not by row of the chunk
  int slabs_per_row;
};

// Tensor maps of one launch.  LOGITS: a0 = Xc (K-major), b0 = W (K-major).
// BWD: a0 = dz (K-major), b0 = W (MN-major), a1 = dz (MN-major view),
// b1 = Xc (MN-major), out = grad_weight (fp32, store / reduce-add of 16 x 128
// slices), pf = grad_weight again with a 256 x 128 box for L2 prefetches.
struct GemmMaps {
  CUtensorMap a0, b0, a1, b1, out;
};

int gemm_smem_bytes();
cudaError_t gemm_prepare(int device);
cudaError_t gemm_max_pairs(int* pairs);   // CTA pairs resident at once (current device)
cudaError_t launch_gemm(const GemmArgs& a, const GemmMaps& m, int grid, cudaStream_t s, bool dependent);

// Host helpers shared by the entry points (flce_api.cu).
struct DeviceState {
  bool ready = false;
  int sms = 0;
  int major = 0;
  int pairs = 0;   // CTA pairs of the GEMM that fit on the device at once
};
cudaError_t device_state(DeviceState* out);
int device_pairs();
int device_sms();
unsigned long long wait_timeout_ns();
bool make_map(CUtensorMap* m, const void* base, unsigned long long inner, unsigned long long outer,
              unsigned long long row_bytes, unsigned box_inner, unsigned box_outer,
              CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);
// Launch a GEMM, bracketed by events when profiling is on.
// dependent: while the previous kernel drains (launch_dependent).
cudaError_t gemm_launch(const GemmArgs& g0, const GemmMaps& m, int grid, cudaStream_t st, bool dependent = false);
void count_launches(long long n);
// Events around a tcgen05 launch of `mode` while profiling is on (begin gives a
// handle for end; a call without profiling costs one lock).
struct ProfScope {
  cudaEvent_t start = nullptr, stop = nullptr;
  bool on = false;
};
ProfScope prof_launch_begin(cudaStream_t st);
void prof_launch_end(const ProfScope& p, int mode, cudaStream_t st);
// Time limit armed by flce_debug_arm_stall for the next tcgen05 launch, or 0; disarms.
unsigned long long take_armed_stall();
bool sizes_ok(long long N, long long H, long long V);

inline size_t al256(size_t x) { return (x + 255) & ~size_t(255); }
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }
inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

// The result of a launch, which does not stay behind as the thread's last error
// (the next call would take it for its own).
inline cudaError_t launch_result(cudaError_t e) {
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// Launch whose blocks may come up while the previous kernel of the stream still
// runs; the kernel has to call ptx::grid_dependency_wait() before it reads or
// writes anything that kernel (or an earlier one) touches.
template <typename... P, typename... A>
cudaError_t launch_dependent_smem(void (*kernel)(P...), unsigned blocks, unsigned threads, size_t smem,
                                  cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return launch_result(cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...));
}
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned blocks, unsigned threads, cudaStream_t st,
                             const A&... args) {
  return launch_dependent_smem(kernel, blocks, threads, 0, st, args...);
}

// Elementwise / bookkeeping kernels (flce_aux.cu).
cudaError_t launch_prep(const int* targets, long long N, int V, int ignore_index,
                        int* hdr, int* idx, int* n_valid_out, int* counters, long long n_counters,
                        cudaStream_t s);
cudaError_t launch_zero_ignored(const int* hdr, const int* idx, long long N, long long row_bytes,
                                void* grad_hidden, cudaStream_t s);
cudaError_t launch_gather(const uint16_t* hidden, const int* targets, const int* hdr,
                          const int* idx, long long c0, int C, int H,
                          uint16_t* xc, int* tc, int v0, int vs, cudaStream_t s);
// Segments of a logit's sum over H.  The tensor core cuts off what its fp32
// accumulator cannot hold, at every 16-wide step, so a sum comes out short by a
// part of itself that grows with its length (0.07e-6 of entropies per K block:
// 1.1e-6 at H = 1024, 5e-6 at 4096).  The log probabilities therefore sum it in
// segments, each from zero, and add these up rounded to nearest.  With
// 2 sqrt(blocks) blocks a segment the error grows with H as that of an fp32
// product on the CUDA cores does; up to 11 blocks it is below 1e-6 anyway.
inline int segment_blocks(long long H) {
  const int blocks = static_cast<int>(cdiv(H, BK));
  const int most = std::max(11, static_cast<int>(2.0 * std::sqrt(static_cast<double>(blocks))));
  return static_cast<int>(cdiv(blocks, cdiv(blocks, most)));   // of equal length
}
// Few tokens: the weight streamed once past all of them (flce_stream.cu).
constexpr int STREAM_MAX_TOKENS = 128;
struct StreamArgs {
  int N, H, V, K;          // K: top alternatives
  int seg_kb;              // K blocks of a segment of a logit's sum
  int ctas;
  float c2;
  int ii;
  unsigned long long timeout_ns;
  int debug_stall;
  const int* targets;
  int* hdr;
  float* zt;               // [N]
  float4* stat;            // [N][ctas] max, sum, weighted sum
  float* zf;               // K > 0: [N][ldz] logits, and
  long long ldz;
  float* tile_max;         // [N][ctas][max_tiles]
  uint32_t* group_max;     // [N][32] largest tile max (as an ordered integer) of each of K groups of tiles, or null
  int max_tiles;           // tiles of a CTA at most
  int* fail;               // [ctas]
  float* logp;
  float* entropy;          // or null
  float* lse;
  int* top_ids;
  float* top_logp;
};
struct StreamMaps {
  CUtensorMap x, w[4];     // w[k]: boxes of 128 >> k weight rows
};
struct StreamLists {
  ListView lists;
  RuleView rules;
};
int stream_ctas(long long V, int sms);
int stream_max_tiles(long long V, int ctas);
int stream_tokens(int N);   // N padded to the tile sizes of the kernel
cudaError_t stream_prepare();
cudaError_t embedding_prepare();   // flce_embedding.cu
cudaError_t launch_stream(const StreamArgs& a, const StreamMaps& m, cudaStream_t s);
// The same with the listed tokens of each row under rules (flce_stream_ruled.cu),
// and the kernel alone with them taken out (flce_stream_taken.cu); both are
// launched while the kernel that makes the lists runs, unless `beside` is false.
cudaError_t stream_ruled_prepare();
cudaError_t stream_taken_prepare();
cudaError_t launch_stream_ruled(const StreamArgs& a, const StreamMaps& m, const StreamLists& l, bool beside,
                                cudaStream_t s);
cudaError_t launch_stream_taken(const StreamArgs& a, const StreamMaps& m, const StreamLists& l, cudaStream_t s);

// Token log probabilities (flce_logprobs.cu).
// The first launch of a call of one chunk and at most FRONT_MAX_TOKENS tokens;
// rowc selects the backward.  Its blocks read N^2 / 2 bytes of targets between
// them (from L2: 134 MB at the most tokens); past that the loss's kernels
// compact the tokens in one block and gather them in another launch.
constexpr long long FRONT_MAX_TOKENS = 16384;
struct FrontArgs {
  const uint16_t* hidden;
  const int* targets;                 // null: every token counts, with target 0
  int N, H, V, ii, C, K;
  int *hdr, *idx, *tc;
  uint16_t* xc;
  int* counters;
  int n_counters;
  float *logp, *lse, *entropy;        // forward outputs
  int* top_ids;
  float* top_logp;
  uint32_t *bound, *group_max;        // K > 0: cleared
  int group_stride;
  DzRow* rowc;                        // backward
  float temperature;
  const float *lse_in, *entropy_in, *grad_logp, *grad_entropy;
  uint16_t* grad_hidden;              // or null
};
cudaError_t launch_probs_front(const FrontArgs& a, cudaStream_t s);
cudaError_t launch_clear_bounds(uint32_t* bound, uint32_t* group_max, int stride, int K, int C, cudaStream_t s);
cudaError_t launch_gather_dz(const uint16_t* hidden, const int* targets, const int* hdr, const int* idx,
                             long long c0, int C, int H, float temperature, const float* lse, const float* entropy,
                             const float* grad_logp, const float* grad_entropy, uint16_t* xc, int* tc, DzRow* rowc,
                             cudaStream_t s);
// The gradient of the distillation loss (flce_distill.cu): that of the log
// probabilities with other row constants, and dz overwritten at listed places.
struct DistillGrad {
  const int* ids;                 // [N][K] teacher tokens
  const float* logp;
  int K, tail;
  const float *lse_in, *rest_logp, *student_logp, *grad_kl;
  int* targets;                   // made from these
  float *lse, *grad;
  uint32_t* patch;                // [N][K] dz at the teacher's tokens, both bf16 parts (the first in the low half)
};
cudaError_t launch_distill_grad_rows(const DistillGrad& d, long long N, int V, float temperature, cudaStream_t s);
cudaError_t launch_distill_patch(const int* hdr, const int* idx, long long c0, int C, int K, int V, long long ldz,
                                 const int* ids, const uint32_t* patch, uint16_t* z, cudaStream_t s);
cudaError_t constrained_prepare();
// The time limit and the tensor maps of a streaming call.
bool stream_setup(StreamArgs* a, StreamMaps* m, const void* hidden, const void* weight, int seg_kb);
cudaError_t launch_dx_reduce(const int* hdr, const int* idx, long long c0, int C, int H, int splits, const float* parts,
                             uint16_t* grad_hidden, cudaStream_t s);
cudaError_t launch_mark_failed(const int* hdr, uint16_t* grad_hidden, float* grad_weight, int gw_bf16,
                               cudaStream_t s);
bool bad_temperature(float t);
constexpr long long PROBS_MAX_V = (1ll << 31) - 512;   // ids rounded up to a tile stay in 32 bits
cudaError_t launch_lse_dz(const int* hdr, long long c0, int C, int V, long long ldz,
                          int nparts, const float2* part, const float* zt, const int* tc,
                          float* rl, uint16_t* z, int reduce_sum, int make_dz,
                          const float* lse_ext, const int* idx, cudaStream_t s);
cudaError_t launch_finalize(const int* hdr, const int* idx, const float* rl,
                            long long N, int reduce_sum, float* loss, int* n_valid_out,
                            float* row_loss, cudaStream_t s);
// Final RMSNorm fused in front of the LM head.
cudaError_t launch_gather_norm(const uint16_t* hidden, const int* targets, const int* hdr, const int* idx,
                               long long c0, int C, int H, const uint16_t* gain, float eps, uint16_t* xc,
                               int* tc, float* rinv, cudaStream_t s);
cudaError_t launch_rmsnorm_bwd(const int* hdr, const int* idx, long long c0, int C, int H,
                               const uint16_t* hidden, const uint16_t* gain, const float* rinv,
                               uint16_t* grad_hidden, float* dgain_partial, cudaStream_t s);
cudaError_t launch_dgain_reduce(const float* partials, long long n_chunks, int H, float* grad_gain,
                                cudaStream_t s);
// Vocabulary-parallel LM head.
cudaError_t launch_shard_stats(const int* hdr, const int* idx, long long c0, int C, int nparts,
                               const float2* part, const float* zt, const int* tc, float* row_max,
                               float* row_sumexp, float* row_zt, cudaStream_t s);
cudaError_t launch_shard_stats_ignored(const int* hdr, const int* idx, long long N, float* row_max,
                                       float* row_sumexp, float* row_zt, cudaStream_t s);
cudaError_t launch_vocab_rescale(const float* m_local, const float* m_global, float* sumexp, long long N,
                                 cudaStream_t s);
cudaError_t launch_vocab_finish(const float* m, const float* sumexp, const float* zt, const int* t, long long N,
                                int ii, int reduce_sum, float* lse, float* row_loss, float* loss, int* n_valid,
                                cudaStream_t s);
cudaError_t launch_scale_grads(uint16_t* grad_hidden, long long n_hidden, float* grad_weight,
                               long long n_weight, const float* scale, cudaStream_t s);
cudaError_t launch_timeout_selftest(int* hdr, unsigned long long timeout_ns,
                                    cudaStream_t s);
// fp32 -> bf16 (round to nearest even), n a multiple of 4, both 16-byte aligned
cudaError_t launch_f32_to_bf16(const float* src, long long n, uint16_t* dst, cudaStream_t s);

}  // namespace flce
