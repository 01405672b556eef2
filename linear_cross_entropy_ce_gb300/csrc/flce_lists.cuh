// Tokens of a row that the logits kernels treat apart: the tokens that a
// penalty or a bias changes, a teacher's alternatives, and the tokens that a
// grammar forbids.
//
// The listed tokens of a row are few, at no fixed places.  A list in ascending
// order, with the place where every tile's (or 128-column part's) tokens begin,
// lets an epilogue see at the cost of two loads whether a piece of a row holds
// any (most do not), and write those logits side by side.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace flce {

struct ListView {
  const int* start;        // entries before each boundary: [boundaries][C] for the chunked form (one every 128
                           // columns, and the end), [rows][boundaries] for the streaming form (one a tile, and the end)
  int boundaries;          // of the streaming form
  const int* id;           // [rows][cap] ascending, each token once
  float* z;                // [rows][cap] their logits, left out of the statistics
  long long cap;
  const uint32_t* mask;    // [N][mask_stride] by token row: bit v % 32 of word v / 32 is set where token v may follow; or null
  long long mask_stride;
};

// What changes the logits of a row's listed tokens.
struct RuleView {
  const int* seen;         // [rows][cap] 0: not in the history; else the times in its output, bit 31 set for those in its prompt
  const float* bias;       // [rows][cap] or null
  const float* repetition; // [N] by token row, or null: none
  const float* frequency;
  const float* presence;
};

struct RowRules {
  float repetition, frequency, presence;
};

__device__ __forceinline__ RowRules row_rules(const RuleView& v, long long token) {
  return RowRules{v.repetition ? v.repetition[token] : 1.f, v.frequency ? v.frequency[token] : 0.f,
                  v.presence ? v.presence[token] : 0.f};
}

// The logit of a listed token under its row's rules.  Each step is rounded to
// fp32 by itself (no fused multiply-add), so that equal logits stay equal
// whoever computes them.
__device__ __forceinline__ float ruled(float z, int seen, float bias, const RowRules& r) {
  if (seen != 0) z = z > 0.f ? __fdiv_rn(z, r.repetition) : __fmul_rn(z, r.repetition);
  const int times = seen & 0x7fffffff;
  if (times != 0) {
    z = __fsub_rn(z, __fmul_rn(r.frequency, static_cast<float>(times)));
    z = __fsub_rn(z, r.presence);
  }
  return __fadd_rn(z, bias);
}

}  // namespace flce
