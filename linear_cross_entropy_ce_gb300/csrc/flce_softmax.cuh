// Softmax statistics of a set of logits at temperature T, and their merge.
// With c2 = log2(e) / T and x = (z - max) c2 <= 0:
//   s = sum 2^x,  d = sum x 2^x
// so that log2 sum 2^(z c2) = max c2 + log2 s, and the entropy is
// ln 2 (log2 s - d / s).
#pragma once

#include "flce_ptx.cuh"

namespace flce {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

struct Stat {
  float m, s, d;   // max (raw), sum 2^x, sum x 2^x with x = (z - m) c2
};

__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b, float c2) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  // a side whose max is -inf holds nothing: its factor is 0 (the clamp also
  // turns -inf - -inf into it)
  const float xa = fmaxf((a.m - r.m) * c2, -1e20f), xb = fmaxf((b.m - r.m) * c2, -1e20f);
  const float fa = ptx::ex2(xa), fb = ptx::ex2(xb);
  r.s = fa * a.s + fb * b.s;
  r.d = fa * fmaf(xa, a.s, a.d) + fb * fmaf(xb, b.s, b.d);
  return r;
}

// fp32 as an unsigned integer of the same order; 0 is below every number.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

}  // namespace flce
