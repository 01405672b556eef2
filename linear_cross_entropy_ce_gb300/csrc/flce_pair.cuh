// Numbers as sums of two fp32 ones, for what is left of terms that nearly cancel:
// exponentials and logarithms to about 2^-28, sums and products to far less, at some
// fp32 instructions each.  (64-bit instructions, conversions among them, take a warp
// 16 cycles of the SM's: with the row's last 40 steps in 64 bits the row kernel of
// 4096 tokens at 512 x 16000 took 34 us, 25 in fp32.)
#pragma once

#include <cuda_runtime.h>
#include <math.h>

namespace flce {

struct Pair {
  float hi, lo;
};

// D. E. Knuth's two-sum: what rounding x + y leaves.
__device__ __forceinline__ float sum_rest(float x, float y, float s) {
  const float b = s - x;
  return (x - (s - b)) + (y - b);
}
__device__ __forceinline__ Pair tidy(float hi, float lo) {   // |lo| far below |hi|
  const float s = hi + lo;
  return Pair{s, (hi - s) + lo};
}
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
  const float s = a.hi + b.hi;
  return tidy(s, sum_rest(a.hi, b.hi, s) + (a.lo + b.lo));
}
__device__ __forceinline__ Pair operator-(const Pair& a) { return Pair{-a.hi, -a.lo}; }
__device__ __forceinline__ Pair operator-(const Pair& a, const Pair& b) { return a + -b; }
__device__ __forceinline__ Pair operator*(const Pair& a, const Pair& b) {
  const float p = a.hi * b.hi;
  return tidy(p, fmaf(a.hi, b.hi, -p) + fmaf(a.hi, b.lo, a.lo * b.hi));
}
__device__ __forceinline__ Pair operator/(const Pair& a, const Pair& b) {
  const float q = a.hi / b.hi;
  return tidy(q, (fmaf(-q, b.hi, a.hi) + fmaf(-q, b.lo, a.lo)) / b.hi);
}

// 2^(j/32), rounded to fp32, and what that leaves.
__device__ const float2 EXP2_32[32] = {
    {1.f, 0.f}, {1.0218972f, -4.81155986e-08f}, {1.04427373f, 4.83347016e-08f}, {1.06714046f, -5.93375198e-08f},
    {1.09050775f, -1.30775399e-08f}, {1.1143868f, -5.43554002e-08f}, {1.13878858f, 5.38622231e-08f},
    {1.1637249f, -4.05144149e-08f}, {1.18920708f, 3.79763527e-08f}, {1.21524739f, -3.26739489e-08f},
    {1.24185777f, 4.4968381e-08f}, {1.26905096f, 1.41933332e-09f}, {1.29683959f, -4.01899953e-08f},
    {1.32523668f, -3.49637332e-08f}, {1.35425556f, -1.01233493e-08f}, {1.38390994f, -5.87557736e-08f},
    {1.41421354f, 2.4203235e-08f}, {1.44518077f, 3.32419994e-08f}, {1.47682619f, -4.50089885e-08f},
    {1.50916445f, -2.49593732e-08f}, {1.54221082f, 8.07090483e-09f}, {1.5759809f, -5.66102543e-08f},
    {1.61049032f, 9.83621717e-09f}, {1.64575553f, -5.12497209e-08f}, {1.68179286f, -2.47553267e-08f},
    {1.71861935f, -4.8496176e-08f}, {1.75625217f, -9.23577037e-09f}, {1.79470909f, -1.14150449e-08f},
    {1.8340081f, -1.1239278e-08f}, {1.87416768f, -4.66300563e-08f}, {1.91520655f, 9.84532811e-09f},
    {1.95714414f, -1.70218044e-08f}};

// exp(x) to about 2^-28 of itself, by a table (P. T. P. Tang, "Table-driven implementation
// of the exponential function in IEEE floating-point arithmetic", 1989): x log2 e =
// n / 32 + r with |r| <= 1 / 64 and its rounding kept, 2^(n/32) from the table, 2^r - 1
// by its Taylor polynomial (the fifth power is below 2^-39).  Where exp(x) is below
// 1e-34, or no number, or far above 1, it is what expf says.
__device__ __forceinline__ Pair exp_pair(float x) {
  if (!(fabsf(x) < 80.f)) return Pair{expf(x), 0.f};
  constexpr float L = 1.44269502f, L_REST = 1.92596299e-08f;   // log2 e
  const float y = x * L, n = rintf(y * 32.f);
  const float r = fmaf(n, -0.03125f, y) + fmaf(x, L_REST, fmaf(x, L, -y));
  const int i = static_cast<int>(n);
  const float2 t = EXP2_32[i & 31];
  const float q = r * fmaf(r, fmaf(r, fmaf(r, 9.61812911e-3f, 5.55041087e-2f), 0.240226507f), 0.693147181f);
  const float c = fmaf(t.x, q, t.y), hi = t.x + c, lo = (t.x - hi) + c;
  const float scale = __int_as_float((127 + (i >> 5)) << 23);
  return Pair{hi * scale, lo * scale};
}

// ln v of a positive v to about 2^-28: an fp32 logarithm l of its mantissa f, and
// what is missing, ln(f e^-l) = f e^-l - 1 to the first order.
__device__ __forceinline__ Pair log_of(const Pair& v) {
  constexpr float LN2_HI = 0.693145752f, LN2_LO = 1.42860677e-6f;   // ln 2, the first of 16 bits: k times it is exact
  int k = 0;
  const float f = frexpf(v.hi, &k), f_lo = ldexpf(v.lo, -k), l = logf(f), kf = static_cast<float>(k);
  const Pair e = exp_pair(-l);
  const float u = fmaf(f, e.hi, -1.f) + fmaf(f, e.lo, f_lo * e.hi), kh = kf * LN2_HI, s = kh + l;
  return tidy(s, sum_rest(kh, l, s) + fmaf(kf, LN2_LO, u));
}

// A running sum whose roundings are kept.
struct PairSum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float x_lo) {
    const float s = hi + x;
    lo += sum_rest(hi, x, s) + x_lo;
    hi = s;
  }
  __device__ __forceinline__ void add_lanes() {   // of all lanes, in every lane
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      add(__shfl_xor_sync(0xffffffffu, hi, o), __shfl_xor_sync(0xffffffffu, lo, o));
  }
  __device__ __forceinline__ Pair value() const { return tidy(hi, lo); }
};

}  // namespace flce
