// gdn_act.h -- elementwise functions of the operators around a recurrent
// layer (the short convolution and the selective scan), in fp32.
#pragma once
#include "gdn_common.h"

namespace gdn {

constexpr float kLog2e = 1.44269504088896341f, kLog2eLow = 1.92596299112661746e-8f, kLn2 = 0.693147180559945309f;

// e^-|v| to a few units in the last place whatever |v|: the product with
// log2(e) is carried with its rounding error (two fma), whose factor is 1 to
// first order.
__device__ __forceinline__ float exp_neg_abs(float v) {
  const float w = -fabsf(v), p = w * kLog2e;
  const float low = fmaf(w, kLog2eLow, fmaf(w, kLog2e, -p));
  const float e = __builtin_amdgcn_exp2f(p);
  const float f = fmaf(e, low * kLn2, e);
  return p > -150.f ? f : e;   // (below: e is zero, and low no number at -inf)
}

struct Sigmoid {
  float s, c;   // sigmoid(v) and 1 - sigmoid(v), each to relative accuracy
};
__device__ __forceinline__ Sigmoid sigmoid_of(float v, float e) {   // e = e^-|v|
  const float r = __builtin_amdgcn_rcpf(1.f + e), q = e * r;
  return v >= 0.f ? Sigmoid{r, q} : Sigmoid{q, r};
}
__device__ __forceinline__ float silu(float v) { return v * sigmoid_of(v, exp_neg_abs(v)).s; }
// silu and its derivative  s (1 + v (1 - s))
__device__ __forceinline__ void silu_grad(float v, float &y, float &dy) {
  const Sigmoid g = sigmoid_of(v, exp_neg_abs(v));
  y = v * g.s;
  dy = fmaf(v * g.s, g.c, g.s);
}

// log(1 + e^v) = max(v, 0) + log1p(e^-|v|), and log1p(e) = 2 atanh(s) with
// s = e / (2 + e) <= 1/3: seven terms of the odd series leave s^14 / 15 <
// 2^-25 of it.  Small steps keep their relative accuracy, which the logarithm
// of a rounded 1 + e would not.
__device__ __forceinline__ float softplus(float v, float e) {
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), p = s * s;
  float q = 1.f / 13;
  q = fmaf(q, p, 1.f / 11);
  q = fmaf(q, p, 1.f / 9);
  q = fmaf(q, p, 1.f / 7);
  q = fmaf(q, p, 1.f / 5);
  q = fmaf(q, p, 1.f / 3);
  q = fmaf(q, p, 1.f);
  return fmaf(2.f * s, q, fmaxf(v, 0.f));
}

// Sequences packed along one row of T tokens: sequence s holds tokens cu[s] ..
// cu[s + 1].  Offsets are held within [0, T], so that offsets that are no
// partition give other results but no access outside the tensors.
struct Sequence {
  int seq, begin, end;
};
__device__ __forceinline__ int offset_at(const int *cu, int s, int T) {
  const int v = cu[s];
  return v < 0 ? 0 : v > T ? T : v;
}
// The sequence of token t, which lies in [0, T); `from`: one at or before it.
// Tokens behind the last offset count as the last sequence's.
__device__ __forceinline__ Sequence sequence_at(const int *cu, int n, int T, int t, int from) {
  int lo = from < n ? from : n - 1, hi = n;   // the last one that begins at t or before
  if (lo + 1 < n && offset_at(cu, lo + 1, T) > t) hi = lo + 1;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (offset_at(cu, mid, T) <= t) lo = mid;
    else hi = mid;
  }
  const int b = offset_at(cu, lo, T), e = offset_at(cu, lo + 1, T);
  return Sequence{lo, b < t ? b : t, e > t ? e : lo + 1 < n ? t + 1 : T};
}

}  // namespace gdn
