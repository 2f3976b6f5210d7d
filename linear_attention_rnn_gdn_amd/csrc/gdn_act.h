// gdn_act.h -- elementwise functions of the operators around a recurrent
// layer (the short convolution and the selective scan), in fp32.
#pragma once
#include "gdn_common.h"

namespace gdn {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f, kLn2Low = -1.9046542e-9f;

// e^w for |w| <= 128 (beyond fp32's range on both sides) to a few units in the
// last place: 2^p e^{w - p ln 2} with p = w log2(e) rounded, and the second
// factor, within 2^-17 of one, to first order.
__device__ __forceinline__ float exp_to_ulps(float w) {
  const float p = w * kLog2e;
  return __builtin_amdgcn_exp2f(p) * (1.f + fmaf(-p, kLn2Low, fmaf(-p, kLn2, w)));
}
// (No number gives zero here, or one of the ends; the sums and products that
// follow carry it.)
__device__ __forceinline__ float exp_neg_abs(float v) { return exp_to_ulps(fmaxf(-fabsf(v), -128.f)); }
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + exp_to_ulps(__builtin_amdgcn_fmed3f(-v, -128.f, 128.f)));
}
// sigmoid of v (1 + a rounding): what the rounding of v log2(e) does to it is
// what another rounding of v would do, so it is as good as v where v is a
// rounded sum (or where the result is rounded to bf16), at half the instructions.
__device__ __forceinline__ float sigmoid_rough(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -kLog2e));
}
template <bool ROUGH> __device__ __forceinline__ float silu(float v) { return v * (ROUGH ? sigmoid_rough(v) : sigmoid(v)); }
// silu and its derivative  s (1 + v (1 - s))
template <bool ROUGH> __device__ __forceinline__ void silu_grad(float v, float &y, float &dy) {
  const float g = ROUGH ? sigmoid_rough(v) : sigmoid(v);
  y = v * g;
  dy = fmaf(y, 1.f - g, g);
}

// log(1 + e^v) = max(v, 0) + log1p(e^-|v|).  With w = 1 + e rounded, log1p(e) =
// log(w) + log1p((e - (w - 1)) / w): the rounding of w, which is all of e where
// a step is small, is added back.  Leaving out the division by w changes that
// by lost (w - 1) / w: at most 2^-24 of log(w), one rounding of it, as lost is
// 2^-24 at most and (w - 1) / w no more than log(w).
__device__ __forceinline__ float softplus(float v, float e) {
  const float w = 1.f + e, lost = e - (w - 1.f);
  return fmaf(__builtin_amdgcn_logf(w), kLn2, lost) + __builtin_elementwise_maximum(v, 0.f);
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
// The sequence of token t, which lies in [0, T).  Tokens behind the last offset
// count as the last sequence's.  OFFSETS: anything that gives offset s in [0, n].
template <typename Offsets>
__device__ __forceinline__ Sequence sequence_of(const Offsets &cu, int n, int T, int t, int lo) {
  const int b = cu(lo), e = cu(lo + 1);
  return Sequence{lo, b < t ? b : t, e > t ? e : lo + 1 < n ? t + 1 : T};
}
// each thread for itself, by halving; `from`: one at or before it
template <typename Offsets>
__device__ __forceinline__ Sequence sequence_at(const Offsets &cu, int n, int T, int t, int from) {
  int lo = from < n ? from : n - 1, hi = n;   // the last one that begins at t or before
  if (lo + 1 < n && cu(lo + 1) > t) hi = lo + 1;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (cu(mid) <= t) lo = mid;
    else hi = mid;
  }
  return sequence_of(cu, n, T, t, lo);
}
// a whole wave for one token: 64 offsets at once
__device__ __forceinline__ Sequence sequence_of_wave(const int *cu, int n, int T, int t, int from, int lane) {
  int lo = from < n ? from : n - 1, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64, at = lo + lane * step;
    const int before = __popcll(__ballot(at < hi && offset_at(cu, at < hi ? at : lo, T) <= t));
    lo += (before > 1 ? before - 1 : 0) * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  const Sequence q = sequence_of([&](int s) { return offset_at(cu, s, T); }, n, T, t, lo);
  return Sequence{__builtin_amdgcn_readfirstlane(q.seq), __builtin_amdgcn_readfirstlane(q.begin), __builtin_amdgcn_readfirstlane(q.end)};
}

}  // namespace gdn
