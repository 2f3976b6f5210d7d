// gdn_common.h -- what the kernel families share: the head dimension, the
// placement of workgroups on the XCDs, and fp32 operands as bf16 planes.
#pragma once
#include "gdn_mfma.h"

namespace gdn {

constexpr int D = 128;        // d_k = d_v

// 1-D workgroup index -> (unit, part) with the `parts` workgroups of a unit on
// one XCD (falls back to unit-major order when units is not a multiple of 8).
__device__ __forceinline__ void xcd_unit(int L, int parts, int units, int &unit, int &part) {
  if ((units & 7) == 0) {
    const int x = L & 7, i = L >> 3;
    unit = (i / parts) * 8 + x;
    part = i % parts;
  } else {
    unit = L / parts;
    part = L % parts;
  }
}

// An fp32 value as NP bf16 planes whose sum is the value: NP = 3 exactly (8 of
// the 24 significant bits each), NP = 2 to 2^-17 relative, NP = 1 to 2^-9.
// The planes but the last are cut off (not rounded) when NP = 3, one AND each,
// because three cut planes hold every bit; with fewer planes each is rounded
// to nearest.  Values come in pairs so that a plane's pair is one word.
template <int NP>
__device__ __forceinline__ void split_pair(float x0, float x1, unsigned (&w)[NP]) {
  if constexpr (NP == 3) {
    const unsigned a0 = __builtin_bit_cast(unsigned, x0), a1 = __builtin_bit_cast(unsigned, x1);
    w[0] = __builtin_amdgcn_perm(a1, a0, 0x07060302u);
    const float r0 = x0 - __builtin_bit_cast(float, a0 & 0xffff0000u);
    const float r1 = x1 - __builtin_bit_cast(float, a1 & 0xffff0000u);
    const unsigned b0 = __builtin_bit_cast(unsigned, r0), b1 = __builtin_bit_cast(unsigned, r1);
    w[1] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
    const float s0 = r0 - __builtin_bit_cast(float, b0 & 0xffff0000u);
    const float s1 = r1 - __builtin_bit_cast(float, b1 & 0xffff0000u);
    w[2] = __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, s1), __builtin_bit_cast(unsigned, s0), 0x07060302u);
  } else {
    w[0] = pk_bf16(x0, x1);
    if constexpr (NP == 2) {
      w[1] = pk_bf16(x0 - __builtin_bit_cast(float, w[0] << 16), x1 - __builtin_bit_cast(float, w[0] & 0xffff0000u));
    }
  }
}

// 8 fp32 values -> NP operand fragments
template <int NP>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&f)[NP]) {
  unsigned w[4][NP];
#pragma unroll
  for (int p = 0; p < 4; ++p) split_pair<NP>(x[2 * p], x[2 * p + 1], w[p]);
#pragma unroll
  for (int n = 0; n < NP; ++n) f[n] = __builtin_bit_cast(bf16x8, uint4{w[0][n], w[1][n], w[2][n], w[3][n]});
}

// c += A B over the planes of both operands, the products of planes i and j
// with i + j < max(NA, NB), smallest first.  What is left out, of a product
// x y: nothing where one operand is one plane and exact (bf16 inputs); with
// three planes of both, x1 y2 + x2 y1 + x2 y2, where cut planes obey
// |x1| < 2^-7 |x| and |x2| < 2^-15 |x|: less than 2^-21 |x y|, always with the
// product's own sign (cutting keeps it).  In a sum that is at most 2^-21 of the
// sum of the terms' sizes: 8 roundings of fp32, and no more than the fp32 sum
// of a few dozen terms itself loses.
template <int NA, int NB>
__device__ __forceinline__ void mma_planes(f32x4 &c, const bf16x8 (&a)[NA], const bf16x8 (&b)[NB]) {
  constexpr int M = NA > NB ? NA : NB;
#pragma unroll
  for (int s = M - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[s - i], c, 0, 0, 0);
}

// Decays.  A sum of log decays along a path is kept in fp64 and in units of
// log2(e), and a weight exp(G_r - G_i) is one exp2 of the difference rounded
// to fp32, so that a strong decay between two tokens costs the weights behind
// it no precision.  A single log decay below -200 is taken as -200: its
// exp is zero in fp32 times any fp32 state, and sums and differences stay
// finite (-inf, a hard reset, among them).
__device__ __forceinline__ double log2_decay(float g) {
  return (double)(g < -200.f ? -200.f : g) * 1.4426950408889634074;
}
__device__ __forceinline__ float decay_between(double to, double from) {
  return __builtin_amdgcn_exp2f((float)(to - from));
}

}  // namespace gdn
