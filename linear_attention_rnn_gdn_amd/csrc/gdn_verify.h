// gdn_verify.h -- verification of a tree of drafted tokens against the
// target's probabilities, from given random numbers.
//
// Row b walks its tree from the root.  At the node reached (probabilities p
// of the next token there) the node's children are looked at in their order:
//   without draft probabilities a child with token x is accepted if
//     u m < p(x),  m = 1 - the probabilities of the children refused before it,
//   and a refused child's token is taken out of p;
//   with draft probabilities q, from which the children were drawn, it is
//   accepted if  u q(x) < p(x), and a refusal leaves p <- max(p - q, 0),
//   scaled to one.
// Where no child is accepted, or there is none, the next token is drawn from
// what is left of p: the lowest v whose running sum passes u times the whole.
//
// Unscaled, the residual after k refusals is max(p - t q, 0) with one number
// t: clamping at zero before taking off more changes nothing, so
//   r_k = max(p - t_k q, 0),  t_k = s_0 + .. + s_{k-1},  s_0 = 1,  s_k = sum r_k
// and a child is accepted if  u s_k q(x) < r_k(x).  A refusal before a further
// child costs one pass over the vocabulary for s_k; all else are reads of
// single probabilities.  A residual without mass is not taken (p stays).
//
// Children have higher numbers than their parent, so one sweep over the nodes
// in order finds the path.  All comparisons and sums are in fp64 of the fp32
// inputs: they decide tokens.
#pragma once
#include "gdn_common.h"

namespace gdn {

constexpr int kVerifyNodes = 64;      // nodes per row: one per lane of a wave
constexpr int VERIFY_PART = 4096;     // tokens of the vocabulary per workgroup and partial sum

struct VerifyPlan {
  double taken;                 // t above
  unsigned long long refused;   // without draft probabilities: the nodes whose tokens are taken out
  int at, pad;                  // the node reached, -1: the root
};

struct VerifyArgs {
  int B, n, V, parts;
  const int *tokens, *parents;
  const float *target, *draft, *uniform;
  int *last, *token, *path;
  VerifyPlan *plan;             // [B]
  double *part;                 // [B, parts]
};

__device__ __forceinline__ double positive(double x) { return x > 0. ? x : 0.; }   // (no number: nothing)

// sum of max(p - t q, 0) over tokens lo .. hi - 1 by THREADS threads, this thread's share
template <int THREADS>
__device__ __forceinline__ double residual_share(const float *p, const float *q, double t, int lo, int hi, int tid) {
  double s = 0.;
  for (int v = lo + tid; v < hi; v += THREADS) {
    double x = (double)p[v];
    if (q) x = fma(-t, (double)q[v], x);
    s += positive(x);
  }
  return s;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

__device__ __forceinline__ double shfl_f64(double x, int lane) { return __shfl(x, lane); }

// The path of one row: one workgroup, every wave the same sweep.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void verify_walk_kernel(VerifyArgs a) {
  constexpr int WAVES = THREADS / 64;
  __shared__ double red[2][WAVES];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.n;
  const int parent = lane < n ? a.parents[(size_t)b * n + lane] : -2;
  const int x = lane < n ? a.tokens[(size_t)b * n + lane] : -1;
  const bool child = parent >= -1 && parent < lane && x >= 0 && x < a.V;
  double px = 0., qx = 0., u = 0.;
  if (child) {
    px = positive((double)a.target[((size_t)b * (n + 1) + parent + 1) * a.V + x]);
    if (a.draft) qx = positive((double)a.draft[((size_t)b * n + parent + 1) * a.V + x]);
    u = (double)a.uniform[(size_t)b * (n + 1) + lane];
  }
  unsigned long long todo = __ballot(child), refused = 0;
  int at = -1, len = 0, turn = 0, mine = -1;   // mine: this lane's entry of the path
  double mass = 1., taken = 0.;
  while (true) {
    const unsigned long long next = __ballot((todo >> lane & 1) && parent == at);
    if (!next) break;
    const int r = __ffsll((long long)next) - 1;
    todo &= ~(1ull << r);
    const double p = shfl_f64(px, r), q = shfl_f64(qx, r), ur = shfl_f64(u, r);
    const int xr = __shfl(x, r);
    bool ok;
    if (a.draft) {
      ok = ur * mass * q < positive(fma(-taken, q, p));
    } else {
      const bool again = __ballot((refused >> lane & 1) && x == xr) != 0;   // a sibling with this token was refused
      const double left = again ? 0. : p;
      ok = ur * mass < left;
      if (!ok) mass -= left;
    }
    if (ok) {
      at = r;
      if (lane == len) mine = r;
      ++len;
      mass = 1.;
      taken = 0.;
      refused = 0;
    } else if (!a.draft) {
      refused |= 1ull << r;
    } else {
      // the sum decides whether the residual is taken, and the next child's test
      const double t = taken + mass;
      const double w = wave_sum(residual_share<THREADS>(a.target + ((size_t)b * (n + 1) + at + 1) * a.V,
                                                        a.draft + ((size_t)b * n + at + 1) * a.V, t, 0, a.V, tid));
      if (lane == 0) red[turn & 1][wave] = w;
      __syncthreads();
      double s = 0.;
      for (int i = 0; i < WAVES; ++i) s += red[turn & 1][i];
      ++turn;
      if (s > 0.) {
        taken = t;
        mass = s;
      }
    }
  }
  if (wave) return;
  if (lane < n) a.path[(size_t)b * n + lane] = mine;
  if (lane == 0) {
    a.last[b] = at;
    a.plan[b] = VerifyPlan{taken, refused, at, 0};
  }
}

// A part's weights: max(p - t q, 0), or p without the refused tokens.
struct Residual {
  const float *p, *q;
  double t;
  const int *tokens;
  unsigned long long refused;   // those in the part
};
__device__ __forceinline__ Residual residual_of(const VerifyArgs &a, int b, int lo, int hi, int lane) {
  const VerifyPlan w = a.plan[b];
  Residual r;
  r.p = a.target + ((size_t)b * (a.n + 1) + w.at + 1) * a.V;
  r.q = a.draft && w.taken > 0. ? a.draft + ((size_t)b * a.n + w.at + 1) * a.V : nullptr;
  r.t = w.taken;
  r.tokens = a.tokens + (size_t)b * a.n;
  const int x = lane < a.n && (w.refused >> lane & 1) ? r.tokens[lane] : -1;
  r.refused = __ballot(x >= lo && x < hi);
  return r;
}
__device__ __forceinline__ double weight(const Residual &r, int v) {
  double x = (double)r.p[v];
  if (r.q) x = fma(-r.t, (double)r.q[v], x);
  for (unsigned long long m = r.refused; m; m &= m - 1)
    if (r.tokens[__ffsll((long long)m) - 1] == v) x = 0.;
  return positive(x);
}

__global__ __launch_bounds__(256) void verify_sum_kernel(VerifyArgs a) {
  __shared__ double red[4];
  const int b = blockIdx.x / a.parts, k = blockIdx.x % a.parts, tid = threadIdx.x, lane = tid & 63;
  const int lo = k * VERIFY_PART, hi = min(a.V, lo + VERIFY_PART);
  const Residual r = residual_of(a, b, lo, hi, lane);
  double s = 0.;
  for (int v = lo + tid; v < hi; v += 256) s += weight(r, v);
  s = wave_sum(s);
  if (lane == 0) red[tid >> 6] = s;
  __syncthreads();
  if (tid == 0) a.part[(size_t)b * a.parts + k] = (red[0] + red[1]) + (red[2] + red[3]);
}

// The token: the part in which the running sum passes u times the whole, then
// the token within it.  Rounding may leave the part's own sums short of the
// mark: its last token with a weight then.
__global__ __launch_bounds__(256) void verify_draw_kernel(VerifyArgs a) {
  constexpr int PER = VERIFY_PART / 256;
  __shared__ double red[4], scan[256];
  __shared__ int found;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const double *part = a.part + (size_t)b * a.parts;
  // thread 0 .. 255: consecutive parts each
  const int per = (a.parts + 255) / 256, k0 = min(a.parts, tid * per), k1 = min(a.parts, k0 + per);
  double s = 0.;
  for (int k = k0; k < k1; ++k) s += part[k];
  scan[tid] = s;
  __syncthreads();
  double before = 0., total = 0.;
  for (int i = 0; i < 256; ++i) {
    if (i == tid) before = total;
    total += scan[i];
  }
  const double mark = (double)a.uniform[(size_t)b * (a.n + 1) + a.n] * total;
  if (tid == 0) found = -1;
  __syncthreads();
  int mine = -1;
  double start = 0., run = before;
  for (int k = k0; k < k1; ++k) {
    if (mine < 0 && run + part[k] > mark && part[k] > 0.) {
      mine = k;
      start = run;
    }
    run += part[k];
  }
  // the first thread whose parts pass the mark; if rounding leaves none, the last one with mass
  const bool pass = mine >= 0;
  __shared__ int first[4];
  __shared__ double from;
  const unsigned long long bal = __ballot(pass);
  if (lane == 0) first[wave] = bal ? wave * 64 + __ffsll((long long)bal) - 1 : 1 << 30;
  __syncthreads();
  const int who = min(min(first[0], first[1]), min(first[2], first[3]));
  if (who == 1 << 30) {   // uniform: no mass (or no number)
    if (tid == 0) a.token[b] = -1;
    return;
  }
  if (tid == who) {
    found = mine;
    from = start;
  }
  __syncthreads();
  const int lo = found * VERIFY_PART, hi = min(a.V, lo + VERIFY_PART);
  const Residual r = residual_of(a, b, lo, hi, lane);
  double w[PER], sum = 0.;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int v = lo + tid * PER + i;
    w[i] = v < hi ? weight(r, v) : 0.;
    sum += w[i];
  }
  double upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 63) red[wave] = upto;
  __syncthreads();
  double run2 = from + (upto - sum);
  for (int i = 0; i < wave; ++i) run2 += red[i];
  int hit = 1 << 30, any = -1;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    run2 += w[i];
    if (w[i] > 0.) {
      any = lo + tid * PER + i;
      if (run2 > mark) hit = min(hit, any);
    }
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    hit = min(hit, __shfl_xor(hit, m));
    any = max(any, __shfl_xor(any, m));
  }
  __shared__ int hits[4], anys[4];
  if (lane == 0) {
    hits[wave] = hit;
    anys[wave] = any;
  }
  __syncthreads();
  if (tid == 0) {
    hit = min(min(hits[0], hits[1]), min(hits[2], hits[3]));
    any = max(max(anys[0], anys[1]), max(anys[2], anys[3]));
    a.token[b] = hit < 1 << 30 ? hit : any;
  }
}

}  // namespace gdn
