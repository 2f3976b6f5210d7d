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
// Unscaled, the residual after k refusals is max(p - t q, 0) with one number t:
// clamping at zero before taking off more changes nothing, so
//   r_k = max(p - t_k q, 0),  t_k = s_0 + .. + s_{k-1},  s_0 = 1,  s_k = sum r_k
// and a child is accepted if  u s_k q(x) < r_k(x).  A refusal before a further
// child costs one pass over the vocabulary for s_k; all else are reads of
// single probabilities.  A residual without mass is not taken (p stays).
//
// Children have higher numbers than their parent, so one sweep over the nodes
// in order finds the path.  All comparisons and sums are in fp64 of the fp32
// inputs: they decide tokens.
//
// Rows are few, so a large vocabulary is cut into parts, a workgroup each,
// whose sums one more workgroup per row joins to find the token's part; of a
// small one a workgroup per row does it all, in one launch.  Latency and
// launches bound both.  Measured: 5 nodes in a chain with draft probabilities,
// 32003 tokens, 12.8 us a call (kernel 12.5); 32 rows of 16 nodes without,
// 131072 tokens, 15.0 us a call (kernels 6.7 + 6.8; 17 MB).  The pass of a
// refusal before a further child adds, at 8192, 32003, 65536 and 131072 tokens,
// 3.0, 8.3, 16 and 30 us to one row, and 3.0, 8.5, 35 and 79 us to 32 rows that
// each have one: it is one workgroup's, and its reads wait for each other.
#pragma once
#include "gdn_common.h"

namespace gdn {

constexpr int kVerifyNodes = 64;      // nodes per row: one per lane of a wave
constexpr int VERIFY_PART = 4096;     // tokens of the vocabulary per workgroup and partial sum

struct VerifyPlan {
  double taken;                 // t above, of the last refusal
  double before;                // t without it, if its residual's mass is not known yet; -1 else
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
// max(p - t q, 0), but p at most: a draft value below zero, or one that is no
// number (fmin takes the other of the two), counts as zero, as in the tests of
// the children.  One instruction more, and behind the loads.
__device__ __forceinline__ double residual(float p, float q, double t) {
  return positive(fmin(fma(-t, (double)q, (double)p), (double)p));
}

// sum of max(p - t q, 0) over tokens lo .. hi - 1 by THREADS threads, this thread's share
// (a token's p and then its q, each waited for before what comes next)
template <int THREADS>
__device__ __forceinline__ double residual_share(const float *p, const float *q, double t, int lo, int hi, int tid) {
  double s = 0.;
  for (int v = lo + tid; v < hi; v += THREADS) {
    s += q ? residual(p[v], q[v], t) : positive((double)p[v]);
  }
  return s;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

// The path of one row, every wave of the workgroup the same sweep.  A refusal
// with no child behind it leaves its residual's mass to the sums that follow.
template <int THREADS, bool DRAFT>
__device__ __forceinline__ VerifyPlan verify_walk(const VerifyArgs &a, int b, int tid, double (&red)[2][THREADS / 64], int &mine) {
  const int lane = tid & 63, wave = tid >> 6, n = a.n;
  const int parent = lane < n ? a.parents[(size_t)b * n + lane] : -2;
  const int x = lane < n ? a.tokens[(size_t)b * n + lane] : -1;
  const bool child = parent >= -1 && parent < lane && x >= 0 && x < a.V;
  double px = 0., qx = 0., u = 0.;
  if (child) {
    px = positive((double)a.target[((size_t)b * (n + 1) + parent + 1) * a.V + x]);
    if constexpr (DRAFT) qx = positive((double)a.draft[((size_t)b * n + parent + 1) * a.V + x]);
    u = (double)a.uniform[(size_t)b * (n + 1) + lane];
  }
  VerifyPlan plan{0., -1., 0, -1, 0};
  unsigned long long todo = __ballot(child);
  int len = 0, turn = 0;
  double mass = 1.;
  mine = -1;   // this lane's entry of the path
  unsigned long long next = __ballot(child && parent == -1);
  while (next) {
    const int r = __ffsll((long long)next) - 1;
    todo &= ~(1ull << r);
    const double p = __shfl(px, r), q = __shfl(qx, r), ur = __shfl(u, r);
    bool ok;
    if constexpr (DRAFT) {
      ok = ur * mass * q < positive(fma(-plan.taken, q, p));
    } else {
      const int xr = __shfl(x, r);
      const bool again = __ballot((plan.refused >> lane & 1) && x == xr) != 0;   // a sibling with this token was refused
      const double left = again ? 0. : p;
      ok = ur * mass < left;
      if (!ok) {
        mass -= left;
        plan.refused |= 1ull << r;
      }
    }
    if (ok) {
      plan = VerifyPlan{0., -1., 0, r, 0};
      if (lane == len) mine = r;
      ++len;
      mass = 1.;
    }
    next = __ballot((todo >> lane & 1) && parent == plan.at);
    if constexpr (DRAFT) {
      if (ok) continue;
      const double t = plan.taken + mass;
      if (!next) {
        plan.before = plan.taken;
        plan.taken = t;
        break;
      }
      // the sum decides whether the residual is taken, and the next child's test
      const double w = wave_sum(residual_share<THREADS>(a.target + ((size_t)b * (n + 1) + plan.at + 1) * a.V,
                                                        a.draft + ((size_t)b * n + plan.at + 1) * a.V, t, 0, a.V, tid));
      if (lane == 0) red[turn & 1][wave] = w;
      __syncthreads();
      double s = 0.;
#pragma unroll
      for (int i = 0; i < THREADS / 64; ++i) s += red[turn & 1][i];
      ++turn;
      if (s > 0.) {
        plan.taken = t;
        mass = s;
      }
    }
  }
  return plan;
}
__device__ __forceinline__ void note_walk(const VerifyArgs &a, int b, int lane, const VerifyPlan &plan, int mine) {
  if (lane < a.n) a.path[(size_t)b * a.n + lane] = mine;
  if (lane == 0) {
    a.last[b] = plan.at;
    a.plan[b] = plan;
  }
}

// With draft probabilities, the walk in a launch of its own: its passes over
// the vocabulary take a whole workgroup per row.
__global__ __launch_bounds__(1024) void verify_walk_kernel(VerifyArgs a) {
  __shared__ double red[2][16];
  int mine;
  const VerifyPlan plan = verify_walk<1024, true>(a, blockIdx.x, threadIdx.x, red, mine);
  if (threadIdx.x < 64) note_walk(a, blockIdx.x, threadIdx.x, plan, mine);
}

// A part's weights: max(p - t q, 0), or p without the refused tokens.
struct Residual {
  const float *p, *q;
  double t;
  const int *tokens;
  unsigned long long refused;   // those in the part
};
__device__ __forceinline__ Residual residual_of(const VerifyArgs &a, const VerifyPlan &w, double taken, int b, int lo, int hi, int lane) {
  Residual r;
  r.p = a.target + ((size_t)b * (a.n + 1) + w.at + 1) * a.V;
  r.q = a.draft && taken > 0. ? a.draft + ((size_t)b * a.n + w.at + 1) * a.V : nullptr;
  r.t = taken;
  r.tokens = a.tokens + (size_t)b * a.n;
  const int x = lane < a.n && (w.refused >> lane & 1) ? r.tokens[lane] : -1;
  r.refused = __ballot(x >= lo && x < hi);
  return r;
}
// COUNT weights, tokens v, v + step, .. below hi (none behind it).  Without draft
// probabilities all are asked for at once; with them each q is read under a test
// for whether there is one, and waited for.
template <int COUNT>
__device__ __forceinline__ void weights(const Residual &r, int v, int step, int hi, double (&w)[COUNT]) {
  float p[COUNT], q[COUNT];
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    const int at = min(v + i * step, hi - 1);
    p[i] = r.p[at];
    q[i] = r.q ? r.q[at] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < COUNT; ++i) w[i] = v + i * step < hi ? residual(p[i], q[i], r.t) : 0.;
  for (unsigned long long m = r.refused; m; m &= m - 1) {   // (uniform, and mostly none)
    const int x = r.tokens[__ffsll((long long)m) - 1];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) w[i] = v + i * step == x ? 0. : w[i];
  }
}
// the sum over a part, by a wave
__device__ __forceinline__ double part_sum(const Residual &r, int lo, int hi, int lane) {
  constexpr int COUNT = 16;
  double s = 0.;
  for (int v = lo; v < hi; v += 64 * COUNT) {
    double w[COUNT];
    weights<COUNT>(r, v + lane, 64, hi, w);
#pragma unroll
    for (int i = 0; i < COUNT; ++i) s += w[i];
  }
  return wave_sum(s);
}

// The sums of the parts, one workgroup each, a quarter per wave.  Without
// draft probabilities every workgroup walks the tree first (a few reads of
// single probabilities), which saves a launch.
template <bool DRAFT>
__global__ __launch_bounds__(256) void verify_sum_kernel(VerifyArgs a) {
  __shared__ double red[4];
  const int b = blockIdx.x / a.parts, k = blockIdx.x % a.parts, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  VerifyPlan plan;
  if constexpr (DRAFT) {
    plan = a.plan[b];
  } else {
    double none[2][4];
    int mine;
    plan = verify_walk<256, false>(a, b, tid, none, mine);
    if (k == 0 && wave == 0) note_walk(a, b, lane, plan, mine);
  }
  constexpr int QUARTER = VERIFY_PART / 4;
  const int lo = min(a.V, k * VERIFY_PART + wave * QUARTER), hi = min(a.V, lo + QUARTER);
  const Residual r = residual_of(a, plan, plan.taken, b, lo, hi, lane);
  const double s = part_sum(r, lo, hi, lane);
  if (lane == 0) red[wave] = s;
  __syncthreads();
  if (tid == 0) a.part[(size_t)b * a.parts + k] = (red[0] + red[1]) + (red[2] + red[3]);
}

__device__ __forceinline__ double wave_scan(double x, int lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// The token: the part in which the running sum passes u times the whole, in it
// the 16 tokens of a thread, among them the token.  Where rounding leaves sums
// on one level short of the mark that the level above had passed, it is the
// last one with a weight.
__global__ __launch_bounds__(256) void verify_draw_kernel(VerifyArgs a) {
  constexpr int PER = VERIFY_PART / 256;
  __shared__ double total[4], from;
  __shared__ int found, hits[4], some[4];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const VerifyPlan plan = a.plan[b];
  double *part = a.part + (size_t)b * a.parts;
  const double u = (double)a.uniform[(size_t)b * (a.n + 1) + a.n];
  const int per = (a.parts + 255) / 256, k0 = min(a.parts, tid * per), k1 = min(a.parts, k0 + per);
  double taken = plan.taken, before, whole;
  if (tid == 0) found = -1;
  for (bool again = false;; again = true) {
    double s = 0.;
    for (int k = k0; k < k1; ++k) s += part[k];
    const double upto = wave_scan(s, lane);
    if (lane == 63) total[wave] = upto;
    __syncthreads();
    before = upto - s;
    whole = 0.;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < wave) before += total[w];
      whole += total[w];
    }
    if (whole > 0. || again || plan.before < 0.) break;   // uniform
    // a residual without mass is not taken: the sums without the last refusal
    taken = plan.before;
    for (int k = wave; k < a.parts; k += 4) {
      const int lo = k * VERIFY_PART, hi = min(a.V, lo + VERIFY_PART);
      const double p = part_sum(residual_of(a, plan, taken, b, lo, hi, lane), lo, hi, lane);
      if (lane == 0) part[k] = p;
    }
    __syncthreads();
  }
  const double mark = u * whole;
  int mine = -1;
  double start = 0., run = before;
  for (int k = k0; k < k1; ++k) {
    if (mine < 0 && part[k] > 0. && run + part[k] > mark) {
      mine = k;
      start = run;
    }
    run += part[k];
  }
  // the first thread with such a part: of a wave, then of the waves
  const unsigned long long pass = __ballot(mine >= 0);
  __shared__ int first[4];
  if (lane == 0) first[wave] = pass ? wave * 64 + __ffsll((long long)pass) - 1 : 256;
  __syncthreads();
  const int who = min(min(first[0], first[1]), min(first[2], first[3]));
  if (who == 256) {   // uniform: no mass (or no number)
    if (tid == 0) a.token[b] = -1;
    return;
  }
  if (tid == who) {
    found = mine;
    from = start;
  }
  __syncthreads();
  const int lo = found * VERIFY_PART, hi = min(a.V, lo + VERIFY_PART);
  const Residual r = residual_of(a, plan, taken, b, lo, hi, lane);
  double w[PER], sum = 0.;
  weights<PER>(r, lo + tid * PER, 1, hi, w);
#pragma unroll
  for (int i = 0; i < PER; ++i) sum += w[i];
  const double upto = wave_scan(sum, lane);
  if (lane == 63) total[wave] = upto;
  __syncthreads();
  run = from + (upto - sum);
  for (int i = 0; i < wave; ++i) run += total[i];
  // this thread's first token with a weight at which the sum passes, and its last with a weight
  int hit = 1 << 30, any = -1;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    run += w[i];
    if (w[i] > 0.) {
      any = lo + tid * PER + i;
      if (run > mark) hit = min(hit, any);
    }
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    hit = min(hit, __shfl_xor(hit, m));
    any = max(any, __shfl_xor(any, m));
  }
  if (lane == 0) {
    hits[wave] = hit;
    some[wave] = any;
  }
  __syncthreads();
  if (tid) return;
  hit = min(min(hits[0], hits[1]), min(hits[2], hits[3]));
  a.token[b] = hit < 1 << 30 ? hit : max(max(some[0], some[1]), max(some[2], some[3]));
}

// All of a row by one workgroup, for small vocabularies: the walk, the sums of
// chunks of 1024 tokens (a wave each; without draft probabilities two at once),
// and the draw by the first wave.
constexpr int VERIFY_CHUNK = 1024, VERIFY_CHUNKS = 32;
template <bool DRAFT>
__global__ __launch_bounds__(1024) void verify_row_kernel(VerifyArgs a) {
  constexpr int PER = VERIFY_CHUNK / 64, PAIR = DRAFT ? 1 : 2;
  __shared__ double red[2][16], sums[VERIFY_CHUNKS];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const double u = (double)a.uniform[(size_t)b * (a.n + 1) + a.n];
  int mine;
  const VerifyPlan plan = verify_walk<1024, DRAFT>(a, b, tid, red, mine);
  if (wave == 0) {
    if (lane < a.n) a.path[(size_t)b * a.n + lane] = mine;
    if (lane == 0) a.last[b] = plan.at;
  }
  const int chunks = (a.V + VERIFY_CHUNK - 1) / VERIFY_CHUNK;
  double taken = plan.taken, own, upto, whole;
  for (bool again = false;; again = true) {
    for (int k = wave; k < chunks; k += 16 * PAIR) {
      float p[PAIR][PER], q[PAIR][PER];
      Residual r[PAIR];
      int hi[PAIR];
#pragma unroll
      for (int m = 0; m < PAIR; ++m) {
        const int lo = (k + 16 * m) * VERIFY_CHUNK;
        hi[m] = min(a.V, lo + VERIFY_CHUNK);
        r[m] = residual_of(a, plan, taken, b, lo, hi[m], lane);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int at = min(lo + lane + i * 64, a.V - 1);   // (a chunk behind the last: read again, and not counted)
          p[m][i] = r[m].p[at];
          q[m][i] = DRAFT && r[m].q ? r[m].q[at] : 0.f;
        }
      }
#pragma unroll
      for (int m = 0; m < PAIR; ++m) {
        double s = 0.;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int v = (k + 16 * m) * VERIFY_CHUNK + lane + i * 64;
          double w = v < hi[m] ? (DRAFT ? residual(p[m][i], q[m][i], taken) : positive((double)p[m][i])) : 0.;
          if constexpr (!DRAFT)
            for (unsigned long long left = r[m].refused; left; left &= left - 1)   // (uniform, and mostly none)
              w = v == r[m].tokens[__ffsll((long long)left) - 1] ? 0. : w;
          s += w;
        }
        s = wave_sum(s);
        if (lane == 0 && k + 16 * m < chunks) sums[k + 16 * m] = s;
      }
    }
    __syncthreads();
    own = lane < chunks ? sums[lane] : 0.;
    upto = wave_scan(own, lane);
    whole = __shfl(upto, 63);
    if (whole > 0. || again || plan.before < 0.) break;   // uniform
    taken = plan.before;   // a residual without mass is not taken
    __syncthreads();
  }
  if (wave) return;
  const double mark = u * whole;
  const unsigned long long pass = __ballot(own > 0. && upto > mark);
  if (!pass) {   // no mass (or no number)
    if (lane == 0) a.token[b] = -1;
    return;
  }
  const int who = __ffsll((long long)pass) - 1;
  const int lo = who * VERIFY_CHUNK, hi = min(a.V, lo + VERIFY_CHUNK);
  double w[PER], sum = 0., run = __shfl(upto - own, who);
  weights<PER>(residual_of(a, plan, taken, b, lo, hi, lane), lo + lane * PER, 1, hi, w);
#pragma unroll
  for (int i = 0; i < PER; ++i) sum += w[i];
  run += wave_scan(sum, lane) - sum;
  int hit = 1 << 30, any = -1;   // the lane's first token at which the sum passes, and its last with a weight
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    run += w[i];
    if (w[i] > 0.) {
      any = lo + lane * PER + i;
      if (run > mark) hit = min(hit, any);
    }
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    hit = min(hit, __shfl_xor(hit, m));
    any = max(any, __shfl_xor(any, m));
  }
  if (lane == 0) a.token[b] = hit < 1 << 30 ? hit : any;
}

}  // namespace gdn
