// gdn_states.h -- kernels on a pool of recurrent states: the single-token
// step, the check of a tree of drafted tokens and the commit of an accepted
// path.
//
// A pool holds states [n_slots][H_v][128][128] in fp32 (row = d_k index); row
// b of a call works on the state in slot slots[b].  Every kernel here reads
// (and, but for the check, writes) 64 KB of state per row and value head and
// computes little on it, so they are built to keep many state bytes in
// flight: a workgroup loads its whole part of a state into registers before
// anything else, and reductions over the state's rows are a few lane
// permutations and one pass through LDS.
#pragma once
#include <type_traits>

#include "gdn_common.h"

namespace gdn {

struct StateArgs {
  int B, n, Hqk, Hv, n_slots;
  int g_fixed;                   // decays: 0 = per token [B, n, H_v], 1 = [H_v]
  const void *q, *k, *v;
  const float *g, *beta;         // beta null: the linear rule (no correction)
  const int *parents, *slots, *last;
  const float *u_in;
  float *state, *u;
  void *o;
  int stream;                    // states are stored past the caches
};

// The slot of row b, or -1 if the row has no state.
__device__ __forceinline__ int row_slot(const StateArgs &a, int b) {
  const int s = a.slots ? a.slots[b] : b;
  return s >= 0 && s < a.n_slots ? s : -1;
}

// Whether an earlier row that writes names the same slot (a thread's share of
// the rows); writes(i): row i writes the state of the slot it names.
template <typename F>
__device__ __forceinline__ bool slot_seen(const StateArgs &a, int b, int slot, int tid, int nthreads, F &&writes) {
  bool seen = false;
  if (a.slots)
    for (int i = tid; i < b; i += nthreads) seen |= a.slots[i] == slot && writes(i);
  return seen;
}

__device__ __forceinline__ float4 ld_state(const float *p) { return *reinterpret_cast<const float4 *>(p); }
// RPT rows of a state, D floats apart.  `stream`: past the caches, for calls
// that write more state than the memory-side cache (256 MB) keeps; a smaller
// pool's states are still there for the next step and are stored plainly.
// Measured with 32 value heads on a pool of as many slots as rows, the same
// call again and again, streamed / plain, us a step and a commit of 6 nodes:
//    32 rows   64 MB   23 /  23    26 /  25      144 rows  288 MB   91 /  95    96 / 103
//    96 rows  192 MB   62 /  62    67 /  65      160 rows  320 MB  102 / 116   107 / 124
//   112 rows  224 MB   71 /  71    78 /  75      192 rows  384 MB  135 / 156   127 / 166
//   128 rows  256 MB   80 /  83    87 /  90      256 rows  512 MB  212 / 213   175 / 221
template <int RPT>
__device__ __forceinline__ void st_state(float *p, const float4 (&x)[RPT], bool stream) {
  if (stream) {
    // (the empty statements keep the compiler from merging the two branches'
    // stores, which would drop the hint)
    asm volatile("");
#pragma unroll
    for (int i = 0; i < RPT; ++i) st16_stream(p + i * D, x[i]);
    asm volatile("");
  } else {
#pragma unroll
    for (int i = 0; i < RPT; ++i) *reinterpret_cast<float4 *>(p + i * D) = x[i];
  }
}
__device__ __forceinline__ float4 fma4(float a, const float4 &x, const float4 &y) {
  return float4{fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w)};
}
__device__ __forceinline__ float4 mul4(float a, const float4 &x) { return float4{a * x.x, a * x.y, a * x.z, a * x.w}; }

// Four consecutive elements of a tensor as fp32, and their store.
__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 ld4(const __bf16 *p) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  return float4{__builtin_bit_cast(float, w.x << 16), __builtin_bit_cast(float, w.x & 0xffff0000u),
                __builtin_bit_cast(float, w.y << 16), __builtin_bit_cast(float, w.y & 0xffff0000u)};
}
__device__ __forceinline__ void st4(float *p, const float4 &x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void st4(__bf16 *p, const float4 &x) {
  *reinterpret_cast<uint2 *>(p) = uint2{pk_bf16(x.x, x.y), pk_bf16(x.z, x.w)};
}

// ----------------------------------------------------------------------------
// The rule for one token:
//   a = e^g S;  u = beta (v - a^T k)  (linear rule: u = v);  S' = a + k u^T;
//   o = S'^T q = e^g S^T q + (q.k) u.
// The second form of o needs the old state only, so S^T k and S^T q are
// reduced together in one pass and the state is read once and written once.
// A workgroup of 256 threads takes COLS columns of one state: each thread
// holds RPT consecutive rows of 4 columns (one 16-byte load per row; a wave's
// load covers whole 128-byte lines).  All sums are fp32.
template <int COLS, typename TI, typename TO>
__global__ __launch_bounds__(256) void step_kernel(StateArgs a) {
  constexpr int LPR = COLS / 4, RG = 256 / LPR, RPT = D / RG;
  __shared__ float ks[D], qs[D];
  __shared__ float4 part[4][2][LPR];
  __shared__ int dup;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  int unit, cpart;
  xcd_unit(blockIdx.x, D / COLS, a.B * a.Hv, unit, cpart);
  const int b = unit / a.Hv, hv = unit % a.Hv, hq = hv / (a.Hv / a.Hqk);
  const int c4 = (tid % LPR) * 4, col = cpart * COLS + c4, r0 = (tid / LPR) * RPT;
  const int slot = row_slot(a, b);
  TO *o = static_cast<TO *>(a.o) + ((size_t)b * a.Hv + hv) * D + col;
  if (slot < 0) {   // uniform: no state, the output row is zero
    if (tid < LPR) st4(o, float4{0.f, 0.f, 0.f, 0.f});
    return;
  }
  float *S = a.state + ((size_t)slot * a.Hv + hv) * (D * D) + (size_t)r0 * D + col;
  float4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = ld_state(S + i * D);
  if (tid == 0) dup = 0;
  const size_t kq = ((size_t)b * a.Hqk + hq) * D;
  if (tid < D) ks[tid] = to_f32(static_cast<const TI *>(a.k)[kq + tid]);
  else qs[tid - D] = to_f32(static_cast<const TI *>(a.q)[kq + tid - D]);
  const float4 v = ld4(static_cast<const TI *>(a.v) + ((size_t)b * a.Hv + hv) * D + col);
  const float eg = decay_between(log2_decay(a.g[a.g_fixed ? hv : (size_t)b * a.Hv + hv]), 0.);
  const float beta = a.beta ? a.beta[(size_t)b * a.Hv + hv] : 0.f;
  __syncthreads();
  if (slot_seen(a, b, slot, tid, 256, [](int) { return true; })) dup = 1;
  float kr[RPT];
  float4 sk{0.f, 0.f, 0.f, 0.f}, sq{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    kr[i] = ks[r0 + i];
    sk = fma4(kr[i], s[i], sk);
    sq = fma4(qs[r0 + i], s[i], sq);
  }
  float qk = ks[lane] * qs[lane] + ks[lane + 64] * qs[lane + 64];
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    qk += __shfl_xor(qk, m);
    if (m >= LPR) {
      sk.x += __shfl_xor(sk.x, m); sk.y += __shfl_xor(sk.y, m); sk.z += __shfl_xor(sk.z, m); sk.w += __shfl_xor(sk.w, m);
      sq.x += __shfl_xor(sq.x, m); sq.y += __shfl_xor(sq.y, m); sq.z += __shfl_xor(sq.z, m); sq.w += __shfl_xor(sq.w, m);
    }
  }
  if (lane < LPR) {
    part[wave][0][lane] = sk;
    part[wave][1][lane] = sq;
  }
  __syncthreads();
  if (dup) {   // uniform: the slot's first row has it
    if (tid < LPR) st4(o, float4{0.f, 0.f, 0.f, 0.f});
    return;
  }
  float4 tk = part[0][0][tid % LPR], tq = part[0][1][tid % LPR];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    tk = fma4(1.f, part[w][0][tid % LPR], tk);
    tq = fma4(1.f, part[w][1][tid % LPR], tq);
  }
  const float4 u = a.beta ? mul4(beta, fma4(-eg, tk, v)) : v;
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = fma4(kr[i], u, mul4(eg, s[i]));
  st_state(S, s, a.stream);
  if (tid < LPR) st4(o, fma4(qk, u, mul4(eg, tq)));
}

// ----------------------------------------------------------------------------
// Trees of up to 64 nodes, one per lane of a wave.  Node r continues node
// parents[r] < r, or the state itself (-1); any other value, or an ancestor
// that has one, makes the node absent.  By doubling of the pointers:
//   anc   the node and its ancestors, as bits      G  the sum of their log decays
struct Path {
  unsigned long long anc;
  double G;        // in units of log2(e)
  bool live;
};
__device__ __forceinline__ Path tree_path(const StateArgs &a, int b, int hv, int lane) {
  const size_t at = (size_t)b * a.n + lane;
  int p = lane < a.n ? a.parents[at] : -2;
  const bool valid = p >= -1 && p < lane;
  Path t;
  t.anc = 1ull << lane;
  t.G = valid ? log2_decay(a.g[a.g_fixed ? hv : at * a.Hv + hv]) : 0.;
  int dead = !valid;
  if (!valid) p = -1;
  while (__ballot(p >= 0)) {
    const int src = p >= 0 ? p : lane;
    const unsigned long long anc = __shfl(t.anc, src);
    const double G = __shfl(t.G, src);
    const int d = __shfl(dead, src), pp = __shfl(p, src);
    if (p >= 0) {
      t.anc |= anc;
      t.G += G;
      dead |= d;
      p = pp;
    }
  }
  t.live = !dead;
  return t;
}

// ----------------------------------------------------------------------------
// Whether row b commits something: its last node lies in the tree, and it and
// all its ancestors are present.  One thread, at most 64 steps.
__device__ __forceinline__ bool row_commits(const StateArgs &a, int b) {
  int at = a.last[b];
  if (at < 0 || at >= a.n) return false;
  while (at >= 0) {
    const int p = a.parents[(size_t)b * a.n + at];
    if (p < -1 || p >= at) return false;
    at = p;
  }
  return true;
}

// The accepted path's commit:  S' = e^{G_a} S + sum_{i on the path to a}
// e^{G_a - G_i} k_i u_i^T, with u_i the corrected values of the check: a
// rank-(path length) update, 2 x 64 KB of state traffic per row and head, so
// it is laid out as the step (each thread RPT rows of 4 columns) and the
// path's k and u pass through LDS in batches of 8 nodes, weights folded into
// k.  All sums are fp32.  Of the rows that name a slot the first one that
// commits something is run: an earlier row's path is looked at only where its
// slot is this one (forks of one sequence), so other calls pay for the slots'
// comparison alone.
template <int COLS, typename TI>
__global__ __launch_bounds__(256) void tree_commit_kernel(StateArgs a) {
  constexpr int LPR = COLS / 4, RG = 256 / LPR, RPT = D / RG, NB = 8;
  __shared__ __attribute__((aligned(16))) float kw[NB][D];
  __shared__ float4 us[NB][LPR];
  __shared__ int dup;
  const int tid = threadIdx.x, lane = tid & 63;
  int unit, cpart;
  xcd_unit(blockIdx.x, D / COLS, a.B * a.Hv, unit, cpart);
  const int b = unit / a.Hv, hv = unit % a.Hv, hq = hv / (a.Hv / a.Hqk);
  const int col = cpart * COLS + (tid % LPR) * 4, r0 = (tid / LPR) * RPT;
  const int slot = row_slot(a, b), last = a.last[b];
  if (slot < 0 || last < 0 || last >= a.n) return;   // uniform: nothing accepted
  float *S = a.state + ((size_t)slot * a.Hv + hv) * (D * D) + (size_t)r0 * D + col;
  float4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = ld_state(S + i * D);
  if (tid == 0) dup = 0;
  const Path t = tree_path(a, b, hv, lane);
  const bool live = __shfl((int)t.live, last);
  const double Ga = __shfl(t.G, last);
  unsigned long long path = __shfl(t.anc, last);
  const float w = decay_between(Ga, t.G);   // this lane's node's weight, if it is on the path
  const float ea = decay_between(Ga, 0.);
  __syncthreads();
  if (slot_seen(a, b, slot, tid, 256, [&](int i) { return row_commits(a, i); })) dup = 1;
  __syncthreads();
  if (dup || !live) return;   // uniform
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = mul4(ea, s[i]);
  const int len = __popcll(path);
  for (int n0 = 0; n0 < len; n0 += NB) {
    const int nb = len - n0 < NB ? len - n0 : NB;
    int node[NB];   // the batch's nodes (uniform)
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      node[i] = path ? __ffsll((long long)path) - 1 : 0;
      path &= path - 1;
    }
    if (n0) __syncthreads();
    // k: thread -> node tid / 32, 4 elements; u: NB x LPR pieces
    {
      const int i = tid >> 5;
      int nd = node[0];
#pragma unroll
      for (int j = 1; j < NB; ++j) nd = i == j ? node[j] : nd;
      const float wi = __shfl(w, nd);
      if (i < nb) {
        const float4 x = ld4(static_cast<const TI *>(a.k) + (((size_t)b * a.n + nd) * a.Hqk + hq) * D + (tid & 31) * 4);
        *reinterpret_cast<float4 *>(&kw[i][(tid & 31) * 4]) = mul4(wi, x);
      }
      if (tid < NB * LPR) {
        const int iu = tid / LPR;
        int nu = node[0];
#pragma unroll
        for (int j = 1; j < NB; ++j) nu = iu == j ? node[j] : nu;
        if (iu < nb)
          us[iu][tid % LPR] = ld4(a.u_in + (((size_t)b * a.n + nu) * a.Hv + hv) * D + cpart * COLS + (tid % LPR) * 4);
      }
    }
    __syncthreads();
    for (int i = 0; i < nb; ++i) {
      const float4 u = us[i][tid % LPR];
#pragma unroll
      for (int r = 0; r < RPT; ++r) s[r] = fma4(kw[i][r0 + r], u, s[r]);
    }
  }
  st_state(S, s, a.stream);
}

// ----------------------------------------------------------------------------
// The check of a drafted tree: every node follows the rule from its parent's
// state, and nothing is written to the pool.  With anc the ancestor relation
// and G the sum of the log decays along a node's path, the rule unrolled
// along the paths is the chunk form with "earlier" replaced by "ancestor":
//   S_ri = beta_r e^{G_r - G_i} k_r.k_i   (i a proper ancestor of r)
//   (I + S) U = diag(beta) (V - diag(e^G) K S0)            (linear rule: U = V)
//   O = diag(e^G) Q S0 + ((Q K^T) o e^{G_r - G_i} o [i = r or ancestor]) U
// Nodes are numbered so that ancestors come first: S is strictly lower
// triangular.  One workgroup per (row, value head, 64 NT columns), four waves
// of 16 NT columns each; columns are independent once the n x n matrices are
// formed.  A wave loads its columns of S0 straight from the pool into the
// matrix cores' B layout (column 2 lr + t of its strip in tile t, so that a
// row's load is one whole line for NT = 2), splits each value once into three
// bf16 planes and multiplies them with K and Q rows from LDS.  The solve runs
// over blocks of 16 nodes: the diagonal blocks are inverted by forward
// substitution (one wave each), the rest are fp32 matrix-core products whose
// B operands are the result tiles as they lie in registers (k index 4 g + i
// of step i: a lane's own element).
template <typename TI> struct TreePitch { static constexpr int v = D + 8; };   // elements of K, Q rows in LDS
template <> struct TreePitch<float> { static constexpr int v = D + 4; };

// workgroups per compute unit: two, but for the largest fp32 trees, which take
// more than half of the LDS (86 or 109 of 160 KB)
template <int MT, typename TI> constexpr int tree_wgs() { return MT == 4 && std::is_same<TI, float>::value ? 1 : 2; }

template <int MT, int NT, typename TI, typename TO, bool DELTA>
__global__ __launch_bounds__(256, (tree_wgs<MT, TI>())) void tree_kernel(StateArgs a) {
  constexpr int N = 16 * MT, KP = TreePitch<TI>::v, SP = N + 4, COLS = 64 * NT;
  constexpr int NPI = std::is_same<TI, float>::value ? 3 : 1;
  __shared__ __attribute__((aligned(16))) TI kl[N * KP], ql[N * KP];
  __shared__ __attribute__((aligned(16))) float Sl[DELTA ? N * SP : 4], Pl[N * SP];
  __shared__ __attribute__((aligned(16))) float Tl[DELTA ? MT * 16 * 20 : 4];
  __shared__ double Gl[N];
  __shared__ unsigned long long Al[N];
  __shared__ float bl[N];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, lr = lane & 15, g = lane >> 4;
  int unit, cpart;
  xcd_unit(blockIdx.x, D / COLS, a.B * a.Hv, unit, cpart);
  const int b = unit / a.Hv, hv = unit % a.Hv, hq = hv / (a.Hv / a.Hqk);
  const int slot = row_slot(a, b);
  const int col = cpart * COLS + wave * 16 * NT + lr * NT;   // this lane's first column
  const size_t orow = ((size_t)b * a.n * a.Hv + hv) * D + col;   // + r * Hv * D
  const size_t ostep = (size_t)a.Hv * D;
  TO *o = static_cast<TO *>(a.o) + orow;
  float *u = a.u + orow;
  auto put = [&](int r, const float (&xo)[NT], const float (&xu)[NT]) {
    TO *po = o + r * ostep;
    float *pu = u + r * ostep;
    if constexpr (NT == 2) {
      *reinterpret_cast<float2 *>(pu) = float2{xu[0], xu[1]};
      if constexpr (std::is_same<TO, float>::value) *reinterpret_cast<float2 *>(po) = float2{xo[0], xo[1]};
      else *reinterpret_cast<unsigned *>(po) = pk_bf16(xo[0], xo[1]);
    } else {
      *pu = xu[0];
      *po = from_f32<TO>(xo[0]);
    }
  };
  if (slot < 0) {   // uniform: no state
    const float z[NT] = {};
    for (int r = g; r < a.n; r += 4) put(r, z, z);
    return;
  }
  // Everything that comes from memory is asked for before anything is waited
  // for, without branches (an absent node's row, or one past the last, is
  // dropped when it arrives): K and Q rows, V in the result layout, and the
  // state's columns, row 32 kb + 8 g + j, columns col .. col + NT - 1.
  constexpr int PER = 16 / sizeof(TI), PIECES = D / PER, LD = N * PIECES / 256;   // 16-byte pieces per row
  static_assert(N * PIECES % 256 == 0, "whole pieces per thread");
  const int pr = tid / PIECES, pc = (tid % PIECES) * PER;
  u32x4 xk[LD], xq[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int r = min(pr + i * (256 / PIECES), a.n - 1);
    const size_t at = (((size_t)b * a.n + r) * a.Hqk + hq) * D + pc;
    xk[i] = *reinterpret_cast<const u32x4 *>(static_cast<const TI *>(a.k) + at);
    xq[i] = *reinterpret_cast<const u32x4 *>(static_cast<const TI *>(a.q) + at);
  }
  float s[4][8][NT];
  const float *S = a.state + ((size_t)slot * a.Hv + hv) * (D * D) + col;
#pragma unroll
  for (int kb = 0; kb < 4; ++kb)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float *p = S + (32 * kb + 8 * g + j) * D;
      if constexpr (NT == 2) {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        s[kb][j][0] = x.x;
        s[kb][j][1] = x.y;
      } else {
        s[kb][j][0] = *p;
      }
    }
  typedef TI VPart __attribute__((ext_vector_type(NT)));
  VPart xv[MT][4];
  const TI *vp = static_cast<const TI *>(a.v) + orow;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      xv[m][i] = *reinterpret_cast<const VPart *>(vp + (size_t)min(16 * m + 4 * g + i, a.n - 1) * ostep);
  // the tree (every wave its own copy)
  const Path path = tree_path(a, b, hv, lane);
  const unsigned long long live = __ballot(path.live);
  if (wave == 0 && lane < N) {
    Gl[lane] = path.live ? path.G : 0.;
    Al[lane] = path.live ? path.anc : 0ull;
    bl[lane] = DELTA && path.live ? a.beta[((size_t)b * a.n + lane) * a.Hv + hv] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int r = pr + i * (256 / PIECES);
    const bool on = live >> r & 1;
    const u32x4 z{0, 0, 0, 0};
    *reinterpret_cast<u32x4 *>(kl + r * KP + pc) = on ? xk[i] : z;
    *reinterpret_cast<u32x4 *>(ql + r * KP + pc) = on ? xq[i] : z;
  }
  __syncthreads();
  // 8 consecutive elements of an LDS row as operand planes
  auto frag = [&](const TI *p, bf16x8 (&f)[NPI]) {
    if constexpr (NPI == 1) {
      f[0] = *reinterpret_cast<const bf16x8 *>(p);
    } else {
      float x[8];
      ld8(p, x);
      split8<3>(x, f);
    }
  };
  // K K^T and Q K^T on and below the diagonal of 16 x 16 tiles, weighted and masked
  constexpr int TILES = MT * (MT + 1) / 2;
  for (int t = wave; t < (DELTA ? 2 : 1) * TILES; t += 4) {
    const bool is_s = t >= TILES;   // the S tiles after the P tiles
    int idx = is_s ? t - TILES : t, mr = 0;
    while (idx > mr) idx -= ++mr;   // row-wise lower triangle: (mr, idx)
    const int mi = idx;
    const TI *rows = (is_s ? kl : ql) + (16 * mr + lr) * KP + 8 * g, *cols = kl + (16 * mi + lr) * KP + 8 * g;
    f32x4 c = zero4();
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      bf16x8 fa[NPI], fb[NPI];
      frag(rows + 32 * kb, fa);
      frag(cols + 32 * kb, fb);
      mma_planes<NPI, NPI>(c, fa, fb);
    }
    const int ci = 16 * mi + lr;
    const double Gi = Gl[ci];
    float *dst = is_s ? Sl : Pl;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * mr + 4 * g + i;
      const bool on = (Al[r] >> ci & 1) && !(is_s && r == ci);
      float x = on ? c[i] * decay_between(Gl[r], Gi) : 0.f;
      if (DELTA && is_s) x *= bl[r];
      dst[r * SP + ci] = x;
    }
  }
  if constexpr (DELTA) {
    __syncthreads();
    // wave m inverts I + S_mm: lane c solves for column c, forward substitution
    if (wave < MT) {
      const float *Sm = Sl + 16 * wave * SP + 16 * wave;
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float acc = r == lr ? 1.f : 0.f;
#pragma unroll
        for (int i = 0; i < r; ++i) acc = fmaf(-Sm[r * SP + i], x[i], acc);
        x[r] = acc;
      }
      if (g == 0)
#pragma unroll
        for (int r = 0; r < 16; ++r) Tl[(16 * wave + r) * 20 + lr] = x[r];
    }
  }
  // Q S0 (and K S0) in the wave's columns
  f32x4 qs[MT][NT], ks[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) qs[m][t] = ks[m][t] = zero4();
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) {
    bf16x8 h[NT][3];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = s[kb][j][t];
      split8<3>(x, h[t]);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      bf16x8 f[NPI];
      frag(ql + (16 * m + lr) * KP + 32 * kb + 8 * g, f);
#pragma unroll
      for (int t = 0; t < NT; ++t) mma_planes<NPI, 3>(qs[m][t], f, h[t]);
      if constexpr (DELTA) {
        frag(kl + (16 * m + lr) * KP + 32 * kb + 8 * g, f);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_planes<NPI, 3>(ks[m][t], f, h[t]);
      }
    }
  }
  __syncthreads();
  // c += M[16 mr ..][16 mi ..] X with M in LDS and X a result tile
  auto mul16 = [&](f32x4 (&c)[NT], const float *M, int pitch, const f32x4 (&x)[NT], float sign) {
    const float4 w = *reinterpret_cast<const float4 *>(M + lr * pitch + 4 * g);
    const float av[4] = {sign * w.x, sign * w.y, sign * w.z, sign * w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) c[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[i], x[t][i], c[t], 0, 0, 0);
  };
  f32x4 U[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    f32x4 R[NT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * m + 4 * g + i;
      float x[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float v = (float)xv[m][i][t];
        x[t] = live >> r & 1 ? v : 0.f;
      }
      const float er = decay_between(Gl[r], 0.), be = bl[r];
#pragma unroll
      for (int t = 0; t < NT; ++t) R[t][i] = DELTA ? be * (x[t] - er * ks[m][t][i]) : x[t];
    }
    if constexpr (DELTA) {
#pragma unroll
      for (int mi = 0; mi < m; ++mi) mul16(R, Sl + 16 * m * SP + 16 * mi, SP, U[mi], -1.f);
#pragma unroll
      for (int t = 0; t < NT; ++t) U[m][t] = zero4();
      mul16(U[m], Tl + 16 * m * 20, 20, R, 1.f);
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t) U[m][t] = R[t];
    }
    f32x4 O[NT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float er = decay_between(Gl[16 * m + 4 * g + i], 0.);
#pragma unroll
      for (int t = 0; t < NT; ++t) O[t][i] = er * qs[m][t][i];
    }
#pragma unroll
    for (int mi = 0; mi <= m; ++mi) mul16(O, Pl + 16 * m * SP + 16 * mi, SP, U[mi], 1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * m + 4 * g + i;
      if (r >= a.n) continue;
      const bool on = live >> r & 1;
      float xo[NT], xu[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        xo[t] = on ? O[t][i] : 0.f;
        xu[t] = on ? U[m][t][i] : 0.f;
      }
      put(r, xo, xu);
    }
  }
}

}  // namespace gdn
