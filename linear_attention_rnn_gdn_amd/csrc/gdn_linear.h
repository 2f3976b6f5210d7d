// gdn_linear.h -- linear attention with a decay per head, in chunks.
//
// The rule:  S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t.  With F the
// running sum of the log decays within a chunk of C tokens, a chunk is
//   out = ((A B^T) o [i <= r] e^{F_r - F_i}) C  +  diag(e^F) A H
//   H'  = e^{F_end} H + B^T diag(e^{F_end - F}) C
// with (A, B, C, H) = (q, k, v, S).  The gradients are the same expression:
//   dq: (dO, v, k, S^T) in token order;
//   dv: (k, q, dO, dS) and dk: (v, dO, q, dS^T) from the last token to the
//   first, F then the sum over the tokens already passed without the row's
//   own (the decay between tokens r and i > r is e^{g_{r+1} + .. + g_i}), so
// one kernel serves all four, its operands and direction given by a role.
//
// A sequence is cut into segments; each (segment, value head) is one walk
// over its chunks with the 128 x 128 state in matrix-core result registers.
// With several segments a first launch folds each segment's own contribution
// to the state, a second carries the states from segment to segment (a scalar
// decay each, so no matrix products), and the walks start from those.
#pragma once
#include <type_traits>

#include "gdn_common.h"

namespace gdn {

typedef short s16x4 __attribute__((ext_vector_type(4)));

struct LinRole {
  const void *a, *b, *c;      // operands [tokens, heads, 128]
  int ga, gb, gc;             // value heads per operand head
  int rev;                    // 1: from the last token to the first
  int trans;                  // 1: the state is the transpose of the stored one
  const float *init;          // state entering the sequence [n_seq, H_v, D, D], null = zero
  const float *seg;           // states entering the other segments [segments, H_v, D, D]
  float *fin;                 // state leaving the sequence, null = not wanted (fold: the segments' contributions)
  float *dec;                 // fold: the segments' decays [segments, H_v]
  void *out;                  // [tokens, H_v, D]
  int out_f32;                // 1: out is fp32 whatever TO
  const void *x;              // with dot: rows to multiply the outputs with, [tokens, heads, 128] (heads as `gx`)
  int gx;
  float *dot;                 // [tokens, H_v] <out_r, x_r>, null = not wanted
  const float *xs, *xs_last;  // with cross: states to multiply each segment's end state with (transposed as `trans`):
  float *cross;               // [segments, H_v], of the segments but the last, and of the last (null = zero)
};

struct LinArgs {
  int Hqk, Hv;
  int T;                      // tokens per sequence (padded batch), or in all (packed)
  int seg_len, J;             // tokens per segment, segments per sequence (padded batch)
  int nseg;                   // segments in all (packed: room for them)
  const int4 *tab;            // packed: (first token, tokens, sequence, segment of it | last << 30) per segment
  const float *g;             // log decays [tokens, H_v] or [H_v]
  int g_fixed;
  int roles;
  LinRole role[3];
};

struct Seg {
  int start, rows, seq;
  bool first, last;
};
// the segment s, or rows = -1 past the last
__device__ __forceinline__ Seg segment(const LinArgs &a, int s) {
  Seg x;
  if (a.tab) {
    const int4 t = a.tab[s];
    x.start = t.x; x.rows = t.y; x.seq = t.z;
    x.first = (t.w & 0x3fffffff) == 0;
    x.last = t.w >> 30 & 1;
  } else {
    x.seq = s / a.J;
    const int j = s % a.J, at = j * a.seg_len;
    x.start = x.seq * a.T + at;
    x.rows = min(a.seg_len, a.T - at);
    x.first = j == 0;
    x.last = j == a.J - 1;
  }
  return x;
}

// Packed sequences' segment table: sequence s covers tokens [cu[s], cu[s+1])
// (offsets clamped into [0, T], a sequence ending no earlier than it starts)
// and has ceil(len / L) segments, an empty one a single segment of no tokens,
// T / L + nseq at most.  One workgroup of 256 threads; thread t takes a
// contiguous block of sequences.  Writes the segments' entries (those past
// the last get rows = -1) and, per sequence, (first segment, segments).
// Entries that would pass nmax (only for offsets that are no partition of
// [0, T]) are dropped, so no access leaves the tables.
__global__ __launch_bounds__(256) void linear_table_kernel(const int *cu, int nseq, int T, int L, int nmax, int4 *tab,
                                                           int2 *seqs) {
  __shared__ int part[257];
  const int t = threadIdx.x;
  const int per = (nseq - 1) / 256 + 1;
  const int s0 = (int)min((int64_t)nseq, (int64_t)t * per), s1 = (int)min((int64_t)nseq, (int64_t)t * per + per);
  auto span = [&](int s, int &st, int &n) {
    st = cu[s] < 0 ? 0 : cu[s] > T ? T : cu[s];
    const int en = cu[s + 1] < st ? st : cu[s + 1] > T ? T : cu[s + 1];
    n = en - st;
    return n ? (n - 1) / L + 1 : 1;
  };
  int mine = 0, st, n;
  for (int s = s0; s < s1; ++s) mine = (int)min((int64_t)nmax, (int64_t)mine + span(s, st, n));
  part[t] = mine;
  __syncthreads();
  if (t == 0) {
    int run = 0;
    for (int i = 0; i < 256; ++i) {
      const int x = part[i];
      part[i] = run;
      run = (int)min((int64_t)nmax, (int64_t)run + x);
    }
    part[256] = run;
  }
  __syncthreads();
  int c = part[t];
  for (int s = s0; s < s1; ++s) {
    const int ns = span(s, st, n), first = c;
    for (int j = 0; j < ns && c < nmax; ++j, ++c)
      tab[c] = int4{st + j * L, min(L, n - j * L), s, j | (j == ns - 1 ? 1 << 30 : 0)};
    seqs[s] = int2{first, c - first};
  }
  for (int i = part[256] + t; i < nmax; i += 256) tab[i] = int4{0, -1, 0, 0};
}

// Transposition of a 4 x 4 block over the lanes 4 q .. 4 q + 3 and a tile's
// four registers: lane s, register i  <->  lane i, register s.
__device__ __forceinline__ float quad_swap(float x, bool two) {
  const int i = __builtin_bit_cast(int, x);
  const int y = two ? __builtin_amdgcn_mov_dpp(i, 0x4e, 0xf, 0xf, true) : __builtin_amdgcn_mov_dpp(i, 0xb1, 0xf, 0xf, true);
  return __builtin_bit_cast(float, y);
}
__device__ __forceinline__ f32x4 quad_transpose(f32x4 v, int lane) {
  const bool o1 = lane & 1, o2 = lane & 2;
#pragma unroll
  for (int p = 0; p < 4; p += 2) {
    const float y = quad_swap(o1 ? v[p] : v[p + 1], false);
    if (o1) v[p] = y;
    else v[p + 1] = y;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const float y = quad_swap(o2 ? v[p] : v[p + 2], true);
    if (o2) v[p] = y;
    else v[p + 2] = y;
  }
  return v;
}

// How a walk is laid out for inputs of type TI: C tokens per chunk and planes
// per input value.  fp32 inputs: three bf16 planes hold every bit, so all
// products run on the bf16 matrix cores (6 of their passes against the 16
// times slower fp32 instruction), with half the chunk to fit the LDS.
template <typename TI> struct LinTile { static constexpr int C = 64, NPI = 1; };
template <> struct LinTile<float> { static constexpr int C = 32, NPI = 3; };

// Four waves; wave w holds columns 16 NTW w + .. of the state, all 128 rows:
// result tile (m, t) has rows 16 m + 4 g + i and the columns
//   dv(lr, t) = 4 NTW (lr / 4) + 4 t + lr % 4,
// so that the wave's NTW tiles give a lane 4 NTW consecutive columns of a
// transposed output tile, and four lanes the four elements of one transposing
// LDS read.
//
// Per chunk: every wave multiplies its state (split into NPO planes) with all
// rows of A (outputs transposed: state as the left operand, straight from its
// result registers); wave w forms the 16-row strip w of the masked scores and
// leaves them in LDS as NPO planes; after a barrier all waves add scores x C
// for their columns, write their outputs, and add B^T (weighted C) to the
// state (weighted C in three planes, so that the state keeps fp32 precision).
// The chunk's operands sit in LDS in row-major order; products over tokens
// read them with the transposing LDS read.  The next chunk's operands are
// loaded into registers while this one is computed.
template <int KIND_FOLD, int NTW, int NPO, typename TI, typename TO>
__global__ __launch_bounds__(256, 2) void linear_kernel(LinArgs p) {
  constexpr bool FOLD = KIND_FOLD;
  using L = LinTile<TI>;
  constexpr int C = L::C, NPI = L::NPI, NR = C / 16, KB = C / 32;
  constexpr int PA = D + 8, PB = D + 16, PP = C + 8;    // row pitches in LDS (elements)
  constexpr int COLS = 64 * NTW;                        // state columns per workgroup
  constexpr int PER = 16 / sizeof(TI), PIECES = D / PER, ROWS = 256 / PIECES, LD = C / ROWS;   // staging loads
  __shared__ __attribute__((aligned(16))) __bf16 al[FOLD ? 1 : NPI][FOLD ? 8 : C * PA];
  __shared__ __attribute__((aligned(16))) __bf16 bl[NPI][C * PB], cl[NPI][C * PB];
  __shared__ __attribute__((aligned(16))) __bf16 pl[FOLD ? 1 : NPO][FOLD ? 8 : C * PP];
  __shared__ double Fl[2][C];
  __shared__ __attribute__((aligned(16))) float fs[2][C], te[2][C];   // e^F, e^{F_end - F}
  __shared__ float fe[2];                                             // e^{F_end}
  __shared__ float dots[FOLD ? 1 : 4][FOLD ? 1 : C];
  __shared__ float crs[4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, lr = lane & 15, g = lane >> 4;

  int unit, part;
  const int R = p.Hv / p.Hqk;
  xcd_unit(blockIdx.x, R * p.roles * (D / COLS), p.nseg * p.Hqk, unit, part);
  const int sidx = unit / p.Hqk, hv = (unit % p.Hqk) * R + part / (p.roles * (D / COLS));
  const int rn = part / (D / COLS) % p.roles;
  // the role's fields, selected one by one: an indexed copy would sit in scratch memory
  LinRole ro;
#define GDN_PICK(f) ro.f = rn == 0 ? p.role[0].f : rn == 1 ? p.role[1].f : p.role[2].f
  GDN_PICK(a); GDN_PICK(b); GDN_PICK(c); GDN_PICK(ga); GDN_PICK(gb); GDN_PICK(gc); GDN_PICK(rev); GDN_PICK(trans);
  GDN_PICK(init); GDN_PICK(seg); GDN_PICK(fin); GDN_PICK(dec); GDN_PICK(out); GDN_PICK(out_f32);
  GDN_PICK(x); GDN_PICK(gx); GDN_PICK(dot); GDN_PICK(xs); GDN_PICK(xs_last); GDN_PICK(cross);
#undef GDN_PICK
  const int col0 = (part % (D / COLS)) * COLS + 16 * NTW * wave;   // this wave's first column
  const Seg sg = segment(p, sidx);
  if (sg.rows < 0) return;
  const bool enters = ro.rev ? sg.last : sg.first, leaves = ro.rev ? sg.first : sg.last;
  if (FOLD && leaves) return;   // its contribution goes nowhere
  const int nch = (sg.rows + C - 1) / C;
  const size_t sth = ((size_t)sidx * p.Hv + hv) * (D * D), sqh = ((size_t)sg.seq * p.Hv + hv) * (D * D);

  f32x4 H[8][NTW];
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int t = 0; t < NTW; ++t) H[m][t] = zero4();
  // this lane's place in a stored state, from a lane index the compiler cannot
  // see through: else it keeps the addresses alive from the first use to the last
  struct Place { int row, col; };
  auto state_place = [&]() __attribute__((always_inline)) -> Place {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int q = l & 15;
    const int along = 4 * (l >> 4), c = col0 + 4 * NTW * (q >> 2);
    return ro.trans ? Place{along, c + (q & 3)} : Place{along + (q & 3), c};
  };
  // state element (row 16 m + 4 g + i, column dv): read along whichever of the two is contiguous
  auto load_state = [&](const float *S, auto &&put) __attribute__((always_inline)) {
    const Place pl = state_place();
    const unsigned at = ro.trans ? pl.col * D + pl.row : pl.row * D + pl.col;
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int t = 0; t < NTW; ++t) {
        const unsigned d = ro.trans ? 4 * t * D + 16 * m : 16 * m * D + 4 * t;
        f32x4 x = *reinterpret_cast<const f32x4 *>(S + (at + d));
        if (!ro.trans) x = quad_transpose(x, lane);
        put(m, t, x);
      }
  };
  if (!FOLD) {
    const float *S = enters ? (ro.init ? ro.init + sqh : nullptr) : ro.seg + sth;
    if (S) load_state(S, [&](int m, int t, const f32x4 &x) { H[m][t] = x; });
  }

  // token of row r of chunk n, in the order of the walk; staging loads
  auto token = [&](int at) __attribute__((always_inline)) { return ro.rev ? sg.start + sg.rows - 1 - at : sg.start + at; };
  const int srow = tid / PIECES, scol = (tid % PIECES) * PER;
  // bytes between tokens; a chunk's first token in memory is uniform, so that
  // a lane's address is a scalar base and a 32-bit offset
  const int na = (p.Hv / ro.ga) * D * (int)sizeof(TI), nb = (p.Hv / ro.gb) * D * (int)sizeof(TI),
            nc = (p.Hv / ro.gc) * D * (int)sizeof(TI);
  const char *pa = static_cast<const char *>(ro.a) + (hv / ro.ga) * D * sizeof(TI);
  const char *pb = static_cast<const char *>(ro.b) + (hv / ro.gb) * D * sizeof(TI);
  const char *pc = static_cast<const char *>(ro.c) + (hv / ro.gc) * D * sizeof(TI);
  auto chunk_base = [&](int n) __attribute__((always_inline)) { return token(ro.rev ? min(n * C + C, sg.rows) - 1 : n * C); };
  u32x4 xa[FOLD ? 1 : LD], xb[LD], xc[LD];
  // (past the segment's end its last row is read, without a branch, and dropped on the way into LDS)
  auto load_chunk = [&](int n) __attribute__((always_inline)) {
    const int lo = chunk_base(n);
    const char *qa = pa + (size_t)lo * na, *qb = pb + (size_t)lo * nb, *qc = pc + (size_t)lo * nc;
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const unsigned d = token(min(n * C + srow + i * ROWS, sg.rows - 1)) - lo, sb = scol * sizeof(TI);
      if constexpr (!FOLD) xa[i] = *reinterpret_cast<const u32x4 *>(qa + (d * na + sb));
      xb[i] = *reinterpret_cast<const u32x4 *>(qb + (d * nb + sb));
      xc[i] = *reinterpret_cast<const u32x4 *>(qc + (d * nc + sb));
    }
  };
  auto put_piece = [&](auto &dst, int pitch, int row, const u32x4 &x) __attribute__((always_inline)) {
    if constexpr (NPI == 1) {
      *reinterpret_cast<u32x4 *>(&dst[0][row * pitch + scol]) = x;
    } else {
      unsigned w0[3], w1[3];
      const f32x4 y = __builtin_bit_cast(f32x4, x);
      split_pair<3>(y[0], y[1], w0);
      split_pair<3>(y[2], y[3], w1);
#pragma unroll
      for (int k = 0; k < NPI; ++k) *reinterpret_cast<u32x2 *>(&dst[k][row * pitch + scol]) = u32x2{w0[k], w1[k]};
    }
  };
  auto store_chunk = [&](int n) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int row = srow + i * ROWS;
      const bool on = n * C + row < sg.rows;
      const u32x4 z{0, 0, 0, 0};
      if constexpr (!FOLD) put_piece(al, PA, row, on ? xa[i] : z);
      put_piece(bl, PB, row, on ? xb[i] : z);
      put_piece(cl, PB, row, on ? xc[i] : z);
    }
  };
  // decays of chunk n: this lane's token's log decay, and (wave 0) the sums
  auto load_decay = [&](int n) __attribute__((always_inline)) -> float {
    const int at = n * C + lane;
    if (lane >= C || at >= sg.rows) return 0.f;
    return p.g[p.g_fixed ? hv : (size_t)token(at) * p.Hv + hv];
  };
  double total = 0.;
  auto put_decay = [&](int buf, float gv) __attribute__((always_inline)) {
    const double own = log2_decay(gv);
    double F = own;
#pragma unroll
    for (int d = 1; d < C; d <<= 1) {
      const double y = __shfl_up(F, d);
      if (lane >= d) F += y;
    }
    const double end = __shfl(F, C - 1);
    total += end;
    if (ro.rev) F -= own;
    if (lane < C) {
      Fl[buf][lane] = F;
      fs[buf][lane] = decay_between(F, 0.);
      te[buf][lane] = decay_between(end, F);
    }
    if (lane == 0) fe[buf] = decay_between(end, 0.);
  };

  // LDS addresses as such (not generic pointers), so that a read's constant
  // part goes into its offset field and all reads share one address register
  typedef const __attribute__((address_space(3))) __bf16 *LdsB;
  typedef __attribute__((address_space(3))) s16x4 *LdsT;
  const LdsB tr_b = (LdsB)&bl[0][0] + (8 * g + (lr >> 2)) * PB + 4 * (lr & 3);
  const LdsB tr_c = (LdsB)&cl[0][0] + (8 * g + (lr >> 2)) * PB + col0 + 4 * NTW * (lr & 3);
  const LdsB row_a = (LdsB)&al[0][0] + lr * PA + 4 * g, row_b = (LdsB)&bl[0][0] + lr * PB + 4 * g;
  const LdsB row_p = (LdsB)&pl[0][0] + lr * PP + 8 * g;
  // 8 tokens x one column of an operand, transposed: tokens 32 kb + 8 g .., column `col` + the lane's
  auto read_tr = [&](LdsB base, int k, int kb, int col) __attribute__((always_inline)) -> bf16x8 {
    const LdsB q = base + k * (C * PB) + 32 * kb * PB + col;
    union { s16x4 h[2]; bf16x8 v; } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsT)q);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsT)(q + 4 * PB));
    return u.v;
  };
  // row lr of strip r, k order of two stacked result tiles: 32 kb + 4 g + {0..3}, 32 kb + 16 + 4 g + {0..3}
  auto read_row = [&](LdsB base, int plane, int pitch, int r, int kb) __attribute__((always_inline)) -> bf16x8 {
    typedef const __attribute__((address_space(3))) u32x2 *P2;
    const LdsB q = base + plane + 16 * r * pitch + 32 * kb;
    union { u32x2 h[2]; bf16x8 v; } u;
    u.h[0] = *(P2)q;
    u.h[1] = *(P2)(q + 16);
    return u.v;
  };

  if (nch > 0) {
    load_chunk(0);
    if (wave == 0) put_decay(0, load_decay(0));
    // scores of the 16 x 16 tiles above the diagonal that a 32-token block of C reads: zero, once
    if constexpr (!FOLD) {
      for (int i = tid; i < NPO * (NR / 2) * 16 * 16; i += 256) {
        const int k = i / (NR / 2 * 256), e = i % (NR / 2 * 256), q = e / 256, r = e / 16 % 16, c = e % 16;
        pl[k][(32 * q + r) * PP + 32 * q + 16 + c] = (__bf16)0.f;
      }
    }
    store_chunk(0);
  }
  float gnext = nch > 1 && wave == 0 ? load_decay(1) : 0.f;
  __syncthreads();

  for (int n = 0; n < nch; ++n) {
    const int buf = n & 1;
    if (n + 1 < nch) load_chunk(n + 1);
    f32x4 O[FOLD ? 1 : NTW][FOLD ? 1 : NR];
    if constexpr (!FOLD) {
      // masked scores, strip `wave` of rows (fewer strips than waves at C = 32)
      if (wave < NR) {
        bf16x8 fa[4][NPI];
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
          for (int k = 0; k < NPI; ++k) fa[kb][k] = read_row(row_a, k * (C * PA), PA, wave, kb);
        const double Fr = Fl[buf][16 * wave + lr];
        for (int mi = 0; mi <= wave; ++mi) {
          f32x4 s = zero4();
#pragma unroll
          for (int kb = 0; kb < 4; ++kb) {
            bf16x8 fb[NPI];
#pragma unroll
            for (int k = 0; k < NPI; ++k) fb[k] = read_row(row_b, k * (C * PB), PB, mi, kb);
            mma_planes<NPI, NPI>(s, fb, fa[kb]);
          }
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int ci = 16 * mi + 4 * g + i;
            x[i] = ci <= 16 * wave + lr ? s[i] * decay_between(Fr, Fl[buf][ci]) : 0.f;
          }
          unsigned w0[NPO], w1[NPO];
          split_pair<NPO>(x[0], x[1], w0);
          split_pair<NPO>(x[2], x[3], w1);
#pragma unroll
          for (int k = 0; k < NPO; ++k)
            *reinterpret_cast<u32x2 *>(&pl[k][(16 * wave + lr) * PP + 16 * mi + 4 * g]) = u32x2{w0[k], w1[k]};
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      // state x A, per token scaled by e^F
#pragma unroll
      for (int t = 0; t < NTW; ++t)
#pragma unroll
        for (int r = 0; r < NR; ++r) O[t][r] = zero4();
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        bf16x8 h[NTW][NPO];
#pragma unroll
        for (int t = 0; t < NTW; ++t) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = H[2 * kb + j / 4][t][j % 4];
          split8<NPO>(x, h[t]);
        }
        bf16x8 f[2][NPI];
#pragma unroll
        for (int k = 0; k < NPI; ++k) f[0][k] = read_row(row_a, k * (C * PA), PA, 0, kb);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if (r + 1 < NR)
#pragma unroll
            for (int k = 0; k < NPI; ++k) f[(r + 1) & 1][k] = read_row(row_a, k * (C * PA), PA, r + 1, kb);
#pragma unroll
          for (int t = 0; t < NTW; ++t) mma_planes<NPO, NPI>(O[t][r], h[t], f[r & 1]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float e = fs[buf][16 * r + lr];
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) O[t][r][i] *= e;
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // (phases kept apart: operands of one only are live)
    // the next chunk's decays, while the scores settle
    if (wave == 0 && n + 1 < nch) {
      put_decay(buf ^ 1, gnext);
      if (n + 2 < nch) gnext = load_decay(n + 2);
    }
    if constexpr (!FOLD) lds_barrier();
    if constexpr (!FOLD) {
      // scores x C
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        bf16x8 cf[NTW][NPI];
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
          for (int k = 0; k < NPI; ++k) cf[t][k] = read_tr(tr_c, k, kb, 4 * t);
#pragma unroll
        for (int r = 2 * kb; r < NR; ++r) {
          bf16x8 ps[NPO];
#pragma unroll
          for (int k = 0; k < NPO; ++k)
            ps[k] = *(const __attribute__((address_space(3))) bf16x8 *)(row_p + k * (C * PP) + 16 * r * PP + 32 * kb);
#pragma unroll
          for (int t = 0; t < NTW; ++t) mma_planes<NPI, NPO>(O[t][r], cf[t], ps);
        }
      }
      // outputs: lane -> token 16 r + lr, columns 4 NTW g .. of the wave's
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int at = n * C + 16 * r + lr;
        const bool on = at < sg.rows;
        const size_t tk = on ? token(at) : 0;
        const int oc = col0 + 4 * NTW * g;
        if (on) {
          const size_t o = (tk * p.Hv + hv) * D + oc;
          if (std::is_same<TO, float>::value || ro.out_f32) {
#pragma unroll
            for (int t = 0; t < NTW; ++t) *reinterpret_cast<f32x4 *>(static_cast<float *>(ro.out) + o + 4 * t) = O[t][r];
          } else {
            unsigned u[2 * NTW];
#pragma unroll
            for (int t = 0; t < NTW; ++t) {
              u[2 * t] = pk_bf16(O[t][r][0], O[t][r][1]);
              u[2 * t + 1] = pk_bf16(O[t][r][2], O[t][r][3]);
            }
            if constexpr (NTW == 2) *reinterpret_cast<uint4 *>(static_cast<__bf16 *>(ro.out) + o) = uint4{u[0], u[1], u[2], u[3]};
            else *reinterpret_cast<uint2 *>(static_cast<__bf16 *>(ro.out) + o) = uint2{u[0], u[1]};
          }
        }
        if (ro.dot) {   // uniform
          float d = 0.f;
          if (on) {
            const TI *x = static_cast<const TI *>(ro.x) + (tk * (p.Hv / ro.gx) + hv / ro.gx) * D + oc;
#pragma unroll
            for (int t = 0; t < NTW; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) d = fmaf(O[t][r][i], to_f32(x[4 * t + i]), d);
          }
          d += __shfl_xor(d, 16);
          d += __shfl_xor(d, 32);
          if (g == 0) dots[wave][16 * r + lr] = d;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // the state
    const float e_end = fe[buf];
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int t = 0; t < NTW; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) H[m][t][i] *= e_end;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      bf16x8 w[NTW][3];   // C's tokens 32 kb .. of the wave's columns, weighted
      float wt[8];
      ld8(&te[buf][32 * kb + 8 * g], wt);
#pragma unroll
      for (int t = 0; t < NTW; ++t) {
        bf16x8 cf[NPI];
#pragma unroll
        for (int k = 0; k < NPI; ++k) cf[k] = read_tr(tr_c, k, kb, 4 * t);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = (float)cf[0][j];
#pragma unroll
          for (int k = 1; k < NPI; ++k) v += (float)cf[k][j];
          x[j] = v * wt[j];
        }
        split8<3>(x, w[t]);
      }
      // (operands read one tile ahead; scheduling fences keep the compiler from reading all of them at once)
      bf16x8 f[2][NPI];
#pragma unroll
      for (int k = 0; k < NPI; ++k) f[0][k] = read_tr(tr_b, k, kb, 0);
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        if (m + 1 < 8)
#pragma unroll
          for (int k = 0; k < NPI; ++k) f[(m + 1) & 1][k] = read_tr(tr_b, k, kb, 16 * (m + 1));
#pragma unroll
        for (int t = 0; t < NTW; ++t) mma_planes<NPI, 3>(H[m][t], f[m & 1], w[t]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    lds_barrier();
    if constexpr (!FOLD) {
      if (ro.dot && tid < C && n * C + tid < sg.rows)
        ro.dot[(size_t)token(n * C + tid) * p.Hv + hv] = (dots[0][tid] + dots[1][tid]) + (dots[2][tid] + dots[3][tid]);
    }
    if (n + 1 < nch) store_chunk(n + 1);
    lds_barrier();
  }

  auto store_state = [&](float *S) __attribute__((always_inline)) {
    const Place pl = state_place();
    const unsigned at = ro.trans ? pl.col * D + pl.row : pl.row * D + pl.col;
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int t = 0; t < NTW; ++t) {
        const unsigned d = ro.trans ? 4 * t * D + 16 * m : 16 * m * D + 4 * t;
        *reinterpret_cast<f32x4 *>(S + (at + d)) = ro.trans ? H[m][t] : quad_transpose(H[m][t], lane);
      }
  };
  if constexpr (FOLD) {
    store_state(ro.fin + sth);
    if (tid == 0 && col0 == 0) ro.dec[(size_t)sidx * p.Hv + hv] = decay_between(total, 0.);
  } else {
    if (ro.fin && leaves) store_state(ro.fin + sqh);
    if (ro.cross) {   // uniform
      const float *S = sg.last ? (ro.xs_last ? ro.xs_last + sqh : nullptr) : ro.xs + sth;
      float d = 0.f;
      if (S)
        load_state(S, [&](int m, int t, const f32x4 &x) {
#pragma unroll
          for (int i = 0; i < 4; ++i) d = fmaf(H[m][t][i], x[i], d);
        });
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) d += __shfl_xor(d, m);
      if (lane == 0) crs[wave] = d;
      __syncthreads();
      if (tid == 0) ro.cross[(size_t)sidx * p.Hv + hv] = (crs[0] + crs[1]) + (crs[2] + crs[3]);
    }
  }
}

// The states entering the segments, from the segments' own contributions B_j
// and decays:  x_0 = init,  x_{j+1} = decay_j x_j + B_j  in the order of the
// walk (x_0 is not written: the walk of that segment reads init).  One thread
// per 4 elements of a state; 8 segments' contributions are loaded at a time,
// so that a sequence of few segments costs one memory latency.
struct ScanRole {
  const float *add, *dec, *init;
  float *x;
  int rev;
};
struct ScanArgs {
  int Hv, J, roles;
  const int2 *seqs;           // packed: (first segment, segments) per sequence
  ScanRole role[2];
};
__global__ __launch_bounds__(256) void linear_scan_kernel(ScanArgs a) {
  constexpr int PARTS = D * D / 1024, NB = 8;
  const int part = blockIdx.x % PARTS;
  int u = blockIdx.x / PARTS;
  ScanRole ro = a.role[0];
  if (u % a.roles) ro = a.role[1];
  u /= a.roles;
  const int hv = u % a.Hv, seq = u / a.Hv;
  const int first = a.seqs ? a.seqs[seq].x : seq * a.J, cnt = a.seqs ? a.seqs[seq].y : a.J;
  const size_t e = (size_t)part * 1024 + threadIdx.x * 4;
  const float *__restrict__ add = ro.add + e;
  float *__restrict__ out = ro.x + e;
  auto at = [&](int j) { return (size_t)(first + (ro.rev ? cnt - 1 - j : j)) * a.Hv + hv; };
  f32x4 x = ro.init ? *reinterpret_cast<const f32x4 *>(ro.init + ((size_t)seq * a.Hv + hv) * (D * D) + e) : zero4();
  for (int j0 = 0; j0 + 1 < cnt; j0 += NB) {
    f32x4 B[NB];
    float f[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const size_t s = at(min(j0 + i, cnt - 2));
      B[i] = *reinterpret_cast<const f32x4 *>(add + s * (D * D));
      f[i] = ro.dec[s];
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (j0 + i + 1 < cnt) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = fmaf(f[i], x[k], B[i][k]);
        *reinterpret_cast<f32x4 *>(out + at(j0 + i + 1) * (D * D)) = x;
      }
  }
}

// ----------------------------------------------------------------------------
// The decays' gradient.  dg_t sums, over every pair of tokens that t lies
// between, the pair's share of the loss: with d_s = <q_s, dq_s> - <k_s, dk_s>
// (unrounded gradients of one value head), dg_t = sum of d_s over s >= t in
// the segment + <S, dS> of the states at the segment's end.  Cutting the sum
// at segments keeps its rounding from growing with the sequence.  One wave
// per (segment, value head), 64 tokens at a time from the last; sums in fp64.
struct DgArgs {
  LinArgs p;
  const float *qd, *kd, *cross;
  float *dg;                  // [tokens, H_v], or null:
  double *part;               // [segments, H_v] sums over the segment's tokens (fixed decays)
};
__global__ __launch_bounds__(256) void linear_dg_kernel(DgArgs a) {
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (unit >= (int64_t)a.p.nseg * a.p.Hv) return;
  const int hv = (int)(unit % a.p.Hv);
  const Seg sg = segment(a.p, (int)(unit / a.p.Hv));
  double carry = a.cross[unit], sum = 0.;
  for (int n = (sg.rows - 1) / 64; sg.rows > 0 && n >= 0; --n) {
    const int r = n * 64 + 63 - lane;   // lane 0: the last token
    const size_t at = ((size_t)sg.start + r) * a.p.Hv + hv;
    double d = r < sg.rows ? (double)a.qd[at] - (double)a.kd[at] : 0.;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double y = __shfl_up(d, m);
      if (lane >= m) d += y;
    }
    d += carry;
    carry = __shfl(d, 63);
    if (r < sg.rows) {
      sum += d;
      if (a.dg) a.dg[at] = (float)d;
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m);
  if (lane == 0) a.part[unit] = sum;
}
// fixed decays: the sum over all segments, one workgroup per value head
__global__ __launch_bounds__(256) void linear_dg_fixed_kernel(const double *part, float *dg, int nseg, int Hv) {
  __shared__ double w[4];
  const int hv = blockIdx.x;
  double s = 0.;
  for (int i = threadIdx.x; i < nseg; i += 256) s += part[(size_t)i * Hv + hv];
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) dg[hv] = (float)((w[0] + w[1]) + (w[2] + w[3]));
}

// Gradients of a query/key head: the sum over the value heads that read it,
// in fp32, rounded once.  One thread per 8 elements.
struct HeadSumArgs {
  const float *src[2];        // [tokens, H_qk, R, D]
  void *dst[2];               // [tokens, H_qk, D]
  size_t n;                   // tokens * H_qk * D / 8
  int R;
};
template <typename TI>
__global__ __launch_bounds__(256) void linear_head_sum_kernel(HeadSumArgs a) {
  constexpr int V = D / 8;
  const float *src = a.src[blockIdx.y];
  TI *dst = static_cast<TI *>(a.dst[blockIdx.y]);
  for (size_t i = blockIdx.x * (size_t)256 + threadIdx.x; i < a.n; i += (size_t)gridDim.x * 256) {
    const float *s = src + (i / V) * a.R * D + (i % V) * 8;
    f32x4 x = zero4(), y = zero4();
    for (int r = 0; r < a.R; ++r) {
      x += *reinterpret_cast<const f32x4 *>(s + (size_t)r * D);
      y += *reinterpret_cast<const f32x4 *>(s + (size_t)r * D + 4);
    }
    if constexpr (std::is_same<TI, float>::value) {
      *reinterpret_cast<f32x4 *>(dst + i * 8) = x;
      *reinterpret_cast<f32x4 *>(dst + i * 8 + 4) = y;
    } else {
      *reinterpret_cast<uint4 *>(dst + i * 8) =
          uint4{pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(y[0], y[1]), pk_bf16(y[2], y[3])};
    }
  }
}

}  // namespace gdn
