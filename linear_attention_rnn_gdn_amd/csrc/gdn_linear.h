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
  const int *order;           // packed: the order in which segments are started
  int alone;                  // packed: one workgroup per compute unit (for the launch)
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
// [0, T]) are dropped, so no access leaves the tables.  `order`: the segments
// by their tokens, longest first (in 32 classes; within one in any order), in
// which the walks are started: a long walk begun last would run alone.
__global__ __launch_bounds__(256) void linear_table_kernel(const int *cu, int nseq, int T, int L, int nmax, int4 *tab,
                                                           int2 *seqs, int *order) {
  constexpr int CLASSES = 32;
  __shared__ int place[CLASSES + 1];
  __shared__ long long waves[4];
  const int t = threadIdx.x, lane = t & 63;
  const int per = (nseq - 1) / 256 + 1;
  const int s0 = (int)min((int64_t)nseq, (int64_t)t * per), s1 = (int)min((int64_t)nseq, (int64_t)t * per + per);
  auto span = [&](int s, int &st, int &n) {
    st = cu[s] < 0 ? 0 : cu[s] > T ? T : cu[s];
    const int en = cu[s + 1] < st ? st : cu[s + 1] > T ? T : cu[s + 1];
    n = en - st;
    return n ? (n - 1) / L + 1 : 1;
  };
  long long mine = 0;   // (64 bits: offsets that are no partition may add up to more than 32 hold)
  int st, n;
  for (int s = s0; s < s1; ++s) mine += span(s, st, n);
  long long upto = mine;   // within the wave, then over the waves
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long long y = __shfl_up(upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 63) waves[t >> 6] = upto;
  __syncthreads();
  long long before = upto - mine, total = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < t >> 6) before += waves[w];
    total += waves[w];
  }
  int c = (int)min(before, (long long)nmax);
  for (int s = s0; s < s1; ++s) {
    const int ns = span(s, st, n), first = c;
    for (int j = 0; j < ns && c < nmax; ++j, ++c)
      tab[c] = int4{st + j * L, min(L, n - j * L), s, j | (j == ns - 1 ? 1 << 30 : 0)};
    seqs[s] = int2{first, c - first};
  }
  for (int64_t i = total + t; i < nmax; i += 256) tab[i] = int4{0, -1, 0, 0};
  // counting sort; class CLASSES: the entries past the last
  if (t <= CLASSES) place[t] = 0;
  __syncthreads();   // (the tables' entries too)
  auto cls = [&](int i) { return i < total ? CLASSES - 1 - (int)min((int64_t)tab[i].y * CLASSES / L, (int64_t)CLASSES - 1) : CLASSES; };
  for (int i = t; i < nmax; i += 256) atomicAdd(&place[cls(i)], 1);
  __syncthreads();
  if (t < 64) {
    int v = t <= CLASSES ? place[t] : 0, w = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(w, d);
      if (lane >= d) w += y;
    }
    if (t <= CLASSES) place[t] = w - v;
  }
  __syncthreads();
  for (int i = t; i < nmax; i += 256) order[atomicAdd(&place[cls(i)], 1)] = i;
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

// Inclusive prefix sum over the wave's lanes by lane permutations of the
// vector ALU (a shuffle through LDS per step would take longer than the rest
// of a chunk's decays), and the value of one lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double x) {
  const long long v = __builtin_bit_cast(long long, x);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (long long)((unsigned long long)(unsigned)hi << 32 | (unsigned)lo));
}
__device__ __forceinline__ double wave_prefix(double x) {
  x += dpp_or_zero<0x111, 0xf>(x);   // row_shr:1 .. 8 within 16 lanes
  x += dpp_or_zero<0x112, 0xf>(x);
  x += dpp_or_zero<0x114, 0xf>(x);
  x += dpp_or_zero<0x118, 0xf>(x);
  x += dpp_or_zero<0x142, 0xa>(x);   // row_bcast:15 into rows 1 and 3
  x += dpp_or_zero<0x143, 0xc>(x);   // row_bcast:31 into rows 2 and 3
  return x;
}
__device__ __forceinline__ double lane_value(double x, int l) {
  const long long v = __builtin_bit_cast(long long, x);
  const int lo = __builtin_amdgcn_readlane((int)v, l), hi = __builtin_amdgcn_readlane((int)(v >> 32), l);
  return __builtin_bit_cast(double, (long long)((unsigned long long)(unsigned)hi << 32 | (unsigned)lo));
}

__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
__device__ __forceinline__ f32x4 load4(const __bf16 *p) {
  const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
  return __builtin_bit_cast(f32x4, u32x4{w[0] << 16, w[0] & 0xffff0000u, w[1] << 16, w[1] & 0xffff0000u});
}

// How a walk is laid out for inputs of type TI: C tokens per chunk and planes
// per input value.  fp32 inputs: three bf16 planes hold every bit (their
// products leave out 2^-21 at most, see mma_planes), so all products run on
// the bf16 matrix cores (6 of their passes against the 16 times slower fp32
// instruction), with half the chunk to fit the LDS.
template <typename TI> struct LinTile { static constexpr int C = 64, NPI = 1; };
template <> struct LinTile<float> { static constexpr int C = 32, NPI = 3; };

// fn(i, j) for every pair of planes that mma_planes multiplies, in its order
template <int NA, int NB, typename F>
__device__ __forceinline__ void each_plane_pair(F &&fn) {
  constexpr int M = NA > NB ? NA : NB;
  auto at = [&](auto s, auto i) __attribute__((always_inline)) {
    if constexpr (i.value < NA && s.value >= i.value && s.value - i.value < NB)
      fn(i, std::integral_constant<int, s.value - i.value>{});
  };
  auto sum = [&](auto s) __attribute__((always_inline)) {
    at(s, std::integral_constant<int, 0>{});
    at(s, std::integral_constant<int, 1>{});
    at(s, std::integral_constant<int, 2>{});
  };
  if constexpr (M > 2) sum(std::integral_constant<int, 2>{});
  if constexpr (M > 1) sum(std::integral_constant<int, 1>{});
  sum(std::integral_constant<int, 0>{});
}
template <int N, typename F>
__device__ __forceinline__ float sum_of(F &&x) {
  float s = x(0);
#pragma unroll
  for (int i = 1; i < N; ++i) s += x(i);
  return s;
}

enum : int { LIN_FWD = 0, LIN_FOLD = 1, LIN_GRAD = 2 };
constexpr int LIN_NW = 8;   // waves per workgroup
// waves per SIMD that the registers are shared out for: two workgroups per
// compute unit for bf16 inputs, one for fp32 ones, for the gradients' sake
// (81,960 bytes of LDS, 40 more than half of it, and 137 registers).  The fp32
// forward takes 80,904 bytes and 126 registers, so that two fit all the same.
template <typename TI> constexpr int lin_waves() { return std::is_same<TI, float>::value ? LIN_NW / 4 : LIN_NW / 2; }
// Eight waves; wave w holds 16 columns of the state, all 128 rows, in eight
// result tiles.  Tile m's row 4 g + i is the state's row
//   32 (m / 2) + 8 g + 4 (m % 2) + i,
// so that a pair of tiles gives lane group g 8 consecutive rows: the pair is
// the operand of the product with A's rows as these lie in memory.
//
// Per chunk: every wave multiplies its state (split into NPO planes) with all
// rows of A (outputs transposed: state as the left operand, straight from its
// result registers); the masked scores' 16 x 16 tiles are dealt out to the
// waves, which leave them in LDS as NPO planes; after a barrier all waves add
// scores x C for their columns, write their outputs, and add B^T (weighted C)
// to the state.  The chunk's operands sit in LDS in row-major order; products
// over tokens read them with the transposing LDS read.  The next chunk's
// operands are loaded into registers while this one is computed.
//
// Roundings: decays are sums in fp64 and weights one exp2 of a rounded
// difference; the state, the scores and all sums are fp32.  As operands the
// weighted C goes in three planes (all 24 bits), state and scores in three
// where the outputs are fp32, and in all three walks of the gradients (dq and
// dk feed the decays' gradient; dv, which does not, is walked by the same
// kernel); in two where a forward's outputs are rounded to bf16 anyway (2^-17
// against the outputs' 2^-8; one plane would add an error as large as the
// outputs' own).
//
// What bounds it (64 tokens x 128 x 128, bf16): 776 matrix-core instructions
// of 16 cycles, 4300 vector and 770 LDS ones per chunk.  With every compute
// unit busy (16 packed sequences, 32 heads, one workgroup per unit) a chunk
// takes about 9,600 cycles, of which the vector ALU is busy 47%, the matrix
// cores 32%, the LDS 42% (a third of that in bank conflicts), and some
// instruction issues in 67%; with three walks and two workgroups per unit (the
// gradients) 55%, 33%, 40% and 80%.  So neither unit is at its limit: vector
// and matrix work hardly overlap, as all waves of a workgroup pass the same
// phase between two barriers, and the phases are fenced from each other.
// Doubling the LDS buffers, reading operands a step ahead and loading two
// chunks ahead each changed nothing; memory is far from its limit (2 to 3
// TB/s).  Measured: 4096 tokens x 32 heads in segments of 512, 49 us (fold 25,
// scan 7).
template <int KIND, int NPO, typename TI, typename TO>
__global__ __launch_bounds__(64 * LIN_NW, lin_waves<TI>()) void linear_kernel(LinArgs p) {
  constexpr bool FOLD = KIND == LIN_FOLD, GRAD = KIND == LIN_GRAD;
  using L = LinTile<TI>;
  constexpr int C = L::C, NPI = L::NPI, NR = C / 16, KB = C / 32;
  constexpr int NW = LIN_NW, NTHR = 64 * NW;
  constexpr int PER = 16 / sizeof(TI), PIECES = D / PER, ROWS = NTHR / PIECES, LD = C / ROWS;   // staging loads
  // operands, rows of 128 in 16-byte pieces; see piece_of()
  __shared__ __attribute__((aligned(256))) __bf16 al[FOLD ? 1 : NPI][FOLD ? 128 : C * D];
  __shared__ __attribute__((aligned(256))) __bf16 bl[NPI][C * D], cl[NPI][C * D];
  __shared__ __attribute__((aligned(256))) __bf16 pl[FOLD ? 1 : NPO][FOLD ? 128 : C * C];
  __shared__ __attribute__((aligned(16))) double Fl[2][C];
  __shared__ __attribute__((aligned(16))) float fs[2][C], te[2][C];   // e^F, e^{F_end - F}
  __shared__ float fe[2];                                             // e^{F_end}
  __shared__ float dots[GRAD ? NW : 1][GRAD ? C : 1];
  __shared__ float crs[NW];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, lr = lane & 15, g = lane >> 4;

  int unit, part;
  const int R = p.Hv / p.Hqk;
  xcd_unit(blockIdx.x, R * p.roles, p.nseg * p.Hqk, unit, part);
  const int sidx = p.order ? p.order[unit / p.Hqk] : unit / p.Hqk, hv = (unit % p.Hqk) * R + part / p.roles;
  const int rn = part % p.roles;
  // the role's fields, selected one by one: an indexed copy would sit in scratch memory
  LinRole ro;
#define GDN_PICK(f) ro.f = rn == 0 ? p.role[0].f : rn == 1 ? p.role[1].f : p.role[2].f
  GDN_PICK(a); GDN_PICK(b); GDN_PICK(c); GDN_PICK(ga); GDN_PICK(gb); GDN_PICK(gc); GDN_PICK(rev); GDN_PICK(trans);
  GDN_PICK(init); GDN_PICK(seg); GDN_PICK(fin); GDN_PICK(dec); GDN_PICK(out); GDN_PICK(out_f32);
  GDN_PICK(x); GDN_PICK(gx); GDN_PICK(dot); GDN_PICK(xs); GDN_PICK(xs_last); GDN_PICK(cross);
#undef GDN_PICK
  const int col0 = 16 * wave;   // this wave's first column
  const Seg sg = segment(p, sidx);
  if (sg.rows < 0) return;
  const bool enters = ro.rev ? sg.last : sg.first, leaves = ro.rev ? sg.first : sg.last;
  if (FOLD && leaves) return;   // its contribution goes nowhere
  const int nch = (sg.rows + C - 1) / C;
  const size_t sth = ((size_t)sidx * p.Hv + hv) * (D * D), sqh = ((size_t)sg.seq * p.Hv + hv) * (D * D);

  f32x4 H[8];
#pragma unroll
  for (int m = 0; m < 8; ++m) H[m] = zero4();
  // this lane's place in a stored state, from a lane index the compiler cannot
  // see through: else it keeps the addresses alive from the first use to the last
  struct Place { int row, col; };
  auto state_place = [&]() __attribute__((always_inline)) -> Place {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int q = l & 15;
    const int along = 8 * (l >> 4), c = col0 + 4 * (q >> 2);
    return ro.trans ? Place{along, c + (q & 3)} : Place{along + (q & 3), c};
  };
  // state element (row state_row(m, g, i), column): read along whichever of the two is contiguous
  // (all loads first, then one branch around the transpositions: a branch per
  // tile would wait for each load by itself)
  auto load_state = [&](const float *S, f32x4 (&x)[8]) __attribute__((always_inline)) {
    const Place pl = state_place();
    const unsigned at = ro.trans ? pl.col * D + pl.row : pl.row * D + pl.col;
    const unsigned dm = ro.trans ? 4 : 4 * D;   // rows: 32 (m / 2) + 4 (m % 2)
#pragma unroll
    for (int m = 0; m < 8; ++m) x[m] = *reinterpret_cast<const f32x4 *>(S + (at + (8 * (m >> 1) + (m & 1)) * dm));
    if (!ro.trans) {
#pragma unroll
      for (int m = 0; m < 8; ++m) x[m] = quad_transpose(x[m], lane);
    }
  };
  // token of row r of chunk n, in the order of the walk; staging loads
  auto token = [&](int at) __attribute__((always_inline)) { return ro.rev ? sg.start + sg.rows - 1 - at : sg.start + at; };
  const int scol = (tid % PIECES) * PER;
  // (opaque at each use: what is derived from it is cheap to form, and would
  // fill registers if kept over the whole loop)
  auto staging_row = [&]() __attribute__((always_inline)) -> int {
    int r = tid / PIECES;
    asm volatile("" : "+v"(r));
    return r;
  };
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
  // token of row r of chunk n, from the chunk's base; rows past the end: the last row
  auto row_token = [&](int n, int r) __attribute__((always_inline)) -> unsigned {
    const int last = min(C, sg.rows - n * C) - 1, d = min(r, last);
    return ro.rev ? last - d : d;
  };
  auto load_chunk = [&](int n) __attribute__((always_inline)) {
    const int srow = staging_row();
    const int lo = chunk_base(n);
    const char *qa = pa + (size_t)lo * na, *qb = pb + (size_t)lo * nb, *qc = pc + (size_t)lo * nc;
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const unsigned d = row_token(n, srow + i * ROWS), sb = scol * sizeof(TI);
      if constexpr (!FOLD) xa[i] = *reinterpret_cast<const u32x4 *>(qa + (__umul24(d, na) + sb));
      xb[i] = *reinterpret_cast<const u32x4 *>(qb + (__umul24(d, nb) + sb));
      xc[i] = *reinterpret_cast<const u32x4 *>(qc + (__umul24(d, nc) + sb));
    }
  };
  // Where piece c of row r lies: its index is XORed with the row's, the row's
  // two low bits above its next two.  16 consecutive rows' pieces of one index
  // are then in 16 different places (row reads), and so are 4 aligned pieces of
  // 4 aligned rows (transposing reads).  Without it the conflicts took 80
  // million cycles of a packed call, with it 48 million of the LDS's 137.
  auto piece_of = [&](int r, int c) __attribute__((always_inline)) -> int {
    return r * D + ((c ^ ((r & 3) << 2 | (r >> 2 & 3))) << 3);
  };
  auto put_piece = [&](auto &dst, int row, const u32x4 &x) __attribute__((always_inline)) {
    const int c = tid % PIECES;
    if constexpr (NPI == 1) {
      *reinterpret_cast<u32x4 *>(&dst[0][piece_of(row, c)]) = x;
    } else {
      const int at = piece_of(row, c >> 1) + 4 * (c & 1);
      unsigned w0[3], w1[3];
      const f32x4 y = __builtin_bit_cast(f32x4, x);
      split_pair<3>(y[0], y[1], w0);
      split_pair<3>(y[2], y[3], w1);
#pragma unroll
      for (int k = 0; k < NPI; ++k) *reinterpret_cast<u32x2 *>(&dst[k][at]) = u32x2{w0[k], w1[k]};
    }
  };
  auto store_chunk = [&](int n) __attribute__((always_inline)) {
    const int srow = staging_row();
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int row = srow + i * ROWS;
      const bool on = n * C + row < sg.rows;
      const u32x4 z{0, 0, 0, 0};
      // (A's and B's rows past the end meet zero rows of C, or give rows of the output that are not written)
      if constexpr (!FOLD) put_piece(al, row, xa[i]);
      put_piece(bl, row, xb[i]);
      put_piece(cl, row, on ? xc[i] : z);
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
    const double F0 = wave_prefix(own);
    const double end = lane_value(F0, C - 1);   // (lanes past the chunk add zero)
    double F = F0;
    total += end;
    if (ro.rev) F -= own;
    if (lane < C) {
      Fl[buf][lane] = F;
      fs[buf][lane] = decay_between(F, 0.);
      te[buf][lane] = decay_between(end, F);
    }
    if (lane == 0) fe[buf] = decay_between(end, 0.);
  };

  // LDS addresses as such (not generic pointers), in bytes: what does not
  // depend on the lane goes into a read's offset field
  typedef const __attribute__((address_space(3))) __bf16 *LdsB;
  auto lds = [](const __bf16 *q) __attribute__((always_inline)) -> unsigned { return (unsigned)(size_t)(LdsB)q; };
  // 8 tokens (32 kb + 8 g ..) x one column, transposed: two reads of 4 tokens,
  // h = 0, 1, at a lane's address ^ (16 h) + 4 rows
  const int tr_row = 8 * g + (lr >> 2), tq = lr & 3;
  unsigned tr_b = 2 * piece_of(tr_row, tq), tr_c0 = 2 * (piece_of(tr_row, (col0 >> 3) + (tq >> 1)) + 4 * (tq & 1));
  auto read_tr = [&](unsigned base, unsigned at, int kb) __attribute__((always_inline)) -> bf16x8 {
    typedef __attribute__((address_space(3))) s16x4 *LdsT;
    union { s16x4 h[2]; bf16x8 v; } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsT)(size_t)(at + (base + 64 * D * kb)));
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsT)(size_t)((at ^ 16) + (base + 64 * D * kb + 8 * D)));
    return u.v;
  };
  // B's columns of tile m (piece q of its 32-column block, the half by m's parity); C's, of the wave's tile
  auto read_b = [&](int k, int kb, int m) __attribute__((always_inline)) -> bf16x8 {
    return read_tr(lds(bl[k]) + 8 * (m & 1), tr_b ^ (64 * (m >> 1)), kb);
  };
  auto read_c = [&](int k, int kb) __attribute__((always_inline)) -> bf16x8 { return read_tr(lds(cl[k]), tr_c0, kb); };
  // row lr of strip r of A or B, columns 32 kb + 8 g ..
  unsigned row0 = 2 * piece_of(lr, g);
  auto read_row = [&](const __bf16 *base, int r, int kb) __attribute__((always_inline)) -> bf16x8 {
    return *(const __attribute__((address_space(3))) bf16x8 *)(size_t)((row0 ^ (64 * kb)) + (lds(base) + 32 * D * r));
  };

  if (nch > 0) load_chunk(0);
  if (!FOLD) {
    const float *S = enters ? (ro.init ? ro.init + sqh : nullptr) : ro.seg + sth;
    if (S) load_state(S, H);
  }

  // element (r, i) of the scores in LDS: rows of C, their 16-byte pieces
  // permuted by the row so that 16 rows' pieces lie in different banks
  auto score_at = [&](int r, int i) __attribute__((always_inline)) -> int {
    return r * C + (((i >> 3) ^ (r & (C / 8 - 1))) << 3) + (i & 7);
  };
  unsigned row_p = 2 * score_at(lr, 8 * g);   // row lr of a strip of scores, columns 8 g ..
  if (nch > 0) {
    if (wave == NW - 1) put_decay(0, load_decay(0));
    // scores of the 16 x 16 tiles above the diagonal that a 32-token block of C reads: zero, once
    if constexpr (!FOLD) {
      for (int i = tid; i < NPO * (NR / 2) * 16 * 4; i += NTHR) {
        const int k = i / (NR / 2 * 64), e = i % (NR / 2 * 64), q = e / 64, r = e / 4 % 16, c = e % 4;
        *reinterpret_cast<u32x2 *>(&pl[k][score_at(32 * q + r, 32 * q + 16 + 4 * c)]) = u32x2{0, 0};
      }
    }
    store_chunk(0);
  }
  float gnext = nch > 1 && wave == NW - 1 ? load_decay(1) : 0.f;
  __syncthreads();

  for (int n = 0; n < nch; ++n) {
    const int buf = n & 1;
    // (per chunk anew: the addresses derived from these are one XOR each, and
    // would fill registers if kept over the whole loop)
    asm volatile("" : "+v"(row0), "+v"(tr_b), "+v"(tr_c0), "+v"(row_p));
    f32x4 O[FOLD ? 1 : NR];
    if constexpr (!FOLD) {
      // masked scores: the tiles on and below the diagonal dealt out to the waves
      constexpr int TILES = NR * (NR + 1) / 2;
#pragma unroll
      for (int i0 = 0; i0 < TILES; i0 += NW) {
        const int ti = i0 + wave;
        if (ti >= TILES) break;
        const int mr = ti < 1 ? 0 : ti < 3 ? 1 : ti < 6 ? 2 : 3, mi = ti - mr * (mr + 1) / 2;
        f32x4 s = zero4();
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          bf16x8 fa[NPI], fb[NPI];
#pragma unroll
          for (int k = 0; k < NPI; ++k) {
            fa[k] = read_row(al[k], mr, kb);
            fb[k] = read_row(bl[k], mi, kb);
          }
          mma_planes<NPI, NPI>(s, fb, fa);
        }
        float x[4];
        const double Fr = Fl[buf][16 * mr + lr];
        double Fi[4];   // (read before the mask, so that it is a select and no branch)
#pragma unroll
        for (int i = 0; i < 4; ++i) Fi[i] = Fl[buf][16 * mi + 4 * g + i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = s[i] * decay_between(Fr, Fi[i]);
          x[i] = 16 * mi + 4 * g + i <= 16 * mr + lr ? y : 0.f;
        }
        unsigned w0[NPO], w1[NPO];
        split_pair<NPO>(x[0], x[1], w0);
        split_pair<NPO>(x[2], x[3], w1);
        const int at = score_at(16 * mr + lr, 16 * mi + 4 * g);
#pragma unroll
        for (int k = 0; k < NPO; ++k) *reinterpret_cast<u32x2 *>(&pl[k][at]) = u32x2{w0[k], w1[k]};
      }
    }
    // the next chunk's operands (the last chunk's again behind it: a load under
    // a condition would keep the registers alive all around the loop)
    __builtin_amdgcn_sched_barrier(0);
    load_chunk(min(n + 1, nch - 1));
    if constexpr (!FOLD) {
      // state x A, per token scaled by e^F
#pragma unroll
      for (int r = 0; r < NR; ++r) O[r] = zero4();
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        bf16x8 h[NPO];
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = H[2 * kb + j / 4][j % 4];
        split8<NPO>(x, h);
        // two strips of rows at a time: products into the same tile stand apart
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          bf16x8 f[2][NPI];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < NPI; ++k) f[j][k] = read_row(al[k], r + j, kb);
          each_plane_pair<NPO, NPI>([&](auto ka, auto kb_) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              O[r + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h[ka], f[j][kb_], O[r + j], 0, 0, 0);
          });
          if (r) __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float e = fs[buf][16 * r + lr];
#pragma unroll
        for (int i = 0; i < 4; ++i) O[r][i] *= e;
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // (phases kept apart: operands of one only are live)
    // the next chunk's decays, while the scores settle
    if (wave == NW - 1 && n + 1 < nch) {
      put_decay(buf ^ 1, gnext);
      if (n + 2 < nch) gnext = load_decay(n + 2);
    }
    if constexpr (!FOLD) lds_barrier();
    if constexpr (!FOLD) {
      // scores x C
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        bf16x8 cf[NPI];
#pragma unroll
        for (int k = 0; k < NPI; ++k) cf[k] = read_c(k, kb);
#pragma unroll
        for (int r = 2 * kb; r < NR; ++r) {
          bf16x8 ps[NPO];
#pragma unroll
          for (int k = 0; k < NPO; ++k)
            ps[k] = *(const __attribute__((address_space(3))) bf16x8 *)(size_t)((row_p ^ (64 * kb)) + (lds(pl[k]) + 32 * C * r));
          mma_planes<NPI, NPO>(O[r], cf, ps);
          if (r & 1) __builtin_amdgcn_sched_barrier(0);
        }
      }
      // outputs: lane -> token 16 r + lr, columns 4 g .. of the wave's
      // (scalar base of the chunk, 32-bit offsets)
      const int lo = chunk_base(n), oc = col0 + 4 * g;
      auto row_of = [&](int r) __attribute__((always_inline)) -> unsigned { return row_token(n, 16 * r + lr); };
      if (std::is_same<TO, float>::value || (GRAD && ro.out_f32)) {
        char *o = static_cast<char *>(ro.out) + ((size_t)lo * p.Hv + hv) * (D * 4);
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if (n * C + 16 * r + lr < sg.rows)
            *reinterpret_cast<f32x4 *>(o + (__umul24(row_of(r), p.Hv * D * 4) + oc * 4)) = O[r];
      } else {
        char *o = static_cast<char *>(ro.out) + ((size_t)lo * p.Hv + hv) * (D * 2);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const u32x2 u{pk_bf16(O[r][0], O[r][1]), pk_bf16(O[r][2], O[r][3])};
          if (n * C + 16 * r + lr < sg.rows)
            *reinterpret_cast<u32x2 *>(o + (__umul24(row_of(r), p.Hv * D * 2) + oc * 2)) = u;
        }
      }
      if constexpr (GRAD) {
        if (ro.dot) {   // uniform
          f32x4 x[NR];
          const int nx = p.Hv / ro.gx;
          const char *q = static_cast<const char *>(ro.x) + ((size_t)lo * nx + hv / ro.gx) * (D * sizeof(TI));
#pragma unroll
          for (int r = 0; r < NR; ++r)
            x[r] = load4(reinterpret_cast<const TI *>(q + (__umul24(row_of(r), nx * D * (int)sizeof(TI)) + oc * (int)sizeof(TI))));
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) d = fmaf(O[r][i], x[r][i], d);
            d += __shfl_xor(d, 16);
            d += __shfl_xor(d, 32);
            if (g == 0) dots[wave][16 * r + lr] = d;
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    asm volatile("" : "+v"(tr_c0), "+v"(tr_b));
    // the state
    const float e_end = fe[buf];
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) H[m][i] *= e_end;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      bf16x8 w[3];   // C's tokens 32 kb .. of the wave's columns, weighted
      float wt[8];
      ld8(&te[buf][32 * kb + 8 * g], wt);
      bf16x8 cf[NPI];
#pragma unroll
      for (int k = 0; k < NPI; ++k) cf[k] = read_c(k, kb);
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = (float)cf[0][j];
#pragma unroll
        for (int k = 1; k < NPI; ++k) v += (float)cf[k][j];
        x[j] = v * wt[j];
      }
      split8<3>(x, w);
      asm volatile("" : "+v"(tr_b));
      // two tiles of rows at a time, their operands read one pair ahead (the
      // scheduling fences keep the compiler from reading all of them at once)
      bf16x8 f[2][2][NPI];
      auto read_pair = [&](int m) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < NPI; ++k) f[m >> 1 & 1][j][k] = read_b(k, kb, m + j);
      };
      read_pair(0);
#pragma unroll
      for (int m = 0; m < 8; m += 2) {
        if (m + 2 < 8) read_pair(m + 2);
        each_plane_pair<NPI, 3>([&](auto ka, auto kw) __attribute__((always_inline)) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            H[m + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[m >> 1 & 1][j][ka], w[kw], H[m + j], 0, 0, 0);
        });
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    lds_barrier();
    if constexpr (GRAD) {
      if (ro.dot && tid < C && n * C + tid < sg.rows)
        ro.dot[(size_t)token(n * C + tid) * p.Hv + hv] = sum_of<NW>([&](int w) { return dots[w][tid]; });
    }
    if (n + 1 < nch) store_chunk(n + 1);
    lds_barrier();
  }

  auto store_state = [&](float *S) __attribute__((always_inline)) {
    const Place pl = state_place();
    const unsigned at = ro.trans ? pl.col * D + pl.row : pl.row * D + pl.col;
    const unsigned dm = ro.trans ? 4 : 4 * D;   // rows: 32 (m / 2) + 4 (m % 2)
    if (!ro.trans) {
#pragma unroll
      for (int m = 0; m < 8; ++m) H[m] = quad_transpose(H[m], lane);
    }
#pragma unroll
    for (int m = 0; m < 8; ++m) *reinterpret_cast<f32x4 *>(S + (at + (8 * (m >> 1) + (m & 1)) * dm)) = H[m];
  };
  if constexpr (FOLD) {
    store_state(ro.fin + sth);
    if (tid == 64 * (NW - 1)) ro.dec[(size_t)sidx * p.Hv + hv] = decay_between(total, 0.);
  } else {
    if (GRAD && ro.cross) {   // uniform
      const float *S = sg.last ? (ro.xs_last ? ro.xs_last + sqh : nullptr) : ro.xs + sth;
      float d = 0.f;
      if (S) {
        f32x4 x[8];
        load_state(S, x);
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) d = fmaf(H[m][i], x[m][i], d);
      }
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) d += __shfl_xor(d, m);
      if (lane == 0) crs[wave] = d;
      __syncthreads();
      if (tid == 0) ro.cross[(size_t)sidx * p.Hv + hv] = sum_of<NW>([&](int w) { return crs[w]; });
    }
    if (ro.fin && leaves) store_state(ro.fin + sqh);
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
