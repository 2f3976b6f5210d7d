// gdn_ssm.h -- the selective state space scan.  Per channel c with N states:
//   d = softplus(dt + dt_bias) (or dt + dt_bias),
//   h_n <- e^{d A_n} h_n + d x B_n,   s = sum_n C_n h_n + D x,   y = s silu(z),
// B and C shared by the channels of a group.
//
// Each of the T x C x N state elements costs one exp2 and four multiply-adds,
// and nothing in them is a matrix product (every channel and state decays by
// its own factor), so the vector ALU bounds all of it: a lane holds one
// channel with its N states in registers, B and C of a token are the same for
// a whole wave and come through scalar loads as scalar operands, and x, dt and
// z are one element per lane.  A wave walks a segment of consecutive tokens.
// Where the sequences alone are too few to fill the chip they are cut into
// segments: a first launch folds each segment into the state at its end (from
// zero, or from the sequence's own state if it begins there) and the sum of d,
// a second carries the states from segment to segment (the decay of a whole
// segment is e^{A sum d}), and the walks start from those.
// Measured at 4096 tokens of 4096 channels with 16 states in bf16: forward
// 135 us a call, gradients 399.  The launches' medians under the profiler, which
// add up to more than a call without it (vector ALU busy; its instructions per
// token and wave): forward folds 57 (91%; 89), scan 12, walks 77 (91%; 121), of
// which 5 N are the recurrence's own; gradients folds 111 (88%; 158), scan 20,
// walks 323 (82%; 449), sums 11.  One token of 256 rows with 4096 channels:
// 28 us, 143 MB, 5.0 TB/s.
#pragma once
#include <type_traits>

#include "gdn_act.h"

namespace gdn {

struct SsmArgs {
  int B, T, C, N, G;            // rows (packed: sequences), tokens per row (packed: in all), channels, states, groups
  int n_slots, softplus;
  int64_t ld_x, ld_dt, ld_z, ld_b, ld_c;   // elements between tokens
  const int *cu, *slots;
  const void *x, *dt, *z, *Bm, *Cm, *dy;
  const float *A, *D, *dt_bias, *h0, *dh_T;
  void *y;
  float *h_T, *state;
  void *dx, *ddt, *dz;
  float *dh0;
  int rows;                     // rows of tokens: B, or 1 where sequences are packed
  int per, tiles;               // waves per group of channels, and in all
  int len, J;                   // tokens per segment, segments per row
  float *end, *sum, *in;        // [rows, J, tiles, N, 64], [rows, J, tiles, 64]: folded segments; states entering them
  int *fresh;                   // [rows, J]: a sequence begins in the segment
  float *rend, *rin;            // the same of the states' cotangents, from the last token to the first
  float *mark, *mark_sum;       // gradients: [rows, J, marks, tiles, N, 64], [rows, J, marks, tiles, 64]: the folded state within
  int marks;                    // a segment in front of each piece of the way back but the first, and the sum of d up to there
  float *part_bc, *part_a;      // gradients: [tokens, tiles, 2 N], [rows, J, N + 2, C]
};

// A pointer whose loads are uniform over the wave: through the scalar cache.
template <typename T> using Uniform = const __attribute__((address_space(4))) T *;
template <typename T> __device__ __forceinline__ Uniform<T> uniform(const T *p) { return (Uniform<T>)(uintptr_t)p; }

// B or C of one token, as it lies in memory: N scalar registers of fp32, half
// as many of pairs of bf16, which are widened by scalar instructions (other
// units than the vector ALU's).
template <int N, typename TI> struct Row {
  static constexpr int WORDS = N * sizeof(TI) / 4;
  unsigned w[WORDS];
  __device__ __forceinline__ void load(const TI *p) {
    const Uniform<unsigned> q = uniform(reinterpret_cast<const unsigned *>(p));
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = q[i];
  }
  __device__ __forceinline__ float at(int n) const {
    if constexpr (WORDS == N) return __builtin_bit_cast(float, w[n]);
    const unsigned v = w[n / 2];
    return n & 1 ? __builtin_bit_cast(float, v & 0xffff0000u) : __builtin_bit_cast(float, v << 16);
  }
  // Waits until the row is here.  Scalar loads return in any order, so a wait
  // is for all of them: what is asked for next has to be asked for behind it.
  __device__ __forceinline__ void wait() const { asm volatile("" ::"s"(w[0]), "s"(w[WORDS - 1])); }
};
// An element at a lane's byte offset from a row that is the same for the whole
// wave: one scalar address per row, and one 32-bit register for all rows.
template <typename T>
__device__ __forceinline__ float get(const T *row, unsigned off) {
  return to_f32(*reinterpret_cast<const T *>(reinterpret_cast<const char *>(row) + off));
}
// (Hides an offset's value, once per group of loads: or the compiler adds it to
// each tensor's address ahead of the loop and then 64-bit addresses per lane to
// those, an instruction of the vector ALU per load.)
__device__ __forceinline__ unsigned fresh_offset(unsigned off) {
  asm volatile("" : "+v"(off));
  return off;
}
template <typename T>
__device__ __forceinline__ T raw(const T *row, unsigned off) {
  return *reinterpret_cast<const T *>(reinterpret_cast<const char *>(row) + off);
}
template <typename T>
__device__ __forceinline__ void put(T *row, unsigned off, float x) {
  *reinterpret_cast<T *>(reinterpret_cast<char *>(row) + off) = from_f32<T>(x);
}

struct Tile {
  int group, c;   // c: this lane's channel (of a lane past the group's last, the last)
  bool on;
};
__device__ __forceinline__ Tile tile_of(const SsmArgs &a, int tile, int lane) {
  const int width = a.C / a.G, i = tile % a.per * 64 + lane;
  const int g = tile / a.per;
  return Tile{g, g * width + min(i, width - 1), i < width};
}

// N consecutive states of one channel in [.., C, N]
template <int N>
__device__ __forceinline__ void load_states(const float *p, float (&h)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = *reinterpret_cast<const float4 *>(p + i);
    h[i] = v.x; h[i + 1] = v.y; h[i + 2] = v.z; h[i + 3] = v.w;
  }
}
template <int N>
__device__ __forceinline__ void store_states(float *p, const float (&h)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(p + i) = float4{h[i], h[i + 1], h[i + 2], h[i + 3]};
}

__device__ __forceinline__ float step_size(const SsmArgs &a, float v) { return a.softplus ? softplus(v, exp_neg_abs(v)) : v; }

// Tokens asked for at once, and worked on without a branch between them, by the
// walk and by the fold of the gradients, which notes states between batches, at
// every 4th or 8th token.  Batches of 4 and of 8 in the walk took, in us: 12
// packed sequences with 16 states 178 and 175; 4096 tokens of 4096 channels in
// bf16 97 and 94 with 8 states, 141 and 139 with 16, 246 and 238 with 32, in fp32
// 105 and 108 with 8, 164 and 158 with 16, 270 and 270 with 32.
constexpr int WALK_BATCH = 8, FOLD_BATCH = 4;

// One wave: 64 channels of one segment.  FOLD: only the segment's end state
// and sum of d.  The elements of the next WALK_BATCH tokens are on their way
// while these are worked on, and so are B and C of the next token.
// A batch in which the segment or a sequence ends is walked token by token.
//
// u B could come from the matrix cores (a lane's channel is a column of
// v_mfma_f32_32x32x2's result, its states the rows), which takes 16
// multiply-adds off the vector ALU; measured, the matrix instruction holds up
// as many cycles of it, and the walk takes as long.
template <int N, typename TI, typename TO, bool FOLD>
__global__ __launch_bounds__(64, 2) void ssm_walk_kernel(SsmArgs a) {
  const int lane = threadIdx.x;
  const int tile = blockIdx.x % a.tiles;
  const int64_t unit = blockIdx.x / a.tiles;   // (row, segment)
  const Tile tl = tile_of(a, tile, lane);
  const int c = tl.c;
  float h[N];
#pragma unroll
  for (int n = 0; n < N; ++n) h[n] = 0.f;
  if (!FOLD && unit >= (int64_t)a.rows * a.J) {   // empty sequences keep their state
    const int s = (int)(unit - (int64_t)a.rows * a.J);
    if (a.T && (!a.cu || offset_at(a.cu, s + 1, a.T) > offset_at(a.cu, s, a.T))) return;
    const size_t at = ((size_t)s * a.C + c) * N;
    if (a.h0) load_states<N>(a.h0 + at, h);
    if (tl.on) store_states<N>(a.h_T + at, h);
    return;
  }
  const int row = (int)(unit / a.J), j = (int)(unit % a.J);
  if (FOLD && j + 1 == a.J) return;   // (nothing comes behind the last one)
  const int t0 = j * a.len, t1 = min(a.T, t0 + a.len);
  Sequence q{row, 0, a.T};
  auto next_sequence = [&](int t, int from) {
    q = sequence_of_wave(a.cu, a.B, a.T, t, from, lane);
  };
  if (a.cu) next_sequence(t0, 0);
  const int64_t r0 = (int64_t)row * a.T + t0;   // the segment's first token
  const bool gated = a.z != nullptr;             // (without a gate x stands in for z, and is not used)
  const int64_t ld_z = gated ? a.ld_z : a.ld_x;
  const TI *x = static_cast<const TI *>(a.x) + r0 * a.ld_x;
  const TI *dt = static_cast<const TI *>(a.dt) + r0 * a.ld_dt;
  const TI *z = static_cast<const TI *>(gated ? a.z : a.x) + r0 * ld_z;
  const TI *Bm = static_cast<const TI *>(a.Bm) + r0 * a.ld_b + tl.group * N;
  const TI *Cm = static_cast<const TI *>(a.Cm) + r0 * a.ld_c + tl.group * N;
  TO *y = static_cast<TO *>(a.y) + r0 * a.C;
  const unsigned ci = c * sizeof(TI), co = c * sizeof(TO);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
  float A[N];   // in units of log2(e)
  load_states<N>(a.A + (size_t)c * N, A);
#pragma unroll
  for (int n = 0; n < N; ++n) A[n] *= kLog2e;
  const size_t su = ((size_t)unit * a.tiles + tile) * 64 + lane;   // among the segments' sums
  const size_t se = ((size_t)unit * a.tiles + tile) * N * 64 + lane;
  auto enter = [&]() {   // the state a sequence starts from
    if (a.h0) {
      load_states<N>(a.h0 + ((size_t)q.seq * a.C + c) * N, h);
#pragma unroll
      for (int n = 0; n < N; ++n) asm volatile("" : "+v"(h[n]));   // (waits here, not at every use behind the join)
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) h[n] = 0.f;
    }
  };
  bool fresh = q.begin == t0;
  if (fresh) enter();
  else if constexpr (!FOLD)
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = a.in[se + n * 64];
  float sum = 0.f;
  struct Batch {
    TI x[WALK_BATCH], dt[WALK_BATCH], z[WALK_BATCH];
  };
  // asks for the elements of the tokens from the pointers' on (past the segment's last: of that one again)
  auto ask = [&](int left, Batch &p) {
    const unsigned off = fresh_offset(ci);
#pragma unroll
    for (int i = 0; i < WALK_BATCH; ++i) {
      const int64_t at = min(i, left - 1);
      p.x[i] = raw(x + at * a.ld_x, off);
      p.dt[i] = raw(dt + at * a.ld_dt, off);
      if constexpr (!FOLD) p.z[i] = raw(z + at * ld_z, off);
    }
  };
  // B and C of a token, and of the next, up to 16 words each.  (At 8 words nearly
  // all of it stays in scalar registers.  At 16, fp32 with 16 states and bf16 with
  // 32, it does not: 224 scalars are kept in lanes of vector registers, and 1115
  // of 3484 and 1103 of 5107 vector instructions of the kernel, as compiled, move
  // them there and back.)
  constexpr bool AHEAD = Row<N, TI>::WORDS <= 16;
  Row<N, TI> B, C, Bn, Cn;
  auto ask_rows = [&](Row<N, TI> &B, Row<N, TI> &C) {
    B.load(Bm);
    if constexpr (!FOLD) C.load(Cm);
  };
  if (AHEAD && t0 < t1) ask_rows(B, C);
  Batch now, next;
  if (t0 < t1) ask(t1 - t0, now);
  for (int t = t0; t < t1; t += WALK_BATCH) {
    const bool whole = t + WALK_BATCH <= t1 && (q.end <= t || q.end >= t + WALK_BATCH);
    x += WALK_BATCH * a.ld_x;
    dt += WALK_BATCH * a.ld_dt;
    z += WALK_BATCH * ld_z;
    if (t + WALK_BATCH < t1) ask(t1 - t - WALK_BATCH, next);
    float xs[WALK_BATCH], d[WALK_BATCH];
#pragma unroll
    for (int i = 0; i < WALK_BATCH; ++i) {
      xs[i] = to_f32(now.x[i]);
      d[i] = step_size(a, to_f32(now.dt[i]) + bias);
    }
    auto token = [&](int i) {
      if constexpr (AHEAD) {
        B.wait();
        if constexpr (!FOLD) C.wait();
        __builtin_amdgcn_sched_barrier(0);
      } else {
        ask_rows(B, C);
      }
      if (t + i + 1 < t1) {
        Bm += a.ld_b;
        Cm += a.ld_c;
      }
      if constexpr (AHEAD) {
        ask_rows(Bn, Cn);
        __builtin_amdgcn_sched_barrier(0);
      }
      const float u = d[i] * xs[i];
      float o[4] = {D * xs[i], 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < N; ++n) {
        h[n] = fmaf(__builtin_amdgcn_exp2f(d[i] * A[n]), h[n], u * B.at(n));
        if constexpr (!FOLD) o[n & 3] = fmaf(C.at(n), h[n], o[n & 3]);
      }
      if constexpr (FOLD) {
        sum += d[i];
      } else {
        float s = (o[0] + o[1]) + (o[2] + o[3]);
        s *= gated ? silu<std::is_same<TO, __bf16>::value>(to_f32(now.z[i])) : 1.f;
        if (tl.on) put(y, fresh_offset(co), s);
        y += a.C;
      }
      if constexpr (AHEAD) {
        B = Bn;
        if constexpr (!FOLD) C = Cn;
      }
    };
    auto sequence_end = [&](int i) {
      if (t + i + 1 != q.end) return;
      if constexpr (!FOLD)
        if (a.h_T && tl.on) store_states<N>(a.h_T + ((size_t)q.seq * a.C + c) * N, h);
      if (q.end < t1) {   // packed: the next sequence
        next_sequence(q.end, q.seq + 1);
        fresh = true;
        sum = 0.f;
        enter();
      }
    };
    if (whole) {
#pragma unroll
      for (int i = 0; i < WALK_BATCH; ++i) token(i);
      sequence_end(WALK_BATCH - 1);
    } else {
#pragma unroll
      for (int i = 0; i < WALK_BATCH; ++i) {
        if (t + i >= t1) break;
        token(i);
        sequence_end(i);
      }
    }
    now = next;
  }
  if constexpr (FOLD) {
    a.sum[su] = sum;
#pragma unroll
    for (int n = 0; n < N; ++n) a.end[se + n * 64] = h[n];
    if (tile == 0 && lane == 0) a.fresh[unit] = fresh;
  }
}

// f + 2^x h: a state carried over many tokens (the sum of d times A, in units of
// log2(e)).  In two halves: where states grow, 2^x alone may pass fp32 while the
// state is zero, or so small that the product does not; x / 2 is held below 128.
__device__ __forceinline__ float carry(float x, float h, float f) {
  const float half = __builtin_amdgcn_exp2f(fminf(0.5f * x, 127.f));
  return fmaf(half, half * h, f);
}

// The states entering the segments (or, REV, the cotangents entering them from
// behind, from the last one on).  A workgroup takes one (row, 64 channels,
// state): its four waves fold a quarter of the segments each, exchange what
// they folded and go over them again from what enters their quarter.  Segment
// j's own state is complete where a sequence begins in it.
// (The scan moves two states per segment, 33 MB in 12 us at 64 segments of 4096 channels; latency bounds it,
// that of the flags too: they are scalar loads under a test, each waited for before the next.)
constexpr int SCAN_AHEAD = 16;   // segments whose states and sums are asked for before they are used
template <int N>
__global__ __launch_bounds__(256) void ssm_scan_kernel(SsmArgs a) {
  __shared__ float folded[2][4][64];
  __shared__ int begins[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t all = (int64_t)a.rows * a.tiles * N;
  const bool rev = blockIdx.x >= all;   // (the second half of the grid, where there is one)
  const int64_t i = blockIdx.x - (rev ? all : 0);
  const int n = (int)(i % N), tile = (int)(i / N % a.tiles), row = (int)(i / N / a.tiles);
  const int c = tile_of(a, tile, lane).c;
  const float A = a.A[(size_t)c * N + n] * kLog2e;
  const float *end = rev ? a.rend : a.end;
  float *in = rev ? a.rin : a.in;
  const int steps = a.J - 1, per = (steps + 3) / 4, k0 = min(steps, wave * per), k1 = min(steps, k0 + per);
  const int64_t first = rev ? a.J - 1 : 0, way = rev ? -1 : 1;   // step k: segment first + way k
  float h = 0.f, sum = 0.f;   // this quarter's own state, and the sum of d over it
  bool begun = false;         // a sequence begins in it
  float e[SCAN_AHEAD], s[SCAN_AHEAD];
  int fresh[SCAN_AHEAD];
  auto ask = [&](int k) {
#pragma unroll
    for (int m = 0; m < SCAN_AHEAD; ++m) {
      const int64_t u = row * (int64_t)a.J + first + way * min(k + m, steps - 1), v = u * a.tiles + tile;
      e[m] = end[(v * N + n) * 64 + lane];
      s[m] = a.sum[v * 64 + lane];
      fresh[m] = !rev && a.fresh[u];
    }
  };
  auto pass = [&](bool write) {
    for (int k = k0; k < k1; k += SCAN_AHEAD) {
      if (!write || k1 - k0 > SCAN_AHEAD) ask(k);   // (the second time a single batch is still here)
#pragma unroll
      for (int m = 0; m < SCAN_AHEAD; ++m) {
        if (k + m >= k1) break;
        h = fresh[m] ? e[m] : carry(s[m] * A, h, e[m]);
        sum += s[m];
        begun = begun || fresh[m];
        if (write) in[(((row * (int64_t)a.J + first + way * (k + m + 1)) * a.tiles + tile) * N + n) * 64 + lane] = h;
      }
    }
  };
  pass(false);
  folded[0][wave][lane] = h;
  folded[1][wave][lane] = sum;
  if (lane == 0) begins[wave] = begun;
  __syncthreads();
  h = rev && a.dh_T ? a.dh_T[((size_t)row * a.C + c) * N + n] : 0.f;
  for (int w = 0; w < wave; ++w) {
    const float f = folded[0][w][lane];
    h = begins[w] ? f : carry(folded[1][w][lane] * A, h, f);
  }
  pass(true);
}

// ----------------------------------------------------------------------------
// One token of every row: 4 states per thread, N / 4 threads per channel, so
// that a wave reads and writes its part of the pool in whole lines; memory
// bound (8 N bytes of state per channel).
template <int N, typename TI, typename TO>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmArgs a) {
  constexpr int L = N / 4;   // threads per channel
  const int tid = threadIdx.x, blocks = (a.C * L + 255) / 256;
  const int b = blockIdx.x / blocks, i = blockIdx.x % blocks * 256 + tid;
  const int c = min(i / L, a.C - 1), n0 = i % L * 4;
  const bool on = i / L < a.C;
  int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) slot = -1;
  float *p = a.state + ((size_t)max(slot, 0) * a.C + c) * N + n0;
  const float4 old = *reinterpret_cast<const float4 *>(p);   // (asked for before the other rows' slots are looked at)
  bool seen = false;
  if (a.slots && slot >= 0)
    for (int r = tid; r < b; r += 256) seen |= a.slots[r] == slot;
  if (__syncthreads_or(seen)) slot = -1;
  TO *y = static_cast<TO *>(a.y) + (size_t)b * a.C + c;
  if (slot < 0) {   // no state: a zero output
    if (on && n0 == 0) *y = from_f32<TO>(0.f);
    return;
  }
  const int g = c / (a.C / a.G);
  const float x = to_f32(static_cast<const TI *>(a.x)[b * a.ld_x + c]);
  const float v = to_f32(static_cast<const TI *>(a.dt)[b * a.ld_dt + c]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
  const TI *Bp = static_cast<const TI *>(a.Bm) + b * a.ld_b + g * N + n0, *Cp = static_cast<const TI *>(a.Cm) + b * a.ld_c + g * N + n0;
  const float4 A = *reinterpret_cast<const float4 *>(a.A + (size_t)c * N + n0);
  const float d = step_size(a, v), u = d * x, dl = d * kLog2e;
  float4 h;
  h.x = fmaf(__builtin_amdgcn_exp2f(dl * A.x), old.x, u * to_f32(Bp[0]));
  h.y = fmaf(__builtin_amdgcn_exp2f(dl * A.y), old.y, u * to_f32(Bp[1]));
  h.z = fmaf(__builtin_amdgcn_exp2f(dl * A.z), old.z, u * to_f32(Bp[2]));
  h.w = fmaf(__builtin_amdgcn_exp2f(dl * A.w), old.w, u * to_f32(Bp[3]));
  float s = fmaf(h.x, to_f32(Cp[0]), h.y * to_f32(Cp[1])) + fmaf(h.z, to_f32(Cp[2]), h.w * to_f32(Cp[3]));
#pragma unroll
  for (int m = 1; m < L; m <<= 1) s += __shfl_xor(s, m);
  if (!on) return;
  *reinterpret_cast<float4 *>(p) = h;
  if (n0) return;
  if (a.D) s = fmaf(a.D[c], x, s);
  if (a.z) s *= silu<std::is_same<TO, __bf16>::value>(to_f32(static_cast<const TI *>(a.z)[b * a.ld_z + c]));
  *y = from_f32<TO>(s);
}

// ----------------------------------------------------------------------------
// The gradients.  With ds = dy silu(z), a_n = e^{d A_n}, h' the state before a
// token and dh the cotangent of the state behind it (from its own output and
// the tokens after it):
//   dh_n = C_n ds + (a_n dh_n of the next token),    g_n = a_n h'_n dh_n,
//   dB_n = sum_c u dh_n,  dC_n = sum_c ds h_n,  dA_n = sum_t d g_n,
//   du = sum_n B_n dh_n,  dd = x du + sum_n A_n g_n,  dx = d du + D ds,  ddt = dd softplus'.
// Folding a segment needs one pass in token order for both directions: with P
// the product of the decays so far, the cotangent that leaves the segment at
// its front is sum_t P_t C_t ds_t.  The states that it passes in front of the
// pieces that the way back takes are noted: with the segment's incoming state
// decayed up to there they are the states themselves.
template <int N> struct SsmBwd {
  static constexpr int NS = N < 16 ? N : 16, WAVES = N / NS, S = NS == 8 ? 8 : 4;   // states and waves per channel, tokens per piece
};

template <int N, typename TI>
__global__ __launch_bounds__(64, 2) void ssm_bwd_fold_kernel(SsmArgs a) {
  using R = Row<N, TI>;
  constexpr bool AHEAD = R::WORDS <= 16;
  const int lane = threadIdx.x, tile = blockIdx.x % a.tiles;
  const int64_t unit = blockIdx.x / a.tiles;
  const Tile tl = tile_of(a, tile, lane);
  const int c = tl.c, row = (int)(unit / a.J), j = (int)(unit % a.J);
  const int t0 = j * a.len, len = min(a.T - t0, a.len);
  const int64_t r0 = (int64_t)row * a.T + t0;
  const bool gated = a.z != nullptr;   // (without a gate x stands in for z, and is not used)
  const int64_t ld_z = gated ? a.ld_z : a.ld_x;
  const TI *x = static_cast<const TI *>(a.x) + r0 * a.ld_x;
  const TI *dt = static_cast<const TI *>(a.dt) + r0 * a.ld_dt;
  const TI *z = static_cast<const TI *>(gated ? a.z : a.x) + r0 * ld_z;
  const TI *dy = static_cast<const TI *>(a.dy) + r0 * a.C;
  const TI *Bm = static_cast<const TI *>(a.Bm) + r0 * a.ld_b + tl.group * N;
  const TI *Cm = static_cast<const TI *>(a.Cm) + r0 * a.ld_c + tl.group * N;
  const unsigned ci = c * sizeof(TI);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
  float A[N], h[N], P[N], Q[N];
  load_states<N>(a.A + (size_t)c * N, A);
  if (j == 0 && a.h0) load_states<N>(a.h0 + ((size_t)row * a.C + c) * N, h);
  else
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    A[n] *= kLog2e;
    P[n] = 1.f;
    Q[n] = 0.f;
  }
  float sum = 0.f;
  struct Batch {
    TI x[FOLD_BATCH], dt[FOLD_BATCH], z[FOLD_BATCH], dy[FOLD_BATCH];
  };
  auto ask = [&](int k, Batch &p) {
    const unsigned off = fresh_offset(ci);
#pragma unroll
    for (int i = 0; i < FOLD_BATCH; ++i) {
      const int64_t at = min(k + i, len - 1);
      p.x[i] = raw(x + at * a.ld_x, off);
      p.dt[i] = raw(dt + at * a.ld_dt, off);
      p.z[i] = raw(z + at * ld_z, off);
      p.dy[i] = raw(dy + at * a.C, off);
    }
  };
  R B, C, Bn, Cn;
  Batch now, next;
  ask(0, now);   // (a segment that is folded has a token)
  if (AHEAD) {
    B.load(Bm);
    C.load(Cm);
  }
  for (int k = 0; k < len; k += FOLD_BATCH) {
    if (k + FOLD_BATCH < len) ask(k + FOLD_BATCH, next);
    if (k && k % SsmBwd<N>::S == 0) {
      const size_t m = ((size_t)unit * a.marks + k / SsmBwd<N>::S - 1) * a.tiles + tile;
      a.mark_sum[m * 64 + lane] = sum;
#pragma unroll
      for (int n = 0; n < N; ++n) a.mark[(m * N + n) * 64 + lane] = h[n];
    }
    float d[FOLD_BATCH], u[FOLD_BATCH], g[FOLD_BATCH];
#pragma unroll
    for (int i = 0; i < FOLD_BATCH; ++i) {   // (a token past the last: no step, no cotangent)
      const bool here = k + i < len;
      d[i] = here ? step_size(a, to_f32(now.dt[i]) + bias) : 0.f;
      u[i] = here ? d[i] * to_f32(now.x[i]) : 0.f;
      g[i] = here ? to_f32(now.dy[i]) : 0.f;
      g[i] *= gated ? silu<false>(to_f32(now.z[i])) : 1.f;   // (it enters dA and dh0, which are fp32)
      sum += d[i];
    }
#pragma unroll
    for (int i = 0; i < FOLD_BATCH; ++i) {
      const int64_t at = min(k + i + (AHEAD ? 1 : 0), len - 1);
      if constexpr (AHEAD) {
        B.wait();
        C.wait();
        __builtin_amdgcn_sched_barrier(0);
        Bn.load(Bm + at * a.ld_b);
        Cn.load(Cm + at * a.ld_c);
        __builtin_amdgcn_sched_barrier(0);
      } else {
        B.load(Bm + at * a.ld_b);
        C.load(Cm + at * a.ld_c);
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float e = __builtin_amdgcn_exp2f(d[i] * A[n]);
        h[n] = fmaf(e, h[n], u[i] * B.at(n));
        P[n] *= e;
        Q[n] = fmaf(P[n], g[i] * C.at(n), Q[n]);
      }
      if constexpr (AHEAD) {
        B = Bn;
        C = Cn;
      }
    }
    now = next;
  }
  const size_t v = (size_t)unit * a.tiles + tile;
  a.sum[v * 64 + lane] = sum;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    a.end[(v * N + n) * 64 + lane] = h[n];
    a.rend[(v * N + n) * 64 + lane] = Q[n];
  }
  if (tile == 0 && lane == 0) a.fresh[unit] = j == 0;
}

// Sums of M values over the wave's 64 lanes: halves, quarters, .. of the
// values go to halves, quarters, .. of the lanes, so that a value costs two
// instructions or three and not twelve.  Behind it lane l holds in v[0] the
// sum of value `reduced_index(l)`; M values of 64 / M lanes each (M <= 64).
__device__ __forceinline__ void swap32(float &x, float &y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y), false, false);
  const unsigned r0 = r[0], r1 = r[1];   // (a bit_cast of a vector's element itself takes element 0)
  x = __builtin_bit_cast(float, r0);
  y = __builtin_bit_cast(float, r1);
}
__device__ __forceinline__ void swap16(float &x, float &y) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y), false, false);
  const unsigned r0 = r[0], r1 = r[1];   // (a bit_cast of a vector's element itself takes element 0)
  x = __builtin_bit_cast(float, r0);
  y = __builtin_bit_cast(float, r1);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
template <int CTRL, int K, int M>
__device__ __forceinline__ void reduce_level(float (&v)[M], bool upper) {
  if constexpr (K >= 1) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float keep = upper ? v[i + K] : v[i], send = upper ? v[i] : v[i + K];
      v[i] = keep + dpp<CTRL>(send);
    }
  } else {
    v[0] += dpp<CTRL>(v[0]);
  }
}
template <int M>
__device__ __forceinline__ void reduce_lanes(float (&v)[M], int lane) {
#pragma unroll
  for (int i = 0; i < M / 2; ++i) {   // lanes 32 .. 63 take the upper half of the values
    swap32(v[i], v[i + M / 2]);
    v[i] += v[i + M / 2];
  }
#pragma unroll
  for (int i = 0; i < M / 4; ++i) {   // odd rows of 16 lanes the upper half of those
    swap16(v[i], v[i + M / 4]);
    v[i] += v[i + M / 4];
  }
  constexpr int Q = M / 4;   // values left over 16 lanes: lanes l and l ^ 8, l and 7 - l of 8, l ^ 2, l ^ 1
  reduce_level<0x128, Q / 2>(v, lane & 8);    // row_ror:8
  reduce_level<0x141, Q / 4>(v, lane & 4);    // row_half_mirror
  reduce_level<0x4e, Q / 8>(v, lane & 2);     // quad_perm 2,3,0,1
  reduce_level<0xb1, Q / 16>(v, lane & 1);    // quad_perm 1,0,3,2
}
template <int M>
__device__ __forceinline__ int reduced_index(int lane) {
  int i = 0, k = M / 2;
#pragma unroll
  for (int bit = 32; bit; bit >>= 1) {
    if (k && (lane & bit)) i += k;
    k >>= 1;
  }
  return i;
}
// the lanes that write a reduced value (the others hold copies)
template <int M> __device__ __forceinline__ bool reduced_writer(int lane) { return (lane & (64 / M - 1)) == 0; }

// The way back over a segment takes pieces of S tokens, whose states a lane
// holds in registers, from the state that the fold noted in front of each.  Of
// 32 states a wave takes 16, and the two waves of a channel exchange their sums
// over states once per piece.  A piece's noted state is asked for while the
// piece behind it is worked on: at 4096 tokens of 4096 channels with 16 states
// this kernel takes 303 us so, and took 422 where it asked for what it needed at once.
// (Asking for the tokens' elements ahead too spills, and gained nothing.)
// Scalar registers are short: 92 of its scalars are kept in lanes of vector
// registers there, and 228 of the loop's 2038 vector instructions, as compiled,
// move them.
//
// A lane's registers stay below 256, two waves per SIMD: with more, copies of
// live values to accumulation registers are placed where paths join, and this
// compiler put them before the lanes that took the other path were switched on
// again (seen in the listing of an earlier form of this kernel; addresses were
// lost).  So there is room for no more tokens, tokens are fenced from each
// other, and what differs between calls (a gate or none) branches on scalars,
// never on lanes.
template <int N, typename TI>
__global__ __launch_bounds__(64 * SsmBwd<N>::WAVES, 2) void ssm_bwd_kernel(SsmArgs a) {
  using K = SsmBwd<N>;
  using R = Row<K::NS, TI>;
  constexpr int S = K::S, NS = K::NS;
  __shared__ float sums[K::WAVES][S][3][K::WAVES > 1 ? 64 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tile = blockIdx.x % a.tiles;
  const int64_t unit = blockIdx.x / a.tiles;
  const Tile tl = tile_of(a, tile, lane);
  const int c = tl.c, row = (int)(unit / a.J), j = (int)(unit % a.J), n0 = wave * NS;
  const int t0 = j * a.len, len = min(a.T - t0, a.len);
  const int64_t r0 = (int64_t)row * a.T + t0;            // the segment's first token
  const bool gated = a.z != nullptr;                      // (without a gate x stands in for z, and is not used)
  const int64_t ld_z = gated ? a.ld_z : a.ld_x;
  const TI *x = static_cast<const TI *>(a.x) + r0 * a.ld_x;
  const TI *dt = static_cast<const TI *>(a.dt) + r0 * a.ld_dt;
  const TI *z = static_cast<const TI *>(gated ? a.z : a.x) + r0 * ld_z;
  const TI *dy = static_cast<const TI *>(a.dy) + r0 * a.C;
  const TI *Bm = static_cast<const TI *>(a.Bm) + r0 * a.ld_b + tl.group * N + n0;
  const TI *Cm = static_cast<const TI *>(a.Cm) + r0 * a.ld_c + tl.group * N + n0;
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
  const size_t v = (size_t)unit * a.tiles + tile, vn = (v * N + n0) * 64 + lane, sn = ((size_t)row * a.C + c) * N + n0;
  const unsigned ci = c * sizeof(TI), cr = reduced_index<NS>(lane) * 4;
  float A[NS], h[NS], dh[NS], dA[NS];   // h: the state in front of the segment
  load_states<NS>(a.A + (size_t)c * N + n0, A);
  if (j > 0)
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = a.in[vn + n * 64];
  else if (a.h0)
    load_states<NS>(a.h0 + sn, h);
  else
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = 0.f;
  if (j + 1 < a.J)
#pragma unroll
    for (int n = 0; n < NS; ++n) dh[n] = a.rin[vn + n * 64];
  else if (a.dh_T)
    load_states<NS>(a.dh_T + sn, dh);
  else
#pragma unroll
    for (int n = 0; n < NS; ++n) dh[n] = 0.f;
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    A[n] *= kLog2e;
    dA[n] = 0.f;
  }
  float dD = 0.f, dbias = 0.f;
  // a token of the way forward
  auto advance = [&](float d, float xi, const R &B, float (&h)[NS]) {
    const float u = d * xi;
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = fmaf(__builtin_amdgcn_exp2f(d * A[n]), h[n], u * B.at(n));
  };
  float front[NS], front_sum = 0.f;
  auto ask_front = [&](int k) {
    if (k <= 0) return;
    const size_t m = ((size_t)unit * a.marks + k / S - 1) * a.tiles + tile;
    front_sum = a.mark_sum[m * 64 + lane];
#pragma unroll
    for (int n = 0; n < NS; ++n) front[n] = a.mark[(m * N + n0 + n) * 64 + lane];
  };
  ask_front((len - 1) / S * S);
  for (int k = (len - 1) / S * S; k >= 0 && len > 0; k -= S) {
    // per token: x, the step, its slope, the cotangent of s, and what s is multiplied with in dz
    float xs[S], ds[S], slope[S], gs[S], ws[S], hs[S + 1][NS];
    R B, C, Bn, Cn;   // of a token, and of the one to be worked on next
    auto row_of = [&](const TI *m, int64_t ld, int i) { return m + (int64_t)min(k + i, len - 1) * ld; };
    {
      TI xr[S], dr[S], gr[S], zr[S];
      const unsigned off = fresh_offset(ci);
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int64_t at = min(k + i, len - 1);
        xr[i] = raw(x + at * a.ld_x, off);
        dr[i] = raw(dt + at * a.ld_dt, off);
        gr[i] = raw(dy + at * a.C, off);
        zr[i] = raw(z + at * ld_z, off);
      }
      // the state in front of the piece (the fold began the row's first segment with h0 itself)
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        hs[0][n] = k ? front[n] : 0.f;
        if (j > 0 || k == 0) hs[0][n] = fmaf(__builtin_amdgcn_exp2f(k ? front_sum * A[n] : 0.f), h[n], hs[0][n]);
      }
      ask_front(k - S);
#pragma unroll
      for (int i = 0; i < S; ++i) {   // a token past the last, or a lane past the last channel: no step, no cotangent
        const bool here = k + i < len;
        const float v = to_f32(dr[i]) + bias;
        slope[i] = a.softplus ? sigmoid(v) : 1.f;
        ds[i] = here ? step_size(a, v) : 0.f;
        xs[i] = here && tl.on ? to_f32(xr[i]) : 0.f;
        const float g = here && tl.on ? to_f32(gr[i]) : 0.f;
        float sg, dsg;
        silu_grad<false>(to_f32(zr[i]), sg, dsg);
        ws[i] = g * dsg;
        gs[i] = gated ? g * sg : g;
      }
    }
    B.load(row_of(Bm, a.ld_b, 0));
#pragma unroll
    for (int i = 0; i < S; ++i) {
      B.wait();
      __builtin_amdgcn_sched_barrier(0);
      if (i + 1 < S) Bn.load(row_of(Bm, a.ld_b, i + 1));
      else C.load(row_of(Cm, a.ld_c, i));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < NS; ++n) hs[i + 1][n] = hs[i][n];
      advance(ds[i], xs[i], B, hs[i + 1]);
      if (i + 1 < S) B = Bn;
      __builtin_amdgcn_sched_barrier(0);
    }
    float sum[S][3];   // over the states: s, du, dd
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
      float r[NS];
      float d = ds[i];
      asm("" : "+v"(d));   // (the decays are formed anew: kept from the way forward they would take S times NS registers)
      B.wait();
      C.wait();
      __builtin_amdgcn_sched_barrier(0);
      if (i) {
        Bn.load(row_of(Bm, a.ld_b, i - 1));
        Cn.load(row_of(Cm, a.ld_c, i - 1));
      }
      __builtin_amdgcn_sched_barrier(0);
      const float u = d * xs[i], g = gs[i];
      float s = 0.f, du = 0.f, dd = 0.f;
      if (k + i < len) {   // (nothing of a token past the last: zero times a state behind a bad last token may be no number)
        float *to = a.part_bc + ((r0 + k + i) * a.tiles + tile) * 2 * N + n0;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          s = fmaf(C.at(n), hs[i + 1][n], s);
          r[n] = g * hs[i + 1][n];
        }
        reduce_lanes<NS>(r, lane);
        const float rc = r[0];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          dh[n] = fmaf(C.at(n), g, dh[n]);
          r[n] = u * dh[n];
          du = fmaf(B.at(n), dh[n], du);
          dh[n] *= __builtin_amdgcn_exp2f(d * A[n]);
          const float q = hs[i][n] * dh[n];
          dd = fmaf(A[n], q, dd);
          dA[n] = fmaf(d, q, dA[n]);
        }
        reduce_lanes<NS>(r, lane);
        if (reduced_writer<NS>(lane)) {
          put(to, cr, r[0]);
          put(to + N, cr, rc);
        }
      }
      asm volatile("" : "+v"(s), "+v"(du), "+v"(dd));   // (summed here, not where they are used)
      sum[i][0] = s;
      sum[i][1] = du;
      sum[i][2] = dd;
      if (i) {
        B = Bn;
        C = Cn;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (K::WAVES > 1) {
      __syncthreads();   // (the last piece's have been read)
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int m = 0; m < 3; ++m) sums[wave][i][m][lane] = sum[i][m];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int m = 0; m < 3; ++m) sum[i][m] = sums[0][i][m][lane] + sums[1][i][m][lane];
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (k + i >= len) break;
      const float g = gs[i], d = ds[i], s = fmaf(D, xs[i], sum[i][0]), du = sum[i][1];
      const float dv = fmaf(xs[i], du, sum[i][2] * kLn2) * slope[i];   // (A is in units of log2(e))
      dbias += dv;
      dD = fmaf(g, xs[i], dD);
      if (tl.on && (K::WAVES == 1 || (i & 1) == wave)) {
        const int64_t at = (r0 + k + i) * a.C;
        put(static_cast<TI *>(a.dx) + at, ci, fmaf(d, du, D * g));
        put(static_cast<TI *>(a.ddt) + at, ci, dv);
        if (gated) put(static_cast<TI *>(a.dz) + at, ci, ws[i] * s);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (!tl.on) return;
  float *pa = a.part_a + (size_t)unit * (N + 2) * a.C + c;
#pragma unroll
  for (int n = 0; n < NS; ++n) pa[(size_t)(n0 + n) * a.C] = dA[n];
  if (wave == 0) {
    pa[(size_t)N * a.C] = dD;
    pa[(size_t)(N + 1) * a.C] = dbias;
  }
  if (j == 0 && a.dh0) store_states<NS>(a.dh0 + sn, dh);
}

constexpr int SUM_AHEAD = 8;   // segments asked for at once
// What is left to sum, in one launch.  The first workgroups: dA, dD and
// ddt_bias over the segments, 64 channels of one of them each, four segments
// side by side.  The others: dB and dC over a group's waves; a wave takes one
// token and group, 16 bytes of the 2 N values per lane, as many of the group's
// waves side by side as that leaves room for.
template <int N, typename TI>
__global__ __launch_bounds__(256) void ssm_sum_kernel(SsmArgs a, float *dA, float *dD, float *dbias, TI *dB, TI *dC, int64_t tokens) {
  constexpr int L = 2 * N / 4, R = 64 / L;   // lanes per row of values, rows at once
  __shared__ double red[4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tiles = (a.C + 63) / 64;
  const int64_t rest = (int64_t)blockIdx.x - (N + 2) * (int64_t)tiles;
  if (rest < 0) {
    const int n = blockIdx.x / tiles, c = blockIdx.x % tiles * 64 + lane;
    const int64_t units = (int64_t)a.rows * a.J, step = (int64_t)(N + 2) * a.C;
    const float *p = a.part_a + (int64_t)n * a.C + min(c, a.C - 1);
    double s = 0.;
    for (int64_t u = wave; u < units; u += 4 * SUM_AHEAD) {
      float v[SUM_AHEAD];
#pragma unroll
      for (int i = 0; i < SUM_AHEAD; ++i) v[i] = p[min(u + 4 * i, units - 1) * step];
#pragma unroll
      for (int i = 0; i < SUM_AHEAD; ++i) s += u + 4 * i < units ? (double)v[i] : 0.;
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave || c >= a.C) return;
    s = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
    if (n < N) dA[(size_t)c * N + n] = (float)s;
    else if (n == N) {
      if (dD) dD[c] = (float)s;
    } else if (dbias) {
      dbias[c] = (float)s;
    }
    return;
  }
  const int64_t i = rest * 4 + wave, t = i / a.G;
  const int g = (int)(i % a.G), n = lane % L * 4;
  if (t >= tokens) return;
  const float *p = a.part_bc + (t * a.tiles + g * a.per) * 2 * N + n;
  float4 s{0.f, 0.f, 0.f, 0.f};
  for (int k = lane / L; k < a.per; k += R) {
    const float4 v = *reinterpret_cast<const float4 *>(p + (size_t)k * 2 * N);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
#pragma unroll
  for (int m = L; m < 64; m <<= 1) {
    s.x += __shfl_xor(s.x, m); s.y += __shfl_xor(s.y, m); s.z += __shfl_xor(s.z, m); s.w += __shfl_xor(s.w, m);
  }
  if (lane >= L) return;
  TI *to = (n < N ? dB : dC) + (t * a.G + g) * N + n % N;
  if constexpr (std::is_same<TI, float>::value) *reinterpret_cast<float4 *>(to) = s;
  else *reinterpret_cast<uint2 *>(to) = uint2{pk_bf16(s.x, s.y), pk_bf16(s.z, s.w)};
}

}  // namespace gdn
