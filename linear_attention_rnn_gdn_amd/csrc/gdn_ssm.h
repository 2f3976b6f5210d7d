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
  float *part_bc, *part_a;      // gradients: [tokens, tiles, 2 N], [rows, J, N + 2, C]
};

// A pointer whose loads are uniform over the wave: through the scalar cache.
template <typename T> using Uniform = const __attribute__((address_space(4))) T *;
template <typename T> __device__ __forceinline__ Uniform<T> uniform(const T *p) { return (Uniform<T>)(uintptr_t)p; }

// B or C of one token
template <int N>
__device__ __forceinline__ void load_row(const float *p, float (&x)[N]) {
  Uniform<float> q = uniform(p);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = q[i];
}
template <int N>
__device__ __forceinline__ void load_row(const __bf16 *p, float (&x)[N]) {
  Uniform<unsigned> q = uniform(reinterpret_cast<const unsigned *>(p));
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const unsigned w = q[i];
    x[2 * i] = __builtin_bit_cast(float, w << 16);
    x[2 * i + 1] = __builtin_bit_cast(float, w & 0xffff0000u);
  }
}

// An element at a lane's byte offset from a row that is the same for the whole
// wave: one scalar address per row, and one 32-bit register for all rows.
template <typename T>
__device__ __forceinline__ float get(const T *row, unsigned off) {
  return to_f32(*reinterpret_cast<const T *>(reinterpret_cast<const char *>(row) + off));
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

constexpr int SSM_BATCH = 8;   // tokens asked for at once

// One wave: 64 channels of one segment.  FOLD: only the segment's end state
// and sum of d.
template <int N, typename TI, typename TO, bool FOLD>
__global__ __launch_bounds__(64) void ssm_walk_kernel(SsmArgs a) {
  const int lane = threadIdx.x;
  const int tile = blockIdx.x % a.tiles;
  const int64_t unit = blockIdx.x / a.tiles;   // (row, segment)
  const Tile tl = tile_of(a, tile, lane);
  const int c = tl.c;
  if (!FOLD && unit >= (int64_t)a.rows * a.J) {   // empty sequences keep their state
    const int s = (int)(unit - (int64_t)a.rows * a.J);
    if (a.T && (!a.cu || offset_at(a.cu, s + 1, a.T) > offset_at(a.cu, s, a.T))) return;
    float h[N] = {};
    const size_t at = ((size_t)s * a.C + c) * N;
    if (a.h0) load_states<N>(a.h0 + at, h);
    if (tl.on) store_states<N>(a.h_T + at, h);
    return;
  }
  const int row = (int)(unit / a.J), j = (int)(unit % a.J);
  if (FOLD && j + 1 == a.J) return;   // (nothing comes behind the last one)
  const int t0 = j * a.len, t1 = min(a.T, t0 + a.len);
  Sequence q{row, 0, a.T};
  if (a.cu) {
    q = sequence_at(a.cu, a.B, a.T, t0, 0);
    q.seq = __builtin_amdgcn_readfirstlane(q.seq);
    q.begin = __builtin_amdgcn_readfirstlane(q.begin);
    q.end = __builtin_amdgcn_readfirstlane(q.end);
  }
  const int64_t r0 = (int64_t)row * a.T;
  const TI *x = static_cast<const TI *>(a.x) + r0 * a.ld_x;
  const TI *dt = static_cast<const TI *>(a.dt) + r0 * a.ld_dt;
  const bool gated = a.z != nullptr;
  const TI *z = gated ? static_cast<const TI *>(a.z) + r0 * a.ld_z : nullptr;
  const TI *Bm = static_cast<const TI *>(a.Bm) + r0 * a.ld_b + tl.group * N;
  const TI *Cm = static_cast<const TI *>(a.Cm) + r0 * a.ld_c + tl.group * N;
  TO *y = static_cast<TO *>(a.y) + r0 * a.C;
  const unsigned ci = c * sizeof(TI), co = c * sizeof(TO);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
  float A[N], h[N];   // A in units of log2(e)
  load_states<N>(a.A + (size_t)c * N, A);
#pragma unroll
  for (int n = 0; n < N; ++n) A[n] *= kLog2e;
  const size_t su = ((size_t)unit * a.tiles + tile) * 64 + lane;   // among the segments' sums
  const size_t se = ((size_t)unit * a.tiles + tile) * N * 64 + lane;
  auto enter = [&]() {   // the state a sequence starts from
    if (a.h0) load_states<N>(a.h0 + ((size_t)q.seq * a.C + c) * N, h);
    else
#pragma unroll
      for (int n = 0; n < N; ++n) h[n] = 0.f;
  };
  bool fresh = q.begin == t0;
  if (fresh) {
    enter();
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = FOLD ? 0.f : a.in[se + n * 64];
  }
  float sum = 0.f;
  int t = t0;
  while (t < t1) {
    const int stop = min(t1, q.end);
    for (; t < stop; t += SSM_BATCH) {
      float xs[SSM_BATCH], ds[SSM_BATCH], zs[SSM_BATCH];
#pragma unroll
      for (int i = 0; i < SSM_BATCH; ++i) {
        const int64_t at = min(t + i, stop - 1);
        xs[i] = get(x + at * a.ld_x, ci);
        ds[i] = get(dt + at * a.ld_dt, ci);
        if constexpr (!FOLD) zs[i] = gated ? get(z + at * a.ld_z, ci) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < SSM_BATCH; ++i) {
        if (t + i >= stop) break;
        float b[N], cc[N];
        load_row<N>(Bm + (int64_t)(t + i) * a.ld_b, b);
        if constexpr (!FOLD) load_row<N>(Cm + (int64_t)(t + i) * a.ld_c, cc);
        const float d = step_size(a, ds[i] + bias), u = d * xs[i];
        float o[4] = {D * xs[i], 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < N; ++n) {
          h[n] = fmaf(__builtin_amdgcn_exp2f(d * A[n]), h[n], u * b[n]);
          if constexpr (!FOLD) o[n & 3] = fmaf(cc[n], h[n], o[n & 3]);
        }
        if constexpr (FOLD) {
          sum += d;
        } else {
          float s = (o[0] + o[1]) + (o[2] + o[3]);
          if (gated) s *= silu(zs[i]);
          if (tl.on) put(y + (int64_t)(t + i) * a.C, co, s);
        }
      }
    }
    t = stop;
    if (stop == q.end) {
      if constexpr (!FOLD)
        if (a.h_T && tl.on) store_states<N>(a.h_T + ((size_t)q.seq * a.C + c) * N, h);
      if (stop < t1) {   // packed: the next sequence
        q = sequence_at(a.cu, a.B, a.T, t, q.seq + 1);
        q.seq = __builtin_amdgcn_readfirstlane(q.seq);
        q.end = __builtin_amdgcn_readfirstlane(q.end);
        fresh = true;
        sum = 0.f;
        enter();
      }
    }
  }
  if constexpr (FOLD) {
    a.sum[su] = sum;
#pragma unroll
    for (int n = 0; n < N; ++n) a.end[se + n * 64] = h[n];
    if (tile == 0 && lane == 0) a.fresh[unit] = fresh;
  }
}

// The states entering the segments: one thread per (row, channel, state),
// from segment to segment.  Segment j's own state is complete where a sequence
// begins in it.
template <int N>
__global__ __launch_bounds__(256) void ssm_scan_kernel(SsmArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), lanes = (int64_t)a.tiles * N;
  if (i >= a.rows * lanes) return;
  const int row = (int)(i / lanes), tile = (int)(i % lanes) / N, n = (int)(i % N);
  const float A = a.A[(size_t)tile_of(a, tile, lane).c * N + n] * kLog2e;
  float h = 0.f;
  for (int j = 0; j + 1 < a.J; ++j) {
    const size_t u = (size_t)row * a.J + j, v = u * a.tiles + tile;
    const float e = a.end[(v * N + n) * 64 + lane], s = a.sum[v * 64 + lane];
    h = a.fresh[u] ? e : fmaf(__builtin_amdgcn_exp2f(s * A), h, e);
    a.in[((v + a.tiles) * N + n) * 64 + lane] = h;
  }
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
  if (a.z) s *= silu(to_f32(static_cast<const TI *>(a.z)[b * a.ld_z + c]));
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
// its front is sum_t P_t C_t ds_t.
template <int N, typename TI>
__global__ __launch_bounds__(64) void ssm_bwd_fold_kernel(SsmArgs a) {
  const int lane = threadIdx.x, tile = blockIdx.x % a.tiles;
  const int64_t unit = blockIdx.x / a.tiles;
  const Tile tl = tile_of(a, tile, lane);
  const int c = tl.c, row = (int)(unit / a.J), j = (int)(unit % a.J);
  const int t0 = j * a.len, t1 = min(a.T, t0 + a.len);
  const int64_t r0 = (int64_t)row * a.T;
  const TI *x = static_cast<const TI *>(a.x) + r0 * a.ld_x;
  const TI *dt = static_cast<const TI *>(a.dt) + r0 * a.ld_dt;
  const bool gated = a.z != nullptr;
  const TI *z = gated ? static_cast<const TI *>(a.z) + r0 * a.ld_z : nullptr;
  const TI *dy = static_cast<const TI *>(a.dy) + r0 * a.C;
  const unsigned ci = c * sizeof(TI);
  const TI *Bm = static_cast<const TI *>(a.Bm) + r0 * a.ld_b + tl.group * N;
  const TI *Cm = static_cast<const TI *>(a.Cm) + r0 * a.ld_c + tl.group * N;
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
  float A[N], h[N], P[N], R[N];
  load_states<N>(a.A + (size_t)c * N, A);
  if (j == 0 && a.h0) load_states<N>(a.h0 + ((size_t)row * a.C + c) * N, h);
  else
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    A[n] *= kLog2e;
    P[n] = 1.f;
    R[n] = 0.f;
  }
  float sum = 0.f;
  for (int t = t0; t < t1; t += SSM_BATCH) {
    float xs[SSM_BATCH], ds[SSM_BATCH], zs[SSM_BATCH], gs[SSM_BATCH];
#pragma unroll
    for (int i = 0; i < SSM_BATCH; ++i) {
      const int64_t at = min(t + i, t1 - 1);
      xs[i] = get(x + at * a.ld_x, ci);
      ds[i] = get(dt + at * a.ld_dt, ci);
      zs[i] = gated ? get(z + at * a.ld_z, ci) : 0.f;
      gs[i] = get(dy + at * a.C, ci);
    }
#pragma unroll
    for (int i = 0; i < SSM_BATCH; ++i) {
      if (t + i >= t1) break;
      float b[N], cc[N];
      load_row<N>(Bm + (int64_t)(t + i) * a.ld_b, b);
      load_row<N>(Cm + (int64_t)(t + i) * a.ld_c, cc);
      const float d = step_size(a, ds[i] + bias), u = d * xs[i];
      const float g = gated ? gs[i] * silu(zs[i]) : gs[i];
      sum += d;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float e = __builtin_amdgcn_exp2f(d * A[n]);
        h[n] = fmaf(e, h[n], u * b[n]);
        P[n] *= e;
        R[n] = fmaf(P[n], g * cc[n], R[n]);
      }
    }
  }
  const size_t v = (size_t)unit * a.tiles + tile;
  a.sum[v * 64 + lane] = sum;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    a.end[(v * N + n) * 64 + lane] = h[n];
    a.rend[(v * N + n) * 64 + lane] = R[n];
  }
  if (tile == 0 && lane == 0) a.fresh[unit] = j == 0;
}

// the cotangents entering the segments from behind, from the last segment on
template <int N>
__global__ __launch_bounds__(256) void ssm_rscan_kernel(SsmArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), lanes = (int64_t)a.tiles * N;
  if (i >= a.rows * lanes) return;
  const int row = (int)(i / lanes), tile = (int)(i % lanes) / N, n = (int)(i % N);
  const int c = tile_of(a, tile, lane).c;
  const float A = a.A[(size_t)c * N + n] * kLog2e;
  float g = a.dh_T ? a.dh_T[((size_t)row * a.C + c) * N + n] : 0.f;
  for (int j = a.J - 1; j > 0; --j) {
    const size_t v = ((size_t)row * a.J + j) * a.tiles + tile;
    g = fmaf(__builtin_amdgcn_exp2f(a.sum[v * 64 + lane] * A), g, a.rend[(v * N + n) * 64 + lane]);
    a.rin[((v - a.tiles) * N + n) * 64 + lane] = g;
  }
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
// holds in registers; the states at the pieces' fronts are kept in LDS (the
// first one's can be read again).  Of 32 states a wave takes 16, and the two
// waves of a channel exchange their sums over states once per piece.
//
// A lane's registers stay below 256, two waves per SIMD: with more, copies of
// live values to accumulation registers are placed where paths join, and this
// compiler put them before the lanes that took the other path were switched on
// again (seen in the listing of an earlier form of this kernel; addresses were
// lost).  So there is room for no more tokens, tokens are fenced from each
// other, and what differs between calls (a gate or none) branches on scalars,
// never on lanes.
template <int N> struct SsmBwd {
  static constexpr int NS = N < 16 ? N : 16, WAVES = N / NS, S = NS == 8 ? 8 : 4, PIECES = 32 / S, LEN = S * PIECES;
};

template <int N, typename TI>
__global__ __launch_bounds__(64 * SsmBwd<N>::WAVES, 2) void ssm_bwd_kernel(SsmArgs a) {
  using K = SsmBwd<N>;
  constexpr int S = K::S, NS = K::NS;
  __shared__ float marks[K::WAVES][K::PIECES - 1][NS][64];
  __shared__ float sums[K::WAVES > 1 ? K::WAVES : 1][S][3][K::WAVES > 1 ? 64 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tile = blockIdx.x % a.tiles;
  const int64_t unit = blockIdx.x / a.tiles;
  const Tile tl = tile_of(a, tile, lane);
  const int c = tl.c, row = (int)(unit / a.J), j = (int)(unit % a.J), n0 = wave * NS;
  const int t0 = j * a.len, t1 = min(a.T, t0 + a.len);
  const int64_t r0 = (int64_t)row * a.T;
  const bool gated = a.z != nullptr;
  const TI *x = static_cast<const TI *>(a.x) + r0 * a.ld_x;
  const TI *dt = static_cast<const TI *>(a.dt) + r0 * a.ld_dt;
  const TI *z = gated ? static_cast<const TI *>(a.z) + r0 * a.ld_z : nullptr;
  const TI *dy = static_cast<const TI *>(a.dy) + r0 * a.C;
  const TI *Bm = static_cast<const TI *>(a.Bm) + r0 * a.ld_b + tl.group * N + n0;
  const TI *Cm = static_cast<const TI *>(a.Cm) + r0 * a.ld_c + tl.group * N + n0;
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
  const size_t v = (size_t)unit * a.tiles + tile, vn = (v * N + n0) * 64 + lane, sn = ((size_t)row * a.C + c) * N + n0;
  float(*mark)[NS][64] = marks[wave];
  const unsigned ci = c * sizeof(TI), cr = reduced_index<NS>(lane) * 4;
  float A[NS], h[NS], dh[NS], dA[NS];
  load_states<NS>(a.A + (size_t)c * N + n0, A);
  auto front = [&]() {
    if (j > 0)
#pragma unroll
      for (int n = 0; n < NS; ++n) h[n] = a.in[vn + n * 64];
    else if (a.h0)
      load_states<NS>(a.h0 + sn, h);
    else
#pragma unroll
      for (int n = 0; n < NS; ++n) h[n] = 0.f;
  };
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
  const int pieces = (t1 - t0 + S - 1) / S;
  // forward over the segment: the state each piece starts from
  front();
  for (int k = 0; k + 1 < pieces; ++k) {
    float xs[S], ds[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int64_t at = t0 + k * S + i;
      xs[i] = get(x + at * a.ld_x, ci);
      ds[i] = get(dt + at * a.ld_dt, ci);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float b[NS];
      load_row<NS>(Bm + (int64_t)(t0 + k * S + i) * a.ld_b, b);
      const float d = step_size(a, ds[i] + bias), u = d * xs[i];
#pragma unroll
      for (int n = 0; n < NS; ++n) h[n] = fmaf(__builtin_amdgcn_exp2f(d * A[n]), h[n], u * b[n]);
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) mark[k][n][lane] = h[n];
  }
  for (int k = pieces - 1; k >= 0; --k) {
    const int tk = t0 + k * S;
    // per token: x, the step and its slope, the cotangent of s, and what s is multiplied with in dz
    float xs[S], ds[S], slope[S], gs[S], ws[S], hs[S + 1][NS];
    {
      float zs[S];
#pragma unroll
      for (int i = 0; i < S; ++i) {   // (a token past the last: no step and no cotangent, so that it changes nothing)
        const int64_t at = min(tk + i, t1 - 1);
        const bool here = tk + i < t1 && tl.on;   // (nor does a lane past the last channel add to dB and dC)
        xs[i] = get(x + at * a.ld_x, ci);
        ds[i] = get(dt + at * a.ld_dt, ci);
        gs[i] = get(dy + at * a.C, ci);
        xs[i] = here ? xs[i] : 0.f;
        gs[i] = here ? gs[i] : 0.f;
        zs[i] = gated ? get(z + at * a.ld_z, ci) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const float e = exp_neg_abs(ds[i] + bias);
        slope[i] = a.softplus ? sigmoid_of(ds[i] + bias, e).s : 1.f;
        ds[i] = a.softplus ? softplus(ds[i] + bias, e) : ds[i] + bias;
        ds[i] = tk + i < t1 ? ds[i] : 0.f;
        float sg, dsg;
        silu_grad(zs[i], sg, dsg);
        ws[i] = gs[i] * dsg;
        gs[i] *= gated ? sg : 1.f;
      }
    }
    if (k) {
#pragma unroll
      for (int n = 0; n < NS; ++n) hs[0][n] = mark[k - 1][n][lane];
    } else {
      front();
#pragma unroll
      for (int n = 0; n < NS; ++n) hs[0][n] = h[n];
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float b[NS];
      load_row<NS>(Bm + (int64_t)min(tk + i, t1 - 1) * a.ld_b, b);
      const float u = ds[i] * xs[i];
#pragma unroll
      for (int n = 0; n < NS; ++n) hs[i + 1][n] = fmaf(__builtin_amdgcn_exp2f(ds[i] * A[n]), hs[i][n], u * b[n]);
      __builtin_amdgcn_sched_barrier(0);
    }
    float sum[S][3];   // over the states: s, du, dd
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
      float b[NS], cc[NS], r[NS];
      int tt = min(tk + i, t1 - 1);
      float d = ds[i];
      // B and the decays are formed anew: kept from the way forward they would take S times as many registers
      asm("" : "+s"(tt));
      asm("" : "+v"(d));
      const int64_t t = tt;
      load_row<NS>(Bm + t * a.ld_b, b);
      load_row<NS>(Cm + t * a.ld_c, cc);
      const float u = d * xs[i], g = gs[i];
      float *to = a.part_bc + ((r0 + t) * a.tiles + tile) * 2 * N + n0;
      float s = 0.f, du = 0.f, dd = 0.f;
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        s = fmaf(cc[n], hs[i + 1][n], s);
        r[n] = g * hs[i + 1][n];
      }
      reduce_lanes<NS>(r, lane);
      const float rc = r[0];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        dh[n] = fmaf(cc[n], g, dh[n]);
        r[n] = u * dh[n];
        du = fmaf(b[n], dh[n], du);
        dh[n] *= __builtin_amdgcn_exp2f(d * A[n]);
        const float q = hs[i][n] * dh[n];
        dd = fmaf(A[n], q, dd);
        dA[n] = fmaf(d, q, dA[n]);
      }
      reduce_lanes<NS>(r, lane);
      if (tk + i < t1 && reduced_writer<NS>(lane)) {
        put(to, cr, r[0]);
        put(to + N, cr, rc);
      }
      asm volatile("" : "+v"(s), "+v"(du), "+v"(dd));   // (summed here, not where they are used)
      sum[i][0] = s;
      sum[i][1] = du;
      sum[i][2] = dd;
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
      if (tk + i >= t1) break;
      const float g = gs[i], d = ds[i], s = fmaf(D, xs[i], sum[i][0]), du = sum[i][1];
      const float dv = fmaf(xs[i], du, sum[i][2] * kLn2) * slope[i];   // (A is in units of log2(e))
      dbias += dv;
      dD = fmaf(g, xs[i], dD);
      if (tl.on && (K::WAVES == 1 || (i & 1) == wave)) {
        const int64_t at = (r0 + tk + i) * a.C;
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

// dB and dC: the sums over a group's waves, one thread per element
template <int N, typename TI>
__global__ __launch_bounds__(256) void ssm_bc_sum_kernel(SsmArgs a, TI *dB, TI *dC, int64_t tokens) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= tokens * a.G * 2 * N) return;
  const int n = (int)(i % (2 * N)), g = (int)(i / (2 * N) % a.G);
  const int64_t t = i / (2 * N) / a.G;
  const float *p = a.part_bc + (t * a.tiles + g * a.per) * 2 * N + n;
  float s = 0.f;
  for (int k = 0; k < a.per; ++k) s += p[(size_t)k * 2 * N];
  const int64_t at = (t * a.G + g) * N + n % N;
  (n < N ? dB : dC)[at] = from_f32<TI>(s);
}

// dA, dD and ddt_bias: the sums over the segments
template <int N>
__global__ __launch_bounds__(256) void ssm_a_sum_kernel(SsmArgs a, float *dA, float *dD, float *dbias) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)(N + 2) * a.C) return;
  const int n = (int)(i / a.C), c = (int)(i % a.C);
  const int64_t units = (int64_t)a.rows * a.J;
  double s = 0.;
  for (int64_t u = 0; u < units; ++u) s += (double)a.part_a[(size_t)u * (N + 2) * a.C + i];
  if (n < N) dA[(size_t)c * N + n] = (float)s;
  else if (n == N) {
    if (dD) dD[c] = (float)s;
  } else if (dbias) {
    dbias[c] = (float)s;
  }
}

}  // namespace gdn
