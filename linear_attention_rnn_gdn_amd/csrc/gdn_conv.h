// gdn_conv.h -- the short causal convolution, one filter of W taps per
// channel:
//   pre[t, c] = bias[c] + sum_w weight[c, w] x[t - (W - 1) + w, c],
//   y = silu(pre), or pre.
// Tokens before a sequence's first are the rows of its window (the last W - 1
// tokens of what came before), or zero.
//
// Every kernel here moves a few bytes per multiply-add, so memory bounds all
// of them; a thread takes VEC neighbouring channels (16 bytes) of a run of
// consecutive tokens and slides the window along in registers, so that a row
// is read once but for the W - 1 rows before each run.
#pragma once
#include <type_traits>

#include "gdn_act.h"

namespace gdn {

struct ConvArgs {
  int B, T, C, n_slots, silu;   // rows (packed: sequences), tokens per row (packed: in all)
  int64_t ld;                   // elements between tokens of x
  const int *cu, *slots;
  const void *x, *h0, *dy, *dh_T;
  const float *weight, *bias;
  void *y, *h_T, *state, *dx, *dh0;
  float *part;                  // gradients of weight and bias: [pieces][W + 1][C]
  int lanes, lane_bits;         // threads of a workgroup side by side in channels (a power of two)
  int run;                      // tokens per thread
  int runs;                     // workgroups per row of tokens
};

template <typename T, int VEC> struct Pack { typedef T type __attribute__((ext_vector_type(VEC))); };
template <typename T> struct Pack<T, 1> { typedef T type; };

template <int VEC, typename T>
__device__ __forceinline__ void widen(const typename Pack<T, VEC>::type &p, float (&x)[VEC]) {
  if constexpr (VEC == 1) x[0] = (float)p;
  else
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = (float)p[i];
}
template <int VEC, typename T>
__device__ __forceinline__ typename Pack<T, VEC>::type narrow(const float (&x)[VEC]) {
  typename Pack<T, VEC>::type p;
  if constexpr (VEC == 1) p = (T)x[0];
  else if constexpr (VEC == 8) p = to_bf16x8(x);
  else
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = x[i];
  return p;
}

// A row of x or, where the token lies before its sequence, of the window;
// `before` = token - first token of the sequence, at least -(W - 1).
template <int W, int VEC, typename T>
__device__ __forceinline__ typename Pack<T, VEC>::type conv_row(const ConvArgs &a, const T *x, int seq, int before, int c) {
  using P = typename Pack<T, VEC>::type;
  if (before >= 0) return *reinterpret_cast<const P *>(x);
  if (!a.h0) return P{};
  return *reinterpret_cast<const P *>(static_cast<const T *>(a.h0) + ((size_t)seq * (W - 1) + (W - 1 + before)) * a.C + c);
}

constexpr int CONV_BATCH = 8, CONV_BWD_BATCH = 4;   // rows asked for at once

template <int W, int VEC, typename T>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a) {
  using P = typename Pack<T, VEC>::type;
  constexpr bool ROUGH = std::is_same<T, __bf16>::value;
  const int tid = threadIdx.x, tiles = (a.C / VEC + a.lanes - 1) / a.lanes;
  const int tile = blockIdx.x % tiles;
  const int64_t piece = blockIdx.x / tiles;
  const int c = (tile * a.lanes + (tid & (a.lanes - 1))) * VEC;
  const int rows = a.cu ? 1 : a.B;
  if (c >= a.C) return;
  if (piece >= (int64_t)rows * a.runs) {   // the windows behind the sequences
    const int per = 256 >> a.lane_bits;
    const int64_t i = (piece - (int64_t)rows * a.runs) * per + (tid >> a.lane_bits);
    if (i >= (int64_t)a.B * (W - 1)) return;
    const int s = (int)(i / (W - 1)), j = (int)(i % (W - 1));
    int begin = 0, end = a.T;
    int64_t row = (int64_t)s * a.T;
    if (a.cu) {
      begin = offset_at(a.cu, s, a.T);
      end = max(begin, offset_at(a.cu, s + 1, a.T));
      row = 0;
    }
    const int t = end - (W - 1) + j;
    const T *x = static_cast<const T *>(a.x) + (row + max(t, 0)) * a.ld + c;
    *reinterpret_cast<P *>(static_cast<T *>(a.h_T) + (size_t)i * a.C + c) = conv_row<W, VEC, T>(a, x, s, t - begin, c);
    return;
  }
  const int row = (int)(piece / a.runs);
  const int64_t at = (int64_t)(piece % a.runs) * (256 >> a.lane_bits) * a.run + (int64_t)(tid >> a.lane_bits) * a.run;
  if (at >= a.T) return;
  const int t0 = (int)at, t1 = (int)min((int64_t)a.T, at + a.run);
  Sequence q{row, 0, a.T};
  if (a.cu) q = sequence_at(a.cu, a.B, a.T, t0, 0);
  const T *x = static_cast<const T *>(a.x) + (int64_t)row * a.T * a.ld + c;
  T *y = static_cast<T *>(a.y) + (int64_t)row * a.T * a.C + c;
  float w[W][VEC], bias[VEC], win[W][VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = a.weight[(size_t)(c + i) * W + k];
  }
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int t = t0 - (W - 1) + k;
    widen<VEC, T>(conv_row<W, VEC, T>(a, x + (int64_t)max(t, 0) * a.ld, q.seq, t - q.begin, c), win[k]);
  }
  for (int tb = t0; tb < t1; tb += CONV_BATCH) {
    P in[CONV_BATCH];
#pragma unroll
    for (int i = 0; i < CONV_BATCH; ++i) in[i] = *reinterpret_cast<const P *>(x + (int64_t)min(tb + i, t1 - 1) * a.ld);
#pragma unroll
    for (int i = 0; i < CONV_BATCH; ++i) {
      const int t = tb + i;
      if (t >= t1) break;
      if (t == q.end) {   // packed: the next sequence
        q = sequence_at(a.cu, a.B, a.T, t, q.seq + 1);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) widen<VEC, T>(conv_row<W, VEC, T>(a, x, q.seq, k - (W - 1), c), win[k]);
      }
      widen<VEC, T>(in[i], win[W - 1]);
      float o[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        float s = bias[v];
#pragma unroll
        for (int k = 0; k < W; ++k) s = fmaf(w[k][v], win[k][v], s);
        o[v] = a.silu ? silu<ROUGH>(s) : s;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) win[k][v] = win[k + 1][v];
      }
      *reinterpret_cast<P *>(y + (int64_t)t * a.C) = narrow<VEC, T>(o);
    }
  }
}

// One token of every row: the row's window in the pool [n_slots, W - 1, C]
// moves on by one token.
template <int W, int VEC, typename T>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a) {
  using P = typename Pack<T, VEC>::type;
  const int tid = threadIdx.x, tiles = (a.C / VEC + 255) / 256;
  const int b = blockIdx.x / tiles, c = (blockIdx.x % tiles * 256 + tid) * VEC;
  int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) slot = -1;
  bool seen = false;   // an earlier row has the slot
  if (a.slots && slot >= 0)
    for (int i = tid; i < b; i += 256) seen |= a.slots[i] == slot;
  if (__syncthreads_or(seen)) slot = -1;
  if (c >= a.C) return;
  P *y = reinterpret_cast<P *>(static_cast<T *>(a.y) + (size_t)b * a.C + c);
  if (slot < 0) {   // no window: a zero output
    *y = P{};
    return;
  }
  T *st = static_cast<T *>(a.state) + (size_t)slot * (W - 1) * a.C + c;
  P in[W];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) in[k] = *reinterpret_cast<const P *>(st + (size_t)k * a.C);
  in[W - 1] = *reinterpret_cast<const P *>(static_cast<const T *>(a.x) + b * a.ld + c);
  float o[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) o[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    float x[VEC];
    widen<VEC, T>(in[k], x);
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] = fmaf(a.weight[(size_t)(c + v) * W + k], x[v], o[v]);
  }
  if (a.silu)
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] = silu<std::is_same<T, __bf16>::value>(o[v]);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) *reinterpret_cast<P *>(st + (size_t)k * a.C) = in[k + 1];
  *y = narrow<VEC, T>(o);
}

// The gradients.  d[t] = dy[t] act'(pre[t]) from the window, as the forward;
//   dx[t] = sum_w weight[w] d[t + W - 1 - w],   dweight[w] = sum_t d[t] x[t - (W - 1) + w],   dbias = sum_t d[t].
// A thread walks its run and the W - 1 tokens behind it, whose d its last dx
// need; the sums of weight and bias take its own tokens only.  They are summed
// over the workgroup's runs in LDS and written as one piece per workgroup; a
// second kernel adds the pieces in a fixed order.
template <int W, int VEC, typename T>
__global__ __launch_bounds__(256, 2) void conv_bwd_kernel(ConvArgs a) {
  using P = typename Pack<T, VEC>::type;
  __shared__ float red[256 * VEC];
  const int tid = threadIdx.x, tiles = (a.C / VEC + a.lanes - 1) / a.lanes;
  const int tile = blockIdx.x % tiles, piece = blockIdx.x / tiles;
  const int c = (tile * a.lanes + (tid & (a.lanes - 1))) * VEC, cc = min(c, a.C - VEC);   // (lanes past the last channel: its rows, not stored)
  const int row = piece / a.runs, per = 256 >> a.lane_bits;
  const int64_t at = (int64_t)(piece % a.runs) * per * a.run + (int64_t)(tid >> a.lane_bits) * a.run;
  const bool on = c < a.C && (at < a.T || at == 0);   // (the first run also of an empty row: it writes dh0)
  float dw[W][VEC] = {}, db[VEC] = {};
  if (on) {
    const int t0 = (int)at, t1 = (int)min((int64_t)a.T, at + a.run), t2 = t1 + W - 1;
    const T *x = static_cast<const T *>(a.x) + (int64_t)row * a.T * a.ld + cc;
    const T *dy = static_cast<const T *>(a.dy) + (int64_t)row * a.T * a.C + cc;
    T *dx = static_cast<T *>(a.dx) + (int64_t)row * a.T * a.C + cc;
    float w[W][VEC], bias[VEC], win[W][VEC], d[W][VEC] = {};   // d[k]: of token t - k
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      bias[i] = a.bias ? a.bias[cc + i] : 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = a.weight[(size_t)(cc + i) * W + k];
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int t = t0 - (W - 1) + k;
      widen<VEC, T>(conv_row<W, VEC, T>(a, x + (int64_t)max(t, 0) * a.ld, row, t, cc), win[k]);
    }
    for (int tb = t0; tb < t2; tb += CONV_BWD_BATCH) {
      P in[CONV_BWD_BATCH], dd[CONV_BWD_BATCH];
#pragma unroll
      for (int i = 0; i < CONV_BWD_BATCH; ++i) {
        const int t = min(min(tb + i, t2 - 1), a.T - 1);
        in[i] = t < 0 ? P{} : *reinterpret_cast<const P *>(x + (int64_t)t * a.ld);
        dd[i] = t < 0 ? P{} : *reinterpret_cast<const P *>(dy + (int64_t)t * a.C);
      }
#pragma unroll
      for (int i = 0; i < CONV_BWD_BATCH; ++i) {
        const int t = tb + i;
        if (t >= t2) break;
#pragma unroll
        for (int v = 0; v < VEC; ++v)
#pragma unroll
          for (int k = W - 1; k > 0; --k) d[k][v] = d[k - 1][v];
        widen<VEC, T>(in[i], win[W - 1]);
        widen<VEC, T>(dd[i], d[0]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          if (a.silu) {
            float s = bias[v], y, g;
#pragma unroll
            for (int k = 0; k < W; ++k) s = fmaf(w[k][v], win[k][v], s);
            silu_grad(s, y, g);
            d[0][v] *= g;
          }
          if (t >= a.T) d[0][v] = 0.f;
          if (t < t1) {
            db[v] += d[0][v];
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][v] = fmaf(d[0][v], win[k][v], dw[k][v]);
          }
#pragma unroll
          for (int k = 0; k < W - 1; ++k) win[k][v] = win[k + 1][v];
        }
        const int to = t - (W - 1);   // its gradient is complete
        if (to < t0 && (t0 || !a.dh0)) continue;
        float o[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          o[v] = 0.f;
#pragma unroll
          for (int k = 0; k < W; ++k) o[v] = fmaf(w[k][v], d[k][v], o[v]);
        }
        if (a.dh_T && to >= a.T - (W - 1)) {
          float e[VEC];
          widen<VEC, T>(*reinterpret_cast<const P *>(static_cast<const T *>(a.dh_T) + ((size_t)row * (W - 1) + to - a.T + W - 1) * a.C + cc), e);
#pragma unroll
          for (int v = 0; v < VEC; ++v) o[v] += e[v];
        }
        T *to_p = to < 0 ? static_cast<T *>(a.dh0) + ((size_t)row * (W - 1) + to + W - 1) * a.C + cc : dx + (int64_t)to * a.C;
        *reinterpret_cast<P *>(to_p) = narrow<VEC, T>(o);
      }
    }
  }
  // red[v][tid]: the workgroup's runs, each sum in turn
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VEC; ++v) red[v * 256 + tid] = k < W ? dw[k < W ? k : 0][v] : db[v];
    __syncthreads();
    for (int i = tid; i < a.lanes * VEC; i += 256) {
      const int v = i & (VEC - 1), l = i / VEC, ch = (tile * a.lanes + l) * VEC + v;
      float s = 0.f;
      for (int r = 0; r < per; ++r) s += red[v * 256 + (r << a.lane_bits) + l];
      if (ch < a.C) a.part[((size_t)piece * (W + 1) + k) * a.C + ch] = s;
    }
  }
}

// The pieces' sums: 64 neighbouring channels of one tap (or of the bias) per
// workgroup, 16 pieces side by side.
__global__ __launch_bounds__(1024) void conv_sum_kernel(const float *part, int pieces, int C, int W, float *dweight, float *dbias) {
  __shared__ double red[16][64];
  const int lane = threadIdx.x & 63, r = threadIdx.x >> 6, tiles = (C + 63) / 64;
  const int k = blockIdx.x / tiles, c = blockIdx.x % tiles * 64 + lane;
  double s = 0.;
  if (c < C)
    for (int p = r; p < pieces; p += 16) s += (double)part[((size_t)p * (W + 1) + k) * C + c];
  red[r][lane] = s;
  __syncthreads();
  if (r || c >= C) return;
  for (int i = 1; i < 16; ++i) s += red[i][lane];
  if (k < W) dweight[(size_t)c * W + k] = (float)s;
  else if (dbias) dbias[c] = (float)s;
}

}  // namespace gdn
