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
// Measured with W = 4 in bf16, 8192 channels: 4096 tokens forward 29 us (134 MB,
// 4.6 TB/s; a large copy reaches 5.0 to 5.2 TB/s here), gradients 50 us and 5 for
// the pieces' sums (202 MB, 3.6 TB/s; the vector ALU is busy 66% of the time),
// one token of 256 rows 9.9 us (34 MB), of 512 rows 13.8 us (67 MB, 4.9 TB/s);
// in fp32 forward 59 us (268 MB, 4.5 TB/s), gradients 91 us with the sums
// (403 MB, 4.4 TB/s, on three waves per SIMD).
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
    for (int i = 0; i < VEC; ++i) p[i] = (T)x[i];
  return p;
}

// A piece at a thread's byte offset from an address of the whole workgroup's.
template <typename P> __device__ __forceinline__ P pick(const void *base, unsigned off) {
  return *reinterpret_cast<const P *>(static_cast<const char *>(base) + off);
}
template <typename P> __device__ __forceinline__ void drop(void *base, unsigned off, const P &p) {
  *reinterpret_cast<P *>(static_cast<char *>(base) + off) = p;
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

// The weights of a workgroup's channels through LDS: they lie as [C][W], and a
// thread's own VEC x W of them, read from memory, would be a line per thread
// and load, many more than all the rest.
template <int W, int VEC> struct Weights {
  static constexpr int OWN = VEC * W, PITCH = OWN % 8 ? OWN : OWN + 4;   // (whole 16 bytes apart, not on the same banks)
  float __attribute__((aligned(16))) lds[64 * PITCH];
  __device__ __forceinline__ void stage(const ConvArgs &a, int first) {   // first channel
    const int n = min(a.lanes * VEC, a.C - first) * W;
    const float *w = a.weight + (size_t)first * W;
    for (int i = threadIdx.x; i < n; i += 256) lds[i / OWN * PITCH + i % OWN] = w[i];
  }
  __device__ __forceinline__ void get(int l, float (&w)[W][VEC]) const {
#pragma unroll
    for (int v = 0; v < VEC; ++v)
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][v] = lds[l * PITCH + v * W + k];
  }
};

constexpr int CONV_OFFSETS = 255, CONV_ONES = 4;
// Rows asked for at once, and again while these are worked on: whole windows,
// which are rings then whose slots are known when the kernel is compiled.
template <int W, int VEC> constexpr int conv_batch() { return (W == 3 ? 3 : 4) * (VEC == 1 ? CONV_ONES : 1); }

template <int W, int VEC, typename T>
__global__ __launch_bounds__(256, 4) void conv_fwd_kernel(ConvArgs a) {
  using P = typename Pack<T, VEC>::type;
  constexpr int BATCH = conv_batch<W, VEC>();
  const int tid = threadIdx.x, tiles = (a.C / VEC + a.lanes - 1) / a.lanes;
  const int tile = blockIdx.x % tiles;
  const int64_t piece = blockIdx.x / tiles;
  const int c = (tile * a.lanes + (tid & (a.lanes - 1))) * VEC;
  const int rows = a.cu ? 1 : a.B;
  __shared__ Weights<W, VEC> all;
  __shared__ int offsets[CONV_OFFSETS + 1];   // of the first packed sequences (all of them, mostly)
  all.stage(a, tile * a.lanes * VEC);
  if (a.cu)
    for (int i = tid; i <= min(a.B, CONV_OFFSETS); i += 256) offsets[i] = offset_at(a.cu, i, a.T);
  __syncthreads();
  auto offset = [&](int s) { return s <= CONV_OFFSETS ? offsets[s] : offset_at(a.cu, s, a.T); };
  if (c >= a.C) return;
  if (piece >= (int64_t)rows * a.runs) {   // the windows behind the sequences
    const int per = 256 >> a.lane_bits;
    const int64_t i = (piece - (int64_t)rows * a.runs) * per + (tid >> a.lane_bits);
    if (i >= (int64_t)a.B * (W - 1)) return;
    const int s = (int)(i / (W - 1)), j = (int)(i % (W - 1));
    int begin = 0, end = a.T;
    int64_t row = (int64_t)s * a.T;
    if (a.cu) {
      begin = offset(s);
      end = max(begin, offset(s + 1));
      row = 0;
    }
    const int t = end - (W - 1) + j;
    const T *x = static_cast<const T *>(a.x) + (row + max(t, 0)) * a.ld + c;
    *reinterpret_cast<P *>(static_cast<T *>(a.h_T) + (size_t)i * a.C + c) = conv_row<W, VEC, T>(a, x, s, t - begin, c);
    return;
  }
  const int row = (int)(piece / a.runs);
  const int64_t first = (piece % a.runs) * (256 >> a.lane_bits) * a.run, at = first + (tid >> a.lane_bits) * a.run;
  if (at >= a.T) return;
  const int t0 = (int)at, t1 = (int)min((int64_t)a.T, at + a.run);
  Sequence q{row, 0, a.T};
  const T *x = static_cast<const T *>(a.x) + (int64_t)row * a.T * a.ld + c;
  // rows from the workgroup's first token on, at 32-bit offsets of this thread's
  const T *xb = static_cast<const T *>(a.x) + ((int64_t)row * a.T + first) * a.ld;
  T *yb = static_cast<T *>(a.y) + ((int64_t)row * a.T + first) * a.C;
  const unsigned step = (unsigned)(a.ld * sizeof(T)), last = (unsigned)(t1 - 1 - first) * step + c * (unsigned)sizeof(T);
  unsigned xo = (unsigned)(t0 - first) * step + c * (unsigned)sizeof(T);
  unsigned yo = ((unsigned)(t0 - first) * a.C + c) * (unsigned)sizeof(T);
  float w[W][VEC], bias[VEC], win[W][VEC];   // token t's x: slot (t - t0) % W
  all.get(tid & (a.lanes - 1), w);
#pragma unroll
  for (int i = 0; i < VEC; ++i) bias[i] = a.bias ? a.bias[c + i] : 0.f;
  P in[BATCH], next[BATCH];
  auto ask = [&](P(&in)[BATCH]) {   // the next tokens (past the run's last: that one)
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      in[i] = pick<P>(xb, min(xo, last));
      xo += step;
    }
  };
  ask(in);
  if (a.cu) q = sequence_at(offset, a.B, a.T, t0, 0);
#pragma unroll
  for (int k = 1; k < W; ++k) {
    const int t = t0 + k - W;
    widen<VEC, T>(conv_row<W, VEC, T>(a, x + (int64_t)max(t, 0) * a.ld, q.seq, t - q.begin, c), win[k]);
  }
  auto token = [&](int i) {
    widen<VEC, T>(in[i], win[i % W]);
    float o[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      float s = bias[v];
#pragma unroll
      for (int k = 0; k < W; ++k) s = fmaf(w[k][v], win[(i + 1 + k) % W][v], s);
      o[v] = a.silu ? silu<true>(s) : s;
    }
    drop<P>(yb, yo, narrow<VEC, T>(o));
    yo += a.C * (unsigned)sizeof(T);
  };
  for (int tb = t0; tb < t1; tb += BATCH) {
    ask(next);
    // Nothing ends among them: mostly, and worth code of its own where a batch is
    // a dozen tokens or so of one channel (61 MB packed, fp32: 17.8 us, 19.7
    // without); of a pack it would take more registers than four waves have.
    if (VEC == 1 && !__any(tb + BATCH > t1 || (q.end > t0 && q.end < tb + BATCH))) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) token(i);
    } else {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        if (tb + i >= t1) break;
        if (tb + i == q.end) {   // packed: the next sequence
          q = sequence_at(offset, a.B, a.T, tb + i, q.seq + 1);
#pragma unroll
          for (int k = 0; k < W - 1; ++k) widen<VEC, T>(conv_row<W, VEC, T>(a, x, q.seq, k - (W - 1), c), win[(i + 1 + k) % W]);
        }
        token(i);
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) in[i] = next[i];
  }
}

// One token of every row: the row's window in the pool [n_slots, W - 1, C]
// moves on by one token.  A thread takes its channels of ROWS rows, which share
// the reads of the weights (all of a thread's own, and so a line each).
template <int W, int VEC, int ROWS, typename T>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a) {
  using P = typename Pack<T, VEC>::type;
  const int tid = threadIdx.x, tiles = (a.C / VEC + 255) / 256;
  const int b0 = blockIdx.x / tiles * ROWS, to = (blockIdx.x % tiles * 256 + tid) * VEC, c = min(to, a.C - VEC);
  // Everything is asked for before the other rows' slots are looked at (a row
  // without a slot reads some window, and leaves it).
  int slot[ROWS];
  P in[ROWS][W];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int b = min(b0 + r, a.B - 1);
    slot[r] = a.slots ? a.slots[b] : b;
    if (slot[r] < 0 || slot[r] >= a.n_slots) slot[r] = -1;
    const T *st = static_cast<const T *>(a.state) + (size_t)max(slot[r], 0) * (W - 1) * a.C + c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[r][k] = *reinterpret_cast<const P *>(st + (size_t)k * a.C);
    in[r][W - 1] = *reinterpret_cast<const P *>(static_cast<const T *>(a.x) + b * a.ld + c);
  }
  float w[W][VEC], bias[VEC];
  const float *wp = a.weight + (size_t)c * W;
  if constexpr (VEC == 1) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][0] = wp[k];
  } else {
#pragma unroll
    for (int i = 0; i < VEC * W; i += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(wp + i);
      w[i % W][i / W] = v.x;
      w[(i + 1) % W][(i + 1) / W] = v.y;
      w[(i + 2) % W][(i + 2) / W] = v.z;
      w[(i + 3) % W][(i + 3) / W] = v.w;
    }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) bias[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    bool seen = false;   // an earlier row has the slot
    if (a.slots && slot[r] >= 0)
      for (int i = tid; i < b0 + r; i += 256) seen |= a.slots[i] == slot[r];
    if (__syncthreads_or(seen)) slot[r] = -1;
  }
  if (to >= a.C) return;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (b0 + r >= a.B) return;
    P *y = reinterpret_cast<P *>(static_cast<T *>(a.y) + (size_t)(b0 + r) * a.C + c);
    if (slot[r] < 0) {   // no window: a zero output
      *y = P{};
      continue;
    }
    float o[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] = bias[v];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      float x[VEC];
      widen<VEC, T>(in[r][k], x);
#pragma unroll
      for (int v = 0; v < VEC; ++v) o[v] = fmaf(w[k][v], x[v], o[v]);
    }
    if (a.silu)
#pragma unroll
      for (int v = 0; v < VEC; ++v) o[v] = silu<true>(o[v]);
    T *st = static_cast<T *>(a.state) + (size_t)slot[r] * (W - 1) * a.C + c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) *reinterpret_cast<P *>(st + (size_t)k * a.C) = in[r][k + 1];
    *y = narrow<VEC, T>(o);
  }
}

// The gradients.  d[t] = dy[t] act'(pre[t]) from the window, as the forward;
//   dx[t] = sum_w weight[w] d[t + W - 1 - w],   dweight[w] = sum_t d[t] x[t - (W - 1) + w],   dbias = sum_t d[t].
// A thread walks its run and the W - 1 tokens behind it, whose d its last dx
// need; the sums of weight and bias take its own tokens only.  They are summed
// over the workgroup's runs in LDS and written as one piece per workgroup; a
// second kernel adds the pieces in a fixed order.
// Tokens go by W at a time, so that the windows of x and d are rings whose
// slots are known when the kernel is compiled and nothing is moved; the rows of
// the next W tokens are on their way meanwhile.
template <int W, int VEC, typename T>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 4 : 3) void conv_bwd_kernel(ConvArgs a) {
  using P = typename Pack<T, VEC>::type;
  __shared__ float red[256 * VEC];
  const int tid = threadIdx.x, tiles = (a.C / VEC + a.lanes - 1) / a.lanes;
  const int tile = blockIdx.x % tiles, piece = blockIdx.x / tiles;
  const int c = (tile * a.lanes + (tid & (a.lanes - 1))) * VEC, cc = min(c, a.C - VEC);   // (lanes past the last channel: its rows, not stored)
  const int row = piece / a.runs, per = 256 >> a.lane_bits;
  const int64_t first = (int64_t)(piece % a.runs) * per * a.run, at = first + (tid >> a.lane_bits) * a.run;
  const bool on = c < a.C && (at < a.T || at == 0);   // (the first run also of an empty row: it writes dh0)
  float dw[W][VEC] = {}, db[VEC] = {};
  __shared__ Weights<W, VEC> all;
  all.stage(a, tile * a.lanes * VEC);
  __syncthreads();
  if (on) {
    const int t0 = (int)at;
    const T *x = static_cast<const T *>(a.x) + (int64_t)row * a.T * a.ld + cc;
    // rows from the workgroup's first token on, at 32-bit offsets of this thread's (none of an empty row)
    const T *xb = static_cast<const T *>(a.x) + ((int64_t)row * a.T + first) * a.ld;
    const T *db_ = static_cast<const T *>(a.dy) + ((int64_t)row * a.T + first) * a.C;
    T *dxb = static_cast<T *>(a.dx) + ((int64_t)row * a.T + first) * a.C;
    const unsigned e = sizeof(T), xs = (unsigned)a.ld * e, ys = (unsigned)a.C * e, co = cc * e;
    const unsigned here = (unsigned)(t0 - first), left = (unsigned)min(a.T - 1 - t0, a.run + 2 * W);   // tokens behind t0 in the row
    const unsigned xlast = (here + left) * xs + co, ylast = (here + left) * ys + co;
    unsigned xo = here * xs + co, yo = here * ys + co, out = yo - (W - 1) * ys;
    float w[W][VEC], bias[VEC], win[W][VEC], d[W][VEC] = {};   // token t's x and d: slot (t - t0) % W
    all.get(tid & (a.lanes - 1), w);
#pragma unroll
    for (int i = 0; i < VEC; ++i) bias[i] = a.bias ? a.bias[cc + i] : 0.f;
    P in[W], dd[W], in_next[W], dd_next[W];
    auto ask = [&](P(&in)[W], P(&dd)[W]) {   // the next W tokens (past the last: that one)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        in[i] = a.T ? pick<P>(xb, min(xo, xlast)) : P{};
        dd[i] = a.T ? pick<P>(db_, min(yo, ylast)) : P{};
        xo += xs;
        yo += ys;
      }
    };
    ask(in, dd);
#pragma unroll
    for (int k = 1; k < W; ++k)
      widen<VEC, T>(conv_row<W, VEC, T>(a, x + (int64_t)max(t0 + k - W, 0) * a.ld, row, t0 + k - W, cc), win[k]);
    for (int r = 0; r <= a.run; r += W) {   // (run is a multiple of W: the last time the W - 1 tokens behind it)
      if (t0 + r >= a.T + W - 1) break;
      const bool own = r < a.run;
      ask(in_next, dd_next);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (i == W - 1 && !own) break;
        const int t = t0 + r + i;
        widen<VEC, T>(in[i], win[i]);
        widen<VEC, T>(dd[i], d[i]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          if (a.silu) {
            float s = bias[v], y, g;
#pragma unroll
            for (int k = 0; k < W; ++k) s = fmaf(w[k][v], win[(i + 1 + k) % W][v], s);
            silu_grad<true>(s, y, g);
            d[i][v] *= g;
          }
          d[i][v] = t < a.T ? d[i][v] : 0.f;
        }
        if (own && t < a.T)   // (none past the last: x there is the last token's again, and zero times that may be no number)
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            db[v] += d[i][v];
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][v] = fmaf(d[i][v], win[(i + 1 + k) % W][v], dw[k][v]);
          }
        const int to = t - (W - 1);   // its gradient is complete
        const unsigned off = out;
        out += ys;
        if (r + i < W - 1 ? t0 || !a.dh0 : to >= a.T) continue;   // (an earlier run's, or none)
        float o[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          o[v] = 0.f;
#pragma unroll
          for (int k = 0; k < W; ++k) o[v] = fmaf(w[k][v], d[(i - k + W) % W][v], o[v]);
        }
        if (a.dh_T && to >= a.T - (W - 1)) {
          float g[VEC];
          widen<VEC, T>(*reinterpret_cast<const P *>(static_cast<const T *>(a.dh_T) + ((size_t)row * (W - 1) + to - a.T + W - 1) * a.C + cc), g);
#pragma unroll
          for (int v = 0; v < VEC; ++v) o[v] += g[v];
        }
        if (to < 0) *reinterpret_cast<P *>(static_cast<T *>(a.dh0) + ((size_t)row * (W - 1) + to + W - 1) * a.C + cc) = narrow<VEC, T>(o);
        else drop<P>(dxb, off, narrow<VEC, T>(o));
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        in[i] = in_next[i];
        dd[i] = dd_next[i];
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
