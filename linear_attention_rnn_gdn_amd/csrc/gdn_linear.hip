// gdn_linear.hip -- C ABI of linear attention with a decay per head in
// chunks (declared in include/gdn.h): argument checks, workspace and launches
// on the caller's stream.  No allocation, no synchronisation.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn.h"
#include "gdn_host.h"
#include "gdn_linear.h"

using namespace gdn;

namespace {

// Tokens per segment: about kWalks (segment, value head) walks in all, one per
// compute unit, but at least one chunk of tokens (two for the gradients), in
// multiples of a chunk, and for the gradients kMaxGradSegment at most (the
// decays' gradient is a sum over a segment).  A segment costs the fold's second
// reading of k and v and a state's traffic (64 KB written, read and written by
// the scan, read again); fewer walks leave compute units idle.  Measured, us a
// call, bf16, 64 / 128 / 256 / 512 / 1024 / 2048 tokens per segment:
//   forward, 4096 tokens x 32 heads   170 / 101 /  77 /  74 / 108 / 198 (512: 256 walks)
//   forward, 2 x 8192 x 32            647 / 410 / 305 / 256 / 232 / 233 (2048)
//   forward, 8192 x 4                  55 /  41 /  47 /  65 / 107 / 197 (128)
//   forward, 2048 x 8                  32 /  36 /  42 /  62 / 106 / 128 (64)
//   gradients, 4096 x 32              430 / 312 / 250 / 228 / 252 / 329
//   gradients, 8192 x 4               115 /  89 /  86 / 103 / 163 / 294
//   gradients, 2048 x 8                68 /  59 /  65 /  97 / 160 / 228
// and fp32, 64 / 128 / 256 / 512 (the rule's):
//   forward, 509 x 2                   29 /  40 /  63 /  67 (64)
//   forward, 2 x 1001 x 4              37 /  44 /  64 / 110 (64)
//   forward, 8192 x 4                  68 /  58 /  71 / 113 (128)
//   forward, 4096 x 32                221 / 162 / 139 / 138 (512)
//   gradients, 509 x 2                 34 /  46 /  71 /  83 (64)
//   gradients, 2 x 1001 x 4            58 /  56 /  79 / 129 (64)
//   gradients, 8192 x 4               170 / 138 / 140 / 153 (128)
//   gradients, 4096 x 32              645 / 517 / 448 / 413 (512)
// Known to be slow: forwards whose (row, value head) pairs number 129 to 255.
// Each sequence is then cut into a long and a short segment, and the fold of the
// long one comes before the walks.  Measured, 4096 tokens x 32 heads, this rule /
// two even segments / one: 5 rows 383 / 325 / 268, 6 rows 462 / 336 / 272, 7 rows
// 536 / 365 / 294, 6 rows fp32 924 / 672 / 537 (4 rows, where the rule's two are
// even: 237, one 265).  The gradients hardly differ: 6 rows 1165 / 1165 / 1162.
constexpr int kWalks = 256, kMaxGradSegment = 2048, kFewWalks = 4 * kWalks, kShort = 256, kLdsToBeAlone = 24 << 10;

struct Plan {
  int L, J, nseg;   // tokens per segment, segments per sequence (padded batch), segments in all
};
Plan plan_of(const gdn_linear_shape &s, bool packed, bool grads) {
  const int64_t tokens = packed ? s.T : (int64_t)s.B * s.T;
  const int64_t chunk = s.dtype == GDN_BF16 ? LinTile<__bf16>::C : LinTile<float>::C;
  int64_t L = (tokens * s.H_v + kWalks - 1) / kWalks;
  L = std::max<int64_t>(std::max<int64_t>(64, grads ? 2 * chunk : chunk), (L + 63) / 64 * 64);
  if (grads) L = std::min<int64_t>(L, kMaxGradSegment);
  L = std::min<int64_t>(L, 1 << 30);
  Plan p{};
  p.L = (int)L;
  p.J = s.T > 0 ? (int)((s.T - 1) / L + 1) : 1;
  p.nseg = packed ? (int)(s.T / L + s.B) : s.B * p.J;
  return p;
}

gdn_status validate_linear(const gdn_linear_shape *s, bool packed, bool grads) {
  if (!s) return GDN_ERR_NULL;
  if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (s->o_dtype != GDN_F32 && s->o_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (s->B < 1 || s->T < 0 || s->H_qk < 1 || s->H_v < 1 || s->H_v % s->H_qk) return GDN_ERR_SHAPE;
  if (s->d_k != D || s->d_v != D || (s->g_fixed & ~1)) return GDN_ERR_SHAPE;
  // a launch holds fewer than 2^32 threads: the scan has 16 workgroups of 256 per
  // sequence, value head and role (2 for gradients), the walks one of 512 per
  // segment, value head and role (3)
  if (s->H_v > (1 << 14) || (int64_t)s->B * s->H_v > (1 << 18)) return GDN_ERR_SHAPE;
  // token indexes are 32-bit, and bytes between tokens fit 24
  if (!packed && (int64_t)s->B * s->T > INT32_MAX) return GDN_ERR_SHAPE;
  const Plan p = plan_of(*s, packed, grads);
  if ((int64_t)p.nseg * s->H_v > (1 << 21)) return GDN_ERR_SHAPE;
  return GDN_OK;
}

struct LinLayout {
  size_t tab, seqs, order, add[2], x[2], dec[2], qd, kd, cross, dq, dk, part, total;
};
LinLayout layout_linear(const gdn_linear_shape &s, bool packed, bool grads) {
  const Plan p = plan_of(s, packed, grads);
  const size_t units = (size_t)p.nseg * s.H_v, tokens = packed ? (size_t)s.T : (size_t)s.B * s.T;
  LinLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes);
    return at;
  };
  if (packed) {
    L.tab = take((size_t)p.nseg * sizeof(int4));
    L.seqs = take((size_t)s.B * sizeof(int2));
    L.order = take((size_t)p.nseg * sizeof(int));
  }
  if (s.T > p.L) {
    for (int r = 0; r < (grads ? 2 : 1); ++r) {
      L.add[r] = take(units * D * D * 4);
      L.x[r] = take(units * D * D * 4);
      L.dec[r] = take(units * 4);
    }
  }
  if (grads) {
    L.qd = take(tokens * s.H_v * 4);
    L.kd = take(tokens * s.H_v * 4);
    L.cross = take(units * 4);
    if (s.H_v != s.H_qk) {
      L.dq = take(tokens * s.H_v * D * 4);
      L.dk = take(tokens * s.H_v * D * 4);
    }
    if (s.g_fixed) L.part = take(units * 8);
  }
  L.total = off;
  return L;
}

template <int KIND, int NPO, typename TI, typename TO>
gdn_status launch_walks(const LinArgs &a, hipStream_t st) {
  const int64_t grid = (int64_t)a.nseg * a.Hv * a.roles;
  const unsigned lds = KIND == LIN_FWD && a.alone ? kLdsToBeAlone : 0;
  hipLaunchKernelGGL((linear_kernel<KIND, NPO, TI, TO>), dim3((unsigned)grid), dim3(64 * LIN_NW), lds, st, a);
  return check_launch();
}

// planes of the state and the scores in the outputs' products
template <typename TI, typename TO> constexpr int out_planes() {
  return std::is_same<TI, float>::value || std::is_same<TO, float>::value ? 3 : 2;
}

gdn_status launch_scan(const gdn_linear_shape &s, const ScanArgs &a, hipStream_t st) {
  const int64_t grid = (int64_t)s.B * s.H_v * a.roles * (D * D / 1024);
  hipLaunchKernelGGL(linear_scan_kernel, dim3((unsigned)grid), dim3(256), 0, st, a);
  return check_launch();
}

struct LinCall {
  const gdn_linear_shape &s;
  const int *cu;
  const void *q, *k, *v;
  const float *g, *h0;
  void *o;
  float *h_T;
  char *ws;
  hipStream_t st;

  LinArgs args(const Plan &p, const LinLayout &L) const {
    LinArgs a{};
    a.Hqk = s.H_qk; a.Hv = s.H_v; a.T = s.T;
    a.seg_len = p.L; a.J = p.J; a.nseg = p.nseg;
    // A few walks of packed sequences, whose lengths differ, run one workgroup
    // per compute unit, by LDS asked for and not used: two would share the unit's
    // instruction rate, and the longest first, one at a time, leave the least
    // idle at the end (5 sequences of 1 .. 16000 tokens, 32 heads: 256 us, two
    // per unit in the order of the batch 313; 16 of 1 .. 8192: 737, 760).  Many
    // walks even out by themselves (256 sequences of 1 .. 300: 620 two per unit,
    // 744 alone), and short ones are bound by their states' bytes (24 of
    // 1 .. 200: 61, 70).
    a.alone = cu && (int64_t)p.nseg * s.H_v <= kFewWalks && s.T / kShort >= s.B;
    a.tab = cu ? reinterpret_cast<const int4 *>(ws + L.tab) : nullptr;
    a.order = cu ? reinterpret_cast<const int *>(ws + L.order) : nullptr;
    a.g = g; a.g_fixed = s.g_fixed;
    return a;
  }

  template <typename TI, typename TO> gdn_status run() const {
    constexpr int NPO = out_planes<TI, TO>();
    const Plan p = plan_of(s, cu, false);
    const LinLayout L = layout_linear(s, cu, false);
    const int R = s.H_v / s.H_qk;
    if (cu) {
      hipLaunchKernelGGL(linear_table_kernel, dim3(1), dim3(256), 0, st, cu, s.B, s.T, p.L, p.nseg,
                         reinterpret_cast<int4 *>(ws + L.tab), reinterpret_cast<int2 *>(ws + L.seqs),
                         reinterpret_cast<int *>(ws + L.order));
      GDN_TRY(check_launch());
    }
    LinArgs a = args(p, L);
    a.roles = 1;
    LinRole r{};
    r.b = k; r.gb = R; r.c = v; r.gc = 1; r.a = q; r.ga = R; r.gx = 1;
    if (s.T > p.L) {
      a.role[0] = r;
      a.role[0].fin = reinterpret_cast<float *>(ws + L.add[0]);
      a.role[0].dec = reinterpret_cast<float *>(ws + L.dec[0]);
      GDN_TRY((launch_walks<LIN_FOLD, 1, TI, float>(a, st)));
      ScanArgs sc{};
      sc.Hv = s.H_v; sc.J = p.J; sc.roles = 1;
      sc.seqs = cu ? reinterpret_cast<const int2 *>(ws + L.seqs) : nullptr;
      sc.role[0] = ScanRole{a.role[0].fin, a.role[0].dec, h0, reinterpret_cast<float *>(ws + L.x[0]), 0};
      GDN_TRY(launch_scan(s, sc, st));
      r.seg = sc.role[0].x;
    }
    r.init = h0; r.out = o; r.fin = h_T;
    a.role[0] = r;
    return launch_walks<LIN_FWD, NPO, TI, TO>(a, st);
  }
};

struct LinBwdCall {
  LinCall f;
  const void *dO;
  const float *dh_T;
  void *dq, *dk, *dv;
  float *dg, *dh0;

  template <typename TI> gdn_status run() const {
    const gdn_linear_shape &s = f.s;
    const Plan p = plan_of(s, false, true);
    const LinLayout L = layout_linear(s, false, true);
    const int R = s.H_v / s.H_qk;
    char *ws = f.ws;
    auto fp = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    LinArgs a = f.args(p, L);
    LinRole fw{}, bw{};   // the state's own walk, and its cotangent's
    fw.b = f.k; fw.gb = R; fw.c = f.v; fw.gc = 1; fw.a = f.q; fw.ga = R; fw.gx = 1;
    bw.b = f.q; bw.gb = R; bw.c = dO; bw.gc = 1; bw.a = f.k; bw.ga = R; bw.gx = 1; bw.rev = 1;
    if (s.T > p.L) {
      a.roles = 2;
      a.role[0] = fw; a.role[1] = bw;
      ScanArgs sc{};
      sc.Hv = s.H_v; sc.J = p.J; sc.roles = 2;
      for (int r = 0; r < 2; ++r) {
        a.role[r].fin = fp(L.add[r]);
        a.role[r].dec = fp(L.dec[r]);
        sc.role[r] = ScanRole{fp(L.add[r]), fp(L.dec[r]), r ? dh_T : f.h0, fp(L.x[r]), r};
      }
      GDN_TRY((launch_walks<LIN_FOLD, 1, TI, float>(a, f.st)));
      GDN_TRY(launch_scan(s, sc, f.st));
    }
    const float *sx = s.T > p.L ? fp(L.x[0]) : nullptr, *dx = s.T > p.L ? fp(L.x[1]) : nullptr;
    a.roles = 3;
    const bool shared = s.H_v != s.H_qk;
    LinRole q{}, v{}, k{};
    q.a = dO; q.ga = 1; q.b = f.v; q.gb = 1; q.c = f.k; q.gc = R; q.trans = 1;
    q.init = f.h0; q.seg = sx;
    q.out = shared ? fp(L.dq) : dq; q.out_f32 = shared;
    q.x = f.q; q.gx = R; q.dot = fp(L.qd);
    q.xs = dx; q.xs_last = dh_T; q.cross = fp(L.cross);
    k.a = f.v; k.ga = 1; k.b = dO; k.gb = 1; k.c = f.q; k.gc = R; k.trans = 1; k.rev = 1;
    k.init = dh_T; k.seg = dx;
    k.out = shared ? fp(L.dk) : dk; k.out_f32 = shared;
    k.x = f.k; k.gx = R; k.dot = fp(L.kd);
    v.a = f.k; v.ga = R; v.b = f.q; v.gb = R; v.c = dO; v.gc = 1; v.rev = 1; v.gx = 1;
    v.init = dh_T; v.seg = dx; v.out = dv; v.fin = dh0;
    a.role[0] = q; a.role[1] = k; a.role[2] = v;
    GDN_TRY((launch_walks<LIN_GRAD, 3, TI, TI>(a, f.st)));
    const int64_t units = (int64_t)p.nseg * s.H_v;
    DgArgs d{};
    d.p = a; d.qd = fp(L.qd); d.kd = fp(L.kd); d.cross = fp(L.cross);
    d.dg = s.g_fixed ? nullptr : dg;
    d.part = s.g_fixed ? reinterpret_cast<double *>(ws + L.part) : nullptr;
    hipLaunchKernelGGL(linear_dg_kernel, dim3((unsigned)((units + 3) / 4)), dim3(256), 0, f.st, d);
    GDN_TRY(check_launch());
    if (s.g_fixed) {
      hipLaunchKernelGGL(linear_dg_fixed_kernel, dim3((unsigned)s.H_v), dim3(256), 0, f.st, d.part, dg, p.nseg, s.H_v);
      GDN_TRY(check_launch());
    }
    if (shared && s.T > 0) {
      HeadSumArgs h{};
      h.src[0] = fp(L.dq); h.src[1] = fp(L.dk);
      h.dst[0] = dq; h.dst[1] = dk;
      h.n = (size_t)s.B * s.T * s.H_qk * D / 8;
      h.R = R;
      const unsigned grid = (unsigned)std::min<size_t>((h.n + 255) / 256, 4096);
      hipLaunchKernelGGL(linear_head_sum_kernel<TI>, dim3(grid, 2), dim3(256), 0, f.st, h);
      GDN_TRY(check_launch());
    }
    return GDN_OK;
  }
};

gdn_status linear_fwd(const gdn_linear_shape *s, bool packed, const int32_t *cu, const void *q, const void *k,
                      const void *v, const float *g, const float *h0, void *o, float *h_T, void *ws, size_t ws_bytes,
                      void *hip_stream) {
  GDN_TRY(validate_linear(s, packed, false));
  const size_t need = layout_linear(*s, packed, false).total;
  if (s->T > 0 && (!q || !k || !v || !g || !o)) return GDN_ERR_NULL;
  if ((packed && !cu) || (need && !ws)) return GDN_ERR_NULL;
  if (s->T == 0 && !h_T) return GDN_OK;
  for (const void *p : {(const void *)cu, q, k, v, (const void *)g, (const void *)h0, (const void *)o,
                        (const void *)h_T, (const void *)ws})
    if (misaligned(p)) return GDN_ERR_ALIGN;
  if (ws_bytes < need) return GDN_ERR_WORKSPACE;
  const LinCall f{*s, packed ? cu : nullptr, q, k, v, g, h0, o, h_T, reinterpret_cast<char *>(ws),
                  reinterpret_cast<hipStream_t>(hip_stream)};
  if (s->dtype == GDN_BF16) return s->o_dtype == GDN_BF16 ? f.run<__bf16, __bf16>() : f.run<__bf16, float>();
  return s->o_dtype == GDN_BF16 ? f.run<float, __bf16>() : f.run<float, float>();
}

}  // namespace

extern "C" {

gdn_status gdn_workspace_size_linear(const gdn_linear_shape *s, int32_t kind, size_t *bytes) {
  if (!bytes) return GDN_ERR_NULL;
  if (kind < GDN_LINEAR_FWD || kind > GDN_LINEAR_BWD) return GDN_ERR_SHAPE;
  const bool packed = kind == GDN_LINEAR_VARLEN, grads = kind == GDN_LINEAR_BWD;
  GDN_TRY(validate_linear(s, packed, grads));
  *bytes = layout_linear(*s, packed, grads).total;
  return GDN_OK;
}

gdn_status gdn_linear_chunk_fwd(const gdn_linear_shape *s, const void *q, const void *k, const void *v, const float *g,
                                const float *h0, void *o, float *h_T, void *ws, size_t ws_bytes, void *hip_stream) {
  return linear_fwd(s, false, nullptr, q, k, v, g, h0, o, h_T, ws, ws_bytes, hip_stream);
}

gdn_status gdn_linear_chunk_fwd_varlen(const gdn_linear_shape *s, const int32_t *cu_seqlens, const void *q,
                                       const void *k, const void *v, const float *g, const float *h0, void *o,
                                       float *h_T, void *ws, size_t ws_bytes, void *hip_stream) {
  return linear_fwd(s, true, cu_seqlens, q, k, v, g, h0, o, h_T, ws, ws_bytes, hip_stream);
}

gdn_status gdn_linear_chunk_bwd(const gdn_linear_shape *s, const void *q, const void *k, const void *v, const float *g,
                                const float *h0, const void *dO, const float *dh_T, void *dq, void *dk, void *dv,
                                float *dg, float *dh0, void *ws, size_t ws_bytes, void *hip_stream) {
  GDN_TRY(validate_linear(s, false, true));
  const size_t need = layout_linear(*s, false, true).total;
  if (s->T > 0 && (!q || !k || !v || !g || !dO || !dq || !dk || !dv || !dg)) return GDN_ERR_NULL;
  if ((s->g_fixed && !dg) || (need && !ws)) return GDN_ERR_NULL;
  for (const void *p : {q, k, v, (const void *)g, (const void *)h0, dO, (const void *)dh_T, (const void *)dq,
                        (const void *)dk, (const void *)dv, (const void *)dg, (const void *)dh0, (const void *)ws})
    if (misaligned(p)) return GDN_ERR_ALIGN;
  if (ws_bytes < need) return GDN_ERR_WORKSPACE;
  const LinBwdCall f{LinCall{*s, nullptr, q, k, v, g, h0, nullptr, nullptr, reinterpret_cast<char *>(ws),
                             reinterpret_cast<hipStream_t>(hip_stream)},
                     dO, dh_T, dq, dk, dv, dg, dh0};
  return s->dtype == GDN_BF16 ? f.run<__bf16>() : f.run<float>();
}

}  // extern "C"
