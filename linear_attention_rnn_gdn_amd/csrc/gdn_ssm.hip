// gdn_ssm.hip -- C ABI of the selective state space scan (declared in
// include/gdn.h): argument checks, workspace and launches on the caller's
// stream.  No allocation, no synchronisation.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn.h"
#include "gdn_host.h"
#include "gdn_ssm.h"

using namespace gdn;

namespace {

constexpr int64_t kMaxWaves = 1ll << 25;   // a launch holds fewer than 2^32 threads
// Segments of a forward pass: as many as give 4096 walks, four per SIMD.  At
// 4096 tokens of 4096 channels with 16 states, and at 12 packed sequences (9925
// tokens) of 2000 channels, 1024 walks took 232 and 284 us, 2048 155 and 190, 4096 139 and
// 175, 8192 152 and 189 (a segment more costs its state's two passes).
constexpr int kWaves = 4096;
// ... of 16 tokens or more: 8, 16, 32 and 64 took 18, 22, 32 and 55 us at 512
// tokens of 512 channels, 47, 37, 38 and 57 at 2048 tokens of them, and 104, 64,
// 53 and 64 at 8192 tokens of 64.
constexpr int kShortest = 16;
// Segments of the gradients have 8, 16, 32 or 64 tokens, by the waves that 32
// would give: fewer than 256, than 1536, than 8192, or more.  Measured, in us:
//   waves of 32 tokens (T x C)      8     16     32     64
//      128   (512 x 512)           41     46     73    131
//      512   (2048 x 512)          72     64     83    139
//     1344   (2048 x 1344)        131    110    116    152
//     2048   (2048 x 2048)        170    140    122    155
//     4096   (2048 x 4096)        333    258    228    232
//     7168   (4096 x 3584)        584    441    387    393
//     8192   (8192 x 2048)        720    513    448    413
// (Short ones fill the chip, long ones need fewer passes over a state.)
constexpr int kFewest = 256, kFew = 1536, kMany = 8192;

int elem(const gdn_ssm_shape &s) { return s.dtype == GDN_BF16 ? 2 : 4; }
int64_t ld(int32_t given, int64_t dense) { return given ? given : dense; }

gdn_status validate_ssm(const gdn_ssm_shape *s) {
  if (!s) return GDN_ERR_NULL;
  if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (s->o_dtype != GDN_F32 && s->o_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (s->B < 1 || s->T < 0 || s->T > 1 << 30 || s->C < 1 || s->C > 1 << 20 || s->G < 1 || s->C % s->G) return GDN_ERR_SHAPE;
  if ((s->N != 8 && s->N != 16 && s->N != 32) || (s->softplus & ~1)) return GDN_ERR_SHAPE;
  for (int32_t l : {s->ld_x, s->ld_dt, s->ld_z})
    if (l && l < s->C) return GDN_ERR_SHAPE;
  // rows of B and C are read in whole words
  for (int32_t l : {s->ld_b, s->ld_c})
    if (l && ((int64_t)l < (int64_t)s->G * s->N || (int64_t)l * elem(*s) % 16)) return GDN_ERR_SHAPE;
  return GDN_OK;
}

gdn_status aligned(const gdn_ssm_shape &s, std::initializer_list<const void *> elements, std::initializer_list<const void *> wide) {
  for (const void *p : elements)
    if (p && (uintptr_t)p % elem(s)) return GDN_ERR_ALIGN;
  for (const void *p : wide)
    if (misaligned(p)) return GDN_ERR_ALIGN;
  return GDN_OK;
}

SsmArgs ssm_args(const gdn_ssm_shape &s, bool packed) {
  SsmArgs a{};
  a.B = s.B; a.T = s.T; a.C = s.C; a.N = s.N; a.G = s.G; a.n_slots = s.n_slots; a.softplus = s.softplus;
  a.ld_x = ld(s.ld_x, s.C); a.ld_dt = ld(s.ld_dt, s.C); a.ld_z = ld(s.ld_z, s.C);
  a.ld_b = ld(s.ld_b, (int64_t)s.G * s.N); a.ld_c = ld(s.ld_c, (int64_t)s.G * s.N);
  a.rows = packed ? 1 : s.B;
  a.per = (s.C / s.G + 63) / 64;
  a.tiles = a.per * s.G;
  return a;
}

template <typename F>
gdn_status with_states(int N, F &&f) {
  return N == 8 ? f(std::integral_constant<int, 8>{}) : N == 16 ? f(std::integral_constant<int, 16>{}) : f(std::integral_constant<int, 32>{});
}
template <typename F>
gdn_status with_types(const gdn_ssm_shape &s, F &&f) {
  if (s.dtype == GDN_BF16) return s.o_dtype == GDN_BF16 ? f(__bf16{}, __bf16{}) : f(__bf16{}, float{});
  return s.o_dtype == GDN_BF16 ? f(float{}, __bf16{}) : f(float{}, float{});
}

// Tokens per segment, segments per row, and where the workspace's pieces lie.
struct Layout {
  int len, J, marks;
  size_t end, in, sum, fresh, rend, rin, mark, mark_sum, part_bc, part_a, total;
};
Layout layout_ssm(const gdn_ssm_shape &s, const SsmArgs &a, bool grads) {
  Layout l{};
  if ((int64_t)a.rows * a.tiles > kMaxWaves) return l;   // (refused by check_sizes: the products below would not fit)
  if (grads) {
    const int64_t waves = (int64_t)a.rows * a.tiles * ((s.T + 31) / 32) * (s.N > 16 ? 2 : 1);
    l.len = waves < kFewest ? 8 : waves < kFew ? 16 : waves < kMany ? 32 : 64;
    l.J = std::max(1, (s.T + l.len - 1) / l.len);
    const int piece = s.N == 8 ? SsmBwd<8>::S : SsmBwd<16>::S;
    l.marks = l.len / piece - 1;
  } else {
    const int64_t walks = (int64_t)a.rows * a.tiles, want = std::max<int64_t>(1, kWaves / walks);
    const int64_t len = (s.T + want - 1) / want;
    l.len = (int)std::max<int64_t>(kShortest, (len + WALK_BATCH - 1) / WALK_BATCH * WALK_BATCH);
    l.J = (int)(((int64_t)s.T + l.len - 1) / l.len);
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes);
    return at;
  };
  const size_t units = (size_t)a.rows * l.J, states = units * a.tiles * s.N * 64 * 4;
  if (l.J > 1 || grads) {
    l.end = take(states);
    l.in = take(states);
    l.sum = take(units * a.tiles * 64 * 4);
    l.fresh = take(units * 4);
    if (grads) {
      l.rend = take(states);
      l.rin = take(states);
    }
  }
  if (grads) {
    l.mark = take(states * l.marks);
    l.mark_sum = take(units * l.marks * a.tiles * 64 * 4);
    l.part_bc = take((size_t)s.B * s.T * a.tiles * 2 * s.N * 4);
    l.part_a = take(units * (s.N + 2) * s.C * 4);
  }
  l.total = off;
  return l;
}
gdn_status check_sizes(const gdn_ssm_shape &s, const SsmArgs &a, const Layout &l) {
  if ((int64_t)a.rows * a.tiles > kMaxWaves) return GDN_ERR_SHAPE;
  if (((int64_t)a.rows * l.J + s.B) * a.tiles * (s.N > 16 ? 2 : 1) > kMaxWaves) return GDN_ERR_SHAPE;
  if ((int64_t)a.rows * a.tiles * s.N > kMaxWaves / 8) return GDN_ERR_SHAPE;
  return GDN_OK;
}
void place(SsmArgs &a, const Layout &l, void *ws) {
  char *p = static_cast<char *>(ws);
  a.len = l.len; a.J = l.J; a.marks = l.marks;
  a.mark = reinterpret_cast<float *>(p + l.mark); a.mark_sum = reinterpret_cast<float *>(p + l.mark_sum);
  a.end = reinterpret_cast<float *>(p + l.end); a.in = reinterpret_cast<float *>(p + l.in);
  a.sum = reinterpret_cast<float *>(p + l.sum); a.fresh = reinterpret_cast<int *>(p + l.fresh);
  a.rend = reinterpret_cast<float *>(p + l.rend); a.rin = reinterpret_cast<float *>(p + l.rin);
  a.part_bc = reinterpret_cast<float *>(p + l.part_bc); a.part_a = reinterpret_cast<float *>(p + l.part_a);
}
unsigned scan_blocks(const SsmArgs &a) { return (unsigned)((int64_t)a.rows * a.tiles * a.N); }

gdn_status ssm_fwd(const gdn_ssm_shape *s, bool packed, const int32_t *cu, const gdn_ssm_inputs *in, const float *h0, void *y, float *h_T,
                   void *ws, size_t ws_bytes, void *hip_stream) {
  GDN_TRY(validate_ssm(s));
  if (!in || !in->A || (packed && !cu)) return GDN_ERR_NULL;
  if (s->T > 0 && (!in->x || !in->dt || !in->B || !in->C || !y)) return GDN_ERR_NULL;
  SsmArgs a = ssm_args(*s, packed);
  const Layout l = layout_ssm(*s, a, false);
  GDN_TRY(check_sizes(*s, a, l));
  GDN_TRY(aligned(*s, {in->x, in->dt, in->z}, {in->B, in->C, in->A, h0, y, h_T, ws}));
  for (const void *p : {(const void *)in->D, (const void *)in->dt_bias, (const void *)cu})
    if (p && (uintptr_t)p % 4) return GDN_ERR_ALIGN;
  if (s->T == 0 && !h_T) return GDN_OK;
  if (l.total && !ws) return GDN_ERR_NULL;
  if (ws_bytes < l.total) return GDN_ERR_WORKSPACE;
  place(a, l, ws);
  a.cu = packed ? cu : nullptr;
  a.x = in->x; a.dt = in->dt; a.z = in->z; a.Bm = in->B; a.Cm = in->C; a.A = in->A; a.D = in->D; a.dt_bias = in->dt_bias;
  a.h0 = h0; a.y = y; a.h_T = h_T;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  const int64_t walks = (int64_t)a.rows * l.J, extra = h_T && (packed || s->T == 0) ? s->B : 0;
  return with_states(s->N, [&](auto n) -> gdn_status {
    constexpr int N = decltype(n)::value;
    return with_types(*s, [&](auto ti, auto to) -> gdn_status {
      using TI = decltype(ti);
      using TO = decltype(to);
      if (l.J > 1) {
        hipLaunchKernelGGL((ssm_walk_kernel<N, TI, float, true>), dim3((unsigned)(walks * a.tiles)), dim3(64), 0, st, a);
        GDN_TRY(check_launch());
        hipLaunchKernelGGL(ssm_scan_kernel<N>, dim3(scan_blocks(a)), dim3(256), 0, st, a);
        GDN_TRY(check_launch());
      }
      hipLaunchKernelGGL((ssm_walk_kernel<N, TI, TO, false>), dim3((unsigned)((walks + extra) * a.tiles)), dim3(64), 0, st, a);
      return check_launch();
    });
  });
}

}  // namespace

extern "C" {

gdn_status gdn_workspace_size_ssm(const gdn_ssm_shape *s, int32_t kind, size_t *bytes) {
  if (!bytes) return GDN_ERR_NULL;
  if (kind < GDN_SSM_FWD || kind > GDN_SSM_BWD) return GDN_ERR_SHAPE;
  GDN_TRY(validate_ssm(s));
  const SsmArgs a = ssm_args(*s, kind == GDN_SSM_VARLEN);
  const Layout l = layout_ssm(*s, a, kind == GDN_SSM_BWD);
  GDN_TRY(check_sizes(*s, a, l));
  *bytes = l.total;
  return GDN_OK;
}

gdn_status gdn_ssm_fwd(const gdn_ssm_shape *s, const gdn_ssm_inputs *in, const float *h0, void *y, float *h_T, void *ws, size_t ws_bytes,
                       void *hip_stream) {
  return ssm_fwd(s, false, nullptr, in, h0, y, h_T, ws, ws_bytes, hip_stream);
}

gdn_status gdn_ssm_fwd_varlen(const gdn_ssm_shape *s, const int32_t *cu_seqlens, const gdn_ssm_inputs *in, const float *h0, void *y,
                              float *h_T, void *ws, size_t ws_bytes, void *hip_stream) {
  return ssm_fwd(s, true, cu_seqlens, in, h0, y, h_T, ws, ws_bytes, hip_stream);
}

gdn_status gdn_ssm_step(const gdn_ssm_shape *s, const gdn_ssm_inputs *in, const int32_t *slots, float *state, void *y, void *hip_stream) {
  GDN_TRY(validate_ssm(s));
  if (s->T != 1 || s->n_slots < 1 || (!slots && s->n_slots < s->B)) return GDN_ERR_SHAPE;
  if (!in || !in->A || !in->x || !in->dt || !in->B || !in->C || !state || !y) return GDN_ERR_NULL;
  GDN_TRY(aligned(*s, {in->x, in->dt, in->z}, {in->B, in->C, in->A, state, y}));
  for (const void *p : {(const void *)in->D, (const void *)in->dt_bias, (const void *)slots})
    if (p && (uintptr_t)p % 4) return GDN_ERR_ALIGN;
  SsmArgs a = ssm_args(*s, false);
  const int64_t blocks = (int64_t)s->B * (((int64_t)s->C * (s->N / 4) + 255) / 256);
  if (blocks > kMaxWaves / 4) return GDN_ERR_SHAPE;
  a.x = in->x; a.dt = in->dt; a.z = in->z; a.Bm = in->B; a.Cm = in->C; a.A = in->A; a.D = in->D; a.dt_bias = in->dt_bias;
  a.slots = slots; a.state = state; a.y = y;
  return with_states(s->N, [&](auto n) -> gdn_status {
    constexpr int N = decltype(n)::value;
    return with_types(*s, [&](auto ti, auto to) -> gdn_status {
      hipLaunchKernelGGL((ssm_step_kernel<N, decltype(ti), decltype(to)>), dim3((unsigned)blocks), dim3(256), 0,
                         reinterpret_cast<hipStream_t>(hip_stream), a);
      return check_launch();
    });
  });
}

gdn_status gdn_ssm_bwd(const gdn_ssm_shape *s, const gdn_ssm_inputs *in, const float *h0, const void *dy, const float *dh_T,
                       const gdn_ssm_grads *out, void *ws, size_t ws_bytes, void *hip_stream) {
  GDN_TRY(validate_ssm(s));
  if (!in || !out || !in->A || !out->dA || !ws) return GDN_ERR_NULL;
  if (s->T > 0 && (!in->x || !in->dt || !in->B || !in->C || !dy || !out->dx || !out->ddt || !out->dB || !out->dC)) return GDN_ERR_NULL;
  if (s->T > 0 && in->z && !out->dz) return GDN_ERR_NULL;
  SsmArgs a = ssm_args(*s, false);
  const Layout l = layout_ssm(*s, a, true);
  GDN_TRY(check_sizes(*s, a, l));
  const int64_t tokens = (int64_t)s->B * s->T, bc = (tokens * s->G + 3) / 4;
  if (bc > kMaxWaves / 4) return GDN_ERR_SHAPE;
  GDN_TRY(aligned(*s, {in->x, in->dt, in->z, dy, out->dx, out->ddt, out->dz}, {in->B, in->C, in->A, h0, dh_T, out->dB, out->dC, out->dA, out->dh0, ws}));
  for (const void *p : {(const void *)in->D, (const void *)in->dt_bias, (const void *)out->dD, (const void *)out->ddt_bias})
    if (p && (uintptr_t)p % 4) return GDN_ERR_ALIGN;
  if (ws_bytes < l.total) return GDN_ERR_WORKSPACE;
  place(a, l, ws);
  a.x = in->x; a.dt = in->dt; a.z = in->z; a.Bm = in->B; a.Cm = in->C; a.A = in->A; a.D = in->D; a.dt_bias = in->dt_bias;
  a.h0 = h0; a.dy = dy; a.dh_T = dh_T; a.dx = out->dx; a.ddt = out->ddt; a.dz = out->dz; a.dh0 = out->dh0;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  const unsigned walks = (unsigned)((int64_t)a.rows * l.J * a.tiles);
  return with_states(s->N, [&](auto n) -> gdn_status {
    constexpr int N = decltype(n)::value;
    auto run = [&](auto ti) -> gdn_status {
      using TI = decltype(ti);
      if (s->T > SsmBwd<N>::S) {   // (one piece needs no marks)
        hipLaunchKernelGGL((ssm_bwd_fold_kernel<N, TI>), dim3(walks), dim3(64), 0, st, a);
        GDN_TRY(check_launch());
      }
      if (l.J > 1) {
        hipLaunchKernelGGL(ssm_scan_kernel<N>, dim3(2 * scan_blocks(a)), dim3(256), 0, st, a);
        GDN_TRY(check_launch());
      }
      hipLaunchKernelGGL((ssm_bwd_kernel<N, TI>), dim3(walks), dim3(64 * SsmBwd<N>::WAVES), 0, st, a);
      GDN_TRY(check_launch());
      const int64_t sums = (int64_t)(N + 2) * ((s->C + 63) / 64) + bc;
      hipLaunchKernelGGL((ssm_sum_kernel<N, TI>), dim3((unsigned)sums), dim3(256), 0, st, a, out->dA, out->dD, out->ddt_bias,
                         static_cast<TI *>(out->dB), static_cast<TI *>(out->dC), tokens);
      return check_launch();
    };
    return s->dtype == GDN_BF16 ? run(__bf16{}) : run(float{});
  });
}

}  // extern "C"
