// gdn_states.hip -- C ABI of the operators on a pool of recurrent states
// (declared in include/gdn.h): argument checks and launches on the caller's
// stream.  No workspace, no allocation, no synchronisation.
#include <hip/hip_runtime.h>

#include "gdn.h"
#include "gdn_host.h"
#include "gdn_states.h"

using namespace gdn;

namespace {

constexpr int64_t kMemoryCache = 256 << 20;   // bytes of the memory-side cache
constexpr int kMaxNodes = 64;   // tree nodes per row: one per lane of a wave

gdn_status validate_pool(const gdn_pool_shape *s, bool slots) {
  if (!s) return GDN_ERR_NULL;
  if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (s->o_dtype != GDN_F32 && s->o_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (s->B < 1 || s->n < 1 || s->n > kMaxNodes || s->H_qk < 1 || s->H_v < 1 || s->H_v % s->H_qk) return GDN_ERR_SHAPE;
  if (s->d_k != D || s->d_v != D || s->n_slots < 1 || (s->g_fixed & ~1)) return GDN_ERR_SHAPE;
  if (!slots && s->n_slots < s->B) return GDN_ERR_SHAPE;
  // a launch holds fewer than 2^32 threads: at most 2 workgroups of 256 per state here
  if ((int64_t)s->B * s->H_v > (1 << 22)) return GDN_ERR_SHAPE;
  return GDN_OK;
}

StateArgs pool_args(const gdn_pool_shape &s) {
  StateArgs a{};
  a.B = s.B; a.n = s.n; a.Hqk = s.H_qk; a.Hv = s.H_v; a.n_slots = s.n_slots; a.g_fixed = s.g_fixed;
  a.stream = (int64_t)s.B * s.H_v * D * D * 4 > kMemoryCache;
  return a;
}

// Columns of a state per workgroup of the step and of the commit: a quarter of
// a state where a call has few, to spread them over the chip, half of one else.
// Measured, us a call with 16 / 32 / 64 / 128 columns per workgroup (step;
// commit of 6 nodes), bf16:
//     32 states   4.0 /  4.0 /  4.2 /  4.7;   4.8 /  5.0 /  5.4 /  6.3
//    128 states   6.3 /  5.3 /  5.3 /  5.7;   7.0 /  6.4 /  6.5 /  7.3
//    512 states  15.1 / 10.4 / 10.3 / 10.0;  16.8 / 13.6 / 12.6 / 12.7
//   2048 states  47.9 / 42.5 / 41.0 / 41.9;  50.4 / 44.9 / 44.3 / 44.6
bool quarter_states(const gdn_pool_shape &s) { return (int64_t)s.B * s.H_v < 128; }

template <typename F>
gdn_status with_types(const gdn_pool_shape &s, F &&f) {
  if (s.dtype == GDN_BF16)
    return s.o_dtype == GDN_BF16 ? f(__bf16{}, __bf16{}) : f(__bf16{}, float{});
  return s.o_dtype == GDN_BF16 ? f(float{}, __bf16{}) : f(float{}, float{});
}

template <int COLS, typename TI, typename TO>
gdn_status launch_step(const StateArgs &a, hipStream_t st) {
  hipLaunchKernelGGL((step_kernel<COLS, TI, TO>), dim3((unsigned)((int64_t)a.B * a.Hv * (D / COLS))), dim3(256), 0, st, a);
  return check_launch();
}

template <int COLS, typename TI>
gdn_status launch_commit(const StateArgs &a, hipStream_t st) {
  hipLaunchKernelGGL((tree_commit_kernel<COLS, TI>), dim3((unsigned)((int64_t)a.B * a.Hv * (D / COLS))), dim3(256), 0, st, a);
  return check_launch();
}

// Two column tiles per wave (a workgroup takes a whole state, and a row's load
// is a whole line) where there are two workgroups per compute unit then, one
// (two workgroups per state) for fewer.  Measured, us a call of 16 nodes, one
// tile / two: 256 states 7.5 / 7.6, 384 9.0 / 10.1, 512 12.7 / 12.2,
// 1024 22.7 / 20.0, 2048 38.2 / 34.5.
template <int MT, typename TI, typename TO, bool DELTA>
gdn_status launch_tree(const StateArgs &a, hipStream_t st) {
  const int64_t units = (int64_t)a.B * a.Hv;
  if (units >= 512)
    hipLaunchKernelGGL((tree_kernel<MT, 2, TI, TO, DELTA>), dim3((unsigned)units), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((tree_kernel<MT, 1, TI, TO, DELTA>), dim3((unsigned)(2 * units)), dim3(256), 0, st, a);
  return check_launch();
}

template <typename TI, typename TO, bool DELTA>
gdn_status run_tree(const StateArgs &a, hipStream_t st) {
  if (a.n <= 16) return launch_tree<1, TI, TO, DELTA>(a, st);
  if (a.n <= 32) return launch_tree<2, TI, TO, DELTA>(a, st);
  if (a.n <= 48) return launch_tree<3, TI, TO, DELTA>(a, st);
  return launch_tree<4, TI, TO, DELTA>(a, st);
}

}  // namespace

extern "C" {

gdn_status gdn_step(const gdn_pool_shape *s, const void *q, const void *k, const void *v, const float *g,
                    const float *beta, const int32_t *slots, float *state, void *o, void *hip_stream) {
  GDN_TRY(validate_pool(s, slots));
  if (s->n != 1) return GDN_ERR_SHAPE;
  if (!q || !k || !v || !g || !state || !o) return GDN_ERR_NULL;
  for (const void *p : {q, k, v, (const void *)g, (const void *)beta, (const void *)slots, (const void *)state,
                        (const void *)o})
    if (misaligned(p)) return GDN_ERR_ALIGN;
  StateArgs a = pool_args(*s);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.slots = slots; a.state = state; a.o = o;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  return with_types(*s, [&](auto ti, auto to) -> gdn_status {
    using TI = decltype(ti);
    using TO = decltype(to);
    return quarter_states(*s) ? launch_step<32, TI, TO>(a, st) : launch_step<64, TI, TO>(a, st);
  });
}

gdn_status gdn_tree_fwd(const gdn_pool_shape *s, const void *q, const void *k, const void *v, const float *g,
                        const float *beta, const int32_t *parents, const int32_t *slots, const float *state, void *o,
                        float *u, void *hip_stream) {
  GDN_TRY(validate_pool(s, slots));
  if (!q || !k || !v || !g || !parents || !state || !o || !u) return GDN_ERR_NULL;
  for (const void *p : {q, k, v, (const void *)g, (const void *)beta, (const void *)parents, (const void *)slots,
                        (const void *)state, (const void *)o, (const void *)u})
    if (misaligned(p)) return GDN_ERR_ALIGN;
  StateArgs a = pool_args(*s);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.parents = parents; a.slots = slots;
  a.state = const_cast<float *>(state); a.o = o; a.u = u;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  return with_types(*s, [&](auto ti, auto to) -> gdn_status {
    using TI = decltype(ti);
    using TO = decltype(to);
    return beta ? run_tree<TI, TO, true>(a, st) : run_tree<TI, TO, false>(a, st);
  });
}

gdn_status gdn_tree_commit(const gdn_pool_shape *s, const void *k, const float *u, const float *g,
                           const int32_t *parents, const int32_t *last, const int32_t *slots, float *state,
                           void *hip_stream) {
  GDN_TRY(validate_pool(s, slots));
  if (!k || !u || !g || !parents || !last || !state) return GDN_ERR_NULL;
  for (const void *p : {k, (const void *)u, (const void *)g, (const void *)parents, (const void *)last,
                        (const void *)slots, (const void *)state})
    if (misaligned(p)) return GDN_ERR_ALIGN;
  StateArgs a = pool_args(*s);
  a.k = k; a.u_in = u; a.g = g; a.parents = parents; a.last = last; a.slots = slots; a.state = state;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  auto run = [&](auto ti) -> gdn_status {
    using TI = decltype(ti);
    return quarter_states(*s) ? launch_commit<32, TI>(a, st) : launch_commit<64, TI>(a, st);
  };
  return s->dtype == GDN_BF16 ? run(__bf16{}) : run(float{});
}

}  // extern "C"
