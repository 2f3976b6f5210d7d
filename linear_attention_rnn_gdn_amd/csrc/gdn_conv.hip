// gdn_conv.hip -- C ABI of the short causal convolution (declared in
// include/gdn.h): argument checks and launches on the caller's stream.  No
// allocation, no synchronisation.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn.h"
#include "gdn_conv.h"
#include "gdn_host.h"

using namespace gdn;

namespace {

constexpr int64_t kMaxBlocks = (1ll << 24) - 1;   // of 256 threads: a launch holds fewer than 2^32
constexpr int kMaxRow = 1 << 20;                  // elements from a token to the next (see lay_out)
// Tokens per thread, rounded down to whole windows.  Forward: at 4096 tokens of
// 8192 channels in bf16 8 took 33 us (each thread reads its W - 1 tokens of
// window too), 16 30 and 32 32.4 (too few waves).
constexpr int kFwdRun = 16;
// Gradients: 16, 32 and 64 took 60.6, 58.7 and 53 us there (a workgroup's sums
// over tokens go through memory), so 64 where that gives 512 workgroups, else
// half, down to 16: 16 and 32 took 19.8 and 22.9 us at 1024 tokens of 2048
// channels, 19.7 and 22 at 300 of 512.  (Halving below 1024 took 59 us instead
// of 53 at the first of these, 19 instead of 19.8 at the last two.)
constexpr int kBwdRun = 64, kBwdShort = 16, kFewPieces = 512;
// Single tokens: two rows per thread in bf16 from so many workgroups of one row
// on, one below and in fp32.  One, two and four rows took, in us: bf16, 64 rows
// of 8192 channels (256 workgroups) 4.4, 5.1 and 6.6, 128 of them (512) 6.2, 6.1
// and 7.5, 192 (768) 8.1 and 8.5, 256 (1024) 10.1, 9.8 and 10.7, 512 (2048)
// 16.4, 13.8 and 14.9; 2048 rows of 4099 channels (single elements) 47 and 40;
// fp32, 256 rows of 4096 channels 7.5, 8.4 and 9.6, 512 rows of 8192 21.0 and 20.6.
constexpr int kManySteps = 1024;

int elem(const gdn_conv_shape &s) { return s.dtype == GDN_BF16 ? 2 : 4; }

gdn_status validate_conv(const gdn_conv_shape *s) {
  if (!s) return GDN_ERR_NULL;
  if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (s->B < 1 || s->B > 1 << 24 || s->T < 0 || s->T > 1 << 30 || s->C < 1 || s->C > kMaxRow || s->W < 2 || s->W > 4) return GDN_ERR_SHAPE;
  if ((s->ld && (s->ld < s->C || s->ld > kMaxRow)) || (s->silu & ~1)) return GDN_ERR_SHAPE;
  return GDN_OK;
}

// every pointer at least an element of its type aligned
gdn_status aligned(const gdn_conv_shape &s, std::initializer_list<const void *> data, std::initializer_list<const void *> f32) {
  for (const void *p : data)
    if (p && (uintptr_t)p % elem(s)) return GDN_ERR_ALIGN;
  for (const void *p : f32)
    if (p && (uintptr_t)p % 4) return GDN_ERR_ALIGN;
  return GDN_OK;
}
// 16-byte pieces where the rows of everything are whole pieces, single elements else
bool wide(const gdn_conv_shape &s, std::initializer_list<const void *> data) {
  const int64_t e = elem(s);
  bool ok = s.C * e % 16 == 0 && s.ld * e % 16 == 0;
  for (const void *p : data) ok = ok && (uintptr_t)p % 16 == 0;
  return ok;
}

ConvArgs conv_args(const gdn_conv_shape &s) {
  ConvArgs a{};
  a.B = s.B; a.T = s.T; a.C = s.C; a.n_slots = s.n_slots; a.silu = s.silu;
  a.ld = s.ld ? s.ld : s.C;
  return a;
}
// 64 threads side by side in channels, fewer where there are fewer, but so many
// that a workgroup's tokens lie within 2^31 bytes: at 64, 4 runs of 64 tokens at
// most, of 2^20 elements of 4 bytes.
void lay_out(ConvArgs &a, int vec, int run, int elem) {
  const int groups = (a.C + vec - 1) / vec;
  const int64_t ld = std::max<int64_t>(a.ld, a.C);
  a.lane_bits = 0;
  while (a.lane_bits < 6 && ((1 << a.lane_bits) < groups || ((int64_t)(256 >> a.lane_bits) * run + 16) * ld * elem >= 1ll << 31)) ++a.lane_bits;
  a.lanes = 1 << a.lane_bits;
  a.run = run;
  const int64_t per = (int64_t)(256 >> a.lane_bits) * run;
  a.runs = (int)((a.T + per - 1) / per);
}
int tiles_of(const ConvArgs &a, int vec) { return (a.C / vec + a.lanes - 1) / a.lanes; }

template <typename F>
gdn_status with_width(int W, F &&f) {
  return W == 2 ? f(std::integral_constant<int, 2>{}) : W == 3 ? f(std::integral_constant<int, 3>{}) : f(std::integral_constant<int, 4>{});
}
template <typename F>
gdn_status with_pack(const gdn_conv_shape &s, bool wide, F &&f) {
  if (s.dtype == GDN_BF16) return wide ? f(std::integral_constant<int, 8>{}, __bf16{}) : f(std::integral_constant<int, 1>{}, __bf16{});
  return wide ? f(std::integral_constant<int, 4>{}, float{}) : f(std::integral_constant<int, 1>{}, float{});
}

template <typename F>
gdn_status with_pack_bwd(const gdn_conv_shape &s, bool wide, F &&f) {
  if (s.dtype == GDN_BF16) return wide ? f(std::integral_constant<int, 4>{}, __bf16{}) : f(std::integral_constant<int, 1>{}, __bf16{});
  return wide ? f(std::integral_constant<int, 4>{}, float{}) : f(std::integral_constant<int, 1>{}, float{});
}

gdn_status conv_fwd(const gdn_conv_shape *s, bool packed, const int32_t *cu, const void *x, const float *weight, const float *bias,
                    const void *h0, void *y, void *h_T, void *hip_stream) {
  GDN_TRY(validate_conv(s));
  if ((s->T > 0 && (!x || !y)) || !weight || (packed && !cu)) return GDN_ERR_NULL;
  GDN_TRY(aligned(*s, {x, h0, y, h_T}, {weight, bias, cu}));
  if (s->T == 0 && !h_T) return GDN_OK;
  ConvArgs a = conv_args(*s);
  a.cu = packed ? cu : nullptr;
  a.x = x; a.weight = weight; a.bias = bias; a.h0 = h0; a.y = y; a.h_T = h_T;
  const int rows = packed ? 1 : s->B;
  return with_pack(*s, wide(*s, {x, h0, y, h_T}), [&](auto vec, auto t) -> gdn_status {
    constexpr int VEC = decltype(vec)::value;
    using T = decltype(t);
    lay_out(a, VEC, kFwdRun / s->W * s->W, sizeof(T));
    const int per = 256 >> a.lane_bits;
    const int64_t windows = h_T ? ((int64_t)s->B * (s->W - 1) + per - 1) / per : 0;
    const int64_t blocks = ((int64_t)rows * a.runs + windows) * tiles_of(a, VEC);
    if (blocks > kMaxBlocks) return GDN_ERR_SHAPE;
    return with_width(s->W, [&](auto w) -> gdn_status {
      hipLaunchKernelGGL((conv_fwd_kernel<decltype(w)::value, VEC, T>), dim3((unsigned)blocks), dim3(256), 0,
                         reinterpret_cast<hipStream_t>(hip_stream), a);
      return check_launch();
    });
  });
}

struct ConvPieces {
  int64_t pieces;
  size_t bytes;
};
ConvPieces pieces_of(const gdn_conv_shape &s, ConvArgs &a, int vec) {
  for (int run = kBwdRun; run >= kBwdShort; run /= 2) {
    lay_out(a, vec, run / s.W * s.W, elem(s));
    if ((int64_t)s.B * a.runs * tiles_of(a, vec) >= kFewPieces) break;
  }
  a.runs = std::max(a.runs, 1);   // (an empty row still writes dh0)
  const int64_t pieces = (int64_t)s.B * a.runs;
  return {pieces, align_up((size_t)pieces * (s.W + 1) * s.C * 4)};
}

}  // namespace

extern "C" {

gdn_status gdn_conv_fwd(const gdn_conv_shape *s, const void *x, const float *weight, const float *bias, const void *h0, void *y,
                        void *h_T, void *hip_stream) {
  return conv_fwd(s, false, nullptr, x, weight, bias, h0, y, h_T, hip_stream);
}

gdn_status gdn_conv_fwd_varlen(const gdn_conv_shape *s, const int32_t *cu_seqlens, const void *x, const float *weight,
                               const float *bias, const void *h0, void *y, void *h_T, void *hip_stream) {
  return conv_fwd(s, true, cu_seqlens, x, weight, bias, h0, y, h_T, hip_stream);
}

gdn_status gdn_conv_step(const gdn_conv_shape *s, const void *x, const float *weight, const float *bias, const int32_t *slots,
                         void *state, void *y, void *hip_stream) {
  GDN_TRY(validate_conv(s));
  if (s->T != 1 || s->n_slots < 1 || (!slots && s->n_slots < s->B)) return GDN_ERR_SHAPE;
  if (!x || !weight || !state || !y) return GDN_ERR_NULL;
  GDN_TRY(aligned(*s, {x, state, y}, {weight, bias, slots}));
  ConvArgs a = conv_args(*s);
  a.x = x; a.weight = weight; a.bias = bias; a.slots = slots; a.state = state; a.y = y;
  return with_pack(*s, wide(*s, {x, state, y, weight}), [&](auto vec, auto t) -> gdn_status {
    constexpr int VEC = decltype(vec)::value;
    using T = decltype(t);
    const int64_t tiles = (s->C / VEC + 255) / 256;
    if (s->B * tiles > kMaxBlocks) return GDN_ERR_SHAPE;
    return with_width(s->W, [&](auto w) -> gdn_status {
      auto run = [&](auto rows) -> gdn_status {
        constexpr int ROWS = decltype(rows)::value;
        hipLaunchKernelGGL((conv_step_kernel<decltype(w)::value, VEC, ROWS, T>), dim3((unsigned)((s->B + ROWS - 1) / ROWS * tiles)),
                           dim3(256), 0, reinterpret_cast<hipStream_t>(hip_stream), a);
        return check_launch();
      };
      if constexpr (sizeof(T) == 2)
        if (s->B * tiles >= kManySteps) return run(std::integral_constant<int, 2>{});
      return run(std::integral_constant<int, 1>{});
    });
  });
}

gdn_status gdn_workspace_size_conv_bwd(const gdn_conv_shape *s, size_t *bytes) {
  if (!bytes) return GDN_ERR_NULL;
  GDN_TRY(validate_conv(s));
  // of the two layouts (16-byte pieces or single elements) that a launch can hold, the larger one
  ConvArgs a = conv_args(*s);
  *bytes = 0;
  for (int vec : {1, 4}) {
    const ConvPieces p = pieces_of(*s, a, vec);
    if (p.pieces * tiles_of(a, vec) <= kMaxBlocks) *bytes = std::max(*bytes, p.bytes);
  }
  return *bytes ? GDN_OK : GDN_ERR_SHAPE;
}

gdn_status gdn_conv_bwd(const gdn_conv_shape *s, const void *x, const float *weight, const float *bias, const void *h0, const void *dy,
                        const void *dh_T, void *dx, float *dweight, float *dbias, void *dh0, void *ws, size_t ws_bytes,
                        void *hip_stream) {
  GDN_TRY(validate_conv(s));
  if ((s->T > 0 && (!x || !dy || !dx)) || !weight || !dweight || !ws) return GDN_ERR_NULL;
  GDN_TRY(aligned(*s, {x, h0, dy, dh_T, dx, dh0}, {weight, bias, dweight, dbias, ws}));
  ConvArgs a = conv_args(*s);
  a.x = x; a.weight = weight; a.bias = bias; a.h0 = h0; a.dy = dy; a.dh_T = dh_T; a.dx = dx; a.dh0 = dh0;
  a.part = static_cast<float *>(ws);
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  return with_pack_bwd(*s, wide(*s, {x, h0, dy, dh_T, dx, dh0}), [&](auto vec, auto t) -> gdn_status {
    constexpr int VEC = decltype(vec)::value;
    using T = decltype(t);
    const ConvPieces p = pieces_of(*s, a, VEC);
    const int64_t blocks = p.pieces * tiles_of(a, VEC);
    if (blocks > kMaxBlocks) return GDN_ERR_SHAPE;
    if (ws_bytes < p.bytes) return GDN_ERR_WORKSPACE;
    GDN_TRY(with_width(s->W, [&](auto w) -> gdn_status {
      hipLaunchKernelGGL((conv_bwd_kernel<decltype(w)::value, VEC, T>), dim3((unsigned)blocks), dim3(256), 0, st, a);
      return check_launch();
    }));
    hipLaunchKernelGGL(conv_sum_kernel, dim3((unsigned)((s->C + 63) / 64 * (s->W + 1))), dim3(1024), 0, st, a.part, (int)p.pieces, s->C,
                       s->W, dweight, dbias);
    return check_launch();
  });
}

}  // extern "C"
