// Host-only harness of the argument checks and workspace sizes of the
// convolution's, the selective scan's and the verification's entry points,
// built with host-side AddressSanitizer and UndefinedBehaviorSanitizer (device
// code is compiled as usual and never launched): every call must be refused
// before a launch.  Exit status 0 when every status is the expected one.  Test
// infrastructure: built and run by tests/test_sanitizers_layers.py.
#include <cstdint>
#include <cstdio>

#include "gdn.h"

static int fails = 0;
static void expect(gdn_status got, gdn_status want, const char *what) {
  if (got != want) {
    std::fprintf(stderr, "FAILED: %s: status %d, expected %d\n", what, (int)got, (int)want);
    ++fails;
  }
}

int main() {
  alignas(16) static char buf[64];
  void *ok = buf, *odd = buf + 4, *half = buf + 1;
  const float *fk = reinterpret_cast<const float *>(buf);
  float *fo = reinterpret_cast<float *>(buf);
  int32_t *ik = reinterpret_cast<int32_t *>(buf);
  const size_t much = (size_t)1 << 60;
  size_t bytes = 0;

  // B, T, C, W, ld, n_slots, silu, dtype
  const int32_t good_conv[][8] = {{1, 0, 1, 2, 0, 1, 1, 1}, {1, 1, 1, 4, 7, 1, 0, 0}, {1, 1 << 30, 64, 4, 0, 1, 1, 1},
                                  {1 << 22, 1, 8, 3, 1 << 20, 1, 0, 1}, {3, 1000, 1 << 20, 4, 1 << 20, 1, 1, 0}};
  for (const auto &g : good_conv) {
    const gdn_conv_shape s{g[0], g[1], g[2], g[3], g[4], g[5], g[6], g[7]};
    expect(gdn_workspace_size_conv_bwd(&s, &bytes), GDN_OK, "conv workspace");
    expect(bytes ? GDN_OK : GDN_ERR_SHAPE, GDN_OK, "conv workspace bytes");
    expect(gdn_conv_bwd(&s, ok, fk, nullptr, nullptr, ok, nullptr, ok, fo, nullptr, nullptr, ok, 0, nullptr), GDN_ERR_WORKSPACE,
           "conv_bwd ws");
  }
  const int32_t bad_conv[][8] = {
      {0, 1, 8, 4, 0, 1, 1, 1},  {-1, 1, 8, 4, 0, 1, 1, 1}, {1, -1, 8, 4, 0, 1, 1, 1},  {1, 1, 0, 4, 0, 1, 1, 1},
      {1, 1, 8, 1, 0, 1, 1, 1},  {1, 1, 8, 5, 0, 1, 1, 1},  {1, 1, 8, 4, 7, 1, 1, 1},   {1, 1, 8, 4, -8, 1, 1, 1},
      {1, 1, 8, 4, 0, 1, 2, 1},  {1, 1, 8, 4, 0, 1, -1, 1}, {1, (1 << 30) + 1, 8, 4, 0, 1, 1, 1},
      {1, 1, (1 << 20) + 1, 4, 0, 1, 1, 1}, {1, 1, 8, 4, (1 << 20) + 1, 1, 1, 1}, {INT32_MAX, 1, 8, 4, 0, 1, 1, 1},
      {1 << 24, 1 << 30, 1 << 20, 4, 0, 1, 1, 1}, {INT32_MAX, INT32_MAX, INT32_MAX, 4, INT32_MAX, INT32_MAX, 1, 1}};
  for (const auto &g : bad_conv) {
    const gdn_conv_shape s{g[0], g[1], g[2], g[3], g[4], g[5], g[6], g[7]};
    expect(gdn_workspace_size_conv_bwd(&s, &bytes), GDN_ERR_SHAPE, "conv workspace shape");
    expect(gdn_conv_fwd(&s, ok, fk, nullptr, nullptr, ok, ok, nullptr), GDN_ERR_SHAPE, "conv_fwd shape");
    expect(gdn_conv_bwd(&s, ok, fk, nullptr, nullptr, ok, nullptr, ok, fo, nullptr, nullptr, ok, much, nullptr), GDN_ERR_SHAPE,
           "conv_bwd shape");
    expect(gdn_conv_step(&s, ok, fk, nullptr, ik, ok, ok, nullptr), GDN_ERR_SHAPE, "conv_step shape");
  }
  const gdn_conv_shape c{4, 10, 64, 4, 0, 8, 1, GDN_BF16};
  gdn_conv_shape one = c;
  one.T = 1;
  expect(gdn_conv_fwd(nullptr, ok, fk, nullptr, nullptr, ok, ok, nullptr), GDN_ERR_NULL, "conv_fwd null shape");
  expect(gdn_conv_fwd(&c, nullptr, fk, nullptr, nullptr, ok, ok, nullptr), GDN_ERR_NULL, "conv_fwd null x");
  expect(gdn_conv_fwd(&c, ok, nullptr, nullptr, nullptr, ok, ok, nullptr), GDN_ERR_NULL, "conv_fwd null weight");
  expect(gdn_conv_fwd(&c, half, fk, nullptr, nullptr, ok, ok, nullptr), GDN_ERR_ALIGN, "conv_fwd misaligned x");
  expect(gdn_conv_fwd_varlen(&c, nullptr, ok, fk, nullptr, nullptr, ok, ok, nullptr), GDN_ERR_NULL, "conv varlen null offsets");
  expect(gdn_conv_step(&c, ok, fk, nullptr, ik, ok, ok, nullptr), GDN_ERR_SHAPE, "conv_step of many tokens");
  expect(gdn_conv_step(&one, ok, fk, nullptr, ik, nullptr, ok, nullptr), GDN_ERR_NULL, "conv_step null state");
  expect(gdn_conv_step(&one, ok, fk, nullptr, ik, half, ok, nullptr), GDN_ERR_ALIGN, "conv_step misaligned state");
  gdn_conv_shape cx = one;
  cx.n_slots = 3;
  expect(gdn_conv_step(&cx, ok, fk, nullptr, nullptr, ok, ok, nullptr), GDN_ERR_SHAPE, "conv_step more rows than slots");
  cx = c;
  cx.dtype = 7;
  expect(gdn_conv_fwd(&cx, ok, fk, nullptr, nullptr, ok, ok, nullptr), GDN_ERR_DTYPE, "conv dtype");
  expect(gdn_workspace_size_conv_bwd(&c, nullptr), GDN_ERR_NULL, "conv size pointer");
  expect(gdn_conv_bwd(&c, ok, fk, nullptr, nullptr, ok, nullptr, ok, nullptr, nullptr, nullptr, ok, much, nullptr), GDN_ERR_NULL,
         "conv_bwd null dweight");

  // B, T, C, N, G, n_slots, softplus, ld_x, ld_dt, ld_z, ld_b, ld_c, dtype, o_dtype
  const gdn_ssm_inputs in{ok, ok, nullptr, ok, ok, fk, nullptr, nullptr};
  const gdn_ssm_grads out{ok, ok, nullptr, ok, ok, fo, nullptr, nullptr, nullptr};
  const int32_t good_ssm[][14] = {{1, 0, 1, 8, 1, 1, 1, 0, 0, 0, 0, 0, 0, 0},       {1, 1, 1, 32, 1, 1, 0, 9, 9, 9, 32, 32, 1, 0},
                                  {2, 5000, 4096, 16, 8, 1, 1, 0, 0, 0, 0, 0, 1, 1}, {1, 1 << 18, 1 << 12, 16, 1, 1, 1, 0, 0, 0, 0, 0, 1, 1},
                                  {1 << 10, 100, 1 << 10, 8, 1, 1, 1, 0, 0, 0, 0, 0, 0, 1}};
  for (const auto &g : good_ssm) {
    const gdn_ssm_shape s{g[0], g[1], g[2], g[3], g[4], g[5], g[6], g[7], g[8], g[9], g[10], g[11], g[12], g[13]};
    for (int32_t kind = GDN_SSM_FWD; kind <= GDN_SSM_BWD; ++kind)
      expect(gdn_workspace_size_ssm(&s, kind, &bytes), GDN_OK, "ssm workspace");
    expect(gdn_ssm_bwd(&s, &in, nullptr, ok, nullptr, &out, ok, bytes - 1, nullptr), GDN_ERR_WORKSPACE, "ssm_bwd ws");
  }
  const int32_t bad_ssm[][14] = {{0, 1, 8, 8, 1, 1, 1, 0, 0, 0, 0, 0, 1, 1},   {1, -1, 8, 8, 1, 1, 1, 0, 0, 0, 0, 0, 1, 1},
                                 {1, 1, 0, 8, 1, 1, 1, 0, 0, 0, 0, 0, 1, 1},   {1, 1, 8, 4, 1, 1, 1, 0, 0, 0, 0, 0, 1, 1},
                                 {1, 1, 8, 64, 1, 1, 1, 0, 0, 0, 0, 0, 1, 1},  {1, 1, 8, 8, 0, 1, 1, 0, 0, 0, 0, 0, 1, 1},
                                 {1, 1, 8, 8, 3, 1, 1, 0, 0, 0, 0, 0, 1, 1},   {1, 1, 8, 8, 1, 1, 2, 0, 0, 0, 0, 0, 1, 1},
                                 {1, 1, 8, 8, 1, 1, 1, 7, 0, 0, 0, 0, 1, 1},   {1, 1, 8, 8, 1, 1, 1, 0, 7, 0, 0, 0, 1, 1},
                                 {1, 1, 8, 8, 1, 1, 1, 0, 0, -1, 0, 0, 1, 1},  {1, 1, 8, 8, 1, 1, 1, 0, 0, 0, 9, 0, 1, 1},
                                 {1, 1, 8, 8, 1, 1, 1, 0, 0, 0, 0, 12, 1, 1},  {1, 1, 8, 8, 2, 1, 1, 0, 0, 0, 8, 0, 1, 1},
                                 {1, INT32_MAX, 8, 8, 1, 1, 1, 0, 0, 0, 0, 0, 1, 1}, {1, 1, (1 << 20) + 1, 8, 1, 1, 1, 0, 0, 0, 0, 0, 1, 1},
                                 {INT32_MAX, 1 << 30, 1 << 20, 32, 1 << 20, 1, 1, 0, 0, 0, 0, 0, 1, 1},
                                 {INT32_MAX, 1, 1, 8, 1, 1, 1, 0, 0, 0, 0, 0, 1, 1}};
  for (const auto &g : bad_ssm) {
    const gdn_ssm_shape s{g[0], g[1], g[2], g[3], g[4], g[5], g[6], g[7], g[8], g[9], g[10], g[11], g[12], g[13]};
    for (int32_t kind : {GDN_SSM_FWD, GDN_SSM_BWD})
      expect(gdn_workspace_size_ssm(&s, kind, &bytes), GDN_ERR_SHAPE, "ssm workspace shape");
    expect(gdn_ssm_fwd(&s, &in, nullptr, ok, fo, ok, much, nullptr), GDN_ERR_SHAPE, "ssm_fwd shape");
    expect(gdn_ssm_bwd(&s, &in, nullptr, ok, nullptr, &out, ok, much, nullptr), GDN_ERR_SHAPE, "ssm_bwd shape");
    expect(gdn_ssm_step(&s, &in, nullptr, fo, ok, nullptr), GDN_ERR_SHAPE, "ssm_step shape");
  }
  const gdn_ssm_shape packed{INT32_MAX, 1 << 30, 1 << 20, 32, 1 << 20, 1, 1, 0, 0, 0, 0, 0, 1, 1};
  expect(gdn_workspace_size_ssm(&packed, GDN_SSM_VARLEN, &bytes), GDN_ERR_SHAPE, "ssm packed workspace");
  expect(gdn_ssm_fwd_varlen(&packed, ik, &in, nullptr, ok, fo, ok, much, nullptr), GDN_ERR_SHAPE, "ssm packed shape");
  const gdn_ssm_shape s{2, 500, 64, 16, 2, 4, 1, 0, 0, 0, 0, 0, GDN_BF16, GDN_F32};
  gdn_ssm_shape tok = s;
  tok.T = 1;
  gdn_ssm_inputs ix = in;
  gdn_ssm_grads ox = out;
  expect(gdn_workspace_size_ssm(&s, 3, &bytes), GDN_ERR_SHAPE, "ssm kind");
  expect(gdn_workspace_size_ssm(&s, 0, nullptr), GDN_ERR_NULL, "ssm size pointer");
  expect(gdn_ssm_fwd(nullptr, &in, nullptr, ok, fo, ok, much, nullptr), GDN_ERR_NULL, "ssm_fwd null shape");
  expect(gdn_ssm_fwd(&s, nullptr, nullptr, ok, fo, ok, much, nullptr), GDN_ERR_NULL, "ssm_fwd null inputs");
  expect(gdn_ssm_fwd(&s, &in, nullptr, nullptr, fo, ok, much, nullptr), GDN_ERR_NULL, "ssm_fwd null y");
  expect(gdn_ssm_fwd(&s, &in, nullptr, ok, fo, nullptr, much, nullptr), GDN_ERR_NULL, "ssm_fwd null ws");
  expect(gdn_ssm_fwd(&s, &in, nullptr, ok, fo, ok, 0, nullptr), GDN_ERR_WORKSPACE, "ssm_fwd ws");
  expect(gdn_ssm_fwd_varlen(&s, nullptr, &in, nullptr, ok, fo, ok, much, nullptr), GDN_ERR_NULL, "ssm varlen null offsets");
  ix.B = odd;
  expect(gdn_ssm_fwd(&s, &ix, nullptr, ok, fo, ok, much, nullptr), GDN_ERR_ALIGN, "ssm_fwd misaligned B");
  ix = in;
  ix.x = half;
  expect(gdn_ssm_fwd(&s, &ix, nullptr, ok, fo, ok, much, nullptr), GDN_ERR_ALIGN, "ssm_fwd misaligned x");
  ix = in;
  ix.z = ok;   // a gate, and nowhere to write its gradient
  expect(gdn_ssm_bwd(&s, &ix, nullptr, ok, nullptr, &out, ok, much, nullptr), GDN_ERR_NULL, "ssm_bwd null dz");
  ox.dB = odd;
  expect(gdn_ssm_bwd(&s, &in, nullptr, ok, nullptr, &ox, ok, much, nullptr), GDN_ERR_ALIGN, "ssm_bwd misaligned dB");
  expect(gdn_ssm_bwd(&s, &in, nullptr, ok, nullptr, nullptr, ok, much, nullptr), GDN_ERR_NULL, "ssm_bwd null outputs");
  expect(gdn_ssm_step(&s, &in, ik, fo, ok, nullptr), GDN_ERR_SHAPE, "ssm_step of many tokens");
  expect(gdn_ssm_step(&tok, &in, ik, nullptr, ok, nullptr), GDN_ERR_NULL, "ssm_step null state");
  tok.n_slots = 1;
  expect(gdn_ssm_step(&tok, &in, nullptr, fo, ok, nullptr), GDN_ERR_SHAPE, "ssm_step more rows than slots");
  tok.o_dtype = 9;
  expect(gdn_ssm_step(&tok, &in, nullptr, fo, ok, nullptr), GDN_ERR_DTYPE, "ssm_step o_dtype");

  const gdn_verify_shape good_verify[] = {{1, 1, 1}, {1, 64, 1 << 24}, {1 << 20, 1, 1}, {2048, 64, 1 << 24}};
  for (const gdn_verify_shape &v : good_verify) {
    expect(gdn_workspace_size_verify(&v, &bytes), GDN_OK, "verify workspace");
    expect(gdn_tree_verify(&v, ik, ik, fk, fk, fk, ik, ik, ik, ok, bytes - 1, nullptr), GDN_ERR_WORKSPACE, "verify ws");
  }
  const gdn_verify_shape bad_verify[] = {{0, 1, 1}, {1, 0, 1}, {1, 65, 1}, {1, 1, 0}, {1, 1, (1 << 24) + 1}, {(1 << 20) + 1, 1, 1},
                                         {2049, 64, 1 << 24}, {INT32_MAX, INT32_MAX, INT32_MAX}};
  for (const gdn_verify_shape &v : bad_verify) {
    expect(gdn_workspace_size_verify(&v, &bytes), GDN_ERR_SHAPE, "verify workspace shape");
    expect(gdn_tree_verify(&v, ik, ik, fk, nullptr, fk, ik, ik, ik, ok, much, nullptr), GDN_ERR_SHAPE, "verify shape");
  }
  const gdn_verify_shape v{2, 4, 100};
  expect(gdn_tree_verify(nullptr, ik, ik, fk, fk, fk, ik, ik, ik, ok, much, nullptr), GDN_ERR_NULL, "verify null shape");
  expect(gdn_tree_verify(&v, ik, ik, nullptr, fk, fk, ik, ik, ik, ok, much, nullptr), GDN_ERR_NULL, "verify null target");
  expect(gdn_tree_verify(&v, ik, ik, fk, fk, fk, ik, ik, ik, odd, much, nullptr), GDN_ERR_ALIGN, "verify misaligned ws");
  expect(gdn_tree_verify(&v, ik, ik, reinterpret_cast<const float *>(half), fk, fk, ik, ik, ik, ok, much, nullptr), GDN_ERR_ALIGN,
         "verify misaligned target");
  if (fails) return 1;
  std::puts("all checks passed");
  return 0;
}
