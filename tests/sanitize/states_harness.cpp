// Host-only harness of the argument checks and workspace sizes of the state
// pool's and of the linear attention's entry points, built with host-side
// AddressSanitizer and UndefinedBehaviorSanitizer (device code is compiled as
// usual and never launched): every call must be refused before a launch.
// Exit status 0 when every status is the expected one.  Test infrastructure:
// built and run by tests/test_sanitizers_states.py.
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
  void *ok = buf, *odd = buf + 4;
  const float *fk = reinterpret_cast<const float *>(buf), *fodd = reinterpret_cast<const float *>(buf + 4);
  float *fo = reinterpret_cast<float *>(buf);
  const int32_t *ik = reinterpret_cast<const int32_t *>(buf);

  const gdn_pool_shape p{4, 1, 16, 32, 128, 128, 8, 0, GDN_BF16, GDN_F32};
  const int32_t bad_pool[][10] = {
      {0, 1, 16, 32, 128, 128, 8, 0, 1, 0},  {4, 0, 16, 32, 128, 128, 8, 0, 1, 0},  {4, 65, 16, 32, 128, 128, 8, 0, 1, 0},
      {4, 1, 0, 32, 128, 128, 8, 0, 1, 0},   {4, 1, 16, 24, 128, 128, 8, 0, 1, 0},  {4, 1, 16, 32, 64, 128, 8, 0, 1, 0},
      {4, 1, 16, 32, 128, 64, 8, 0, 1, 0},   {4, 1, 16, 32, 128, 128, 0, 0, 1, 0},  {4, 1, 16, 32, 128, 128, 8, 2, 1, 0},
      {INT32_MAX, 1, 1, INT32_MAX, 128, 128, INT32_MAX, 0, 1, 0}};
  for (const auto &b : bad_pool) {
    const gdn_pool_shape s{b[0], b[1], b[2], b[3], b[4], b[5], b[6], b[7], b[8], b[9]};
    expect(gdn_step(&s, ok, ok, ok, fk, fk, ik, fo, ok, nullptr), GDN_ERR_SHAPE, "step shape");
    expect(gdn_tree_fwd(&s, ok, ok, ok, fk, fk, ik, ik, fk, ok, fo, nullptr), GDN_ERR_SHAPE, "tree shape");
    expect(gdn_tree_commit(&s, ok, fk, fk, ik, ik, ik, fo, nullptr), GDN_ERR_SHAPE, "commit shape");
  }
  expect(gdn_step(nullptr, ok, ok, ok, fk, fk, ik, fo, ok, nullptr), GDN_ERR_NULL, "step null shape");
  expect(gdn_step(&p, ok, ok, ok, nullptr, fk, ik, fo, ok, nullptr), GDN_ERR_NULL, "step null g");
  expect(gdn_step(&p, ok, odd, ok, fk, fk, ik, fo, ok, nullptr), GDN_ERR_ALIGN, "step misaligned k");
  expect(gdn_tree_fwd(&p, ok, ok, ok, fk, fk, nullptr, ik, fk, ok, fo, nullptr), GDN_ERR_NULL, "tree null parents");
  expect(gdn_tree_fwd(&p, ok, ok, ok, fk, fodd, ik, ik, fk, ok, fo, nullptr), GDN_ERR_ALIGN, "tree misaligned beta");
  expect(gdn_tree_commit(&p, ok, fk, fk, ik, nullptr, ik, fo, nullptr), GDN_ERR_NULL, "commit null last");
  gdn_pool_shape d = p;
  d.o_dtype = 9;
  expect(gdn_step(&d, ok, ok, ok, fk, fk, ik, fo, ok, nullptr), GDN_ERR_DTYPE, "step o_dtype");
  d = p;
  d.B = 9;
  expect(gdn_step(&d, ok, ok, ok, fk, fk, nullptr, fo, ok, nullptr), GDN_ERR_SHAPE, "more rows than slots");

  size_t bytes = 0;
  for (int32_t kind = GDN_LINEAR_FWD; kind <= GDN_LINEAR_BWD; ++kind) {
    // every supported size computes, the largest among them
    const int32_t good[][7] = {{1, 0, 1, 1, 128, 128, 0},      {1, 1, 1, 1, 128, 128, 1},   {2, 1000, 4, 8, 128, 128, 0},
                               {1, INT32_MAX, 1, 1, 128, 128, 1}, {1 << 12, 1 << 18, 1, 1, 128, 128, 0},
                               {1, 100, 1, 1 << 14, 128, 128, 1}};
    for (const auto &g : good)
      for (int32_t dt = 0; dt < 2; ++dt) {
        const gdn_linear_shape s{g[0], g[1], g[2], g[3], g[4], g[5], g[6], dt, 1 - dt};
        expect(gdn_workspace_size_linear(&s, kind, &bytes), GDN_OK, "linear workspace");
      }
    const int32_t bad[][7] = {{0, 10, 1, 1, 128, 128, 0},  {1, -1, 1, 1, 128, 128, 0},  {1, 10, 2, 3, 128, 128, 0},
                              {1, 10, 0, 1, 128, 128, 0},  {1, 10, 1, 1, 64, 128, 0},   {1, 10, 1, 1, 128, 256, 0},
                              {1, 10, 1, 1, 128, 128, 2},  {1, 10, 1, (1 << 14) + 1, 128, 128, 0},
                              {INT32_MAX, INT32_MAX, 1, 1 << 14, 128, 128, 0}};
    for (const auto &g : bad) {
      const gdn_linear_shape s{g[0], g[1], g[2], g[3], g[4], g[5], g[6], 1, 0};
      expect(gdn_workspace_size_linear(&s, kind, &bytes), GDN_ERR_SHAPE, "linear shape");
    }
  }
  const gdn_linear_shape s{2, 5000, 4, 8, 128, 128, 0, GDN_BF16, GDN_BF16};
  expect(gdn_workspace_size_linear(&s, 3, &bytes), GDN_ERR_SHAPE, "linear kind");
  expect(gdn_workspace_size_linear(&s, 0, nullptr), GDN_ERR_NULL, "linear size pointer");
  expect(gdn_workspace_size_linear(&s, GDN_LINEAR_FWD, &bytes), GDN_OK, "linear forward workspace");
  expect(gdn_linear_chunk_fwd(&s, ok, ok, ok, fk, nullptr, nullptr, nullptr, ok, bytes, nullptr), GDN_ERR_NULL, "fwd null o");
  expect(gdn_linear_chunk_fwd(&s, ok, ok, odd, fk, nullptr, ok, nullptr, ok, bytes, nullptr), GDN_ERR_ALIGN, "fwd misaligned");
  expect(gdn_linear_chunk_fwd(&s, ok, ok, ok, fk, nullptr, ok, nullptr, ok, bytes - 1, nullptr), GDN_ERR_WORKSPACE, "fwd ws");
  expect(gdn_linear_chunk_fwd_varlen(&s, nullptr, ok, ok, ok, fk, nullptr, ok, nullptr, ok, (size_t)1 << 40, nullptr),
         GDN_ERR_NULL, "varlen null offsets");
  expect(gdn_linear_chunk_bwd(&s, ok, ok, ok, fk, nullptr, ok, nullptr, ok, ok, nullptr, fo, nullptr, ok, (size_t)1 << 40, nullptr),
         GDN_ERR_NULL, "bwd null dv");
  expect(gdn_linear_chunk_bwd(&s, ok, ok, ok, fk, nullptr, ok, nullptr, ok, ok, ok, fo, nullptr, ok, 0, nullptr),
         GDN_ERR_WORKSPACE, "bwd ws");
  if (fails) return 1;
  std::puts("all checks passed");
  return 0;
}
