// gdn_verify.hip -- C ABI of the verification of drafted tokens (declared in
// include/gdn.h): argument checks and launches on the caller's stream.  No
// allocation, no synchronisation.
#include <hip/hip_runtime.h>

#include "gdn.h"
#include "gdn_host.h"
#include "gdn_verify.h"

using namespace gdn;

namespace {

// One launch, a workgroup per row, for vocabularies of 2^15 tokens at most and,
// without draft probabilities, at most 32 rows; else the sums by parts and the
// draw in launches of their own.  Measured, one launch against several, in us
// on the device (each launch less also saves 3 us of the host's time), 8 nodes
// a row (4 of 512 rows of 65536 tokens), in a chain, where no refusal needs a
// pass over the vocabulary, or a tree, half of whose nodes continue the one
// before and half branch off any earlier one (with draft probabilities 0.3 to
// 0.7 passes a row, and up to 4 of the row that has most):
//   tokens                        8192          32003         65536
//   draft, chain, 1 row         9.6 / 15.1   13.1 / 14.6    19.1 / 15.1
//                32 rows       10.7 / 17.3   20.1 / 20.6    33.4 / 22.0
//               512 rows       24.4 / 31.1   55.5 / 60.9    96.2 / 86.0
//   draft, tree,  1 row        10.7 / 16.2   12.1 / 13.9    19.1 / 14.8
//                32 rows       15.6 / 21.2   29.7 / 43.4    69.5 / 66.7
//               512 rows       33.7 / 39.2  104.6 / 103.2  153.3 / 154.8
//   no draft, tree, 1 row       7.8 /  9.4    8.2 /  9.2    12.0 /  9.2
//                  32 rows     10.6 / 10.6   11.3 / 10.5    14.5 / 11.1
//                 512 rows     22.1 / 16.4   25.2 / 24.4    41.3 / 39.4
constexpr int kRowTokens = 1 << 15, kRowRows = 32;
static_assert(kRowTokens <= VERIFY_CHUNKS * VERIFY_CHUNK, "the sums of a row's chunks lie in LDS");

gdn_status validate_verify(const gdn_verify_shape *s) {
  if (!s) return GDN_ERR_NULL;
  if (s->B < 1 || s->n < 1 || s->n > kVerifyNodes || s->V < 1 || s->V > 1 << 24) return GDN_ERR_SHAPE;
  // a launch holds fewer than 2^32 threads
  if (s->B > 1 << 20 || (int64_t)s->B * ((s->V + VERIFY_PART - 1) / VERIFY_PART) > (1 << 23)) return GDN_ERR_SHAPE;
  return GDN_OK;
}
size_t plan_bytes(const gdn_verify_shape &s) { return align_up((size_t)s.B * sizeof(VerifyPlan)); }
int parts_of(const gdn_verify_shape &s) { return (s.V + VERIFY_PART - 1) / VERIFY_PART; }
size_t bytes_of(const gdn_verify_shape &s) { return plan_bytes(s) + align_up((size_t)s.B * parts_of(s) * 8); }

}  // namespace

extern "C" {

gdn_status gdn_workspace_size_verify(const gdn_verify_shape *s, size_t *bytes) {
  if (!bytes) return GDN_ERR_NULL;
  GDN_TRY(validate_verify(s));
  *bytes = bytes_of(*s);
  return GDN_OK;
}

gdn_status gdn_tree_verify(const gdn_verify_shape *s, const int32_t *tokens, const int32_t *parents, const float *target,
                           const float *draft, const float *uniform, int32_t *last, int32_t *token, int32_t *path, void *ws,
                           size_t ws_bytes, void *hip_stream) {
  GDN_TRY(validate_verify(s));
  if (!tokens || !parents || !target || !uniform || !last || !token || !path || !ws) return GDN_ERR_NULL;
  for (const void *p : {(const void *)tokens, (const void *)parents, (const void *)target, (const void *)draft, (const void *)uniform,
                        (const void *)last, (const void *)token, (const void *)path})
    if (p && (uintptr_t)p % 4) return GDN_ERR_ALIGN;
  if (misaligned(ws)) return GDN_ERR_ALIGN;
  if (ws_bytes < bytes_of(*s)) return GDN_ERR_WORKSPACE;
  VerifyArgs a{};
  a.B = s->B; a.n = s->n; a.V = s->V; a.parts = parts_of(*s);
  a.tokens = tokens; a.parents = parents; a.target = target; a.draft = draft; a.uniform = uniform;
  a.last = last; a.token = token; a.path = path;
  a.plan = static_cast<VerifyPlan *>(ws);
  a.part = reinterpret_cast<double *>(static_cast<char *>(ws) + plan_bytes(*s));
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  if (s->V <= kRowTokens && (draft || s->B <= kRowRows)) {
    if (draft) hipLaunchKernelGGL(verify_row_kernel<true>, dim3((unsigned)s->B), dim3(1024), 0, st, a);
    else hipLaunchKernelGGL(verify_row_kernel<false>, dim3((unsigned)s->B), dim3(1024), 0, st, a);
    return check_launch();
  }
  const dim3 parts((unsigned)(s->B * a.parts));
  if (draft) {
    hipLaunchKernelGGL(verify_walk_kernel, dim3((unsigned)s->B), dim3(1024), 0, st, a);
    GDN_TRY(check_launch());
    hipLaunchKernelGGL(verify_sum_kernel<true>, parts, dim3(256), 0, st, a);
  } else {
    hipLaunchKernelGGL(verify_sum_kernel<false>, parts, dim3(256), 0, st, a);
  }
  GDN_TRY(check_launch());
  hipLaunchKernelGGL(verify_draw_kernel, dim3((unsigned)s->B), dim3(256), 0, st, a);
  return check_launch();
}

}  // extern "C"
