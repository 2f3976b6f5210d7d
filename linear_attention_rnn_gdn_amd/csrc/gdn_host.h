// gdn_host.h -- host-side helpers shared by the library's entry points:
// alignment of workspace pieces and pointers, launch status.
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gdn.h"

namespace gdn {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool misaligned(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }

inline gdn_status check_launch() { return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

#define GDN_TRY(x)                       \
  do {                                   \
    gdn_status st_ = (x);                \
    if (st_ != GDN_OK) return st_;       \
  } while (0)

}  // namespace gdn
