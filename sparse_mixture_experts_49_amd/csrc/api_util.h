// Helpers shared by the C ABI's source files: the thread-local error message,
// argument checks, workspace carving and the overlap test.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/moe_mi355x.h"

namespace moe {
namespace api {

inline thread_local char g_err[512] = "";

inline int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return status;
}

inline int ok() {
  g_err[0] = '\0';
  return MOE_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define MOE_REQUIRE_PTR(p, name)                                                       \
  do {                                                                                 \
    if (!(p)) return fail(MOE_ERR_INVALID, "%s must not be NULL", name);               \
    if (!aligned16(p)) return fail(MOE_ERR_INVALID, "%s must be 16-byte aligned", name); \
  } while (0)
#define MOE_OPTIONAL_PTR(p, name)                                                      \
  do {                                                                                 \
    if ((p) && !aligned16(p)) return fail(MOE_ERR_INVALID, "%s must be 16-byte aligned", name); \
  } while (0)

inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// ---- aliasing -------------------------------------------------------------
// Outputs (the workspace included) must be disjoint from each other and from
// every input; a call that would write over its own operands is refused.

struct Span {
  const void* p;
  size_t n;
  const char* name;
};

struct Spans {
  Span s[40];
  int n = 0;
  void add(const void* p, size_t bytes, const char* name) {
    if (p && bytes && n < 40) s[n++] = Span{p, bytes, name};
  }
};

inline bool overlaps(const Span& a, const Span& b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

inline int check_alias(const Spans& outs, const Spans& ins) {
  for (int i = 0; i < outs.n; ++i) {
    for (int j = i + 1; j < outs.n; ++j)
      if (overlaps(outs.s[i], outs.s[j]))
        return fail(MOE_ERR_INVALID, "%s overlaps %s", outs.s[i].name, outs.s[j].name);
    for (int j = 0; j < ins.n; ++j)
      if (overlaps(outs.s[i], ins.s[j]))
        return fail(MOE_ERR_INVALID, "%s overlaps %s", outs.s[i].name, ins.s[j].name);
  }
  return MOE_OK;
}

inline int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace api
}  // namespace moe
