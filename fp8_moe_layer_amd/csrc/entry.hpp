// entry.hpp -- host-side checks shared by the C entry points of the dense
// operators, of the norms and of the 4-bit products.
#pragma once

#include "../../include/fp8moe.h"
#include "internal.hpp"

namespace fp8moe {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int32_t type_bytes(int32_t type) { return type == MOE_T_F32 ? 4 : 2; }

// Longest row stride: a tile's rows (256) stay within the kernels' buffer
// descriptors (2^30 bytes).
constexpr int64_t kMaxRowBytes = (int64_t)1 << 22;

// A caller's array: where it starts and how many bytes it spans.
struct Span {
  const void *p;
  int64_t bytes;
};
inline bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
// Does one of the outputs share memory with an input or another output?
template <int NO, int NI>
bool clash(const Span (&out)[NO], const Span (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
    for (int j = 0; j < NI; ++j)
      if (overlap(out[i], in[j])) return true;
  }
  return false;
}
inline int64_t span_rows(int64_t rows, int64_t ld, int64_t cols, int64_t size) {
  return rows > 0 ? ((rows - 1) * ld + cols) * size : 0;
}

template <int N>
bool all_aligned(const void *const (&p)[N], size_t a) {
  for (const void *q : p)
    if (!aligned(q, a)) return false;
  return true;
}

inline moe_status check_rows(const char *fn, int32_t T, int64_t ld, int32_t cols, int32_t size) {
  if (T < 0 || T > MOE_MAX_TOKENS)
    return fail_status(MOE_ERR_SHAPE, "%s: T=%d must be in [0, %d]", fn, T, MOE_MAX_TOKENS);
  if (ld < cols || ld * size % 16 || ld * size > kMaxRowBytes)
    return fail_status(MOE_ERR_SHAPE,
                       "%s: row stride %lld must be at least the row length %d, a multiple of 16 "
                       "bytes and at most %lld bytes", fn, (long long)ld, cols,
                       (long long)kMaxRowBytes);
  return MOE_OK;
}

// An optional workspace: NULL, or at least `need` bytes.
inline moe_status check_workspace(const char *fn, const void *workspace, size_t bytes, size_t need) {
  if (!workspace) return MOE_OK;
  if (bytes < need)
    return fail_status(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, bytes, need);
  if (!aligned(workspace, 256))
    return fail_status(MOE_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  return MOE_OK;
}

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace fp8moe
