// norm.hip -- C entry points of the norms around a block (include/fp8moe.h):
// host-side validation and kernel enqueueing.
#include "norm.hpp"

#include <float.h>

#include "common.hpp"
#include "dense.hpp"
#include "entry.hpp"

using namespace fp8moe;

namespace {

// The end of an entry point that enqueued work (the debug build waits for it).
moe_status finish(hipError_t e, const char *fn) {
  if (e != hipSuccess)
    return fail_status(MOE_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
#ifdef FP8MOE_DEBUG
  if (debug_take_norm())
    return fail_status(MOE_ERR_DEVICE_CHECK, "%s: the check words could not be read", fn);
#endif
  return ok_status();
}

moe_status check_dims(const char *fn, const moe_norm_dims *m) {
  if (!m) return fail_status(MOE_ERR_NULL, "%s: dims is required", fn);
  if (m->type < MOE_T_F32 || m->type > MOE_T_F16 || (m->w_type != MOE_T_F32 && m->w_type != m->type))
    return fail_status(MOE_ERR_UNSUPPORTED, "%s: type=%d, w_type=%d (fp32 or the same type)", fn,
                       m->type, m->w_type);
  if (m->T < 0 || m->T > MOE_MAX_TOKENS || m->d < 16 || m->d % 16 || m->d > MOE_MAX_HIDDEN)
    return fail_status(MOE_ERR_SHAPE, "%s: T=%d (in [0, %d]), d=%d (a multiple of 16 in [16, %d])",
                       fn, m->T, MOE_MAX_TOKENS, m->d, MOE_MAX_HIDDEN);
  if (m->gate_rows < 0 || (m->gate_rows > 0 && m->T % m->gate_rows) ||
      (m->gate_rows > m->T && m->gate_rows > 1))
    return fail_status(MOE_ERR_SHAPE, "%s: gate_rows=%d must divide T=%d", fn, m->gate_rows, m->T);
  if (!(m->eps >= FLT_MIN && m->eps <= FLT_MAX))
    return fail_status(MOE_ERR_SHAPE, "%s: eps must be a positive normal number", fn);
  return MOE_OK;
}

// An array of rows: where it is, its row stride and what it holds.
moe_status check_array(const char *fn, const char *name, const void *p, int64_t ld, int32_t rows,
                       int32_t d, int32_t size) {
  moe_status s = check_rows(fn, rows, ld, d, size);
  if (s) return s;
  if (!p && rows > 0) return fail_status(MOE_ERR_NULL, "%s: %s is required", fn, name);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_norm_residual(const moe_norm_dims *dims, const void *x, int64_t ldx, const void *y,
                             int64_t ldy, const void *w_post, const void *gate, int64_t ldg,
                             const void *w_next, void *r, void *n, float *rstd_y, float *rstd_r,
                             void *stream) {
  const char *fn = "moe_norm_residual";
  moe_status s = check_dims(fn, dims);
  if (s) return s;
  const moe_norm_dims &m = *dims;
  const int32_t size = type_bytes(m.type), wsize = type_bytes(m.w_type);
  if ((s = check_array(fn, "x", x, ldx, m.T, m.d, size))) return s;
  const bool sum = r != nullptr || y != nullptr;
  if (sum && (s = check_array(fn, "y", y, ldy, m.T, m.d, size))) return s;
  if (m.T > 0 && sum && !r) return fail_status(MOE_ERR_NULL, "%s: r is required with y", fn);
  if (!sum && m.T > 0 && (w_post || gate || rstd_y || m.gate_rows))
    return fail_status(MOE_ERR_NULL, "%s: w_post, gate and rstd_y need y", fn);
  if ((m.gate_rows > 0) != (gate != nullptr))
    return fail_status(MOE_ERR_NULL, "%s: gate and gate_rows are given together or not at all", fn);
  if (gate && (s = check_rows(fn, m.gate_rows, ldg, m.d, wsize))) return s;
  if (m.T == 0) return ok_status();
  if (!sum && !w_next) return fail_status(MOE_ERR_NULL, "%s: w_next is required without y", fn);
  if ((w_next != nullptr) != (n != nullptr) || (rstd_r && !w_next) || (rstd_y && !w_post))
    return fail_status(MOE_ERR_NULL, "%s: n and rstd_r go with w_next, rstd_y with w_post", fn);
  if (!all_aligned({x, y, w_post, gate, w_next, r, n}, 16) || !all_aligned({rstd_y, rstd_r}, 4))
    return fail_status(MOE_ERR_ALIGN, "%s: every array must be 16-byte, rstd 4-byte aligned", fn);
  const int64_t rows = (int64_t)m.T * m.d * size, vec = (int64_t)m.d * wsize;
  const Span out[] = {{r, rows}, {n, rows}, {rstd_y, (int64_t)m.T * 4}, {rstd_r, (int64_t)m.T * 4}};
  const Span in[] = {{x, span_rows(m.T, ldx, m.d, size)}, {y, span_rows(m.T, ldy, m.d, size)},
                     {w_post, vec}, {gate, span_rows(m.gate_rows, ldg, m.d, wsize)}, {w_next, vec}};
  if (clash(out, in))
    return fail_status(MOE_ERR_SHAPE, "%s: an output overlaps an input or another output", fn);
  const NormForward p{m.T, m.d, m.type, m.w_type, m.gate_rows, m.scale, m.offset, m.eps, x, ldx, y,
                      ldy, w_post, gate, ldg, w_next, r, n, rstd_y, rstd_r};
  return finish(launch_norm_forward(p, as_stream(stream)), fn);
}

size_t moe_norm_residual_backward_workspace_bytes(const moe_norm_dims *dims) {
  if (check_dims("moe_norm_residual_backward_workspace_bytes", dims)) return 0;
  (void)ok_status();
  return norm_backward_workspace(dims->T, dims->d, dims->gate_rows);
}

moe_status moe_norm_residual_backward(const moe_norm_dims *dims, const void *dr, int64_t lddr,
                                      const void *dn, int64_t lddn, const void *x, int64_t ldx,
                                      const void *y, int64_t ldy, const float *rstd_y,
                                      const float *rstd_r, const void *w_post, const void *gate,
                                      int64_t ldg, const void *w_next, void *dx, void *dy,
                                      void *dw_post, void *dgate, void *dw_next, void *workspace,
                                      size_t workspace_bytes, void *stream) {
  const char *fn = "moe_norm_residual_backward";
  moe_status s = check_dims(fn, dims);
  if (s) return s;
  const moe_norm_dims &m = *dims;
  const int32_t size = type_bytes(m.type), wsize = type_bytes(m.w_type);
  const bool sum = y != nullptr || dy != nullptr;
  if (dr && (s = check_array(fn, "dr", dr, lddr, m.T, m.d, size))) return s;
  if (w_next && ((s = check_array(fn, "dn", dn, lddn, m.T, m.d, size)) ||
                 (s = check_array(fn, "x", x, ldx, m.T, m.d, size))))
    return s;
  if (sum && (s = check_array(fn, "y", y, ldy, m.T, m.d, size))) return s;
  if ((m.gate_rows > 0) != (gate != nullptr))
    return fail_status(MOE_ERR_NULL, "%s: gate and gate_rows are given together or not at all", fn);
  if (gate && (s = check_rows(fn, m.gate_rows, ldg, m.d, wsize))) return s;
  if (!sum && m.T > 0 && (w_post || gate))
    return fail_status(MOE_ERR_NULL, "%s: w_post and gate need y", fn);
  if ((w_post != nullptr) != (dw_post != nullptr) || (gate != nullptr) != (dgate != nullptr) ||
      (w_next != nullptr) != (dw_next != nullptr))
    return fail_status(MOE_ERR_NULL, "%s: every vector has its gradient and the other way round", fn);
  if (m.T > 0) {
    if (!dx || (sum && !dy)) return fail_status(MOE_ERR_NULL, "%s: dx, and dy with y, are required", fn);
    if (!dr && !w_next) return fail_status(MOE_ERR_NULL, "%s: dr is required without w_next", fn);
    if ((w_post && !rstd_y) || (w_next && !rstd_r))
      return fail_status(MOE_ERR_NULL, "%s: rstd_y goes with w_post, rstd_r with w_next", fn);
  }
  if (!all_aligned({dr, dn, x, y, w_post, gate, w_next, dx, dy, dw_post, dgate, dw_next}, 16) ||
      !all_aligned({rstd_y, rstd_r}, 4))
    return fail_status(MOE_ERR_ALIGN, "%s: every array must be 16-byte, rstd 4-byte aligned", fn);
  const size_t need = norm_backward_workspace(m.T, m.d, m.gate_rows);
  if (need && (!workspace || workspace_bytes < need))
    return fail_status(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn,
                       workspace ? workspace_bytes : (size_t)0, need);
  if (!aligned(workspace, 256))
    return fail_status(MOE_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  const int64_t rows = (int64_t)m.T * m.d * size, vec = (int64_t)m.d * wsize;
  const Span out[] = {{dx, rows}, {dy, rows}, {dw_post, vec}, {dgate, m.gate_rows * vec},
                      {dw_next, vec}, {workspace, (int64_t)need}};
  const Span in[] = {{dr, dr ? span_rows(m.T, lddr, m.d, size) : 0},
                     {dn, w_next ? span_rows(m.T, lddn, m.d, size) : 0},
                     {x, w_next ? span_rows(m.T, ldx, m.d, size) : 0},
                     {y, span_rows(m.T, ldy, m.d, size)},
                     {rstd_y, w_post ? (int64_t)m.T * 4 : 0}, {rstd_r, w_next ? (int64_t)m.T * 4 : 0},
                     {w_post, vec}, {gate, span_rows(m.gate_rows, ldg, m.d, wsize)}, {w_next, vec}};
  if (clash(out, in))
    return fail_status(MOE_ERR_SHAPE,
                       "%s: an output or the workspace overlaps an input or another output", fn);
  // without a sum its scale is not read (the kernel multiplies it with zeros for y)
  const float scale = y ? m.scale : 1.0f;
  const NormBackward p{m.T, m.d, m.type, m.w_type, m.gate_rows, scale, m.offset, dr, lddr, dn, lddn,
                       x, ldx, y, ldy, rstd_y, rstd_r, w_post, gate, ldg, w_next, dx, dy, dw_post,
                       dgate, dw_next, static_cast<float *>(workspace)};
  return finish(launch_norm_backward(p, as_stream(stream)), fn);
}

}  // extern "C"
