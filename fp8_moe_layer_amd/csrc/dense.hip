// dense.hip -- C entry points of the dense feed-forward operators
// (include/fp8moe.h): host-side validation and kernel enqueueing.  No
// allocation, no synchronisation, no state kept between calls.
#include "../../include/fp8moe.h"
#include "dense.hpp"
#include "entry.hpp"

using namespace fp8moe;

static_assert(MOE_T_F32 == kTypeF32 && MOE_T_BF16 == kTypeBf16 && MOE_T_F16 == kTypeF16, "types");
static_assert(MOE_MAX_I8_K == kMaxI8K, "K limit");
static_assert(MOE_DENSE_MATMUL_I8 == kOpMatmulI8 && MOE_DENSE_GATED_I8 == kOpGatedI8 &&
                  MOE_DENSE_GATED == kOpGated && MOE_DENSE_GATED_BACKWARD == kOpGatedBackward, "ops");
static_assert(MOE_FORM_NONE == kFormNone && MOE_FORM_STREAM == kFormStream && MOE_FORM_CUT == kFormCut &&
                  MOE_FORM_TILE == kFormTile && MOE_FORM_PAIR == kFormPair &&
                  MOE_FORM_PAIR_SECOND == kFormPairSecond, "forms");

namespace {

// The end of an entry point that enqueued work (in the debug build: wait for
// it and report the device checks that failed).
moe_status finish(hipError_t e, const char *fn) {
  if (e != hipSuccess)
    return fail_status(MOE_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
#ifdef FP8MOE_DEBUG
  const uint32_t b = debug_take_dense();
  if (b)
    return fail_status(MOE_ERR_DEVICE_CHECK, "%s: device checks failed (0x%x):%s%s", fn, b,
                       (b & 2u) ? " non-finite value in a row to quantise;" : "",
                       (b & 0x80000000u) ? " the check words could not be read;" : "");
#endif
  return ok_status();
}

moe_status check_product_dims(const char *fn, int32_t K, int32_t N) {
  if (K < 16 || K % 16 || K > MOE_MAX_I8_K || N < 1 || N > MOE_MAX_TOKENS)
    return fail_status(MOE_ERR_SHAPE, "%s: K=%d (a multiple of 16 in [16, %d]), N=%d (in [1, %d])",
                       fn, K, MOE_MAX_I8_K, N, MOE_MAX_TOKENS);
  return MOE_OK;
}

moe_status check_gated_dims(const char *fn, int32_t d, int32_t f) {
  if (d < 64 || d % 64 || d > MOE_MAX_HIDDEN)
    return fail_status(MOE_ERR_SHAPE, "%s: d=%d must be a multiple of 64 in [64, %d]", fn, d,
                       MOE_MAX_HIDDEN);
  if (f < 64 || f % 64 || f > MOE_MAX_FFN)
    return fail_status(MOE_ERR_SHAPE, "%s: f=%d must be a multiple of 64 in [64, %d]", fn, f,
                       MOE_MAX_FFN);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_quantize_rows_i8(const void *x, int32_t x_type, int64_t ldx, int32_t rows,
                                int32_t cols, int8_t *q, float *scale, void *stream) {
  const char *fn = "moe_quantize_rows_i8";
  if (x_type < MOE_T_F32 || x_type > MOE_T_F16)
    return fail_status(MOE_ERR_UNSUPPORTED, "%s: x_type=%d", fn, x_type);
  if (cols < 16 || cols % 16 || cols > MOE_MAX_I8_K)
    return fail_status(MOE_ERR_SHAPE, "%s: cols=%d must be a multiple of 16 in [16, %d]", fn, cols,
                       MOE_MAX_I8_K);
  const int32_t size = type_bytes(x_type);
  moe_status s = check_rows(fn, rows, ldx, cols, size);
  if (s) return s;
  if (rows == 0) return ok_status();
  if (!x || !q || !scale) return fail_status(MOE_ERR_NULL, "%s: x, q and scale are required", fn);
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4))
    return fail_status(MOE_ERR_ALIGN, "%s: x and q must be 16-byte and scale 4-byte aligned", fn);
  const Span out[] = {{q, (int64_t)rows * cols}, {scale, (int64_t)rows * 4}};
  const Span in[] = {{x, span_rows(rows, ldx, cols, size)}};
  if (clash(out, in)) return fail_status(MOE_ERR_SHAPE, "%s: q, scale and x overlap", fn);
  return finish(launch_quantize_i8(x, x_type, ldx, rows, cols, q, scale, as_stream(stream)), fn);
}

moe_status moe_matmul_i8(const int8_t *xq, int64_t ldx, const float *sx, const int8_t *wq,
                         const float *sw, const float *bias, int32_t T, int32_t K, int32_t N,
                         int32_t y_type, void *y, void *workspace, size_t workspace_bytes,
                         void *stream) {
  const char *fn = "moe_matmul_i8";
  if (y_type < MOE_T_F32 || y_type > MOE_T_F16)
    return fail_status(MOE_ERR_UNSUPPORTED, "%s: y_type=%d", fn, y_type);
  moe_status s = check_product_dims(fn, K, N);
  if (s || (s = check_rows(fn, T, ldx, K, 1))) return s;
  if (T == 0) return ok_status();
  if (!xq || !sx || !wq || !sw || !y)
    return fail_status(MOE_ERR_NULL, "%s: xq, sx, wq, sw and y are required", fn);
  if (!all_aligned({xq, wq, y}, 16) || !all_aligned({sx, sw, bias}, 4))
    return fail_status(MOE_ERR_ALIGN, "%s: xq, wq and y must be 16-byte, scales and bias 4-byte "
                       "aligned", fn);
  const size_t need = matmul_i8_workspace(T, K, N);
  if ((s = check_workspace(fn, workspace, workspace_bytes, need))) return s;
  const Span out[] = {{y, (int64_t)T * N * type_bytes(y_type)}, {workspace, (int64_t)need}};
  const Span in[] = {{xq, span_rows(T, ldx, K, 1)}, {sx, (int64_t)T * 4}, {wq, (int64_t)N * K},
                     {sw, (int64_t)N * 4},          {bias, (int64_t)N * 4}};
  if (clash(out, in)) return fail_status(MOE_ERR_SHAPE, "%s: y or the workspace overlaps an input or the other", fn);
  const I8Product p{xq, ldx, sx, wq, sw, bias, T, K, N, y_type, y, workspace};
  return finish(launch_matmul_i8(p, as_stream(stream)), fn);
}

moe_status moe_gated_ffn_i8(const int8_t *xq, int64_t ldx, const float *sx, const int8_t *w_gate,
                            const float *s_gate, const int8_t *w_up, const float *s_up, int32_t T,
                            int32_t d, int32_t f, int32_t h_type, void *h, void *workspace,
                            size_t workspace_bytes, void *stream) {
  const char *fn = "moe_gated_ffn_i8";
  if (h_type < MOE_T_F32 || h_type > MOE_T_F16)
    return fail_status(MOE_ERR_UNSUPPORTED, "%s: h_type=%d", fn, h_type);
  moe_status s = check_gated_dims(fn, d, f);
  if (s || (s = check_rows(fn, T, ldx, d, 1))) return s;
  if (T == 0) return ok_status();
  if (!xq || !sx || !w_gate || !s_gate || !w_up || !s_up || !h)
    return fail_status(MOE_ERR_NULL, "%s: xq, sx, w_gate, s_gate, w_up, s_up and h are required",
                       fn);
  if (!all_aligned({xq, w_gate, w_up, h}, 16) || !all_aligned({sx, s_gate, s_up}, 4))
    return fail_status(MOE_ERR_ALIGN, "%s: xq, w_gate, w_up and h must be 16-byte, scales 4-byte "
                       "aligned", fn);
  const size_t need = gated_i8_workspace(T, d, f);
  if ((s = check_workspace(fn, workspace, workspace_bytes, need))) return s;
  const int64_t wb = (int64_t)f * d;
  const Span out[] = {{h, (int64_t)T * f * type_bytes(h_type)}, {workspace, (int64_t)need}};
  const Span in[] = {{xq, span_rows(T, ldx, d, 1)}, {sx, (int64_t)T * 4}, {w_gate, wb}, {w_up, wb},
                     {s_gate, (int64_t)f * 4},      {s_up, (int64_t)f * 4}};
  if (clash(out, in)) return fail_status(MOE_ERR_SHAPE, "%s: h or the workspace overlaps an input or the other", fn);
  const I8Gated p{xq, ldx, sx, w_gate, w_up, s_gate, s_up, T, d, f, h_type, h, workspace};
  return finish(launch_gated_i8(p, as_stream(stream)), fn);
}

moe_status moe_gated_ffn(const void *x, int64_t ldx, const void *w_gate, const void *w_up,
                         int32_t type, int32_t T, int32_t d, int32_t f, void *h, float *gate,
                         float *up, void *workspace, size_t workspace_bytes, void *stream) {
  const char *fn = "moe_gated_ffn";
  if (type != MOE_T_BF16 && type != MOE_T_F16)
    return fail_status(MOE_ERR_UNSUPPORTED, "%s: type=%d (MOE_T_BF16 or MOE_T_F16)", fn, type);
  moe_status s = check_gated_dims(fn, d, f);
  if (s || (s = check_rows(fn, T, ldx, d, 2))) return s;
  if ((gate == nullptr) != (up == nullptr) && T > 0)
    return fail_status(MOE_ERR_NULL, "%s: gate and up are given together or not at all", fn);
  if (T == 0) return ok_status();
  if (!x || !w_gate || !w_up || !h)
    return fail_status(MOE_ERR_NULL, "%s: x, w_gate, w_up and h are required", fn);
  if (!all_aligned({x, w_gate, w_up, h, gate, up}, 16))
    return fail_status(MOE_ERR_ALIGN, "%s: every array must be 16-byte aligned", fn);
  const int64_t wb = (int64_t)f * d * 2, hb = (int64_t)T * f * 2;
  const size_t need = gated_workspace(T, d, f);
  if ((s = check_workspace(fn, workspace, workspace_bytes, need))) return s;
  const Span out[] = {{h, hb}, {gate, 2 * hb}, {up, 2 * hb}, {workspace, (int64_t)need}};
  const Span in[] = {{x, span_rows(T, ldx, d, 2)}, {w_gate, wb}, {w_up, wb}};
  if (clash(out, in))
    return fail_status(MOE_ERR_SHAPE, "%s: an output overlaps an input or another output", fn);
  const Gated16 p{x, ldx, w_gate, w_up, T, d, f, type, h, gate, up, workspace};
  return finish(launch_gated(p, as_stream(stream)), fn);
}

size_t moe_matmul_i8_workspace_bytes(int32_t T, int32_t K, int32_t N) {
  const char *fn = "moe_matmul_i8_workspace_bytes";
  if (check_product_dims(fn, K, N) || check_rows(fn, T, K, K, 1)) return 0;
  (void)ok_status();
  return matmul_i8_workspace(T, K, N);
}

size_t moe_gated_ffn_i8_workspace_bytes(int32_t T, int32_t d, int32_t f) {
  const char *fn = "moe_gated_ffn_i8_workspace_bytes";
  if (check_gated_dims(fn, d, f) || check_rows(fn, T, d, d, 1)) return 0;
  (void)ok_status();
  return gated_i8_workspace(T, d, f);
}

size_t moe_gated_ffn_workspace_bytes(int32_t T, int32_t d, int32_t f) {
  const char *fn = "moe_gated_ffn_workspace_bytes";
  if (check_gated_dims(fn, d, f) || check_rows(fn, T, d, d, 2)) return 0;
  (void)ok_status();
  return gated_workspace(T, d, f);
}

size_t moe_gated_ffn_backward_workspace_bytes(int32_t T, int32_t d, int32_t f) {
  const char *fn = "moe_gated_ffn_backward_workspace_bytes";
  if (check_gated_dims(fn, d, f) || check_rows(fn, T, d, d, 2)) return 0;
  (void)ok_status();
  return gated_backward_workspace(T, d, f);
}

moe_status moe_gated_ffn_backward(const void *dh, int64_t lddh, const void *x, int64_t ldx,
                                  const void *w_gate, const void *w_up, const float *gate,
                                  const float *up, int32_t type, int32_t T, int32_t d, int32_t f,
                                  void *dx, void *dw_gate, void *dw_up, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  const char *fn = "moe_gated_ffn_backward";
  if (type != MOE_T_BF16 && type != MOE_T_F16)
    return fail_status(MOE_ERR_UNSUPPORTED, "%s: type=%d (MOE_T_BF16 or MOE_T_F16)", fn, type);
  moe_status s = check_gated_dims(fn, d, f);
  if (s || (s = check_rows(fn, T, ldx, d, 2)) || (s = check_rows(fn, T, lddh, f, 2))) return s;
  if (!w_gate || !w_up || !dw_gate || !dw_up)
    return fail_status(MOE_ERR_NULL, "%s: w_gate, w_up, dw_gate and dw_up are required", fn);
  if (T > 0 && (!dh || !x || !gate || !up || !dx))
    return fail_status(MOE_ERR_NULL, "%s: dh, x, gate, up and dx are required", fn);
  if (!all_aligned({dh, x, w_gate, w_up, gate, up, dx, dw_gate, dw_up}, 16))
    return fail_status(MOE_ERR_ALIGN, "%s: every array must be 16-byte aligned", fn);
  const size_t need = gated_backward_workspace(T, d, f);
  if (!workspace || workspace_bytes < need)
    return fail_status(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn,
                       workspace ? workspace_bytes : (size_t)0, need);
  if (!aligned(workspace, 256))
    return fail_status(MOE_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  const int64_t wb = (int64_t)f * d * 2, hb = (int64_t)T * f * 2;
  const Span out[] = {{dx, (int64_t)T * d * 2}, {dw_gate, wb}, {dw_up, wb},
                      {workspace, (int64_t)need}};
  const Span in[] = {{dh, span_rows(T, lddh, f, 2)}, {x, span_rows(T, ldx, d, 2)}, {w_gate, wb},
                     {w_up, wb}, {gate, 2 * hb}, {up, 2 * hb}};
  if (clash(out, in))
    return fail_status(MOE_ERR_SHAPE,
                       "%s: an output or the workspace overlaps an input or another output", fn);
  const Gated16Backward p{dh, lddh, x, ldx, w_gate, w_up, gate, up, T, d, f, type,
                          dx, dw_gate, dw_up, (char *)workspace};
  return finish(launch_gated_backward(p, as_stream(stream)), fn);
}

moe_status moe_dense_form(int32_t op, int32_t T, int32_t inner, int32_t outputs, int32_t workspace,
                          int32_t *forms) {
  const char *fn = "moe_dense_form";
  if (op < MOE_DENSE_MATMUL_I8 || op > MOE_DENSE_GATED_BACKWARD)
    return fail_status(MOE_ERR_UNSUPPORTED, "%s: op=%d", fn, op);
  moe_status s = op == MOE_DENSE_MATMUL_I8 ? check_product_dims(fn, inner, outputs)
                                           : check_gated_dims(fn, inner, outputs);
  if (s || (s = check_rows(fn, T, inner, inner, op < MOE_DENSE_GATED ? 1 : 2))) return s;
  if (!forms) return fail_status(MOE_ERR_NULL, "%s: forms is required", fn);
  int32_t form[2];
  dense_form(op, T, inner, outputs, workspace != 0, form);
  forms[0] = form[0];
  forms[1] = form[1];
  return ok_status();
}

}  // extern "C"
