// mx4.hip -- C entry points of the 4-bit operators (include/fp8moe.h): host-side
// validation and kernel enqueueing.
#include "mx4.hpp"

#include "common.hpp"
#include "dense.hpp"
#include "entry.hpp"

using namespace fp8moe;

static_assert(MOE_MX4_GROUP == kMxGroup && MOE_MX4_MAX_TOKENS == kMx4MaxTokens &&
                  MOE_MX4_MAX_SHARED == kMx4MaxShared && MOE_MAX_EXPERTS == kMaxExperts &&
                  MOE_MAX_K == kMaxK && MOE_MX4_FORM_STREAM == kMx4Stream &&
                  MOE_MX4_FORM_TILE == kMx4Tile, "limits and forms");

namespace {

// The end of an entry point that enqueued work (in the debug build: wait for it
// and report the device checks that failed).
moe_status finish(hipError_t e, const char *fn) {
  if (e != hipSuccess)
    return fail_status(MOE_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
#ifdef FP8MOE_DEBUG
  const uint32_t b = debug_take_mx4();
  if (b)
    return fail_status(MOE_ERR_DEVICE_CHECK, "%s: device checks failed (0x%x):%s%s%s", fn, b,
                       (b & 1u) ? " k_per_token outside [1, k_max];" : "",
                       (b & 2u) ? " non-finite router logit;" : "",
                       (b & 0x80000000u) ? " the check words could not be read;" : "");
#endif
  return ok_status();
}

moe_status check_matrix(const char *fn, int32_t rows, int32_t cols) {
  if (rows < 0 || rows > MOE_MAX_TOKENS || cols < MOE_MX4_GROUP || cols % MOE_MX4_GROUP ||
      cols > MOE_MAX_MX4_K)
    return fail_status(MOE_ERR_SHAPE, "%s: rows=%d (in [0, %d]), cols=%d (a multiple of %d up to %d)",
                       fn, rows, MOE_MAX_TOKENS, cols, MOE_MX4_GROUP, MOE_MAX_MX4_K);
  return MOE_OK;
}

moe_status check_types(const char *fn, int32_t x_type, int32_t y_type) {
  if ((x_type != MOE_T_BF16 && x_type != MOE_T_F16) || (y_type != x_type && y_type != MOE_T_F32))
    return fail_status(MOE_ERR_UNSUPPORTED,
                       "%s: x_type=%d (MOE_T_BF16 or MOE_T_F16), y_type=%d (the same or MOE_T_F32)",
                       fn, x_type, y_type);
  return MOE_OK;
}

moe_status check_block(const char *fn, int32_t d, int32_t f) {
  if (d < 32 || d % 32 || d > MOE_MAX_HIDDEN || f < 32 || f % 32 || f > MOE_MAX_FFN)
    return fail_status(MOE_ERR_SHAPE, "%s: d=%d, f=%d must be multiples of 32 in [32, %d] and [32, %d]",
                       fn, d, f, MOE_MAX_HIDDEN, MOE_MAX_FFN);
  return MOE_OK;
}

// A required workspace (of no bytes: none).
moe_status need_workspace(const char *fn, const void *workspace, size_t bytes, size_t need) {
  if (need && !workspace)
    return fail_status(MOE_ERR_WORKSPACE, "%s: a workspace of %zu bytes is needed", fn, need);
  return check_workspace(fn, workspace, bytes, need);
}

moe_status check_layer(const char *fn, const moe_dims *m) {
  if (!m) return fail_status(MOE_ERR_NULL, "%s: dims is required", fn);
  if (m->flags) return fail_status(MOE_ERR_UNSUPPORTED, "%s: flags=0x%x must be 0", fn, m->flags);
  if (m->T < 0 || m->T > MOE_MX4_MAX_TOKENS)
    return fail_status(MOE_ERR_SHAPE, "%s: T=%d must be in [0, %d]", fn, m->T, MOE_MX4_MAX_TOKENS);
  const moe_status s = check_block(fn, m->d, m->f);
  if (s) return s;
  if (m->E < 1 || m->E > MOE_MAX_EXPERTS || m->k_max < 1 || m->k_max > MOE_MAX_K || m->k_max > m->E ||
      m->n_shared < 0 || m->n_shared > MOE_MX4_MAX_SHARED)
    return fail_status(MOE_ERR_SHAPE, "%s: E=%d (in [1, %d]), k_max=%d (in [1, min(E, %d)]), n_shared=%d "
                       "(in [0, %d])", fn, m->E, MOE_MAX_EXPERTS, m->k_max, MOE_MAX_K, m->n_shared,
                       MOE_MX4_MAX_SHARED);
  return MOE_OK;
}

size_t layer_workspace(const moe_dims &m) {
  Mx4Moe p{};
  p.T = m.T, p.d = m.d, p.f = m.f, p.E = m.E, p.S = m.n_shared, p.k_max = m.k_max;
  return mx4_moe_workspace(p);
}

int64_t code_bytes(int32_t rows, int32_t cols) { return (int64_t)rows * (cols / 2); }
int64_t scale_bytes(int32_t rows, int32_t cols) { return (int64_t)rows * (cols / MOE_MX4_GROUP); }

}  // namespace

extern "C" {

moe_status moe_quantize_rows_mx4(const void *x, int32_t x_type, int64_t ldx, int32_t rows,
                                 int32_t cols, uint8_t *codes, uint8_t *scales, void *stream) {
  const char *fn = "moe_quantize_rows_mx4";
  if (x_type < MOE_T_F32 || x_type > MOE_T_F16)
    return fail_status(MOE_ERR_UNSUPPORTED, "%s: x_type=%d", fn, x_type);
  const int32_t size = type_bytes(x_type);
  moe_status s = check_matrix(fn, rows, cols);
  if (s || (s = check_rows(fn, rows, ldx, cols, size))) return s;
  if (rows == 0) return ok_status();
  if (!x || !codes || !scales)
    return fail_status(MOE_ERR_NULL, "%s: x, codes and scales are required", fn);
  if (!all_aligned({x, codes}, 16))
    return fail_status(MOE_ERR_ALIGN, "%s: x and codes must be 16-byte aligned", fn);
  const Span out[] = {{codes, code_bytes(rows, cols)}, {scales, scale_bytes(rows, cols)}};
  const Span in[] = {{x, span_rows(rows, ldx, cols, size)}};
  if (clash(out, in)) return fail_status(MOE_ERR_SHAPE, "%s: codes, scales and x overlap", fn);
  return finish(launch_quantize_mx4(x, x_type, ldx, rows, cols, codes, scales, as_stream(stream)), fn);
}

moe_status moe_dequantize_rows_mx4(const uint8_t *codes, const uint8_t *scales, int32_t rows,
                                   int32_t cols, int32_t y_type, void *y, void *stream) {
  const char *fn = "moe_dequantize_rows_mx4";
  if (y_type < MOE_T_F32 || y_type > MOE_T_F16)
    return fail_status(MOE_ERR_UNSUPPORTED, "%s: y_type=%d", fn, y_type);
  moe_status s = check_matrix(fn, rows, cols);
  if (s) return s;
  if (rows == 0) return ok_status();
  if (!codes || !scales || !y)
    return fail_status(MOE_ERR_NULL, "%s: codes, scales and y are required", fn);
  if (!all_aligned({codes, y}, 16))
    return fail_status(MOE_ERR_ALIGN, "%s: codes and y must be 16-byte aligned", fn);
  const Span out[] = {{y, (int64_t)rows * cols * type_bytes(y_type)}};
  const Span in[] = {{codes, code_bytes(rows, cols)}, {scales, scale_bytes(rows, cols)}};
  if (clash(out, in)) return fail_status(MOE_ERR_SHAPE, "%s: y overlaps an input", fn);
  return finish(launch_dequantize_mx4(codes, scales, rows, cols, y_type, y, as_stream(stream)), fn);
}

int64_t moe_packed_mx4_bytes(int32_t rows, int32_t cols) {
  if (rows < 1) rows = -1;
  if (check_matrix("moe_packed_mx4_bytes", rows, cols)) return 0;
  (void)ok_status();
  return Mx4Layout(rows, cols).bytes();
}

moe_status moe_pack_mx4(const uint8_t *codes, const uint8_t *scales, int32_t rows, int32_t cols,
                        void *packed, void *stream) {
  const char *fn = "moe_pack_mx4";
  if (rows < 1) rows = -1;
  moe_status s = check_matrix(fn, rows, cols);
  if (s) return s;
  if (!codes || !scales || !packed)
    return fail_status(MOE_ERR_NULL, "%s: codes, scales and packed are required", fn);
  if (!all_aligned({codes, packed}, 16))
    return fail_status(MOE_ERR_ALIGN, "%s: codes and packed must be 16-byte aligned", fn);
  const Span out[] = {{packed, Mx4Layout(rows, cols).bytes()}};
  const Span in[] = {{codes, code_bytes(rows, cols)}, {scales, scale_bytes(rows, cols)}};
  if (clash(out, in)) return fail_status(MOE_ERR_SHAPE, "%s: packed overlaps an input", fn);
  return finish(launch_pack_mx4(codes, scales, rows, cols, (uint8_t *)packed, as_stream(stream)), fn);
}

size_t moe_matmul_mx4_workspace_bytes(int32_t T, int32_t K, int32_t N) {
  const char *fn = "moe_matmul_mx4_workspace_bytes";
  if (check_matrix(fn, N < 1 ? -1 : N, K) || check_rows(fn, T, K, K, 2)) return 0;
  (void)ok_status();
  return mx4_product_workspace(T, K, N, false);
}

moe_status moe_matmul_mx4(const void *x, int64_t ldx, const void *w, const float *bias, int32_t x_type,
                          int32_t T, int32_t K, int32_t N, int32_t y_type, void *y, void *workspace,
                          size_t workspace_bytes, void *stream) {
  const char *fn = "moe_matmul_mx4";
  moe_status s = check_types(fn, x_type, y_type);
  if (s || (s = check_matrix(fn, N < 1 ? -1 : N, K)) || (s = check_rows(fn, T, ldx, K, 2))) return s;
  if (T == 0) return ok_status();
  if (!x || !w || !y) return fail_status(MOE_ERR_NULL, "%s: x, w and y are required", fn);
  if (!all_aligned({x, w, y}, 16) || !aligned(bias, 4))
    return fail_status(MOE_ERR_ALIGN, "%s: x, w and y must be 16-byte, bias 4-byte aligned", fn);
  const size_t need = mx4_product_workspace(T, K, N, false);
  if ((s = need_workspace(fn, workspace, workspace_bytes, need))) return s;
  const Span out[] = {{y, (int64_t)T * N * type_bytes(y_type)}, {workspace, (int64_t)need}};
  const Span in[] = {{x, span_rows(T, ldx, K, 2)}, {w, Mx4Layout(N, K).bytes()}, {bias, (int64_t)N * 4}};
  if (clash(out, in))
    return fail_status(MOE_ERR_SHAPE, "%s: y or the workspace overlaps an input or the other", fn);
  const Mx4Product p{x, ldx, (const uint8_t *)w, nullptr, bias, T, K, N, x_type, y_type, y, workspace};
  return finish(launch_mx4_product(p, as_stream(stream)), fn);
}

size_t moe_ffn_mx4_workspace_bytes(int32_t T, int32_t d, int32_t f) {
  const char *fn = "moe_ffn_mx4_workspace_bytes";
  if (check_block(fn, d, f) || check_rows(fn, T, d, d, 2)) return 0;
  (void)ok_status();
  return mx4_product_workspace(T, d, f, true);
}

moe_status moe_ffn_mx4(const void *x, int64_t ldx, const void *w_gate, const void *w_up, int32_t type,
                       int32_t T, int32_t d, int32_t f, void *h, void *workspace, size_t workspace_bytes,
                       void *stream) {
  const char *fn = "moe_ffn_mx4";
  moe_status s = check_types(fn, type, type);
  if (s || (s = check_block(fn, d, f)) || (s = check_rows(fn, T, ldx, d, 2))) return s;
  if (T == 0) return ok_status();
  if (!x || !w_gate || !w_up || !h)
    return fail_status(MOE_ERR_NULL, "%s: x, w_gate, w_up and h are required", fn);
  if (!all_aligned({x, w_gate, w_up, h}, 16))
    return fail_status(MOE_ERR_ALIGN, "%s: every array must be 16-byte aligned", fn);
  const int64_t wb = Mx4Layout(f, d).bytes();
  const size_t need = mx4_product_workspace(T, d, f, true);
  if ((s = need_workspace(fn, workspace, workspace_bytes, need))) return s;
  const Span out[] = {{h, (int64_t)T * f * 2}, {workspace, (int64_t)need}};
  const Span in[] = {{x, span_rows(T, ldx, d, 2)}, {w_gate, wb}, {w_up, wb}};
  if (clash(out, in))
    return fail_status(MOE_ERR_SHAPE, "%s: h or the workspace overlaps an input or the other", fn);
  const Mx4Product p{x, ldx, (const uint8_t *)w_gate, (const uint8_t *)w_up, nullptr, T, d, f, type,
                     type, h, workspace};
  return finish(launch_mx4_product(p, as_stream(stream)), fn);
}

moe_status moe_mx4_form(int32_t gated, int32_t T, int32_t inner, int32_t outputs, int32_t *forms) {
  const char *fn = "moe_mx4_form";
  moe_status s = gated ? check_block(fn, inner, outputs) : check_matrix(fn, outputs < 1 ? -1 : outputs, inner);
  if (s || (s = check_rows(fn, T, inner, inner, 2))) return s;
  if (!forms) return fail_status(MOE_ERR_NULL, "%s: forms is required", fn);
  int32_t form[3];
  mx4_form(T, inner, outputs, gated != 0, form);
  for (int i = 0; i < 3; ++i) forms[i] = form[i];
  return ok_status();
}

size_t moe_mx4_workspace_bytes(const moe_dims *dims) {
  if (check_layer("moe_mx4_workspace_bytes", dims)) return 0;
  (void)ok_status();
  return layer_workspace(*dims);
}

moe_status moe_mx4_forward(const moe_dims *dims, int32_t type, const void *x, int64_t ldx,
                           const float *w_router, const float *router_bias,
                           const int32_t *k_per_token, const moe_mx4_weights *w,
                           const float *logits_override, void *out, int32_t *topk_ids_out,
                           float *topk_w_out, void *workspace, size_t workspace_bytes, void *stream) {
  const char *fn = "moe_mx4_forward";
  moe_status s = check_layer(fn, dims);
  if (s || (s = check_types(fn, type, type)) || (s = check_rows(fn, dims->T, ldx, dims->d, 2))) return s;
  const moe_dims &m = *dims;
  if (m.T == 0) return ok_status();
  if (!x || !out || !w || !w->w_gate || !w->w_up || !w->w_down ||
      (m.n_shared > 0 && (!w->ws_gate || !w->ws_up || !w->ws_down)))
    return fail_status(MOE_ERR_NULL, "%s: x, out and the experts' matrices are required", fn);
  if (!w_router && !logits_override)
    return fail_status(MOE_ERR_NULL, "%s: w_router or logits_override is required", fn);
  if (!all_aligned({x, out, w_router, w->w_gate, w->w_up, w->w_down, w->ws_gate, w->ws_up, w->ws_down}, 16) ||
      !all_aligned({router_bias, k_per_token, logits_override, topk_ids_out, topk_w_out}, 4))
    return fail_status(MOE_ERR_ALIGN, "%s: x, out, w_router and the matrices must be 16-byte, the other "
                       "arrays 4-byte aligned", fn);
  const size_t need = layer_workspace(m);
  if (!workspace || workspace_bytes < need)
    return fail_status(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn,
                       workspace ? workspace_bytes : (size_t)0, need);
  if (!aligned(workspace, 256))
    return fail_status(MOE_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  const int64_t gu = Mx4Layout(m.f, m.d).bytes(), dn = Mx4Layout(m.d, m.f).bytes();
  const int64_t slots = (int64_t)m.T * m.k_max * 4, scores = (int64_t)m.T * m.E * 4;
  const Span outs[] = {{out, (int64_t)m.T * m.d * 2}, {topk_ids_out, slots}, {topk_w_out, slots},
                       {workspace, (int64_t)need}};
  const Span ins[] = {{x, span_rows(m.T, ldx, m.d, 2)},
                      {logits_override ? nullptr : w_router, (int64_t)m.E * m.d * 4},
                      {logits_override ? nullptr : router_bias, (int64_t)m.E * 4},
                      {k_per_token, (int64_t)m.T * 4}, {logits_override, scores},
                      {w->w_gate, m.E * gu}, {w->w_up, m.E * gu}, {w->w_down, m.E * dn},
                      {w->ws_gate, m.n_shared * gu}, {w->ws_up, m.n_shared * gu},
                      {w->ws_down, m.n_shared * dn}};
  if (clash(outs, ins))
    return fail_status(MOE_ERR_SHAPE, "%s: an output or the workspace overlaps an input or another output", fn);
  auto u8 = [](const void *p) { return static_cast<const uint8_t *>(p); };
  const Mx4Moe p{x, ldx, m.T, m.d, m.f, m.E, m.n_shared, m.k_max, type, w_router, router_bias,
                 logits_override, k_per_token, u8(w->w_gate), u8(w->w_up), u8(w->w_down), u8(w->ws_gate),
                 u8(w->ws_up), u8(w->ws_down), out, topk_ids_out, topk_w_out, (char *)workspace};
  return finish(launch_mx4_moe(p, as_stream(stream)), fn);
}

}  // extern "C"
