// norm.hpp -- launch interface between the norms' entry points (norm.hip) and
// their kernels (kernels_norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8moe {

// r = x + scale * gate(t) * norm(y; w_post), n = norm(r; w_next); see
// moe_norm_residual.  y == nullptr: n = norm(x; w_next).
struct NormForward {
  int32_t T, d, type, w_type, gate_rows;
  float scale, offset, eps;
  const void *x;
  int64_t ldx;  // elements, as every ld
  const void *y;
  int64_t ldy;
  const void *w_post, *gate;
  int64_t ldg;
  const void *w_next;
  void *r, *n;
  float *rstd_y, *rstd_r;
};
hipError_t launch_norm_forward(const NormForward &p, hipStream_t stream);

struct NormBackward {
  int32_t T, d, type, w_type, gate_rows;
  float scale, offset;
  const void *dr;
  int64_t lddr;
  const void *dn;
  int64_t lddn;
  const void *x;
  int64_t ldx;
  const void *y;
  int64_t ldy;
  const float *rstd_y, *rstd_r;
  const void *w_post, *gate;
  int64_t ldg;
  const void *w_next;
  void *dx, *dy, *dw_post, *dgate, *dw_next;
  float *workspace;
};
size_t norm_backward_workspace(int32_t T, int32_t d, int32_t gate_rows);
hipError_t launch_norm_backward(const NormBackward &p, hipStream_t stream);
uint32_t debug_take_norm();

}  // namespace fp8moe
