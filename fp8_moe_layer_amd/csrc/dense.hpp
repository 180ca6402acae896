// dense.hpp -- launch interface between the dense feed-forward entry points
// (dense.hip) and their kernels (kernels_dense.hip).  Every launcher enqueues
// on `stream` and returns the hipError_t of the launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8moe {

// Element types of activations and outputs (MOE_T_* of the C ABI).
enum : int32_t { kTypeF32 = 0, kTypeBf16 = 1, kTypeF16 = 2 };

// Longest K of the int8 product: 65536 * 128 * 128 = 2^30 fits the 32-bit sums.
constexpr int32_t kMaxI8K = 65536;

hipError_t launch_quantize_i8(const void *x, int32_t type, int64_t ldx, int32_t rows, int32_t cols,
                              int8_t *q, float *scale, hipStream_t stream);

// y[t][n] = sum_k xq[t][k] * wq[n][k] * sx[t] * sw[n] (+ bias[n]).
struct I8Product {
  const int8_t *xq;
  int64_t ldx;
  const float *sx;
  const int8_t *wq;
  const float *sw, *bias;
  int32_t T, K, N, out_type;
  void *y;
  void *workspace;  // matmul_i8_workspace bytes or NULL
};
size_t matmul_i8_workspace(int32_t T, int32_t K, int32_t N);
hipError_t launch_matmul_i8(const I8Product &p, hipStream_t stream);

// h = SiLU(g) * u from int8 operands.
struct I8Gated {
  const int8_t *xq;
  int64_t ldx;
  const float *sx;
  const int8_t *w_gate, *w_up;
  const float *s_gate, *s_up;
  int32_t T, d, f, out_type;
  void *h;
  void *workspace;  // gated_i8_workspace bytes or NULL
};
size_t gated_i8_workspace(int32_t T, int32_t d, int32_t f);
hipError_t launch_gated_i8(const I8Gated &p, hipStream_t stream);

// h = SiLU(x Wg^T) * (x Wu^T) in 16-bit types; gate, up: the two products
// kept (fp32) for the backward pass, or both NULL.
struct Gated16 {
  const void *x;
  int64_t ldx;  // elements
  const void *w_gate, *w_up;
  int32_t T, d, f, type;
  void *h;
  float *gate, *up;
  void *workspace;  // gated_workspace bytes or NULL
};
size_t gated_workspace(int32_t T, int32_t d, int32_t f);
hipError_t launch_gated(const Gated16 &p, hipStream_t stream);

struct Gated16Backward {
  const void *dh;
  int64_t lddh;
  const void *x;
  int64_t ldx;
  const void *w_gate, *w_up;
  const float *gate, *up;
  int32_t T, d, f, type;
  void *dx, *dw_gate, *dw_up;
  char *workspace;
};
size_t gated_backward_workspace(int32_t T, int32_t d, int32_t f);
hipError_t launch_gated_backward(const Gated16Backward &p, hipStream_t stream);

// Which kernels the sizes take (MOE_DENSE_* and MOE_FORM_* of the C ABI); the
// launchers above go by the same choice.
enum : int32_t { kOpMatmulI8 = 0, kOpGatedI8 = 1, kOpGated = 2, kOpGatedBackward = 3 };
enum : int32_t {
  kFormNone = 0,
  kFormStream = 1,       // + 0..3
  kFormCut = 8,
  kFormTile = 16,        // + 0..4
  kFormPair = 24,        // + 0..4
  kFormPairSecond = 32,  // + 0..4
};
void dense_form(int32_t op, int32_t T, int32_t inner, int32_t outputs, bool workspace,
                int32_t (&form)[2]);

uint32_t debug_take_dense();

}  // namespace fp8moe
