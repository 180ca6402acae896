/* Runs the host-side code of the dense feed-forward entry points
 * (include/fp8moe.h) that needs no GPU, for a build with AddressSanitizer and
 * UndefinedBehaviourSanitizer on the host: the workspace sizes, and with them
 * the choice of tile and of the parts of K, over a sweep of sizes up to the
 * limits, and validation (every call below fails it or has no tokens, so
 * nothing is enqueued).  Prints "dense host driver ok" and exits 0 on success. */
#include <stdio.h>
#include <stdlib.h>

#include "../../include/fp8moe.h"

#define CHECK(c)                                                      \
  do {                                                                \
    if (!(c)) {                                                       \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
      exit(1);                                                        \
    }                                                                 \
  } while (0)

int main(void) {
  const int Ts[] = {0, 1, 9, 17, 32, 33, 64, 100, 513, 4096, MOE_MAX_TOKENS};
  const int ds[] = {64, 192, 2048, 14336, MOE_MAX_HIDDEN};
  const int Ns[] = {1, 63, 2051, 70000, MOE_MAX_TOKENS};
  const int Ks[] = {16, 80, 4096, 14336, MOE_MAX_I8_K};
  for (unsigned i = 0; i < sizeof Ts / sizeof Ts[0]; ++i) {
    for (unsigned j = 0; j < sizeof ds / sizeof ds[0]; ++j)
      for (unsigned k = 0; k < sizeof ds / sizeof ds[0]; ++k) {
        const int T = Ts[i], d = ds[j], f = ds[k];
        CHECK(moe_gated_ffn_workspace_bytes(T, d, f) <= (size_t)16 << 20);
        CHECK(moe_gated_ffn_i8_workspace_bytes(T, d, f) <= (size_t)16 << 20);
        const size_t b = moe_gated_ffn_backward_workspace_bytes(T, d, f);
        CHECK(b >= (size_t)T * 4 * (size_t)f && b <= (size_t)T * 4 * (size_t)f + ((size_t)17 << 20));
      }
    for (unsigned j = 0; j < sizeof Ks / sizeof Ks[0]; ++j)
      for (unsigned k = 0; k < sizeof Ns / sizeof Ns[0]; ++k)
        CHECK(moe_matmul_i8_workspace_bytes(Ts[i], Ks[j], Ns[k]) <= (size_t)16 << 20);
  }
  CHECK(moe_matmul_i8_workspace_bytes(-1, 64, 64) == 0 && moe_last_error()[0]);
  CHECK(moe_gated_ffn_workspace_bytes(4, 100, 64) == 0 && moe_last_error()[0]);

  int8_t *q = (int8_t *)(uintptr_t)0x10000000;
  float *s = (float *)(uintptr_t)0x20000000, *y = (float *)(uintptr_t)0x30000000;
  CHECK(moe_quantize_rows_i8(y, MOE_T_F32, 64, 4, 64, NULL, s, NULL) == MOE_ERR_NULL);
  CHECK(moe_quantize_rows_i8(y, MOE_T_F32, 60, 4, 64, q, s, NULL) == MOE_ERR_SHAPE);
  CHECK(moe_quantize_rows_i8(y, 9, 64, 4, 64, q, s, NULL) == MOE_ERR_UNSUPPORTED);
  CHECK(moe_quantize_rows_i8(NULL, MOE_T_F16, 64, 0, 64, NULL, NULL, NULL) == MOE_OK);
  CHECK(moe_matmul_i8(q, 64, s, q, s, NULL, 4, 64, 4, MOE_T_BF16, q, NULL, 0, NULL) == MOE_ERR_SHAPE);
  CHECK(moe_matmul_i8(q, 64, s, q, s, NULL, 4, 60, 4, MOE_T_BF16, y, NULL, 0, NULL) == MOE_ERR_SHAPE);
  CHECK(moe_matmul_i8(q, 16384, s, q, s, NULL, 64, 16384, 64, MOE_T_F32, y, y, 16, NULL) ==
        MOE_ERR_WORKSPACE);
  CHECK(moe_gated_ffn_i8(q, 64, s, q, s, q, NULL, 4, 64, 64, MOE_T_F32, y, NULL, 0, NULL) ==
        MOE_ERR_NULL);
  CHECK(moe_gated_ffn(q, 64, q, q, MOE_T_F32, 4, 64, 64, y, NULL, NULL, NULL, 0, NULL) ==
        MOE_ERR_UNSUPPORTED);
  CHECK(moe_gated_ffn(q, 64, q, q, MOE_T_F16, 4, 64, 64, y, s, NULL, NULL, 0, NULL) == MOE_ERR_NULL);
  CHECK(moe_gated_ffn_backward(q, 64, q, 64, q, q, s, s, MOE_T_F16, 4, 64, 64, y, y, y, NULL, 0,
                               NULL) == MOE_ERR_WORKSPACE);
  puts("dense host driver ok");
  return 0;
}
