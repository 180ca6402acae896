/* Runs the host-side code of the norms' and the 4-bit operators' entry points
 * (include/fp8moe.h) that needs no GPU, for a build with AddressSanitizer and
 * UndefinedBehaviourSanitizer on the host: the workspace and packed sizes, and with
 * them the choice of form and of the parts of K, over a sweep of sizes up to the
 * limits, and validation (every call below fails it or has no tokens, so nothing is
 * enqueued).  Prints "mx4 host driver ok" and exits 0 on success. */
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
  const int Ts[] = {0, 1, 4, 5, 16, 17, 32, 33, 100, 513, 4096, MOE_MAX_TOKENS};
  const int Ks[] = {32, 160, 4096, 14336, MOE_MAX_MX4_K};
  const int Ns[] = {1, 33, 2051, 70000, MOE_MAX_TOKENS};
  const int ds[] = {32, 96, 2048, 14336, MOE_MAX_HIDDEN};
  const int64_t GB = (int64_t)1 << 30;
  for (unsigned i = 0; i < sizeof Ts / sizeof Ts[0]; ++i) {
    const int T = Ts[i];
    for (unsigned j = 0; j < sizeof Ks / sizeof Ks[0]; ++j)
      for (unsigned k = 0; k < sizeof Ns / sizeof Ns[0]; ++k)
        CHECK((int64_t)moe_matmul_mx4_workspace_bytes(T, Ks[j], Ns[k]) <= 8 * GB);
    for (unsigned j = 0; j < sizeof ds / sizeof ds[0]; ++j)
      for (unsigned k = 0; k < sizeof ds / sizeof ds[0]; ++k) {
        CHECK((int64_t)moe_ffn_mx4_workspace_bytes(T, ds[j], ds[k]) <= 8 * GB);
        for (int E = 1; E <= MOE_MAX_EXPERTS && T <= MOE_MX4_MAX_TOKENS; E *= 8) {
          moe_dims m = {T, ds[j], ds[k], E, E < 32 ? E : 32, E % 3 ? 0 : MOE_MX4_MAX_SHARED, 16, 0};
          const size_t n = moe_mx4_workspace_bytes(&m);
          CHECK(n >= (size_t)T * m.k_max * 4 * (size_t)m.f && n <= ((size_t)1 << 30));
        }
      }
    for (int d = 16; d <= MOE_MAX_HIDDEN; d *= 4)
      for (int g = 0; g < 3; ++g) {
        moe_norm_dims m = {T, d, MOE_T_BF16, MOE_T_F32, g == 2 ? T : g, 1.0f, 0.0f, 1e-6f};
        const size_t n = moe_norm_residual_backward_workspace_bytes(&m);
        CHECK(T == 0 ? n == 0 : n > 0 && n <= (size_t)512 * 3 * 4 * (size_t)d);
      }
  }
  CHECK(moe_packed_mx4_bytes(MOE_MAX_TOKENS, MOE_MAX_MX4_K) > 64 * GB);
  CHECK(moe_packed_mx4_bytes(-4, 64) == 0 && moe_last_error()[0]);
  CHECK(moe_matmul_mx4_workspace_bytes(4, 100, 64) == 0 && moe_last_error()[0]);
  CHECK(moe_ffn_mx4_workspace_bytes(-1, 64, 64) == 0 && moe_last_error()[0]);
  CHECK(moe_mx4_workspace_bytes(NULL) == 0 && moe_last_error()[0]);
  CHECK(moe_norm_residual_backward_workspace_bytes(NULL) == 0 && moe_last_error()[0]);

  uint8_t *c = (uint8_t *)(uintptr_t)0x10000000, *s = (uint8_t *)(uintptr_t)0x20000000;
  float *y = (float *)(uintptr_t)0x30000000;
  CHECK(moe_quantize_rows_mx4(y, MOE_T_F32, 64, 4, 64, NULL, s, NULL) == MOE_ERR_NULL);
  CHECK(moe_quantize_rows_mx4(y, MOE_T_F32, 64, 4, 48, c, s, NULL) == MOE_ERR_SHAPE);
  CHECK(moe_quantize_rows_mx4(NULL, MOE_T_F16, 64, 0, 64, NULL, NULL, NULL) == MOE_OK);
  CHECK(moe_dequantize_rows_mx4(c, s, 4, 64, 5, y, NULL) == MOE_ERR_UNSUPPORTED);
  CHECK(moe_pack_mx4(c, s, 4, 64, c, NULL) == MOE_ERR_SHAPE);
  CHECK(moe_matmul_mx4(c, 64, s, NULL, MOE_T_BF16, 4, 64, 32, MOE_T_F16, y, NULL, 0, NULL) ==
        MOE_ERR_UNSUPPORTED);
  CHECK(moe_matmul_mx4_workspace_bytes(16, 14336, 64) > 0);
  CHECK(moe_matmul_mx4(c, 14336, s, NULL, MOE_T_BF16, 16, 14336, 64, MOE_T_F32, y, NULL, 0, NULL) ==
        MOE_ERR_WORKSPACE);
  CHECK(moe_ffn_mx4(c, 64, s, s, MOE_T_F32, 4, 64, 64, y, NULL, 0, NULL) == MOE_ERR_UNSUPPORTED);
  moe_dims m = {4, 64, 64, 8, 2, 0, 16, 0};
  moe_mx4_weights w = {c, c, c, NULL, NULL, NULL};
  CHECK(moe_mx4_forward(&m, MOE_T_BF16, y, 64, y, NULL, NULL, &w, NULL, s, NULL, NULL, NULL, 0, NULL) ==
        MOE_ERR_WORKSPACE);
  m.n_shared = 1;
  CHECK(moe_mx4_forward(&m, MOE_T_BF16, y, 64, y, NULL, NULL, &w, NULL, s, NULL, NULL, NULL, 0, NULL) ==
        MOE_ERR_NULL);
  moe_norm_dims d = {4, 64, MOE_T_F32, MOE_T_F32, 0, 1.0f, 0.0f, 1e-6f};
  CHECK(moe_norm_residual(&d, y, 64, NULL, 0, NULL, NULL, 0, NULL, NULL, NULL, NULL, NULL, NULL) == MOE_ERR_NULL);
  CHECK(moe_norm_residual_backward(&d, y, 64, NULL, 0, NULL, 0, NULL, 0, NULL, NULL, NULL, NULL, 0, NULL, c,
                                   NULL, NULL, NULL, NULL, NULL, 0, NULL) == MOE_ERR_WORKSPACE);
  puts("mx4 host driver ok");
  return 0;
}
