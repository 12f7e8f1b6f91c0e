/* Host-side argument checks of the row, norm and 8-bit block entry points, built
 * with AddressSanitizer and UndefinedBehaviorSanitizer on the host code
 * (tests/test_layer_sanitizers.py). Every call here is rejected (or, with nothing to
 * do, finished) before any HIP runtime call, so no GPU is needed. The pointers are
 * made-up addresses that are never dereferenced. Exit status: the number of failed
 * checks. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "grouped_gemm.h"

static int failures = 0;

static void expect(const char *what, int64_t got, int64_t want) {
  if (got != want) {
    printf("FAIL %s: %lld, expected %lld\n", what, (long long)got, (long long)want);
    ++failures;
  }
}

/* Arrays 2^56 bytes apart: no size within the limits reaches from one to the next. */
#define P(i) ((void *)((uintptr_t)(i) << 56))
#define I(i) ((int32_t *)P(i))
#define F(i) ((float *)P(i))
#define CHECK(want, call) expect(#call, call, want)

int main(void) {
  const int64_t big[] = {INT64_MIN, INT32_MIN, -1, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX - 4096, INT64_MAX};
  const int32_t odd[] = {INT32_MIN, -16, -1, 1 << 30, INT32_MAX - 15, INT32_MAX};
  /* every size at its extremes: refused, and nothing overflows on the way */
  for (unsigned i = 0; i < sizeof big / sizeof *big; ++i) {
    const int64_t T = big[i];
    const gg_status_t want = T < 0 ? GG_ERR_INVALID_VALUE : GG_ERR_UNSUPPORTED;
    CHECK(want, gg_fp8_quantize(P(1), P(2), F(3), T, GG_MAX_K, NULL));
    CHECK(want, gg_expert_sort(P(1), 0, F(2), I(3), I(4), I(5), F(6), P(7), T, 2, 4, NULL));
    CHECK(want, gg_expert_sort(P(1), 1, F(2), I(3), I(4), I(5), F(6), P(7), T, INT32_MAX, 4, NULL));
    CHECK(want, gg_expert_spread(P(1), I(2), P(3), P(4), P(5), 8, T, 1, 1 << 30, INT32_MAX, 5, NULL));
    CHECK(want, gg_expert_spread(P(1), I(2), P(3), NULL, NULL, 0, 5, 1, T < 0 ? T : T / 32 * 16 + 2147483648, 0, 5, NULL));
    if (T > INT32_MAX || T < 0) {
      CHECK(want, gg_expert_spread(P(1), I(2), P(3), NULL, NULL, 0, 5, 1, 64, 0, T, NULL));
      CHECK(want, gg_expert_combine(P(1), 0, I(2), F(3), P(4), 0, 5, 2, 64, T, NULL));
      CHECK(want, gg_expert_combine_grad(P(1), P(2), 1, I(3), F(4), P(5), F(6), 5, 2, 64, T, NULL));
    }
    CHECK(want, gg_expert_combine(P(1), 1, I(2), F(3), P(4), 1, T, 1, GG_MAX_N, 5, NULL));
    CHECK(want, gg_expert_combine_grad(P(1), P(2), 0, I(3), F(4), P(5), F(6), T, 1, GG_MAX_N, 5, NULL));
    CHECK(want, gg_rms_norm_fp8(P(1), P(2), P(3), P(4), F(5), P(6), P(7), T, 16384, 1e-6f, NULL));
    CHECK(want, gg_rms_norm_grad(P(1), P(2), P(3), P(4), P(5), F(6), P(7), T, 16384, 1e-6f, NULL));
    if (T < 0) CHECK(0, gg_expert_sort_workspace(T, 4));
    CHECK(T < 0 ? 0 : gg_rms_norm_grad_workspace(1 << 20, 16384), gg_rms_norm_grad_workspace(T, 16384));
  }
  for (unsigned i = 0; i < sizeof odd / sizeof *odd; ++i) {
    const int32_t n = odd[i], up = n < 0 ? n : n / 16 * 16;
    const gg_status_t want = n < 0 ? GG_ERR_INVALID_VALUE : GG_ERR_UNSUPPORTED;
    CHECK(want, gg_fp8_quantize(P(1), P(2), F(3), INT32_MAX, up, NULL));
    CHECK(want, gg_fp8_quantize_weights(P(1), P(2), F(3), 0, n, GG_MAX_K, GG_MAX_N, NULL));
    CHECK(want, gg_fp8_quantize_weights(P(1), P(2), F(3), 0, 1024, up, GG_MAX_N, NULL));
    CHECK(want, gg_fp8_quantize_weights(P(1), P(2), F(3), 1, 1024, GG_MAX_N, up, NULL));
    CHECK(want, gg_grouped_gemm_fp8_block(P(1), F(2), P(3), F(4), I(5), F(6), n, 256, 256, 29, 0, NULL));
    CHECK(want, gg_grouped_gemm_fp8_block_bf16out(P(1), F(2), P(3), F(4), I(5), P(6), 1024, up, 256, 29, 0, NULL));
    CHECK(want, gg_grouped_gemm_fp8_block_swiglu(P(1), F(2), P(3), F(4), I(5), P(6), 1024, 256, up, 29, 0, NULL));
    CHECK(want, gg_expert_sort(P(1), 0, NULL, I(3), I(4), I(5), NULL, P(7), 5, 2, n, NULL));
    CHECK(want, gg_expert_combine(P(1), 0, I(2), F(3), P(4), 0, INT32_MAX, 1, up, 5, NULL));
    CHECK(want, gg_rms_norm_fp8(P(1), P(2), P(3), P(4), F(5), P(6), P(7), 5, up, 1e-6f, NULL));
    CHECK(want, gg_rms_norm_grad(P(1), P(2), P(3), P(4), P(5), F(6), P(7), 5, up, 1e-6f, NULL));
  }
  CHECK(GG_ERR_INVALID_VALUE, gg_rms_norm_fp8(P(1), P(2), P(3), P(4), F(5), P(6), P(7), 5, 64, NAN, NULL));
  CHECK(GG_ERR_INVALID_VALUE, gg_expert_spread(P(1), I(2), P(3), P(4), P(5), 5, 5, 2, 64, 1, 10, NULL));
  /* an output over the last byte of another array, and one right behind it */
  CHECK(GG_ERR_INVALID_VALUE, gg_fp8_quantize(P(1), (char *)P(1) + 3 * 64 * 2 - 16, F(3), 3, 64, NULL));
  CHECK(GG_ERR_INVALID_VALUE, gg_expert_combine(P(1), 0, I(2), NULL, (char *)P(1) + 10 * 64 * 2 - 16, 0, 5, 2, 64, 10, NULL));
  /* nothing to do */
  CHECK(GG_OK, gg_fp8_quantize(NULL, NULL, NULL, 0, 64, NULL));
  CHECK(GG_OK, gg_expert_spread(NULL, NULL, NULL, NULL, NULL, 0, 0, 2, 64, 0, 0, NULL));
  CHECK(GG_OK, gg_expert_combine(NULL, 0, NULL, NULL, NULL, 0, 0, 2, 64, 0, NULL));
  CHECK(GG_OK, gg_expert_combine_grad(NULL, NULL, 0, NULL, NULL, NULL, NULL, 0, 2, 64, 0, NULL));
  CHECK(GG_OK, gg_rms_norm_fp8(NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, 64, 0.0f, NULL));
  CHECK(GG_OK, gg_grouped_gemm_fp8_block(NULL, NULL, P(3), F(4), I(5), NULL, 4, 256, 256, 0, 0, NULL));
  printf("layer checks: %d failure(s)\n", failures);
  return failures;
}
