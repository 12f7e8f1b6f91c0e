/* Host-side argument checks of the gradients and the 4-bit operators, built with
 * AddressSanitizer and UndefinedBehaviorSanitizer on the host code
 * (tests/test_operator_sanitizers.py). Every call here is rejected (or, with no
 * rows, finished) before any HIP runtime call, so no GPU is needed. The pointers
 * are made-up addresses that are never dereferenced. Exit status: the number of
 * failed checks. */
#include <stdint.h>
#include <stdio.h>

#include "grouped_gemm.h"

static int failures = 0;

static void expect(const char *what, const char *which, gg_status_t got, gg_status_t want) {
  if (got != want) {
    printf("FAIL %s: %s: status %d, expected %d\n", what, which, (int)got, (int)want);
    ++failures;
  }
}

/* Arrays 2^56 bytes apart: no size within the limits reaches from one to the next. */
#define HOME(i) ((uintptr_t)(i) << 56)
#define P(x) ((void *)(uintptr_t)(x))
#define OFF(x) ((const int32_t *)(uintptr_t)(x))

struct args {
  uintptr_t in1, in2, in3, in4, off, out, h;
  int32_t E, K, N, M, bm;
};

static gg_status_t dgrad(struct args a) {
  return gg_grouped_gemm_bf16_dgrad(P(a.in1), P(a.in2), OFF(a.off), (float *)P(a.out), a.E, a.K, a.N,
                                    a.M, a.bm, NULL);
}
static gg_status_t dgrad_bf16(struct args a) {
  return gg_grouped_gemm_bf16_dgrad_bf16out(P(a.in1), P(a.in2), OFF(a.off), P(a.out), a.E, a.K, a.N,
                                            a.M, a.bm, NULL);
}
static gg_status_t dgrad_swiglu(struct args a) {
  return gg_grouped_gemm_bf16_dgrad_swiglu(P(a.in1), P(a.in2), OFF(a.off), P(a.in3), P(a.out), P(a.h),
                                           a.E, a.K, a.N, a.M, a.bm, NULL);
}
static gg_status_t wgrad(struct args a) {
  return gg_grouped_gemm_bf16_wgrad(P(a.in1), P(a.in2), OFF(a.off), (float *)P(a.out), 0, a.E, a.K, a.N,
                                    a.M, NULL);
}
static gg_status_t wgrad_add(struct args a) {
  return gg_grouped_gemm_bf16_wgrad(P(a.in1), P(a.in2), OFF(a.off), (float *)P(a.out), 1, a.E, a.K, a.N,
                                    a.M, NULL);
}
static gg_status_t wgrad_bf16(struct args a) {
  return gg_grouped_gemm_bf16_wgrad_bf16out(P(a.in1), P(a.in2), OFF(a.off), P(a.out), a.E, a.K, a.N, a.M,
                                            NULL);
}
static gg_status_t mx4(struct args a) {
  return gg_grouped_gemm_mx4(P(a.in1), P(a.in2), P(a.in3), P(a.in4), OFF(a.off), (float *)P(a.out), a.E,
                             a.K, a.N, a.M, a.bm, NULL);
}
static gg_status_t mx4_bf16(struct args a) {
  return gg_grouped_gemm_mx4_bf16out(P(a.in1), P(a.in2), P(a.in3), P(a.in4), OFF(a.off), P(a.out), a.E,
                                     a.K, a.N, a.M, a.bm, NULL);
}
static gg_status_t mx4_swiglu(struct args a) {
  return gg_grouped_gemm_mx4_swiglu(P(a.in1), P(a.in2), P(a.in3), P(a.in4), OFF(a.off), P(a.out), a.E,
                                    a.K, a.N, a.M, a.bm, NULL);
}

enum kind { DGRAD, DGRAD_SWIGLU, WGRAD, MX4 };

int main(void) {
  const struct {
    const char *name;
    gg_status_t (*fn)(struct args);
    enum kind kind;
  } fns[] = {{"dgrad", dgrad, DGRAD},
             {"dgrad bf16", dgrad_bf16, DGRAD},
             {"dgrad swiglu", dgrad_swiglu, DGRAD_SWIGLU},
             {"wgrad", wgrad, WGRAD},
             {"wgrad accumulate", wgrad_add, WGRAD},
             {"wgrad bf16", wgrad_bf16, WGRAD},
             {"mx4", mx4, MX4},
             {"mx4 bf16", mx4_bf16, MX4},
             {"mx4 swiglu", mx4_swiglu, MX4}};
  for (size_t i = 0; i < sizeof(fns) / sizeof(fns[0]); ++i) {
    const struct args good = {HOME(1), HOME(2), HOME(3), HOME(4), HOME(5), HOME(6),
                              HOME(7), 4,       256,     256,     29,      0};
    const enum kind kind = fns[i].kind;
    struct args a;
#define CASE(text, change, want)                       \
  do {                                                 \
    a = good;                                          \
    change;                                            \
    expect(fns[i].name, text, fns[i].fn(a), want);     \
  } while (0)
    CASE("null offsets", a.off = 0, GG_ERR_INVALID_VALUE);
    CASE("null output", a.out = 0, GG_ERR_INVALID_VALUE);
    CASE("null first input", a.in1 = 0, GG_ERR_INVALID_VALUE);
    CASE("null second input", a.in2 = 0, GG_ERR_INVALID_VALUE);
    CASE("misaligned offsets", a.off += 2, GG_ERR_MISALIGNED);
    CASE("misaligned input", a.in1 += 8, GG_ERR_MISALIGNED);
    CASE("misaligned output", a.out += 8, GG_ERR_MISALIGNED);
    CASE("output over the first input", a.out = a.in1, GG_ERR_INVALID_VALUE);
    CASE("output over the second input's end", a.out = a.in2 + 16, GG_ERR_INVALID_VALUE);
    CASE("output over the offsets", a.out = a.off, GG_ERR_INVALID_VALUE);
    CASE("E = 0", a.E = 0, GG_ERR_INVALID_VALUE);
    CASE("E < 0", a.E = INT32_MIN, GG_ERR_INVALID_VALUE);
    CASE("K = 0", a.K = 0, GG_ERR_INVALID_VALUE);
    CASE("K < 0", a.K = INT32_MIN, GG_ERR_INVALID_VALUE);
    CASE("N < 0", a.N = INT32_MIN, GG_ERR_INVALID_VALUE);
    CASE("M_cap < 0", a.M = INT32_MIN, GG_ERR_INVALID_VALUE);
    CASE("E too large", a.E = GG_MAX_EXPERTS + 1, GG_ERR_UNSUPPORTED);
    CASE("E largest int", a.E = INT32_MAX, GG_ERR_UNSUPPORTED);
    CASE("M_cap near the end", a.M = INT32_MAX - 255, GG_ERR_UNSUPPORTED);
    CASE("M_cap at the end", a.M = INT32_MAX, GG_ERR_UNSUPPORTED);
    CASE("K past its limit", a.K = 1 << 25, GG_ERR_UNSUPPORTED);
    CASE("N past its limit", a.N = 1 << 25, GG_ERR_UNSUPPORTED);
    CASE("largest multiples of 32", (a.K = a.N = INT32_MAX - 31, a.E = GG_MAX_EXPERTS, a.M = INT32_MAX - 256),
         GG_ERR_UNSUPPORTED);
    CASE("N not a multiple of 8", a.N = 100, GG_ERR_MISALIGNED);
    CASE("K not a multiple of 8", a.K = 100, GG_ERR_MISALIGNED);
    if (kind != WGRAD) {
      CASE("bm = 24", a.bm = 24, GG_ERR_INVALID_VALUE);
      CASE("bm < 0", a.bm = INT32_MIN, GG_ERR_INVALID_VALUE);
      CASE("no rows", a.M = 0, GG_OK);
      CASE("no rows, null arrays of rows", (a.M = 0, a.in1 = a.out = a.h = 0), GG_OK);
      /* the tile bound at its end, then past it */
      CASE("largest bound", (a.M = 1 << 28, a.K = a.N = 15 * 256, a.out = a.off), GG_ERR_INVALID_VALUE);
      CASE("past the largest bound", (a.M = 1 << 28, a.K = a.N = 16 * 256), GG_ERR_UNSUPPORTED);
      CASE("widest columns",
           (a.E = 1, a.M = 1, a.K = kind == MX4 ? GG_MAX_K : GG_MAX_N, a.N = kind == MX4 ? GG_MAX_N : GG_MAX_DGRAD_N,
            a.out = a.off),
           GG_ERR_INVALID_VALUE);
      CASE("all limits at once",
           (a.E = GG_MAX_EXPERTS, a.M = 1 << 15, a.bm = 256, a.K = kind == MX4 ? GG_MAX_K : GG_MAX_N / 8,
            a.N = kind == MX4 ? GG_MAX_N / 8 : GG_MAX_DGRAD_N, a.out = a.off),
           GG_ERR_INVALID_VALUE);
    } else {
      CASE("longest rows", (a.E = 1, a.K = GG_MAX_K, a.N = 8, a.M = INT32_MAX - 256, a.out = a.off),
           GG_ERR_INVALID_VALUE);
      CASE("tiles past a launch", (a.E = GG_MAX_EXPERTS, a.K = a.N = GG_MAX_K), GG_ERR_UNSUPPORTED);
      CASE("largest grid", (a.E = 1023, a.K = 128, a.N = 16383 * 256, a.out = a.off), GG_ERR_INVALID_VALUE);
    }
    if (kind == DGRAD_SWIGLU) {
      CASE("null C", a.in3 = 0, GG_ERR_INVALID_VALUE);
      CASE("misaligned H", a.h += 8, GG_ERR_MISALIGNED);
      CASE("H over dC", a.h = a.out, GG_ERR_INVALID_VALUE);
      CASE("H over C", a.h = a.in3, GG_ERR_INVALID_VALUE);
      CASE("dC over C from its second row", a.out = a.in3 + 1024, GG_ERR_INVALID_VALUE);
    }
    if (kind == MX4) {
      CASE("null weight codes", a.in3 = 0, GG_ERR_INVALID_VALUE);
      CASE("null weight scales", a.in4 = 0, GG_ERR_INVALID_VALUE);
      CASE("K not a multiple of 32", a.K = 264, GG_ERR_MISALIGNED);
      CASE("output over the weights' scales", a.out = a.in4, GG_ERR_INVALID_VALUE);
    }
  }

  const char *q = "quantize", *w = "quantize weights", *d = "dequantize";
  expect(q, "rows < 0", gg_mx4_quantize(P(16), P(HOME(2)), P(HOME(3)), INT64_MIN, 64, NULL), GG_ERR_INVALID_VALUE);
  expect(q, "rows past int32", gg_mx4_quantize(P(16), P(HOME(2)), P(HOME(3)), INT64_MAX, 64, NULL), GG_ERR_UNSUPPORTED);
  expect(q, "largest launch, null values", gg_mx4_quantize(NULL, P(32), P(48), (1 << 24) - 1, 8192, NULL),
         GG_ERR_INVALID_VALUE);
  expect(q, "past the largest launch", gg_mx4_quantize(NULL, P(32), P(48), 1 << 24, 8192, NULL), GG_ERR_UNSUPPORTED);
  expect(q, "largest rows over each other", gg_mx4_quantize(P(16), P(32), P(48), INT32_MAX, 32, NULL),
         GG_ERR_INVALID_VALUE);
  expect(q, "longest rows over each other", gg_mx4_quantize(P(16), P(32), P(48), 1, GG_MAX_K, NULL),
         GG_ERR_INVALID_VALUE);
  expect(q, "misaligned", gg_mx4_quantize(P(24), P(32), P(48), 3, 64, NULL), GG_ERR_MISALIGNED);
  expect(q, "K largest int", gg_mx4_quantize(P(16), P(32), P(48), 3, INT32_MAX - 31, NULL), GG_ERR_UNSUPPORTED);
  expect(q, "nothing to do", gg_mx4_quantize(NULL, NULL, NULL, 0, 64, NULL), GG_OK);
  expect(w, "null", gg_mx4_quantize_weights(P(16), NULL, P(48), 2, 64, 8, NULL), GG_ERR_INVALID_VALUE);
  expect(w, "largest ints", gg_mx4_quantize_weights(P(16), P(32), P(48), INT32_MAX, INT32_MAX - 31, INT32_MAX - 7, NULL),
         GG_ERR_UNSUPPORTED);
  expect(w, "limits at once", gg_mx4_quantize_weights(P(16), P(32), P(48), GG_MAX_EXPERTS, GG_MAX_K, GG_MAX_N, NULL),
         GG_ERR_UNSUPPORTED);
  expect(w, "largest launch over each other", gg_mx4_quantize_weights(P(16), P(32), P(48), 1023, 1 << 21, 256, NULL),
         GG_ERR_INVALID_VALUE);
  expect(w, "misaligned N", gg_mx4_quantize_weights(P(16), P(32), P(48), 2, 64, 12, NULL), GG_ERR_MISALIGNED);
  expect(d, "batch < 0", gg_mx4_dequantize(P(16), P(32), P(48), INT32_MIN, 3, 64, NULL), GG_ERR_INVALID_VALUE);
  expect(d, "batch too large", gg_mx4_dequantize(P(16), P(32), P(48), INT32_MAX, 3, 64, NULL), GG_ERR_UNSUPPORTED);
  expect(d, "largest batch over each other", gg_mx4_dequantize(P(16), P(32), P(48), 65535, INT32_MAX, 32, NULL),
         GG_ERR_INVALID_VALUE);
  expect(d, "nothing to do", gg_mx4_dequantize(NULL, NULL, NULL, 0, 3, 64, NULL), GG_OK);
  printf("operator checks: %d failure(s)\n", failures);
  return failures;
}
