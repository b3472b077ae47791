/*
 * Sanitizer driver for the host side of dispatch, combine, their gradients, the
 * grouped products and their activations (include/moe.h): linked by
 * tests/test_sanitizers_tokens.py against a host-only build of their
 * translation units under AddressSanitizer and UndefinedBehaviorSanitizer.
 * It calls the size helpers over a sweep that holds the ends of int32, and
 * every entry point with each argument in turn at the ends of its type, beside
 * one that is refused last, so that no call reaches a launch (no device is
 * touched: the pointers below are never dereferenced).
 */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "moe.h"

static int failures = 0;
#define CHECK(c)                                                      \
  do {                                                                \
    if (!(c)) {                                                       \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
      ++failures;                                                     \
    }                                                                 \
  } while (0)

#define FAKE ((void*)0x10000)
#define FAKE_OFF(n) ((void*)(0x10000 + (n)))
#define COUNT(a) (sizeof a / sizeof a[0])

static const int32_t kSizes[] = {INT32_MIN, -1, 0, 1, 2, 8, 16, 17, 64, 512, 513, 1 << 16, (1 << 16) + 16, 1 << 17,
                                 1 << 22, (1 << 26) - 1, 1 << 26, 1 << 30, INT32_MAX - 15, INT32_MAX};
static const int64_t kStrides[] = {INT64_MIN, -16, 0, 1, 64, 1 << 20, 1 << 21, (int64_t)1 << 31, (int64_t)1 << 32,
                                   ((int64_t)1 << 60) + 64, ((int64_t)1 << 61) + 64, ((int64_t)1 << 62) + 64,
                                   ((int64_t)1 << 63) - 64, INT64_MAX};

static void helpers(void) {
  const size_t n = COUNT(kSizes);
  for (size_t a = 0; a < n; ++a)
    for (size_t b = 0; b < n; ++b)
      for (size_t c = 0; c < n; ++c) {
        const int32_t M = kSizes[a], k = kSizes[b], E = kSizes[c];
        const size_t bytes = moe_dispatch_workspace_size(M, k, E);
        if (M < 0 || k < 1 || k > 16 || E < 1 || E > 512 || (int64_t)M * k >= 1 << 26 || (int64_t)M * k <= 4096)
          CHECK(bytes == 0);
        else
          CHECK(bytes == (((size_t)M * k + 1023) / 1024 + 1) * E * 4);
        for (size_t d = 0; d < n; ++d)
          for (size_t e = 0; e < n; e += 1 + (a + b) % 3) {
            const int32_t K = kSizes[d], rows = kSizes[e];
            const size_t need = moe_grouped_int8_workspace_size(M, E, k, K, rows);  // N takes k's values
            if (M < 0 || M >= 1 << 26 || E < 1 || E > 512 || k < 1 || k % 8 || K < 1 || K % 16 || K > 1 << 16 ||
                (int64_t)k * K >= (int64_t)1 << 31 || rows < 0 || rows >= 1 << 26)
              CHECK(need == 0);
            else
              CHECK(need == 0 || need == ((size_t)rows * K + 255) / 256 * 256 + (size_t)rows * 4);
          }
      }
  CHECK(moe_dispatch_workspace_size((1 << 26) - 1, 1, 512) == (size_t)65537 * 512 * 4);
  CHECK(moe_grouped_int8_workspace_size((1 << 26) - 1, 1, 8, 1 << 16, (1 << 26) - 1) ==
        (((size_t)1 << 26) - 1) * 65536 + (((size_t)1 << 26) - 1) * 4);
}

/* Every value of an argument, with `last` refused behind it: never MOE_OK. */
#define EACH(base_of, call, last, field, values)              \
  for (size_t i_ = 0; i_ < COUNT(values); ++i_) {             \
    base_of(&a);                                              \
    last;                                                     \
    a.field = values[i_];                                     \
    const moe_status_t rc = call(&a, NULL);                   \
    CHECK(rc == MOE_ERR_INVALID_ARG || rc == MOE_ERR_UNSUPPORTED || rc == MOE_ERR_WORKSPACE_TOO_SMALL); \
  }
#define CASE(base_of, call, setup, code) \
  do {                                   \
    base_of(&a);                         \
    setup;                               \
    CHECK(call(&a, NULL) == (code));     \
  } while (0)

static void dispatch_base(moe_dispatch_args_t* a) {
  memset(a, 0, sizeof *a);
  a->M = 10, a->top_k = 2, a->E = 4;
  a->ids = FAKE, a->x = FAKE, a->x_stride = 128, a->row_bytes = 128, a->rows = FAKE, a->rows_stride = 128;
  a->offsets = FAKE, a->positions = FAKE, a->pairs = FAKE;
}

static void dispatch(void) {
  moe_dispatch_args_t a;
#define LAST a.offsets = (int32_t*)FAKE_OFF(1)
  EACH(dispatch_base, moe_dispatch, LAST, M, kSizes)
  EACH(dispatch_base, moe_dispatch, LAST, top_k, kSizes)
  EACH(dispatch_base, moe_dispatch, LAST, E, kSizes)
  EACH(dispatch_base, moe_dispatch, LAST, first_expert, kSizes)
  EACH(dispatch_base, moe_dispatch, LAST, row_bytes, kSizes)
#undef LAST
  EACH(dispatch_base, moe_dispatch, a.rows = NULL, x_stride, kStrides)
  /* the largest count of pairs, and strides refused behind it */
  CASE(dispatch_base, moe_dispatch, (a.M = (1 << 26) - 1, a.top_k = 1, a.E = 512), MOE_ERR_INVALID_ARG);
  CASE(dispatch_base, moe_dispatch,
       (a.M = (1 << 22) - 1, a.top_k = 16, a.E = 512, a.workspace = FAKE, a.workspace_bytes = 65536 * 512 * 4),
       MOE_ERR_WORKSPACE_TOO_SMALL);
  for (size_t i = 0; i < COUNT(kStrides); ++i)
    if (kStrides[i] < 128 || kStrides[i] % 16 || kStrides[i] >= 1 << 22)
      CASE(dispatch_base, moe_dispatch, a.rows_stride = kStrides[i],
           kStrides[i] < 128 || kStrides[i] % 16 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
  CHECK(moe_dispatch(NULL, NULL) == MOE_ERR_INVALID_ARG);
}

/* What a stride of elements of `size` bytes is refused with; MOE_OK: it is not. */
static moe_status_t stride_status(int64_t stride, int64_t width, int size) {
  if (stride < width || stride % (16 / size)) return MOE_ERR_INVALID_ARG;
  return stride >= ((int64_t)1 << 22) / size ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

static void combine_base(moe_combine_args_t* a) {
  memset(a, 0, sizeof *a);
  a->M = 10, a->top_k = 2, a->H = 64, a->R = 20;
  a->rows = FAKE, a->rows_stride = 64, a->positions = FAKE, a->weights = FAKE, a->y = FAKE, a->y_stride = 64;
}

static void combine(void) {
  moe_combine_args_t a;
  for (size_t i = 0; i < COUNT(kSizes); ++i) {
    if (kSizes[i] == 0) continue; /* no tokens: nothing to do */
    CASE(combine_base, moe_combine, (a.y = NULL, a.M = kSizes[i]),
         kSizes[i] >= 1 << 25 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG);
  }
  EACH(combine_base, moe_combine, a.y = NULL, top_k, kSizes)
  EACH(combine_base, moe_combine, a.y = NULL, H, kSizes)
  EACH(combine_base, moe_combine, a.y = NULL, R, kSizes)
  for (int f32 = 0; f32 < 2; ++f32)
    for (size_t i = 0; i < COUNT(kStrides); ++i) {
      const moe_status_t want = stride_status(kStrides[i], 64, f32 ? 4 : 2);
      CASE(combine_base, moe_combine,
           (a.y = FAKE_OFF(2), a.rows_type = f32 ? MOE_OUT_FP32 : MOE_OUT_BF16, a.rows_stride = kStrides[i]),
           want == MOE_OK ? MOE_ERR_INVALID_ARG : want);
      if (want != MOE_OK)
        CASE(combine_base, moe_combine, (a.y_type = f32 ? MOE_OUT_FP32 : MOE_OUT_BF16, a.y_stride = kStrides[i]), want);
    }
  CASE(combine_base, moe_combine, a.M = 0, MOE_OK);
  CHECK(moe_combine(NULL, NULL) == MOE_ERR_INVALID_ARG);
}

static void grad_base(moe_combine_grad_args_t* a) {
  memset(a, 0, sizeof *a);
  a->M = 10, a->top_k = 2, a->H = 64, a->R = 20;
  a->dy = FAKE, a->dy_stride = 64, a->rows = FAKE, a->rows_stride = 64, a->positions = FAKE, a->weights = FAKE;
  a->drows = FAKE, a->drows_stride = 64, a->dweights = FAKE;
}

static void grad(void) {
  moe_combine_grad_args_t a;
  for (size_t i = 0; i < COUNT(kSizes); ++i) {
    if (kSizes[i] == 0) continue;
    CASE(grad_base, moe_combine_grad, (a.drows = FAKE_OFF(8), a.M = kSizes[i]),
         kSizes[i] >= 1 << 25 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG);
  }
  EACH(grad_base, moe_combine_grad, a.drows = FAKE_OFF(8), top_k, kSizes)
  EACH(grad_base, moe_combine_grad, a.drows = FAKE_OFF(8), H, kSizes)
  EACH(grad_base, moe_combine_grad, a.drows = FAKE_OFF(8), R, kSizes)
  for (int f32 = 0; f32 < 2; ++f32) {
    const moe_out_t type = f32 ? MOE_OUT_FP32 : MOE_OUT_BF16;
    for (size_t i = 0; i < COUNT(kStrides); ++i) {
      const moe_status_t want = stride_status(kStrides[i], 64, f32 ? 4 : 2), rest = want ? want : MOE_ERR_INVALID_ARG;
      CASE(grad_base, moe_combine_grad, (a.drows = FAKE_OFF(8), a.dy_type = type, a.dy_stride = kStrides[i]), rest);
      CASE(grad_base, moe_combine_grad, (a.drows = FAKE_OFF(8), a.rows_type = type, a.rows_stride = kStrides[i]), rest);
      if (want != MOE_OK)
        CASE(grad_base, moe_combine_grad, (a.drows_type = type, a.drows_stride = kStrides[i]), want);
    }
  }
  CASE(grad_base, moe_combine_grad, a.M = 0, MOE_OK);
  CASE(grad_base, moe_combine_grad, (a.drows = NULL, a.dweights = NULL, a.rows = NULL), MOE_ERR_INVALID_ARG);
  CHECK(moe_combine_grad(NULL, NULL) == MOE_ERR_INVALID_ARG);
}

static void product_base(moe_grouped_int8_args_t* a) {
  const moe_rows_t in = {FAKE, 128, 10, 1, NULL}, out = {FAKE, 64, 10, 1, NULL};
  memset(a, 0, sizeof *a);
  a->R = 10, a->E = 4, a->N = 64, a->K = 128;
  a->offsets = FAKE, a->in = in, a->in_scale = FAKE, a->w = FAKE, a->w_scale = FAKE, a->out = out;
}

static void product(void) {
  moe_grouped_int8_args_t a;
  for (size_t i = 0; i < COUNT(kSizes); ++i) {
    if (kSizes[i] == 0) continue; /* no rows: nothing to do */
    CASE(product_base, moe_grouped_gemm_int8, (a.out.data = NULL, a.R = kSizes[i]),
         kSizes[i] >= 1 << 26 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG);
  }
  EACH(product_base, moe_grouped_gemm_int8, a.out.data = NULL, E, kSizes)
  EACH(product_base, moe_grouped_gemm_int8, a.out.data = NULL, N, kSizes)
  EACH(product_base, moe_grouped_gemm_int8, a.out.data = NULL, K, kSizes)
  EACH(product_base, moe_grouped_gemm_int8, a.out.data = NULL, in.rows, kSizes)
  EACH(product_base, moe_grouped_gemm_int8, (a.out.data = NULL, a.in.ids = FAKE), in.rows, kSizes)
  EACH(product_base, moe_grouped_gemm_int8, (a.out.data = NULL, a.in.ids = FAKE), in.div, kSizes)
  EACH(product_base, moe_grouped_gemm_int8, a.out.data = NULL, in.stride, kStrides)
  EACH(product_base, moe_grouped_gemm_int8, (a.out.data = NULL, a.in_scale = NULL), in.stride, kStrides)
  for (int f32 = 0; f32 < 2; ++f32)
    for (size_t i = 0; i < COUNT(kStrides); ++i)
      if (kStrides[i] < 64 || kStrides[i] % (f32 ? 4 : 8) || kStrides[i] >= 1 << 20)
        CASE(product_base, moe_grouped_gemm_int8,
             (a.out_type = f32 ? MOE_OUT_FP32 : MOE_OUT_BF16, a.out.stride = kStrides[i]),
             kStrides[i] < 64 || kStrides[i] % (f32 ? 4 : 8) ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
  CASE(product_base, moe_grouped_gemm_int8,
       (a.R = (1 << 26) - 1, a.in.rows = a.out.rows = a.R, a.K = 65536, a.in.stride = 65536, a.in_scale = NULL,
        a.workspace = FAKE, a.workspace_bytes = (size_t)1 << 42),
       MOE_ERR_WORKSPACE_TOO_SMALL);
  CASE(product_base, moe_grouped_gemm_int8, a.R = 0, MOE_OK);
  CHECK(moe_grouped_gemm_int8(NULL, NULL) == MOE_ERR_INVALID_ARG);
}

static void bf16_base(moe_grouped_args_t* a) {
  const moe_rows_t in = {FAKE, 128, 10, 1, NULL}, out = {FAKE, 64, 10, 1, NULL};
  memset(a, 0, sizeof *a);
  a->R = 10, a->E = 4, a->N = 64, a->K = 128;
  a->offsets = FAKE, a->in = in, a->w = FAKE, a->out = out;
}

static void wgrad_base(moe_grouped_wgrad_args_t* a) {
  const moe_rows_t dy = {FAKE, 64, 10, 1, NULL}, in = {FAKE, 128, 10, 1, NULL};
  memset(a, 0, sizeof *a);
  a->R = 10, a->E = 4, a->N = 64, a->K = 128;
  a->offsets = FAKE, a->dy = dy, a->in = in, a->dw = FAKE;
}

static void bf16_products(void) {
  {
    moe_grouped_args_t a;
    for (size_t i = 0; i < COUNT(kSizes); ++i)
      if (kSizes[i] != 0) /* no rows: nothing to do */
        CASE(bf16_base, moe_grouped_gemm, (a.out.data = NULL, a.R = kSizes[i]),
             kSizes[i] >= 1 << 26 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG);
    EACH(bf16_base, moe_grouped_gemm, a.out.data = NULL, E, kSizes)
    EACH(bf16_base, moe_grouped_gemm, a.out.data = NULL, N, kSizes)
    EACH(bf16_base, moe_grouped_gemm_dgrad, a.out.data = NULL, K, kSizes)
    EACH(bf16_base, moe_grouped_gemm, (a.out.data = NULL, a.in.ids = FAKE), in.rows, kSizes)
    EACH(bf16_base, moe_grouped_gemm, (a.out.data = NULL, a.in.ids = FAKE), in.div, kSizes)
    EACH(bf16_base, moe_grouped_gemm, a.out.data = NULL, in.stride, kStrides)
    for (size_t i = 0; i < COUNT(kStrides); ++i)
      if (kStrides[i] < 64 || kStrides[i] % 4 || kStrides[i] >= 1 << 20)
        CASE(bf16_base, moe_grouped_gemm, (a.out_type = MOE_OUT_FP32, a.out.stride = kStrides[i]),
             kStrides[i] < 64 || kStrides[i] % 4 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
  }
  moe_grouped_wgrad_args_t a;
#define LAST a.in.data = NULL
  EACH(wgrad_base, moe_grouped_gemm_wgrad, LAST, R, kSizes)
  EACH(wgrad_base, moe_grouped_gemm_wgrad, LAST, E, kSizes)
  EACH(wgrad_base, moe_grouped_gemm_wgrad, LAST, N, kSizes)
  EACH(wgrad_base, moe_grouped_gemm_wgrad, LAST, K, kSizes)
  EACH(wgrad_base, moe_grouped_gemm_wgrad, LAST, dy.stride, kStrides)
#undef LAST
}

static void vectors(void) {
  for (size_t i = 0; i < COUNT(kSizes); ++i) {
    const int32_t n = kSizes[i];
    if (n != 0) {
      CHECK(moe_route_topk_grad(FAKE, FAKE, FAKE, n, 8, 2, NULL, NULL) != MOE_OK);
      CHECK(moe_quant_int8(FAKE, 64, n, 64, FAKE, NULL, NULL) != MOE_OK);
      CHECK(moe_swiglu_int8(FAKE, 128, NULL, n, 64, NULL, FAKE, NULL, NULL) != MOE_OK);
      CHECK(moe_swiglu_checkpoint(FAKE, 128, NULL, n, 64, NULL, NULL, NULL, NULL, NULL) != MOE_OK);
      CHECK(moe_swiglu_checkpoint_grad(FAKE, FAKE, FAKE, NULL, n, 64, NULL, NULL, NULL, NULL, NULL) != MOE_OK);
    }
    CHECK(moe_swiglu_checkpoint(FAKE, INT64_MAX, NULL, 4, n, NULL, NULL, NULL, NULL, NULL) != MOE_OK);
    CHECK(moe_swiglu_checkpoint_grad(FAKE, FAKE, FAKE, NULL, 4, n, NULL, NULL, NULL, NULL, NULL) != MOE_OK);
    CHECK(moe_route_topk_grad(FAKE, FAKE, FAKE, 4, n, 2, NULL, NULL) != MOE_OK);
    CHECK(moe_route_topk_grad(FAKE, FAKE, FAKE, 4, 8, n, NULL, NULL) != MOE_OK);
    CHECK(moe_quant_int8(FAKE, INT64_MAX, 4, n, FAKE, NULL, NULL) != MOE_OK);
    CHECK(moe_swiglu_int8(FAKE, INT64_MAX, NULL, 4, n, NULL, FAKE, NULL, NULL) != MOE_OK);
  }
  for (size_t i = 0; i < COUNT(kStrides); ++i) {
    CHECK(moe_quant_int8(FAKE, kStrides[i], 4, 64, FAKE, NULL, NULL) != MOE_OK);
    CHECK(moe_swiglu_int8(FAKE, kStrides[i], NULL, 4, 64, NULL, FAKE, NULL, NULL) != MOE_OK);
  }
}

int main(void) {
  helpers();
  dispatch();
  combine();
  grad();
  product();
  bf16_products();
  vectors();
  if (failures) {
    fprintf(stderr, "%d checks failed\n", failures);
    return 1;
  }
  printf("abi tokens sanitizer driver ok\n");
  return 0;
}
