/* Host-side checks of the entry points between the layer and the rest of a
 * model, built with AddressSanitizer and UndefinedBehaviorSanitizer on the
 * library's host code (test_abi_model_operators.py). Every call is rejected
 * before any HIP call. */
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "moe_w4a16.h"

static int fails = 0;
#define CHECK(cond)                                                 \
  do {                                                              \
    if (!(cond)) {                                                  \
      fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #cond);       \
      ++fails;                                                      \
    }                                                               \
  } while (0)

static unsigned char buf[4096] __attribute__((aligned(256)));
#define V ((void*)buf)
#define I ((int32_t*)buf)
#define F ((float*)buf)
#define D ((double*)buf)
#define U16 ((uint16_t*)buf)
#define U8 ((uint8_t*)buf)
#define N_MANY 8193

static const void* grads[N_MANY];
static void* outs[N_MANY];
static int64_t sizes[N_MANY];
static int32_t kinds[N_MANY];

int main(void) {
  const int32_t ext[] = {INT_MIN, -1, 0, 1, 2, 8, 64, 65, 1023, 1024, 1025, 32768, 32769, 1 << 24, (1 << 24) + 1,
                         1 << 30, INT_MAX};
  const int n = (int)(sizeof ext / sizeof ext[0]);
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      for (int k = 0; k < n; ++k) {
        /* without logits nothing is launched */
        int st = moe_route_scored(0, ext[i], ext[j], ext[k], 0, 0, 1, 1, 1, 1, 1.0f, 0, 16, I, F, I, I, I, I, INT64_MAX, 0);
        CHECK(st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED || (st == MOE_OK && ext[i] == 0));
        st = moe_route_scored(0, 4, 1024, 8, 1, F, ext[i], ext[j], ext[k], 0, 1.0f, U8, 16, I, F, I, I, I, I, 1 << 20, 0);
        CHECK(st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED);
        st = moe_route_scored(F, 4, 64, 4, 1, F, 1, 1, 1, 0, 1.0f, U8, ext[i], I, F, I, I, I, 0, ext[j], 0);
        CHECK(st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED);
        st = moe_route_scored_backward(0, ext[i], ext[j], ext[k], 1, 1, 1.0f, I, F, F, F, 0);
        CHECK(st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED || (st == MOE_OK && ext[i] == 0));
        /* without a weight nothing is launched */
        st = moe_add_rms_norm(U16, ext[k], V, INT64_MAX, 0, ext[i], ext[j], 0, 0.0f, 0, 0, U16, INT64_MIN, U8, 1, F,
                              ext[k], F, 0);
        CHECK(st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED || (st == MOE_OK && ext[i] == 0));
        const int64_t w = moe_add_rms_norm_workspace_bytes(ext[i], ext[j]);
        CHECK(w == -1 || w > 0);
        st = moe_add_rms_norm_backward(U16, INT64_MAX, V, ext[k], 1, F, ext[i], ext[j], U16, 0, 0, V, INT64_MAX, F, V,
                                       w > 0 ? w - 1 : 0, 0);
        CHECK(st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED || st == MOE_ERR_WORKSPACE);
      }
  for (int i = 0; i < N_MANY; ++i) {
    grads[i] = outs[i] = (void*)(uintptr_t)(((uint64_t)i + 1) << 42); /* the largest tensors, end to end */
    sizes[i] = (int64_t)1 << 40;
    kinds[i] = MOE_DTYPE_F32;
  }
  CHECK(moe_grad_sumsq(grads, sizes, kinds, N_MANY, D, V, INT64_MAX, 0) == MOE_ERR_UNSUPPORTED);
  CHECK(moe_grad_sumsq(grads, sizes, kinds, 8192, D, V, moe_grad_norm_workspace_bytes(8192) - 1, 0) == MOE_ERR_WORKSPACE);
  CHECK(moe_grad_clip(grads, outs, sizes, kinds, 8192, D, -0.5f, F, 0) == MOE_ERR_INVALID_ARG);
  CHECK(moe_grad_clip(grads, outs, sizes, kinds, 8192, D, NAN, F, 0) == MOE_ERR_INVALID_ARG);
  outs[0] = (void*)((uintptr_t)grads[8191] + 8); /* found among all of them */
  sizes[0] = 1;
  CHECK(moe_grad_clip(grads, outs, sizes, kinds, 8192, D, 1.0f, F, 0) == MOE_ERR_INVALID_ARG);
  outs[0] = (void*)((uintptr_t)grads[4000] - 4);
  sizes[0] = 2;
  CHECK(moe_grad_clip(grads, outs, sizes, kinds, 8192, D, 1.0f, F, 0) == MOE_ERR_INVALID_ARG);
  if (fails) return 1;
  printf("model operator checks passed\n");
  return 0;
}
