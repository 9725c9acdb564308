/* Host-side checks of the operators' entry points, built with
 * AddressSanitizer and UndefinedBehaviorSanitizer on the library's host code
 * (test_abi_operators.py). Every call is rejected before any HIP call; the
 * sizes are the largest that the size arithmetic meets. */
#include <limits.h>
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
#define U16 ((uint16_t*)buf)

int main(void) {
  const int32_t ext[] = {INT_MIN, -1, 0, 1, 7, 8, 1023, 1024, 1025, 65535, 65536, 1 << 20, (1 << 20) + 1, 1 << 24,
                         (1 << 24) + 1, 1 << 30, INT_MAX};
  const int n = (int)(sizeof ext / sizeof ext[0]);
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      for (int k = 0; k < n; ++k) {
        const int64_t w = moe_balance_workspace_bytes(ext[i], ext[j], ext[k]);
        CHECK(w == -1 || w > 0);
        /* a workspace one byte short, or sizes that are refused */
        const int st = moe_balance_loss(F, I, ext[i], ext[j], 1, I, ext[k], 0, I, F, I, F, V, w > 0 ? w - 1 : 0, 0);
        CHECK(st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED || st == MOE_ERR_WORKSPACE);
        CHECK(moe_balance_loss_backward(0, ext[i], ext[j], ext[k], I, 1, 0, I, I, F, F, 0) != MOE_ERR_HIP);
        for (int r = 8; r <= 128; r += 120)
          for (int back = 0; back < 2; ++back) {
            /* rows, adapters, widths */
            const int64_t l = moe_lora_workspace_bytes(ext[i], ext[j], ext[k], ext[(k + 5) % n], r, back);
            CHECK(l == -1 || l > 0 || ext[i] == 0);
            const int32_t K = ext[k], N = ext[(k + 5) % n];
            const int64_t short_by_one = l > 0 ? l - 1 : 0;
            const int fs =
                back ? moe_lora_backward(V, N, 1, U16, K, I, F, ext[i], ext[j], K, N, r, U16, U16, F, U16, K, U16, K, F,
                                         F, V, short_by_one, 0)
                     : moe_lora_forward(U16, K, I, ext[i], ext[j], K, N, r, U16, U16, F, V, N, V, N, 1, F, V,
                                        short_by_one, 0);
            CHECK(fs != MOE_ERR_HIP);
            CHECK(fs != MOE_OK || ext[i] == 0);
          }
      }
  CHECK(moe_lora_forward(U16, INT64_MAX, I, 4, 1, 8, 8, 8, U16, U16, F, V, INT64_MAX, V, INT64_MIN, 0, F, V, 0, 0) ==
        MOE_ERR_INVALID_ARG);
  CHECK(moe_lora_forward(U16, INT64_MAX - 7, I, 4, 1, 8, 8, 8, U16, U16, F, V, 8, V, 8, 0, F, V, 0, 0) ==
        MOE_ERR_WORKSPACE);
  if (fails) return 1;
  printf("operator checks passed\n");
  return 0;
}
