/* The row operators and the MXFP4 operators from C: the header's declarations
 * compile and link as C99 and C++, and their checks behave as it states.  Every
 * call made here returns before anything touches a GPU. */
#include <stdint.h>
#include <stdio.h>

#include "moe.h"

static int failures = 0;

#define EXPECT(cond)                                   \
  do {                                                 \
    if (!(cond)) {                                     \
      printf("FAILED line %d: %s\n", __LINE__, #cond); \
      ++failures;                                      \
    }                                                  \
  } while (0)

int main(void) {
  /* Never dereferenced. */
  char *a = (char *)(uintptr_t)0x100000000u;
  char *b = (char *)(uintptr_t)0x200000000u;
  char *c = (char *)(uintptr_t)0x300000000u;
  char *d = (char *)(uintptr_t)0x400000000u;
  const int32_t *inv = (const int32_t *)(uintptr_t)0x500000000u;
  const float *w = (const float *)(uintptr_t)0x600000000u;

  EXPECT(moe_permute(NULL, 4, 256, 2, inv, b, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_permute(a, 4, 255, 2, inv, b, NULL) == MOE_ERR_UNSUPPORTED);
  EXPECT(moe_permute(a, 4, 256, 2, inv, a + 512, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_permute_backward(a, 3, 4, 64, 2, inv, b, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_unpermute(a, MOE_T_FP32, 4, 6, 2, inv, w, b, NULL) == MOE_ERR_UNSUPPORTED);
  EXPECT(moe_unpermute(a, MOE_T_BF16, 4, 64, 2, inv, NULL, b, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_unpermute_backward(a, b, MOE_T_BF16, 4, 64, 2, inv, w, NULL, NULL, NULL) ==
         MOE_ERR_INVALID_ARG);
  EXPECT(moe_quantize_mxfp4(a, MOE_T_FP16, 4, 48, 1, NULL, (uint8_t *)b, (uint8_t *)c,
                            MOE_SCALES_ROW_MAJOR, NULL) == MOE_ERR_UNSUPPORTED);
  EXPECT(moe_quantize_mxfp4(a, MOE_T_FP16, 4, 64, 2, NULL, (uint8_t *)b, (uint8_t *)c,
                            MOE_SCALES_GROUP_MAJOR, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_dequantize_mxfp4((uint8_t *)a, (uint8_t *)b, 2, 4, 64, MOE_T_BF16, c, NULL) ==
         MOE_ERR_INVALID_ARG);
  EXPECT(moe_mxfp4_weight_bytes(2, 128, 256) == 2 * 16384);
  EXPECT(moe_mxfp4_weight_scale_bytes(2, 136, 288) == 2 * 2 * 2 * 1024);
  EXPECT(moe_mxfp4_prepack((uint8_t *)a, (uint8_t *)b, 1, 12, 256, (uint8_t *)c, (uint8_t *)d,
                           NULL) == MOE_ERR_UNSUPPORTED);
  EXPECT(moe_mxfp4_workspace_bytes(0, 1, 128, 256) == 0);
  EXPECT(moe_mxfp4_gemm((uint8_t *)a, (uint8_t *)b, NULL, 4, 2, 128, 256, (uint8_t *)c,
                        (uint8_t *)d, MOE_T_BF16, (void *)inv, (void *)w, NULL) ==
         MOE_ERR_INVALID_ARG);
  EXPECT(moe_mxfp4_check_error(NULL, NULL) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_mxfp4_clear_error(a + 16, NULL) == MOE_ERR_ALIGNMENT);
  if (failures == 0) printf("abi ok\n");
  return failures != 0;
}
