/* Plain C99 user of the feed-forward products and the gradient norm: the public
 * header alone, argument errors, sizes and empty calls, with no GPU needed.
 * Exit code 0 on success. */
#include <stdio.h>

#include "mpnum.h"

#define CHECK(cond)                                          \
  do {                                                       \
    if (!(cond)) {                                           \
      fprintf(stderr, "failed: %s (line %d)\n", #cond, __LINE__); \
      return 1;                                              \
    }                                                        \
  } while (0)

int main(void) {
  void* a = (void*)4096;
  mp_grad g = {a, a, 100, MP_F32, MP_F32};
  CHECK(sizeof(mp_grad) == 32);
  CHECK(linear_swiglu(NULL, MP_BF16, 4, 64, 256, a, a, a, MP_BF16, 128, NULL, NULL, NULL, 256, NULL, NULL, NULL) == MP_EINVAL);
  CHECK(linear_swiglu(a, MP_BF16, 4, 72, 256, a, a, a, MP_BF16, 128, NULL, NULL, NULL, 256, NULL, NULL, NULL) == MP_ESHAPE);
  CHECK(linear_swiglu(a, MP_BF16, 0, 64, 256, a, a, a, MP_BF16, 128, NULL, NULL, NULL, 256, NULL, NULL, NULL) == MP_OK);
  CHECK(linear_swiglu_workspace_size(4, 64, 256) >= 4 * 256 * 4 && linear_swiglu_workspace_size(0, 64, 256) == 0);
  CHECK(linear_swiglu_backward(a, MP_BF16, 4, 64, 256, a, a, a, NULL, NULL, 256, NULL, NULL, a, a, a, NULL, 0, NULL) ==
        MP_EWORKSPACE);
  CHECK(linear_swiglu_backward(a, MP_BF16, 4, 64, 256, a, a, a, NULL, NULL, 256, NULL, NULL, NULL, NULL, NULL, NULL, 0,
                               NULL) == MP_OK);
  CHECK(mp_grad_norm_workspace_size(&g, 1) >= 64);
  CHECK(mp_grad_norm(&g, 1, NULL, NULL, a, 1 << 20, NULL) == MP_EINVAL);
  CHECK(mp_grad_norm(&g, 1, NULL, (float*)a, a, 8, NULL) == MP_EWORKSPACE);
  CHECK(mp_grad_clip(&g, 1, (const float*)a, 0.0f, NULL) == MP_EINVAL);
  g.out_dtype = MP_F16;
  CHECK(mp_grad_clip(&g, 1, (const float*)a, 1.0f, NULL) == MP_EINVAL); /* in place into another type */
  CHECK(mp_grad_clip(NULL, 0, (const float*)a, 1.0f, NULL) == MP_OK);
  CHECK(mp_launch_count() == 0);
  printf("products abi ok\n");
  return 0;
}
