/* Plain C99 client of the paged-cache part of the C ABI: built by tests/test_kv_host.py with
 * gcc -std=c99 -pedantic.  Prints the layout of fp8_kv_cache for the binding's test and checks
 * that bad arguments are refused before any CUDA call, so it runs without a GPU. */
#include <stddef.h>
#include <stdio.h>
#include "fp8lin.h"
int main(void) {
  fp8_kv_cache c = {0};
  static double mem[64];
  c.num_pages = 4, c.page_size = 16, c.heads = 2, c.head_dim = 64;
  c.page_stride = 2 * 16 * 64, c.head_stride = 16 * 64, c.token_stride = 64;
  c.fmt = FP8_E4M3, c.scale_fmt = FP8_SCALE_FP32;
  if (fp8_paged_attention_ws_bytes(3, 8, &c) != 0) return 1;                  /* no memory yet */
  if (fp8_kv_write(mem, 128, 64, mem, 128, 64, 4, (const int64_t*)mem, &c, NULL) != FP8_ERR_INVALID_ARG) return 2;
  if (fp8_kv_read(&c, (const int32_t*)mem, 4, 4, (const int32_t*)mem, 1, 4, mem, mem, NULL) != FP8_ERR_INVALID_ARG) return 3;
  if (fp8_paged_attention(mem, 512, 64, 1, 8, &c, (const int32_t*)mem, 4, 4, (const int32_t*)mem, 0.125f, 0, mem, NULL, mem,
                          sizeof mem, NULL) != FP8_ERR_INVALID_ARG) return 4;
  if (fp8_qk_norm_rope(mem, 128, 64, mem, 128, 64, 4, 2, 2, 60, NULL, NULL, 1e-6f, NULL, 0, 0, 0, NULL, mem, 128, 64, mem,
                       128, 64, NULL) != FP8_ERR_SHAPE) return 5;
  printf("%d %d %d %d %d\n", (int)sizeof c, (int)offsetof(fp8_kv_cache, v_scale), (int)offsetof(fp8_kv_cache, num_pages),
         (int)offsetof(fp8_kv_cache, token_stride), (int)offsetof(fp8_kv_cache, scale_fmt));
  return 0;
}
