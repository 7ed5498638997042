// host_sanitize_cache.cpp -- drives the host side of the paged cache's entry points (argument
// checks, workspace plans, launch plans) under AddressSanitizer and UndefinedBehaviorSanitizer
// on the CPU.  Every call is refused or answered before any HIP call.  Built and run by
// tests/test_host_sanitize_cache.py; prints one line per checked value.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "spec_cache.h"

int main() {
  unsigned long long acc = 0;
  const int32_t v[] = {INT_MIN, -1, 0, 1, 2, 16, 64, 128, 256, 1024, 1025, 1 << 20, INT_MAX};
  for (int32_t B : v)
    for (int32_t N : v)
      for (int32_t H : v)
        for (int32_t W : v) {
          acc += sv_attention_workspace_bytes(B, N, H, 1, 64, 16, W, SV_BF16);
          acc += sv_attention_workspace_bytes(B, N, 8, H, 256, W, N, SV_F32);
          acc += sv_attention_workspace_bytes(B, 1, 64, 64, H, 64, W, SV_BF16);
          const char *p = sv_attention_launch_plan(N, H, B, 128, (sv_dtype)(W & 3));
          for (; p && *p; ++p) acc += (unsigned char)*p;
        }
  for (int32_t S : v)
    for (int32_t P : v) acc += sv_resize_workspace_bytes(S, P);
  int32_t a[64] = {0};
  char ws[512];
  void *W = (void *)(((uintptr_t)ws + 255) & ~(uintptr_t)255);
  int64_t big = INT64_MAX;
  printf("scale %d\n", (int)spec_paged_attention(W, 64, 64, W, W, SV_F32, a, a, a, a, 1, 1, 1, 1, 64, 16, 1, 1, 1.0f / 0.0f, 0, 0, W, a, W, 256, nullptr));
  printf("stride %d\n", (int)spec_paged_attention(W, big, big, W, W, SV_F32, a, a, a, a, 1, 1, 1, 1, 64, 16, 1, 1, 1.0f, 0, 0, W, a, W, 256, nullptr));
  printf("small %d\n", (int)spec_paged_attention(W, 64, 64, W, W, SV_BF16, a, a, a, a, 1, 1, 1, 1, 64, 16, 1, 1, 1.0f, 0, 0, W, a, W, 16, nullptr));
  printf("append %d\n", (int)spec_cache_append(W, big, 3, W, 64, 64, SV_BF16, W, W, a, a, a, 1, 1, 1, 64, 16, 1, 1, a, nullptr));
  printf("commit %d\n", (int)spec_cache_commit(W, W, SV_BF16, a, a, a + 16, a + 32, 1, 4, 2, 1, 64, 16, 1, 1, a, a + 48, nullptr));
  printf("resize %d\n", (int)spec_cache_resize(a, a, a, a, a, a, W, W, SV_BF16, INT_MAX, 1, INT_MAX, 64, 16, 1, 1, a, W, 256, nullptr));
  printf("fork %d\n", (int)spec_cache_fork(a, a, a, a, a, a, INT_MAX, INT_MAX, 1, 1, a, nullptr));
  printf("checksum %llu\n", acc);
  return 0;
}
