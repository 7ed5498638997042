// host_sanitize_step.cpp -- drives the host side of the entry points of positions, of the cache in
// 4 bits and of filtered sampling under AddressSanitizer and UndefinedBehaviorSanitizer on the CPU.
// Every call is refused or answered before any HIP call.  Built and run by
// tests/test_host_sanitize_step.py; prints one line per checked value.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "spec_cache.h"
#include "spec_filter.h"

int main() {
  unsigned long long acc = 0;
  const int32_t v[] = {INT_MIN, -1, 0, 1, 2, 16, 64, 128, 256, 1024, 1025, 1 << 20, 1 << 24, INT_MAX};
  int32_t a[64] = {0};
  char ws[512];
  void *W = (void *)(((uintptr_t)ws + 255) & ~(uintptr_t)255);
  const int64_t big = INT64_MAX;
  sv_rotary rot = {(const float *)W, 64, 1, 1.0f};
  sv_policy pol = {1.0f, 5, 0.9f, 0.1f, nullptr, nullptr, nullptr, nullptr};
  for (int32_t B : v)
    for (int32_t N : v)
      for (int32_t H : v) {
        acc += sv_attention4_workspace_bytes(B, N, H, 1, 64, 16, N);
        acc += sv_attention4_workspace_bytes(B, N, 8, H, 256, 64, H);
        acc += sv_filter_workspace_bytes(B, N, (sv_dtype)(H & 3));
        const char *p = sv_attention4_launch_plan(N, H, B, 128);
        for (; p && *p; ++p) acc += (unsigned char)*p;
        for (int32_t P : v) {
          rot.rot_dim = P;
          // no rows' status: refused whatever the sizes
          acc += spec_cache_append_rotary(W, big, 3, W, 64, big, W, 64, 64, SV_BF16, W, nullptr, W, nullptr, &rot, a, a, a, a, a, a, B, N, H, P, 64, 16, P, N,
                                          (char *)W, nullptr, nullptr) != SV_OK;
          acc += spec_cache_append_rotary(nullptr, 0, 0, W, big, 64, W, 64, 64, SV_BF16, W, W, W, W, nullptr, a, a, a, a, a, a, B, N, 0, H, 128, 64, P, N,
                                          nullptr, nullptr, nullptr) != SV_OK;
          acc += spec_cache_read(W, W, W, W, SV_BF16, a, a, a, B, N, H, 64, 16, P, B, W, W, nullptr, nullptr) != SV_OK;
          acc += spec_cache_commit4(W, W, W, W, a, a, a, a, a, P, B, N, H, 64, 16, P, N, a, nullptr, nullptr) != SV_OK;
          acc += spec_cache_resize4(a, a, a, a, a, a, W, W, W, W, P, B, H, 64, 16, P, N, nullptr, W, 512, nullptr) != SV_OK;
          acc += spec_paged_attention4(W, big, 8, W, W, W, W, a, a, a, a, a, B, N, H, P, 64, 16, P, N, 1.0f, 0, 0, W, nullptr, W, 256, nullptr, nullptr, 0, nullptr) != SV_OK;
          acc += spec_sample_filtered(W, SV_F32, nullptr, B, N, &pol, a, nullptr, W, 256, nullptr, nullptr, 0, nullptr) != SV_OK;
          acc += spec_filter_logits(W, SV_BF16, B, N, &pol, W, nullptr, W, 256, nullptr, nullptr, 0, nullptr) != SV_OK;
        }
      }
  rot.rot_dim = 64;
  printf("factor %d\n", (int)(rot.factor = 1.0f / 0.0f, spec_cache_append_rotary(W, 64, 64, W, 64, 64, W, 64, 64, SV_F32, W, nullptr, W, nullptr, &rot, a, a, a, a, a, a,
                                                                                1, 1, 1, 1, 64, 16, 1, 1, W, a, nullptr)));
  rot.factor = 1.0f;
  printf("stride %d\n", (int)spec_cache_append_rotary(W, big, big, W, 64, 64, W, 64, 64, SV_F32, W, nullptr, W, nullptr, &rot, a, a, a, a, a, a, 1, 1, 1, 1, 64, 16, 1, 1,
                                                      W, a, nullptr));
  printf("scale %d\n", (int)spec_paged_attention4(W, 64, 64, W, W, W, W, a, a, a, a, a, 1, 1, 1, 1, 64, 16, 1, 1, 1.0f / 0.0f, 0, 0, W, a, W, 256, nullptr, nullptr, 0, nullptr));
  printf("small %d\n", (int)spec_paged_attention4(W, 64, 64, W, W, W, W, a, a, a, a, nullptr, 1, 1, 1, 1, 64, 16, 1, 1, 1.0f, 0, 0, W, a, W, 16, nullptr, nullptr, 0, nullptr));
  pol.top_p = 0.0f;
  printf("policy %d\n", (int)spec_sample_filtered(W, SV_F32, (float *)W, 1, 1, &pol, a, a, W, 256, nullptr, nullptr, 0, nullptr));
  printf("checksum %llu\n", acc);
  return 0;
}
