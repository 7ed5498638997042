// sv_cache.h -- what the paged cache's kernels share: where a pool's slots lie, the host's checks
// of its sizes, and the plan of a resize's workspace.
#pragma once

#include "sv_common.h"

#include "spec_cache.h"

namespace sv {

// Where slots of one sequence lie.
struct Pool {
  int page_shift, P, W;
  unsigned Hkv, D;
};
// Bytes of one page of one layer, and of one head in it.
template <typename T>
SVD size_t head_bytes(const Pool &p) { return ((size_t)p.D << p.page_shift) * sizeof(T); }

constexpr int COMMIT_R = 2;  // units of keys, and of values, that a thread of a commit holds

}  // namespace sv

namespace sv_host {

using namespace sv;

// Most workgroups of NT threads: a launch has fewer than 2^32 threads.
constexpr long long MAX_WGS = 0xffffffffLL / NT;

inline bool pool_ok(int32_t Hkv, int32_t D, int32_t page, int32_t P, int32_t W) {
  return Hkv >= 1 && D >= 16 && D <= COMMIT_R * NT && D % 16 == 0 && page >= 16 && page <= 256 && (page & (page - 1)) == 0 &&
         P >= 1 && W >= 1 && (long long)W * page <= 0x7fffffffLL - 4096;
}

inline Pool pool_of(int32_t Hkv, int32_t D, int32_t page, int32_t P, int32_t W) {
  return Pool{__builtin_ctz((unsigned)page), P, W, (unsigned)Hkv, (unsigned)D};
}

// Whether two arrays of n int32 share memory.
inline bool overlap(const int32_t *x, const int32_t *y, int32_t n) {
  return x && y && (uintptr_t)x < (uintptr_t)(y + n) && (uintptr_t)y < (uintptr_t)(x + n);
}
// Whether row codes [B] lie on what several workgroups read of a sequence: its pages, lengths, counts, nodes' entries.
inline bool codes_on_inputs(const int32_t *codes, int32_t B, int32_t N, int32_t W, const int32_t *table, const int32_t *cache_len,
                            const int32_t *n_new, const int32_t *parent, const int32_t *positions) {
  const uintptr_t c0 = (uintptr_t)codes, c1 = c0 + (uintptr_t)B * 4;
  auto on = [&](const int32_t *p, int32_t n) { return p && c0 < (uintptr_t)p + (uintptr_t)B * (uintptr_t)n * 4 && (uintptr_t)p < c1; };
  return on(table, W) || overlap(codes, cache_len, B) || overlap(codes, n_new, B) || on(parent, N) || on(positions, N);
}

template <typename A>
sv_status launch(const void *fn, A &a, long long grid, int block, void *stream, unsigned lds = 0) {
  sv_host::Launcher L{(hipStream_t)stream, nullptr, 0};
  L.block = block;
  L.lds = lds;
  void *args[] = {&a};
  L.go(fn, (unsigned)grid, args);
  return L.e == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

struct ResizePlan {
  size_t alloc, old, copies, n_copy, total;
};
inline ResizePlan resize_plan(int32_t S, int32_t P) {
  ResizePlan p;
  size_t o = 0;
  p.alloc = o; o = align256(o + (size_t)P * 4);
  p.old = o; o = align256(o + (size_t)P * 4);
  p.copies = o; o = align256(o + (size_t)S * 16);
  p.n_copy = o; o = align256(o + 4);
  p.total = o;
  return p;
}

}  // namespace sv_host
