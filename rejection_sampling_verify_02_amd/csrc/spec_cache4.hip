// spec_cache4.hip -- a cache in 4 bits through the rest of a round: an accepted path's entries moved
// together, and kept slots copied where a shared page is replaced (include/spec_cache.h).  The
// books are those of spec_cache.hip; only what lies in a slot differs.

#include "sv_fp4.h"

namespace sv {

struct Commit4Args {
  char *k_codes, *k_scales, *v_codes, *v_scales;
  const int32_t *page_table, *cache_len, *accepted_len, *path, *prior;
  int N;
  unsigned B, LH;  // layers times heads
  int32_t *new_len, *row_status;
  Pool pool;
};

// One workgroup moves one head's entries of one sequence in one layer, in batches of as many as
// its threads hold in registers: everything a batch moves is read before any of it is written, and
// later batches read nothing that earlier ones wrote, since sources lie behind their targets.  An
// entry is D / 32 blocks of a key, 16 pieces of a value and 2 D / 32 scale bytes, an item each
// (16 trees of 32 nodes, 32 layers, 8 heads of 128: 18 us for 5.6 MB, the bf16 cache's commit 23;
// bound by the partial lines that it touches).
constexpr int COMMIT4_R = 2;  // items a thread holds

__global__ __launch_bounds__(NT) void k_cache_commit4(const Commit4Args a) {
  __shared__ int s_slot[SV_CACHE_MAX_NEW], s_page[SV_CACHE_MAX_NEW];  // of the sources
  __shared__ int s_first;
  const int tid = threadIdx.x;
  const int b = (int)(blockIdx.x % a.B);
  const unsigned lh = blockIdx.x / a.B;
  const int len = a.cache_len[b], acc = a.accepted_len[b];
  const int sh = a.pool.page_shift, page = 1 << sh, D = (int)a.pool.D;
  const int32_t *table = a.page_table + (size_t)b * a.pool.W;

  if (tid == 0) s_first = acc;
  int code = a.prior ? min(a.prior[b], 0) : 0, top = 0;  // top: the last node kept
  if (code != 0) {
    // an earlier call refused the sequence: its pages may not be its own
  } else if (acc < 0) {
    code = acc;
  } else if (len < 0 || acc > a.N - 1) {
    code = SV_ROW_BAD_LENGTH;
  } else {
    top = acc;
    if (a.path && acc > 0) {
      const int32_t *path = a.path + (size_t)b * a.N;
      bool bad = false;
      for (int j = tid; j < acc; j += NT) {
        const int x = path[j], y = j ? path[j - 1] : 0;
        bad |= x <= y || x >= a.N;
      }
      top = path[acc - 1];
      if (__syncthreads_or(bad)) code = SV_ROW_BAD_TREE;
    }
    if (code == 0 && (long long)len + top + 1 > ((long long)a.pool.W << sh)) code = SV_ROW_BAD_LENGTH;
    if (code == 0) {
      bool bad = false;
      for (int i = (len >> sh) + tid; i <= (len + top) >> sh; i += NT) bad |= (unsigned)table[i] >= (unsigned)a.pool.P;
      if (__syncthreads_or(bad)) code = SV_ROW_BAD_PAGE;
    }
  }
  if (lh == 0 && tid == 0) {
    a.row_status[b] = code;
    a.new_len[b] = (code == 0) ? len + 1 + acc : len;
  }
  if (code != 0 || !a.path || top == acc) return;  // entries that lie together already
  for (int j = tid; j < acc; j += NT) {
    const int x = a.path[(size_t)b * a.N + j];
    s_slot[j] = len + x;
    s_page[j] = table[(len + x) >> sh];
    if (x != j + 1) atomicMin(&s_first, j);
  }
  __syncthreads();

  const unsigned l = lh / a.pool.Hkv, h = lh % a.pool.Hkv;
  const size_t lay = (size_t)l * a.pool.P, cb = f4_codes(a.pool), sb = f4_scales(a.pool);
  auto head = [&](int p) { return (lay + (size_t)p) * a.pool.Hkv + h; };
  const int U = D / F4_BLOCK, items = 3 * U + 16, per = COMMIT4_R * NT / items;
  for (int j0 = s_first; j0 < acc; j0 += per) {
    const int n = min(per, acc - j0) * items;
    u32x4 w[COMMIT4_R];
    // Where item y of the entry at (page p, slot t) lies, and what of it is moved.
    auto move = [&](int r, bool put, int p, int t, int y) {
      const size_t ph = head(p);
      if (y < U) {
        u32x4 *at = reinterpret_cast<u32x4 *>(a.k_codes + ph * cb + f4_key(a.pool, y, t));
        if (put) *at = w[r];
        else w[r] = *at;
      } else if (y < U + 16) {
        char *at = a.v_codes + ph * cb + f4_value(a.pool, t, y - U);
        if (D == 64) {
          if (put) *reinterpret_cast<uint16_t *>(at) = (uint16_t)w[r].x;
          else w[r].x = *reinterpret_cast<uint16_t *>(at);
        } else {
          if (put) *reinterpret_cast<unsigned *>(at) = w[r].x;
          else w[r].x = *reinterpret_cast<unsigned *>(at);
          if (D == 256) {
            if (put) *reinterpret_cast<unsigned *>(at + 4) = w[r].y;
            else w[r].y = *reinterpret_cast<unsigned *>(at + 4);
          }
        }
      } else {
        const int u = y - U - 16;
        unsigned char *at = reinterpret_cast<unsigned char *>((u < U ? a.k_scales : a.v_scales) + ph * sb + f4_scale(a.pool, u < U ? u : u - U, t));
        if (put) *at = (unsigned char)w[r].x;
        else w[r].x = *at;
      }
    };
#pragma unroll
    for (int r = 0; r < COMMIT4_R; ++r) {
      const int x = tid + r * NT;
      if (x < n) {
        const int j = j0 + x / items;
        move(r, false, s_page[j], s_slot[j] & (page - 1), x % items);
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < COMMIT4_R; ++r) {
      const int x = tid + r * NT;
      if (x < n) {
        const int s = len + 1 + j0 + x / items;
        move(r, true, table[s >> sh], s & (page - 1), x % items);
      }
    }
    __syncthreads();
  }
}

struct Copy4Args {
  char *k_codes, *k_scales, *v_codes, *v_scales;
  const int4 *copies;
  const int32_t *n_copy;
  unsigned L;
  Pool pool;
};

constexpr int COPY4_WGS = 1024;  // 4 a CU, whatever there is to copy: the host does not know

// The kept slots of a page into another: a workgroup moves one head of one layer at a time, in
// units of 16 bytes, the ends of rows in smaller ones.  Bound by bytes: 128 pages in 32 layers of 8
// heads of 128, 267 MB read and written in 54 us, a copy's rate.
__global__ __launch_bounds__(NT) void k_cache_copy4(const Copy4Args a) {
  const unsigned per = a.L * a.pool.Hkv;
  const unsigned long long items = (unsigned long long)*a.n_copy * per;
  const int tid = threadIdx.x, D = (int)a.pool.D, U = D / F4_BLOCK, S = 512 / D, B = D / 32;
  const size_t cb = f4_codes(a.pool), sb = f4_scales(a.pool);
  for (unsigned long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int4 c = a.copies[it / per];
    const unsigned lh = (unsigned)(it % per), l = lh / a.pool.Hkv, h = lh % a.pool.Hkv;
    const size_t src = ((size_t)l * a.pool.P + c.x) * a.pool.Hkv + h, dst = ((size_t)l * a.pool.P + c.y) * a.pool.Hkv + h;
    const int kept = c.z, nk = U * kept, nv = kept / S * 16;
    for (int x = tid; x < nk + nv; x += NT) {
      const size_t o = x < nk ? f4_key(a.pool, x / kept, x % kept) : (unsigned)(x - nk) * 16u;
      char *p = x < nk ? a.k_codes : a.v_codes;
      *reinterpret_cast<u32x4 *>(p + dst * cb + o) = *reinterpret_cast<const u32x4 *>(p + src * cb + o);
    }
    // values of the last unit's kept slots, two bytes at a time
    for (int x = tid; x < kept % S * 16 * (B / 2); x += NT) {
      const int y = x / (B / 2);
      const size_t o = f4_value(a.pool, kept / S * S + y / 16, y % 16) + (unsigned)(x % (B / 2)) * 2u;
      *reinterpret_cast<uint16_t *>(a.v_codes + dst * cb + o) = *reinterpret_cast<const uint16_t *>(a.v_codes + src * cb + o);
    }
    // scales: rows of bytes, eight at a time
    const int n8 = kept / 8, row = n8 + kept % 8;
    for (int x = tid; x < 2 * U * row; x += NT) {
      const int u = x / row, y = x % row;
      char *p = u < U ? a.k_scales : a.v_scales;
      const size_t o = f4_scale(a.pool, u < U ? u : u - U, y < n8 ? y * 8 : n8 * 8 + y - n8);
      if (y < n8) *reinterpret_cast<uint2 *>(p + dst * sb + o) = *reinterpret_cast<const uint2 *>(p + src * sb + o);
      else p[dst * sb + o] = p[src * sb + o];
    }
  }
}

}  // namespace sv

// ======================================================================== host side

namespace {

using namespace sv;
using namespace sv_host;

bool pool4_ok(int32_t Hkv, int32_t D, int32_t page, int32_t P, int32_t W) {
  return (D == 64 || D == 128 || D == 256) && pool_ok(Hkv, D, page, P, W);
}

bool aligned4(const void *kc, const void *ks, const void *vc, const void *vs) {
  return !(((uintptr_t)kc | (uintptr_t)vc) & 15) && !(((uintptr_t)ks | (uintptr_t)vs) & 7);
}

}  // namespace

extern "C" {

sv_status spec_cache_commit4(void *k_codes, void *k_scales, void *v_codes, void *v_scales, const int32_t *page_table,
                             const int32_t *cache_len, const int32_t *accepted_len, const int32_t *path_nodes,
                             const int32_t *prior, int32_t L, int32_t B, int32_t N, int32_t Hkv, int32_t D, int32_t page_size,
                             int32_t num_pages, int32_t table_width, int32_t *new_len, int32_t *row_status, void *stream) {
  if (B < 1 || L < 1 || N < 1 || N > SV_CACHE_MAX_NEW || !pool4_ok(Hkv, D, page_size, num_pages, table_width)) return SV_ERR_SHAPE;
  const long long LH = (long long)L * Hkv;
  if (B > MAX_WGS || LH > 0x7fffffffLL || (path_nodes && LH > MAX_WGS / B)) return SV_ERR_SHAPE;  // chains: one a sequence
  if (!k_codes || !k_scales || !v_codes || !v_scales || !page_table || !cache_len || !accepted_len || !new_len || !row_status) return SV_ERR_NULL;
  if (!aligned4(k_codes, k_scales, v_codes, v_scales)) return SV_ERR_ALIGN;
  // With paths several workgroups read a sequence's lengths: what they read is not written here.
  for (const int32_t *in : {cache_len, accepted_len})
    for (const int32_t *to : {(const int32_t *)new_len, (const int32_t *)row_status})
      if (path_nodes && overlap(in, to, B)) return SV_ERR_PARAM;
  if (overlap(prior, new_len, B) || overlap(prior, row_status, B)) return SV_ERR_PARAM;
  Commit4Args a = {static_cast<char *>(k_codes), static_cast<char *>(k_scales), static_cast<char *>(v_codes),
                   static_cast<char *>(v_scales), page_table, cache_len, accepted_len, path_nodes, prior, N, (unsigned)B,
                   (unsigned)LH, new_len, row_status, pool_of(Hkv, D, page_size, num_pages, table_width)};
  return launch((const void *)&k_cache_commit4, a, path_nodes ? LH * B : B, NT, stream);
}

sv_status spec_cache_resize4(int32_t *page_table, int32_t *seq_pages, int32_t *ref_count, int32_t *free_map,
                             const int32_t *keep_len, const int32_t *want_len, void *k_codes, void *k_scales, void *v_codes,
                             void *v_scales, int32_t L, int32_t S, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                             int32_t table_width, int32_t *row_status, void *workspace, size_t workspace_bytes, void *stream) {
  if (L < 1 || !pool4_ok(Hkv, D, page_size, num_pages, table_width) || (long long)L * Hkv > 0x7fffffffLL) return SV_ERR_SHAPE;
  if (!k_codes || !k_scales || !v_codes || !v_scales) return SV_ERR_NULL;
  if (!aligned4(k_codes, k_scales, v_codes, v_scales)) return SV_ERR_ALIGN;
  // the books, which leave the copies to make in the workspace
  const sv_status st = spec_cache_resize(page_table, seq_pages, ref_count, free_map, keep_len, want_len, nullptr, nullptr, SV_BF16,
                                         0, S, 1, 16, page_size, num_pages, table_width, row_status, workspace, workspace_bytes, stream);
  if (st != SV_OK) return st;
  const ResizePlan p = resize_plan(S, num_pages);
  const char *base = static_cast<const char *>(workspace);
  Copy4Args c = {static_cast<char *>(k_codes), static_cast<char *>(k_scales), static_cast<char *>(v_codes), static_cast<char *>(v_scales),
                 (const int4 *)(base + p.copies), (const int32_t *)(base + p.n_copy), (unsigned)L,
                 pool_of(Hkv, D, page_size, num_pages, table_width)};
  return launch((const void *)&k_cache_copy4, c, COPY4_WGS, NT, stream);
}

}  // extern "C"
