// spec_cache.hip -- the paged key-value cache of a speculative decoding round: new entries
// appended, an accepted path's entries moved together, pages taken, shared, copied and given
// back (include/spec_cache.h has the layout and the semantics).
//
// All of it is data movement; the floor of each call is its bytes, and below some megabytes
// the launch.  Every kernel checks what it indexes with, so bad tables cost a row code and
// never an access outside the pool.

#include "sv_cache.h"

namespace sv {

// ---------------------------------------------------------------- append

struct AppendArgs {
  const char *k, *v;
  long long k_sb, k_sn, v_sb, v_sn;  // bytes
  char *k_pages, *v_pages;
  const int32_t *page_table, *cache_len, *n_new, *prior;
  int N, chunks;
  int32_t *row_status;
  Pool pool;
};

// Slots a workgroup writes, whole value units (8 prompts of up to 1000 tokens, 36.9 MB read and
// written: 16 slots 11.6, 32 10.0, 64 11.4 us; a copy of those bytes takes 7.7).
constexpr int APPEND_SLOTS = 32;

// One workgroup writes up to APPEND_SLOTS slots of one head.  Keys: a thread moves 16 bytes
// (E values of d of one slot), neighbours along d in the source.  Values: a thread gathers
// the E slots of one d into 16 bytes; neighbours along d, so the loads of a wave cover whole
// rows of the source and its stores whole lines of the page; only a unit that the new slots
// share with older ones is written element by element.
template <typename T>
__global__ __launch_bounds__(NT) void k_cache_append(const AppendArgs a) {
  constexpr int E = 16 / (int)sizeof(T);
  const int tid = threadIdx.x;
  const int chunk = (int)(blockIdx.x % (unsigned)a.chunks);
  const unsigned bh = blockIdx.x / (unsigned)a.chunks;
  const int h = (int)(bh % a.pool.Hkv), b = (int)(bh / a.pool.Hkv);
  const int len = a.cache_len[b], m = a.n_new ? a.n_new[b] : a.N;
  const int sh = a.pool.page_shift, page = 1 << sh, D = (int)a.pool.D;
  const int32_t *table = a.page_table + (size_t)b * a.pool.W;

  int code = a.prior ? min(a.prior[b], 0) : 0;
  if (code != 0) {
    // an earlier call refused the sequence: its pages may not be its own
  } else if (len < 0 || m < 0 || m > a.N || (long long)len + m > ((long long)a.pool.W << sh)) {
    code = SV_ROW_BAD_LENGTH;
  } else if (m > 0) {
    const int p0 = len >> sh, p1 = (len + m - 1) >> sh;
    bool bad = false;
    for (int i = p0 + tid; i <= p1; i += NT) bad |= (unsigned)table[i] >= (unsigned)a.pool.P;
    if (__syncthreads_or(bad)) code = SV_ROW_BAD_PAGE;
  }
  if (chunk == 0 && h == 0 && tid == 0) a.row_status[b] = code;
  if (code != 0) return;
  // chunks start at multiples of APPEND_SLOTS, so that a value unit has one writer
  const int c0 = (len / APPEND_SLOTS + chunk) * APPEND_SLOTS;
  const int s0 = max(len, c0), s1 = min(len + m, c0 + APPEND_SLOTS);
  if (s0 >= s1) return;

  const size_t hb = head_bytes<T>(a.pool);
  const int U = D / E;
  const char *ks = a.k + (long long)b * a.k_sb + (size_t)h * D * sizeof(T);
  for (int x = tid; x < (s1 - s0) * U; x += NT) {
    const int s = s0 + x / U, u = x % U;
    const u32x4 w = *reinterpret_cast<const u32x4 *>(ks + (long long)(s - len) * a.k_sn + u * 16);
    const size_t base = ((size_t)table[s >> sh] * a.pool.Hkv + h) * hb;
    *reinterpret_cast<u32x4 *>(a.k_pages + base + ((size_t)u * page + (s & (page - 1))) * 16) = w;
  }
  const char *vs = a.v + (long long)b * a.v_sb + (size_t)h * D * sizeof(T);
  const int u0 = s0 / E, u1 = (s1 - 1) / E;
  for (int x = tid; x < (u1 - u0 + 1) * D; x += NT) {
    const int u = u0 + x / D, d = x % D, f = u * E;
    T e[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int s = min(max(f + j, s0), s1 - 1);
      e[j] = *reinterpret_cast<const T *>(vs + (long long)(s - len) * a.v_sn + (size_t)d * sizeof(T));
    }
    const size_t base = ((size_t)table[f >> sh] * a.pool.Hkv + h) * hb;
    T *out = reinterpret_cast<T *>(a.v_pages + base + ((size_t)((f & (page - 1)) / E) * D + d) * 16);
    if (f >= s0 && f + E <= s1) {
      u32x4 w;
      __builtin_memcpy(&w, e, 16);
      *reinterpret_cast<u32x4 *>(out) = w;
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (f + j >= s0 && f + j < s1) out[j] = e[j];
    }
  }
}

// ---------------------------------------------------------------- commit

struct CommitArgs {
  char *k_pages, *v_pages;
  const int32_t *page_table, *cache_len, *accepted_len, *path, *prior;
  int N;
  unsigned B, LH;  // layers times heads
  int32_t *new_len, *row_status;
  Pool pool;
};

// One workgroup moves one head's entries of one sequence in one layer, in batches of whole
// target units of values (COMMIT_R * NT / D of them): everything a batch moves is read before
// any of it is written.  Later batches read nothing that earlier ones wrote, since sources lie
// behind their targets (path_nodes[j] >= j + 1, increasing).  A value unit is put together in
// registers and written whole, slots that are no targets as they were: 16-byte stores in place
// of single elements 16 bytes apart (16 trees, 32 layers: 43 us, so 23, the
// bytes' 4.4; every moved value element is 2 bytes of a 64-byte line that is read and written).
template <typename T>
__global__ __launch_bounds__(NT) void k_cache_commit(const CommitArgs a) {
  constexpr int E = 16 / (int)sizeof(T);
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

  const size_t hb = head_bytes<T>(a.pool);
  const unsigned l = lh / a.pool.Hkv, h = lh % a.pool.Hkv;
  const size_t lay = (size_t)l * a.pool.P;
  auto base = [&](int p) { return ((lay + (size_t)p) * a.pool.Hkv + h) * hb; };
  const int U = D / E, per = COMMIT_R * NT / D;  // target units a batch
  const int t_end = len + 1 + acc;               // targets are slots len + 1 + j
  for (int u0 = (len + 1 + s_first) / E; u0 * E < t_end; u0 += per) {
    const int lo = max(u0 * E, len + 1 + s_first), hi = min((u0 + per) * E, t_end);
    u32x4 kw[COMMIT_R], vw[COMMIT_R];
#pragma unroll
    for (int r = 0; r < COMMIT_R; ++r) {
      const int x = tid + r * NT;
      if (x < (hi - lo) * U) {
        const int j = lo + x / U - (len + 1), s = s_slot[j];
        kw[r] = *reinterpret_cast<const u32x4 *>(a.k_pages + base(s_page[j]) + ((size_t)(x % U) * page + (s & (page - 1))) * 16);
      }
      if (x < per * D) {
        const int u = u0 + x / D, d = x % D, f = u * E;
        if (f < hi) {
          const size_t o = ((size_t)((f & (page - 1)) / E) * D + d) * 16;
          u32x4 w = *reinterpret_cast<const u32x4 *>(a.v_pages + base(table[f >> sh]) + o);
          T e[E];
          __builtin_memcpy(e, &w, 16);
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (f + i >= lo && f + i < hi) {
              const int j = f + i - (len + 1), t = s_slot[j] & (page - 1);
              e[i] = *reinterpret_cast<const T *>(a.v_pages + base(s_page[j]) + ((size_t)(t / E) * D + d) * 16 + (size_t)(t % E) * sizeof(T));
            }
          __builtin_memcpy(&w, e, 16);
          vw[r] = w;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < COMMIT_R; ++r) {
      const int x = tid + r * NT;
      if (x < (hi - lo) * U) {
        const int s = lo + x / U;
        *reinterpret_cast<u32x4 *>(a.k_pages + base(table[s >> sh]) + ((size_t)(x % U) * page + (s & (page - 1))) * 16) = kw[r];
      }
      if (x < per * D) {
        const int u = u0 + x / D, d = x % D, f = u * E;
        if (f < hi)
          *reinterpret_cast<u32x4 *>(a.v_pages + base(table[f >> sh]) + ((size_t)((f & (page - 1)) / E) * D + d) * 16) = vw[r];
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- resize

struct ResizeArgs {
  int32_t *page_table, *seq_pages, *ref_count;
  unsigned *free_map;
  const int32_t *keep_len, *want_len;
  int S, P, W, page_shift;
  int32_t *row_status;
  // workspace
  int32_t *alloc;   // [P] the fresh pages in order
  int32_t *old;     // [P] the pages they replaced (-1: none)
  int4 *copies;     // [S] page to copy from, page to copy to, slots to copy
  int32_t *n_copy;
};

constexpr int RZ_NT = 1024, RZ_NW = RZ_NT / WAVE;

// Exclusive prefix over the workgroup of 1024, and the total.
SVD unsigned rz_scan(unsigned v, unsigned *s_w, unsigned &total) {
  const int lane = lane_id(), wid = (int)threadIdx.x / WAVE;
  const unsigned inc = scan_add_u(v);
  if (lane == WAVE - 1) s_w[wid] = inc;
  __syncthreads();
  unsigned before = 0, tot = 0;
#pragma unroll
  for (int k = 0; k < RZ_NW; ++k) {
    before += (k < wid) ? s_w[k] : 0u;
    tot += s_w[k];
  }
  __syncthreads();
  total = tot;
  return before + inc - v;
}
// In place, x[0 .. n) becomes its exclusive prefix and x[n] the total.
SVD unsigned rz_prefix(unsigned *x, int n, unsigned *s_w) {
  unsigned run = 0;
  for (int i0 = 0; i0 < n; i0 += RZ_NT) {
    const int i = i0 + (int)threadIdx.x;
    unsigned tot;
    const unsigned ex = rz_scan(i < n ? x[i] : 0u, s_w, tot);
    if (i < n) x[i] = run + ex;
    run += tot;
  }
  if (threadIdx.x == 0) x[n] = run;
  __syncthreads();
  return run;
}
// The i with x[i] <= e < x[i + 1] in a prefix over n.
SVD int rz_find(const unsigned *x, int n, unsigned e) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (x[m] <= e) lo = m;
    else hi = m;
  }
  return lo;
}
SVD int ld_ref(const int32_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
SVD unsigned ld_map(const unsigned *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// One holder less; a page without holders is marked free.
SVD void give_back(const ResizeArgs &a, int p) {
  if (atomicSub(&a.ref_count[p], 1) == 1) atomicOr(&a.free_map[p >> 5], 1u << (p & 31));
}
// A barrier behind which the workgroup's own atomics and stores have been done.  (Its loads of
// what it changes go past the L1; no other workgroup reads the books, so that nothing needs to
// be written back beyond the L2.)
SVD void rz_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x70);  // vmcnt 0, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The pool's books are a few kilobytes and every sequence's pages depend on those of the
// sequences before it, so one workgroup does them.  Bound: a chain of about ten rounds to
// memory.  Each round runs over the table entries it concerns laid end to end, whoever's they
// are, a thread an entry, which it keeps in registers (256 sequences whose pages grow and
// shrink: 9.4 us; a wave a sequence, 16 sequences after one another, 54).  Which pages are
// picked does not depend on the order in which atomics land: the counts are sums, and picking
// reads the map only after all of them.
__global__ __launch_bounds__(RZ_NT) void k_cache_resize(const ResizeArgs a) {
  extern __shared__ unsigned s_dyn[];
  __shared__ unsigned s_w[RZ_NW];
  __shared__ int s_ncopy, s_served;
  const int tid = threadIdx.x, S = a.S;
  const int sh = a.page_shift, page = 1 << sh;
  // per sequence: the first entry this call reads (to give back, or at or behind keep_len), the
  // pages it is to hold (-1: it is left as it is), and prefixes of its entries read, entries to
  // replace and entries to add
  int *s_lo = (int *)s_dyn, *s_goal = s_lo + S;
  unsigned *s_ent = s_dyn + 2 * S, *s_swap = s_ent + S + 1, *s_add = s_swap + S + 1;
  int *s_bad = (int *)(s_add + S + 1);
  if (tid == 0) s_ncopy = s_served = 0;

  for (int b = tid; b < S; b += RZ_NT) {
    const int keep = a.keep_len[b], want = a.want_len[b], held = a.seq_pages[b];
    const int goal = (int)(((long long)want + page - 1) >> sh);
    int lo = 0, g = -1, ent = 0, add = 0, code = 0;
    if (want >= 0) {
      if (held < 0 || held > a.W || goal > a.W || keep < 0 || (long long)keep > ((long long)held << sh)) {
        code = SV_ROW_BAD_LENGTH;
      } else {
        g = goal;
        lo = min(goal, keep >> sh);
        ent = held - lo;
        add = max(0, goal - held);  // none for want <= keep: goal <= held then
      }
    }
    s_lo[b] = lo;
    s_goal[b] = g;
    s_ent[b] = (unsigned)ent;
    s_add[b] = (unsigned)add;
    s_swap[b] = 0u;
    s_bad[b] = code;
  }
  __syncthreads();
  const unsigned n_ent = rz_prefix(s_ent, S, s_w);
  auto row_of = [&](int b) { return a.page_table + (size_t)b * a.W; };

  // ---- the entries' pages.  A thread keeps its first entry; most calls have no more.
  struct Entry {
    int b, i, page;
  };
  auto entry_at = [&](unsigned e) {
    Entry t;
    t.b = rz_find(s_ent, S, e);
    t.i = s_lo[t.b] + (int)(e - s_ent[t.b]);
    t.page = row_of(t.b)[t.i];
    return t;
  };
  Entry mine = {0, 0, 0};
  if ((unsigned)tid < n_ent) mine = entry_at(tid);
  auto entry = [&](unsigned e) { return e == (unsigned)tid ? mine : entry_at(e); };
  for (unsigned e = tid; e < n_ent; e += RZ_NT) {
    const Entry t = entry(e);
    if ((unsigned)t.page >= (unsigned)a.P || ld_ref(&a.ref_count[t.page]) <= 0) s_bad[t.b] = SV_ROW_BAD_PAGE;  // whoever writes: the same
  }
  __syncthreads();
  for (int b = tid; b < S; b += RZ_NT) {
    a.row_status[b] = s_bad[b];
    if (s_bad[b]) {
      s_goal[b] = -1;
      s_add[b] = 0u;
    }
  }
  __syncthreads();

  // ---- pages behind the goal given back
  for (unsigned e = tid; e < n_ent; e += RZ_NT) {
    const Entry t = entry(e);
    if (s_goal[t.b] >= 0 && t.i >= s_goal[t.b]) {
      give_back(a, t.page);
      row_of(t.b)[t.i] = -1;
    }
  }
  rz_sync();

  // ---- entries to replace: others hold the page too, and the sequence is to write behind keep_len
  auto swaps = [&](const Entry &t) {
    return t.i < s_goal[t.b] && a.want_len[t.b] > a.keep_len[t.b] && ld_ref(&a.ref_count[t.page]) > 1;
  };
  for (unsigned e = tid; e < n_ent; e += RZ_NT) {
    const Entry t = entry(e);
    if (swaps(t)) atomicAdd(&s_swap[t.b], 1u);
  }
  __syncthreads();
  const unsigned n_add = rz_prefix(s_add, S, s_w), n_swap = rz_prefix(s_swap, S, s_w);
  const unsigned need_all = n_add + n_swap;

  // ---- the lowest free pages, need_all of them or as many as there are
  unsigned found = 0;
  const int words = (a.P + 31) >> 5;
  for (int w0 = 0; w0 < words && found < need_all; w0 += RZ_NT) {
    unsigned bits = (w0 + tid < words) ? ld_map(&a.free_map[w0 + tid]) : 0u;
    if (w0 + tid == words - 1 && (a.P & 31)) bits &= (1u << (a.P & 31)) - 1u;
    unsigned tot;
    unsigned at = found + rz_scan((unsigned)__popc(bits), s_w, tot);
    for (; bits && at < need_all; bits &= bits - 1, ++at) a.alloc[at] = (w0 + tid) * 32 + __ffs((int)bits) - 1;
    found += tot;
  }
  found = min(found, need_all);
  // A sequence's pages are those from s_swap + s_add on, replaced entries first, if the free
  // pages reach to its last one (then they reach all sequences before it).
  auto end_of = [&](int b) { return s_swap[b + 1] + s_add[b + 1]; };
  auto some = [&](int b) { return end_of(b) > s_swap[b] + s_add[b]; };
  auto fits = [&](int b) { return end_of(b) <= found; };
  for (int b = tid; b < S; b += RZ_NT)
    if (some(b) && fits(b)) atomicMax(&s_served, (int)end_of(b));
  rz_sync();

  // ---- handed out.  The books of the fresh pages are kept back until all of it is done: what
  // swaps says of an entry must be what was counted, also where the map calls a page free that
  // has holders (counted pages and taken ones would be different ones then, and a page that is
  // already gone could be taken again).
  auto take = [&](int b, int i, unsigned at, int old) {
    const int fresh = a.alloc[at];
    row_of(b)[i] = fresh;
    a.old[at] = old;
    return fresh;
  };
  if (n_swap > 0) {
    unsigned seen = 0;  // entries replaced so far, in the order of all entries
    for (unsigned e0 = 0; e0 < n_ent; e0 += RZ_NT) {
      const unsigned e = e0 + tid;
      Entry t = {0, 0, 0};
      bool it = false;
      if (e < n_ent) {
        t = entry(e);
        it = swaps(t);
      }
      unsigned tot;
      const unsigned at = seen + rz_scan(it ? 1u : 0u, s_w, tot);
      if (it && fits(t.b)) {
        const int keep = a.keep_len[t.b], fresh = take(t.b, t.i, at + s_add[t.b], t.page);
        if (t.i == keep >> sh && (keep & (page - 1))) a.copies[atomicAdd(&s_ncopy, 1)] = make_int4(t.page, fresh, keep & (page - 1), 0);
      }
      seen += tot;
    }
  }
  for (unsigned e = tid; e < n_add; e += RZ_NT) {
    const int b = rz_find(s_add, S, e);
    if (fits(b)) take(b, a.seq_pages[b] + (int)(e - s_add[b]), s_swap[b + 1] + e, -1);
  }
  __syncthreads();
  for (int k = tid; k < s_served; k += RZ_NT) {
    const int fresh = a.alloc[k];
    atomicAnd(&a.free_map[fresh >> 5], ~(1u << (fresh & 31)));
    __hip_atomic_store(&a.ref_count[fresh], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  for (int b = tid; b < S; b += RZ_NT) {
    const int goal = s_goal[b];
    if (goal < 0) continue;
    if (some(b) && !fits(b)) {
      a.row_status[b] = SV_ROW_NO_PAGES;
      a.seq_pages[b] = min(a.seq_pages[b], goal);
    } else {
      a.seq_pages[b] = goal;
    }
  }
  rz_sync();
  // ---- replaced pages lose a holder (only now: the counts above are those after giving back)
  if (n_swap > 0)
    for (int k = tid; k < s_served; k += RZ_NT)
      if (a.old[k] >= 0) give_back(a, a.old[k]);
  if (tid == 0) *a.n_copy = s_ncopy;
}

// Dynamic LDS of k_cache_resize.
inline unsigned resize_lds(int S) { return (unsigned)(6 * S + 3) * 4; }

struct CopyArgs {
  char *k_pages, *v_pages;
  const int4 *copies;
  const int32_t *n_copy;
  unsigned L;
  Pool pool;
};

constexpr int COPY_WGS = 1024;  // 4 a CU, whatever there is to copy: the host does not know

// The kept slots of a page into another: a workgroup moves one head of one layer at a time,
// COPY_STEP 16-byte units a thread in flight (16 prompts continued seven ways in 32 layers,
// 1.01 GB read and written: 186 us, 5.4 TB/s; bound by memory).  Keys: t runs fastest, kept * 16 bytes together.
// Values: whole units lie together; of the last one only the kept elements are written.
constexpr int COPY_STEP = 4;

template <typename T>
__global__ __launch_bounds__(NT) void k_cache_copy(const CopyArgs a) {
  constexpr int E = 16 / (int)sizeof(T);
  const unsigned per = a.L * a.pool.Hkv;
  const unsigned long long items = (unsigned long long)*a.n_copy * per;
  const int tid = threadIdx.x, page = 1 << a.pool.page_shift, D = (int)a.pool.D, U = D / E;
  const size_t hb = head_bytes<T>(a.pool);
  for (unsigned long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int4 c = a.copies[it / per];
    const unsigned lh = (unsigned)(it % per), l = lh / a.pool.Hkv, h = lh % a.pool.Hkv;
    const size_t src = (((size_t)l * a.pool.P + c.x) * a.pool.Hkv + h) * hb, dst = (((size_t)l * a.pool.P + c.y) * a.pool.Hkv + h) * hb;
    const int kept = c.z, nk = U * kept, nv = (kept / E) * D;
    for (int x0 = tid; x0 < nk + nv; x0 += COPY_STEP * NT) {
      u32x4 w[COPY_STEP];
      size_t at[COPY_STEP];
#pragma unroll
      for (int j = 0; j < COPY_STEP; ++j) {
        const int x = min(x0 + j * NT, nk + nv - 1);
        at[j] = (x < nk) ? ((size_t)(x / kept) * page + x % kept) * 16 : (size_t)(x - nk) * 16;
        w[j] = *reinterpret_cast<const u32x4 *>((x < nk ? a.k_pages : a.v_pages) + src + at[j]);
      }
#pragma unroll
      for (int j = 0; j < COPY_STEP; ++j)
        if (x0 + j * NT < nk + nv) *reinterpret_cast<u32x4 *>((x0 + j * NT < nk ? a.k_pages : a.v_pages) + dst + at[j]) = w[j];
    }
    if (kept % E)
      for (int d = tid; d < D; d += NT) {
        const size_t o = ((size_t)(kept / E) * D + d) * 16;
        const u32x4 w = *reinterpret_cast<const u32x4 *>(a.v_pages + src + o);
        T e[E];
        __builtin_memcpy(e, &w, 16);
        T *out = reinterpret_cast<T *>(a.v_pages + dst + o);
#pragma unroll
        for (int j = 0; j < E - 1; ++j)
          if (j < kept % E) out[j] = e[j];
      }
  }
}

// ---------------------------------------------------------------- fork

struct ForkArgs {
  int32_t *page_table, *seq_pages, *ref_count, *cache_len;
  const int32_t *src, *dst;
  int F, S, P, W;
  int32_t *pair_status;
};

// One wave a pair.  Pairs do not touch what other pairs read: a target holds no pages, is no
// pair's source, and of pairs with one target only the first is made.  (A target's own row
// may be read by the checks of a pair that is refused whatever they find.)
__global__ __launch_bounds__(NT) void k_cache_fork(const ForkArgs a) {
  const int lane = lane_id(), f = (int)(blockIdx.x * NW) + (int)threadIdx.x / WAVE;
  if (f >= a.F) return;
  const int s = a.src[f], d = a.dst[f];
  int code = 0, held = 0;
  bool bad = (unsigned)s >= (unsigned)a.S || (unsigned)d >= (unsigned)a.S;
  for (int i = lane; i < a.F; i += WAVE) bad |= a.src[i] == d || (i < f && a.dst[i] == d);
  if (__any(bad)) {
    code = SV_ROW_BAD_FORK;
  } else if (a.seq_pages[d] != 0) {
    code = SV_ROW_BAD_FORK;
  } else {
    held = a.seq_pages[s];
    const int32_t *row = a.page_table + (size_t)s * a.W;
    if (held < 0 || held > a.W) {
      code = SV_ROW_BAD_LENGTH;
    } else {
      bool off = false;
      for (int i = lane; i < held; i += WAVE) {
        const unsigned p = (unsigned)row[i];
        off |= p >= (unsigned)a.P || ld_ref(&a.ref_count[p]) <= 0;
      }
      if (__any(off)) code = SV_ROW_BAD_PAGE;
    }
  }
  if (lane == 0) a.pair_status[f] = code;
  if (code != 0) return;
  const int32_t *row = a.page_table + (size_t)s * a.W;
  int32_t *to = a.page_table + (size_t)d * a.W;
  for (int i = lane; i < held; i += WAVE) {
    const int p = row[i];
    to[i] = p;
    atomicAdd(&a.ref_count[p], 1);
  }
  if (lane == 0) {
    a.seq_pages[d] = held;
    a.cache_len[d] = a.cache_len[s];
  }
}

}  // namespace sv

// ======================================================================== host side

namespace {

using namespace sv;
using namespace sv_host;

}  // namespace

extern "C" {

sv_status spec_cache_append(const void *k, int64_t k_stride_b, int64_t k_stride_n, const void *v, int64_t v_stride_b,
                            int64_t v_stride_n, sv_dtype dtype, void *k_pages, void *v_pages,
                            const int32_t *page_table, const int32_t *cache_len, const int32_t *n_new, int32_t B,
                            int32_t N, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                            int32_t table_width, int32_t *row_status, void *stream) {
  return spec_cache_append_after(k, k_stride_b, k_stride_n, v, v_stride_b, v_stride_n, dtype, k_pages, v_pages, page_table,
                                 cache_len, n_new, nullptr, B, N, Hkv, D, page_size, num_pages, table_width, row_status, stream);
}

sv_status spec_cache_append_after(const void *k, int64_t k_stride_b, int64_t k_stride_n, const void *v,
                                  int64_t v_stride_b, int64_t v_stride_n, sv_dtype dtype, void *k_pages, void *v_pages,
                                  const int32_t *page_table, const int32_t *cache_len, const int32_t *n_new,
                                  const int32_t *prior, int32_t B, int32_t N, int32_t Hkv, int32_t D, int32_t page_size,
                                  int32_t num_pages, int32_t table_width, int32_t *row_status, void *stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  const int esz = dtype == SV_BF16 ? 2 : 4;
  if (B < 1 || N < 1 || N > SV_CACHE_MAX_NEW || !pool_ok(Hkv, D, page_size, num_pages, table_width)) return SV_ERR_SHAPE;
  AppendArgs a = {};
  a.chunks = (N + APPEND_SLOTS - 2) / APPEND_SLOTS + 1;  // the first may begin anywhere in a chunk
  const long long heads = (long long)B * Hkv;
  if (heads > MAX_WGS / a.chunks) return SV_ERR_SHAPE;
  const long long grid = heads * a.chunks;
  if (!k || !v || !k_pages || !v_pages || !page_table || !cache_len || !row_status) return SV_ERR_NULL;
  a.k = static_cast<const char *>(k);
  a.v = static_cast<const char *>(v);
  a.k_sb = (long long)((unsigned long long)k_stride_b * esz);
  a.k_sn = (long long)((unsigned long long)k_stride_n * esz);
  a.v_sb = (long long)((unsigned long long)v_stride_b * esz);
  a.v_sn = (long long)((unsigned long long)v_stride_n * esz);
  if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)a.k_sb | (uintptr_t)a.k_sn |
       (uintptr_t)a.v_sb | (uintptr_t)a.v_sn) & 15)
    return SV_ERR_ALIGN;
  if (overlap(prior, row_status, B)) return SV_ERR_PARAM;
  a.k_pages = static_cast<char *>(k_pages);
  a.v_pages = static_cast<char *>(v_pages);
  a.page_table = page_table;
  a.cache_len = cache_len;
  a.n_new = n_new;
  a.prior = prior;
  a.N = N;
  a.row_status = row_status;
  a.pool = pool_of(Hkv, D, page_size, num_pages, table_width);
  return launch(esz == 2 ? (const void *)&k_cache_append<uint16_t> : (const void *)&k_cache_append<float>, a, grid, NT, stream);
}

sv_status spec_cache_commit(void *k_pages, void *v_pages, sv_dtype dtype, const int32_t *page_table,
                            const int32_t *cache_len, const int32_t *accepted_len, const int32_t *path_nodes, int32_t L,
                            int32_t B, int32_t N, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                            int32_t table_width, int32_t *new_len, int32_t *row_status, void *stream) {
  return spec_cache_commit_after(k_pages, v_pages, dtype, page_table, cache_len, accepted_len, path_nodes, nullptr, L, B, N, Hkv,
                                 D, page_size, num_pages, table_width, new_len, row_status, stream);
}

sv_status spec_cache_commit_after(void *k_pages, void *v_pages, sv_dtype dtype, const int32_t *page_table,
                                  const int32_t *cache_len, const int32_t *accepted_len, const int32_t *path_nodes,
                                  const int32_t *prior, int32_t L, int32_t B, int32_t N, int32_t Hkv, int32_t D,
                                  int32_t page_size, int32_t num_pages, int32_t table_width, int32_t *new_len,
                                  int32_t *row_status, void *stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (B < 1 || L < 1 || N < 1 || N > SV_CACHE_MAX_NEW || !pool_ok(Hkv, D, page_size, num_pages, table_width)) return SV_ERR_SHAPE;
  const long long LH = (long long)L * Hkv;
  if (B > MAX_WGS || LH > 0x7fffffffLL || (path_nodes && LH * B > MAX_WGS)) return SV_ERR_SHAPE;  // chains: one a sequence
  if (!k_pages || !v_pages || !page_table || !cache_len || !accepted_len || !new_len || !row_status) return SV_ERR_NULL;
  if (((uintptr_t)k_pages | (uintptr_t)v_pages) & 15) return SV_ERR_ALIGN;
  // With paths several workgroups read a sequence's lengths: what they read is not written here.
  for (const int32_t *in : {cache_len, accepted_len})
    for (const int32_t *to : {(const int32_t *)new_len, (const int32_t *)row_status})
      if (path_nodes && overlap(in, to, B)) return SV_ERR_PARAM;
  if (overlap(prior, new_len, B) || overlap(prior, row_status, B)) return SV_ERR_PARAM;
  CommitArgs a = {};
  a.k_pages = static_cast<char *>(k_pages);
  a.v_pages = static_cast<char *>(v_pages);
  a.page_table = page_table;
  a.cache_len = cache_len;
  a.accepted_len = accepted_len;
  a.path = path_nodes;
  a.prior = prior;
  a.N = N;
  a.B = (unsigned)B;
  a.LH = (unsigned)LH;
  a.new_len = new_len;
  a.row_status = row_status;
  a.pool = pool_of(Hkv, D, page_size, num_pages, table_width);
  // chains move nothing: one workgroup a sequence writes the lengths
  return launch(dtype == SV_BF16 ? (const void *)&k_cache_commit<uint16_t> : (const void *)&k_cache_commit<float>, a,
                path_nodes ? LH * B : B, NT, stream);
}

size_t sv_resize_workspace_bytes(int32_t S, int32_t num_pages) {
  if (S < 1 || S > SV_CACHE_MAX_SEQS || num_pages < 1) return 256;
  return resize_plan(S, num_pages).total;
}

sv_status spec_cache_resize(int32_t *page_table, int32_t *seq_pages, int32_t *ref_count, int32_t *free_map,
                            const int32_t *keep_len, const int32_t *want_len, void *k_pages, void *v_pages,
                            sv_dtype dtype, int32_t L, int32_t S, int32_t Hkv, int32_t D, int32_t page_size,
                            int32_t num_pages, int32_t table_width, int32_t *row_status, void *workspace,
                            size_t workspace_bytes, void *stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (S < 1 || S > SV_CACHE_MAX_SEQS || L < 0 || !pool_ok(L ? Hkv : 1, L ? D : 16, page_size, num_pages, table_width) ||
      (long long)L * Hkv > 0x7fffffffLL || (long long)S * table_width > 0x7fffffffLL)  // entries are counted in 32 bits
    return SV_ERR_SHAPE;
  if (!page_table || !seq_pages || !ref_count || !free_map || !keep_len || !want_len || !row_status || !workspace ||
      (L > 0 && (!k_pages || !v_pages)))
    return SV_ERR_NULL;
  if (L > 0 && (((uintptr_t)k_pages | (uintptr_t)v_pages) & 15)) return SV_ERR_ALIGN;
  const ResizePlan p = resize_plan(S, num_pages);
  if (workspace_bytes < p.total || ((uintptr_t)workspace & 255)) return SV_ERR_WORKSPACE;
  char *base = static_cast<char *>(workspace);
  ResizeArgs a = {page_table, seq_pages, ref_count, (unsigned *)free_map, keep_len, want_len, S, num_pages, table_width,
                  __builtin_ctz((unsigned)page_size), row_status, (int32_t *)(base + p.alloc), (int32_t *)(base + p.old),
                  (int4 *)(base + p.copies), (int32_t *)(base + p.n_copy)};
  const sv_status st = launch((const void *)&k_cache_resize, a, 1, RZ_NT, stream, resize_lds(S));
  if (st != SV_OK || L == 0) return st;
  CopyArgs c = {static_cast<char *>(k_pages), static_cast<char *>(v_pages), a.copies, a.n_copy, (unsigned)L,
                pool_of(Hkv, D, page_size, num_pages, table_width)};
  return launch(dtype == SV_BF16 ? (const void *)&k_cache_copy<uint16_t> : (const void *)&k_cache_copy<float>, c, COPY_WGS,
                NT, stream);
}

sv_status spec_cache_fork(int32_t *page_table, int32_t *seq_pages, int32_t *ref_count, int32_t *cache_len,
                          const int32_t *src, const int32_t *dst, int32_t F, int32_t S, int32_t num_pages,
                          int32_t table_width, int32_t *pair_status, void *stream) {
  if (F < 1 || F > SV_CACHE_MAX_SEQS || S < 1 || S > SV_CACHE_MAX_SEQS || num_pages < 1 || table_width < 1) return SV_ERR_SHAPE;
  if (!page_table || !seq_pages || !ref_count || !cache_len || !src || !dst || !pair_status) return SV_ERR_NULL;
  ForkArgs a = {page_table, seq_pages, ref_count, cache_len, src, dst, F, S, num_pages, table_width, pair_status};
  return launch((const void *)&k_cache_fork, a, (F + NW - 1) / NW, NT, stream);
}

}  // extern "C"
