// spec_attention.hip -- attention of a round's new tokens over a paged key-value cache.
//
// For node i of sequence b and query head h: out = softmax(scale q.k) v over the slots the
// node sees (include/spec_cache.h).  All query rows of one key head, row r = node * group +
// head in group, read the same keys and values, so a unit of work is (sequence, key head,
// row tile of RT = 16 R rows) and streams the sequence's slots once, 32 at a time:
//   S^T = K Q^T   keys as the matrix instruction's A operand, query rows as its columns
//   O^T += V^T P^T
// With rows as columns a lane owns one query row of each 16-row tile, in both products:
// the row's running maximum and sum live in that lane's registers, rescaling is one factor
// a lane, and the weights leave the first product in exactly the lanes and order in which
// the second one takes them, so nothing goes through LDS inside the loop (the order of the
// 16 slots of a score tile is chosen for that: SlotMap).  The cache's layout puts the 16
// bytes each lane needs together, so keys and values go from HBM to the lanes that multiply
// them with no staging either.
//
// Bound: with few rows the cache's bytes (2 D Hkv element sizes a token), read once; every
// wave keeps the next tile's keys and this tile's values in flight.  The tiles of all units
// are laid end to end and cut into equal shares, one a workgroup, whatever the lengths of
// the sequences (a share may end in the middle of one unit and go on with the next); the
// four waves of a workgroup take tiles in turn and join in LDS, and units that more than one
// workgroup streamed are joined by k_attn_join.  Sums run in a fixed order: same call, same
// bits.

#include "sv_common.h"

#include "spec_cache.h"

namespace sv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int TILE = 32;  // slots a wave takes at a time

struct AttnArgs {
  const char *q, *k_pages, *v_pages;
  long long q_sb, q_sn;  // bytes
  const int32_t *page_table, *cache_len, *n_new, *parent;
  int B, N, Hq, Hkv, group, page_shift, P, W;
  float c2;  // scale * log2 e: scores are kept as powers of two
  int window, sinks;
  char *out;
  int32_t *row_status;
  int n_rt;        // row tiles of a unit
  unsigned grid;   // workgroups (a multiple of LANES)
  // workspace: per workgroup two segments (the one it goes on with, the one it begins)
  float *part_o;   // [2 grid][RT][D]
  float2 *part_ml; // [2 grid][RT] maximum and sum
  uint4 *desc;     // [units] first workgroup, workgroups, valid rows
};

// A row tile's nodes and the tiles of slots they see.
struct Span {
  int i0, i1;          // nodes of the tile that are new tokens (i0 > i1: none)
  int from;            // the first slot of the window (0: no window)
  int first, n_sink;   // the tile it lies in, tiles of sinks before that
  int tiles;
};

struct Seq {
  int len, m;
  bool ok;  // lengths fit; the pages and the tree are checked elsewhere
};

SVD Seq seq_of(const AttnArgs &a, int b) {
  Seq s;
  s.len = a.cache_len[b];
  s.m = a.n_new ? a.n_new[b] : a.N;
  s.ok = s.len >= 0 && s.m >= 0 && s.m <= a.N && (long long)s.len + s.m <= ((long long)a.W << a.page_shift);
  return s;
}

// Every unit has at least one tile, so that some workgroup writes its rows.
template <int RT>
SVD Span span_of(const AttnArgs &a, const Seq &s, int rt) {
  Span p;
  p.i0 = rt * RT / a.group;
  p.i1 = min(s.m - 1, (rt * RT + RT - 1) / a.group);
  p.from = p.first = p.n_sink = 0;
  p.tiles = 1;
  if (!s.ok || p.i0 > p.i1) {
    p.i0 = 1;
    p.i1 = 0;
    return p;
  }
  const int end = s.len + (a.parent ? s.m : p.i1 + 1);
  if (a.window > 0) {  // the least position in the tile: a node's depth is at least 1 behind node 0
    const int pos = s.len + (a.parent ? (p.i0 > 0) : p.i0);
    p.from = max(0, pos - a.window + 1);
    p.first = p.from / TILE;
    p.n_sink = min((int)(((long long)a.sinks + TILE - 1) / TILE), p.first);
  }
  p.tiles = p.n_sink + (end + TILE - 1) / TILE - p.first;
  return p;
}
template <int RT>
SVD unsigned seq_tiles(const AttnArgs &a, int b) {
  const Seq s = seq_of(a, b);
  unsigned t = 0;
  for (int rt = 0; rt < a.n_rt; ++rt) t += (unsigned)span_of<RT>(a, s, rt).tiles;
  return t * (unsigned)a.Hkv;
}

SVD float xor_max(float x) {  // over the four lanes of a column (lane % 16 equal)
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
SVD float xor_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}
SVD unsigned xor_or(unsigned x) {
  x |= (unsigned)__shfl_xor((int)x, 16);
  return x | (unsigned)__shfl_xor((int)x, 32);
}

// Bits of the slots [a, b) among the 32 from t0 on.
SVD unsigned slots32(int t0, int a, int b) {
  const int lo = min(max(a - t0, 0), 32), hi = min(max(b - t0, 0), 32);
  return (hi > lo) ? (unsigned)(((1ull << hi) - 1ull) >> lo << lo) : 0u;
}
// 32 bits of a bit string of `words` words from bit j0 on (j0 > -32; zeros around it).
SVD unsigned anc32(const unsigned *w, int words, int j0) {
  const int k = j0 >> 5, sh = j0 & 31;
  const unsigned lo = (k >= 0 && k < words) ? w[k] : 0u, hi = (k + 1 >= 0 && k + 1 < words) ? w[k + 1] : 0u;
  return (unsigned)((((unsigned long long)hi << 32) | lo) >> sh);
}

template <typename T>
struct Mma;

// bf16: a 16-byte unit is 8 elements, one operand of a 16x16x32 instruction.  Score tile t2
// (0, 1) holds slots 8 (m / 4) + 4 t2 + m % 4, m its row: lane group g then has slots 8 g ..
// 8 g + 7 in the order of a value unit.
template <>
struct Mma<uint16_t> {
  static constexpr int E = 8, VT = 1;  // elements a unit; value units a lane needs per 16 d
  SVD static int key_slot(int t2, int m) { return 8 * (m >> 2) + 4 * t2 + (m & 3); }
  SVD static int val_slot(int, int g) { return 8 * g; }           // first slot of the lane's unit
  SVD static unsigned lane_bits(unsigned x, int g) { return (x >> (8 * g)) & 0xffu; }  // a tile's bits to score order
  SVD static f32x4 qk(u32x4 k, u32x4 q, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k), __builtin_bit_cast(bf16x8, q), c, 0, 0, 0);
  }
  struct P {
    bf16x8 w;
  };
  // The weights are rounded to bf16 (at most 2^-9 relative each, as the inputs themselves
  // are); their sum is taken in f32 before the rounding.
  SVD static P weights(const f32x4 (&s)[2]) {
    P p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p.w[i] = (__bf16)s[0][i];
      p.w[4 + i] = (__bf16)s[1][i];
    }
    return p;
  }
  SVD static f32x4 pv(const u32x4 (&v)[1], const P &p, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v[0]), p.w, c, 0, 0, 0);
  }
  SVD static bool non_finite(u32x4 v) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) bad |= (v[j] & 0x7f800000u) == 0x7f800000u || (v[j] & 0x7f80u) == 0x7f80u;
    return bad;
  }
  // Elements e >= n of the unit become zero.
  SVD static u32x4 cut(u32x4 v, int n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (n >= 2 * j + 2) ? v[j] : (n == 2 * j + 1) ? (v[j] & 0xffffu) : 0u;
    return v;
  }
  // Unit of f(element) with f in {0, 1}, as weights of the same type.
  template <typename F>
  SVD static u32x4 flags(u32x4 v, F f) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = (f(__uint_as_float(v[j] << 16)) ? 0x3f80u : 0u) | (f(__uint_as_float(v[j] & 0xffff0000u)) ? 0x3f800000u : 0u);
    return r;
  }
  SVD static void store4(char *p, float a, float b, float c, float d) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<bf16x4 *>(p) = bf16x4{(__bf16)a, (__bf16)b, (__bf16)c, (__bf16)d};
  }
};

// f32: a unit is 4 elements, one element each for four 16x16x4 instructions (instruction j
// of a step contracts over element j of every lane group's unit).  Score tile t2 holds slots
// 16 t2 + m; the value unit of lane group g for it is slots 16 t2 + 4 g .. + 3.
template <>
struct Mma<float> {
  static constexpr int E = 4, VT = 2;
  SVD static int key_slot(int t2, int m) { return 16 * t2 + m; }
  SVD static int val_slot(int t2, int g) { return 16 * t2 + 4 * g; }
  SVD static unsigned lane_bits(unsigned x, int g) { return ((x >> (4 * g)) & 0xfu) | (((x >> (16 + 4 * g)) & 0xfu) << 4); }
  SVD static f32x4 qk(u32x4 k, u32x4 q, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[j]), __uint_as_float(q[j]), c, 0, 0, 0);
    return c;
  }
  struct P {
    f32x4 w[2];
  };
  SVD static P weights(const f32x4 (&s)[2]) { return P{{s[0], s[1]}}; }
  SVD static f32x4 pv(const u32x4 (&v)[2], const P &p, f32x4 c) {
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(v[t2][j]), p.w[t2][j], c, 0, 0, 0);
    return c;
  }
  SVD static bool non_finite(u32x4 v) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) bad |= (v[j] & 0x7f800000u) == 0x7f800000u;
    return bad;
  }
  SVD static u32x4 cut(u32x4 v, int n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (n > j) ? v[j] : 0u;
    return v;
  }
  template <typename F>
  SVD static u32x4 flags(u32x4 v, F f) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = f(__uint_as_float(v[j])) ? 0x3f800000u : 0u;
    return r;
  }
  SVD static void store4(char *p, float a, float b, float c, float d) {
    *reinterpret_cast<f32x4 *>(p) = f32x4{a, b, c, d};
  }
};

// Workgroups resident on a CU (their waves' registers bound them: the output tile, the query
// rows, one tile of keys and one of values), which is also how many the grid has per CU.
template <typename T, int D, int R>
constexpr int attn_occ() {
  constexpr int regs = R * (D / 4) + R * (D * (int)sizeof(T) / 16) + 2 * (D * (int)sizeof(T) / 8) + 8 * R + 48;
  return regs <= 168 ? 3 : regs <= 256 ? 2 : 1;
}

template <typename T, int D, int R>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(attn_occ<T, D, R>()))) void k_attn(const AttnArgs a) {
  typedef Mma<T> M;
  constexpr int RT = 16 * R, E = M::E, ESZ = (int)sizeof(T);
  constexpr int KS = D / (4 * E);  // key units a lane holds of a 16-slot score tile
  constexpr int DT = D / 16;       // 16-wide tiles of the output's d
  constexpr int PADD = D + 4;      // rows of the LDS join tile, padded against bank conflicts
  constexpr unsigned MIN_SHARE = 4;  // a tile for each wave

  __shared__ float s_o[NW * RT * PADD];
  __shared__ float s_m[NW * RT], s_l[NW * RT];
  __shared__ int s_par[SV_CACHE_MAX_NEW];
  __shared__ uint16_t s_dep[RT];
  __shared__ unsigned s_anc[RT * (SV_CACHE_MAX_NEW / 32)];
  __shared__ unsigned s_w[NW];
  __shared__ unsigned s_at[2];
  __shared__ int s_bad;

  const int tid = threadIdx.x, lane = lane_id(), wid = tid / WAVE;
  const int m = lane & 15, g = lane >> 4;
  const int page = 1 << a.page_shift;
  // Consecutive shares on one XCD: the row tiles of a key head read the same keys and values
  // through that XCD's L2.
  const unsigned w = (blockIdx.x % LANES) * (a.grid / LANES) + blockIdx.x / LANES;

  // ---- this workgroup's share of all tiles
  unsigned T_all = 0, v = 0, ex = 0;
  for (int b0 = 0; b0 < a.B; b0 += NT) {
    v = (b0 + tid < a.B) ? seq_tiles<RT>(a, b0 + tid) : 0u;
    unsigned tot;
    ex = block_excl_scan(v, s_w, tot);
    T_all += tot;
  }
  const unsigned share = max((T_all + a.grid - 1) / a.grid, MIN_SHARE);
  if ((unsigned long long)w * share >= T_all) return;
  unsigned pos = w * share;
  const unsigned pos_end = min(T_all, pos + share);
  if (a.B <= NT) {
    if (pos >= ex && pos < ex + v) {
      s_at[0] = (unsigned)tid;
      s_at[1] = pos - ex;
    }
  } else {
    unsigned run = 0;
    for (int b0 = 0; run <= pos; b0 += NT) {
      v = (b0 + tid < a.B) ? seq_tiles<RT>(a, b0 + tid) : 0u;
      unsigned tot;
      ex = run + block_excl_scan(v, s_w, tot);
      if (pos >= ex && pos < ex + v) {
        s_at[0] = (unsigned)(b0 + tid);
        s_at[1] = pos - ex;
      }
      run += tot;
    }
  }
  __syncthreads();
  int b = (int)s_at[0];
  unsigned off = s_at[1];  // tiles of sequence b before pos

  const unsigned long long page_bytes = (unsigned long long)a.Hkv * page * D * ESZ;
  const unsigned head_bytes = (unsigned)page * D * ESZ;

  Seq sq = seq_of(a, b);
  int tree_b = -1;  // the sequence whose parents and depths are in LDS
  while (pos < pos_end) {
    // ---- the unit and the tiles of it that are this workgroup's
    unsigned per_head = 0;
    for (int rt = 0; rt < a.n_rt; ++rt) per_head += (unsigned)span_of<RT>(a, sq, rt).tiles;
    if (off >= per_head * (unsigned)a.Hkv) {
      off -= per_head * (unsigned)a.Hkv;
      sq = seq_of(a, ++b);
      continue;
    }
    const int h = (int)(off / per_head);
    unsigned l0 = off - (unsigned)h * per_head;
    int rt = 0;
    Span sp = span_of<RT>(a, sq, 0);
    while (l0 >= (unsigned)sp.tiles) {
      l0 -= (unsigned)sp.tiles;
      sp = span_of<RT>(a, sq, ++rt);
    }
    const int l1 = (int)min((unsigned)sp.tiles, l0 + (pos_end - pos));
    const bool whole = l0 == 0 && l1 == sp.tiles;
    const int unit = (b * a.Hkv + h) * a.n_rt + rt;
    const int32_t *table = a.page_table + (size_t)b * a.W;
    const int32_t *par = a.parent ? a.parent + (size_t)b * a.N : nullptr;
    const bool live = sp.i0 <= sp.i1;
    const int end_all = sq.len + sq.m;

    // ---- what makes the whole sequence invalid: the same test in every workgroup of it
    __syncthreads();  // the previous segment is done with the LDS
    if (tid == 0) s_bad = sq.ok ? 0 : -SV_ROW_BAD_LENGTH;
    if (par && sq.ok && tree_b != b)
      for (int i = tid; i < sq.m; i += NT) s_par[i] = par[i];
    __syncthreads();
    if (sq.ok && sq.m > 0) {
      if (par) {
        bool bad = false;
        for (int i = tid; i < sq.m; i += NT) bad |= (i == 0) ? s_par[0] != -1 : (s_par[i] < 0 || s_par[i] >= i);
        if (bad) atomicMax(&s_bad, 64 - SV_ROW_BAD_TREE);
      }
      int p0 = 0, np = 0;  // pages of the sinks, then from the window on
      const int first = (a.window > 0) ? max(0, sq.len - a.window + 1) : 0;
      p0 = first >> a.page_shift;
      const int ps = min((min(a.sinks, first) + page - 1) >> a.page_shift, p0);
      np = ((end_all + page - 1) >> a.page_shift) - p0 + ps;
      bool bad = false;
      for (int i = tid; i < np; i += NT) bad |= (unsigned)table[i < ps ? i : i - ps + p0] >= (unsigned)a.P;
      if (bad) atomicMax(&s_bad, -SV_ROW_BAD_PAGE);
    }
    __syncthreads();
    const int code = s_bad > 64 ? 64 - s_bad : -s_bad;  // a bad tree before a bad page
    if (tid == 0 && h == 0 && rt == 0 && l0 == 0) a.row_status[b] = code;

    f32x4 o[R][DT];
    float rm[R], rl[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rm[r] = -INFINITY;
      rl[r] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[r][d] = f32x4{0, 0, 0, 0};
    }

    if (live && code == 0) {
      // ---- depths of the rows' nodes and the nodes they see, where tiles of this segment need them
      const int i0 = sp.i0, words = (sq.m + 31) >> 5;
      const int last_tile = (l1 - 1 < sp.n_sink) ? l1 - 1 : l1 - 1 - sp.n_sink + sp.first;
      const bool masks = a.window > 0 || (last_tile + 1) * TILE > sq.len;
      if (par && masks) {
        const int n_nodes = sp.i1 - i0 + 1;
        for (int i = tid; i < n_nodes * words; i += NT) s_anc[i] = 0u;
        __syncthreads();
        for (int i = tid; i < n_nodes; i += NT) {
          int dep_i = 0;
          for (int j = s_par[i0 + i]; j >= 0; j = s_par[j]) ++dep_i;
          s_dep[i] = (uint16_t)dep_i;
          int d = dep_i;  // depth of j
          for (int j = i0 + i; j >= 0; j = s_par[j], --d)
            if (a.window <= 0 || dep_i - d < a.window || sq.len + d < a.sinks) s_anc[i * words + (j >> 5)] |= 1u << (j & 31);
        }
        __syncthreads();
        tree_b = b;
      }

      // ---- query rows
      u32x4 qf[R][KS];
      int node[R], dep[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = rt * RT + 16 * r + m;
        const int i = row / a.group, hh = row - i * a.group;
        const bool in = i < sq.m;
        node[r] = in ? i : sp.i1;
        dep[r] = (par && masks) ? (int)s_dep[node[r] - i0] : node[r];
        const char *qp = a.q + (long long)b * a.q_sb + (long long)(in ? i : 0) * a.q_sn + (size_t)(h * a.group + hh) * D * ESZ;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const u32x4 x = *reinterpret_cast<const u32x4 *>(qp + (4 * s + g) * 16);
          qf[r][s] = in ? x : u32x4{0, 0, 0, 0};
        }
      }

      const char *kh = a.k_pages + (size_t)h * head_bytes;
      const char *vh = a.v_pages + (size_t)h * head_bytes;
      auto tile_of = [&](int l) { return l < sp.n_sink ? l : l - sp.n_sink + sp.first; };
      // The pages of a tile's two halves (a page has at least 16 slots).  A half that no row
      // sees may have no page any more (behind the sequence, or left of the window): the
      // other half's page stands in for it.
      auto pages_of = [&](int l, int &pa, int &pb) {
        const int t0 = tile_of(l) * TILE, t1 = t0 + TILE / 2;
        const bool ha = t0 < a.sinks || t1 > sp.from;
        const bool hb = t1 < end_all && (t1 < a.sinks || t1 + TILE / 2 > sp.from);
        const int ia = t0 >> a.page_shift, ib = t1 >> a.page_shift;
        pa = table[ha ? ia : ib];
        pb = (hb && ib != ia) ? table[ib] : pa;
      };
      auto load_k = [&](int l, int pa, int pb, u32x4 (&k)[2][KS]) {
        const int t0 = tile_of(l) * TILE;
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
          const int sl = M::key_slot(t2, m);
          const char *p = kh + (unsigned long long)(unsigned)(sl < 16 ? pa : pb) * page_bytes + ((unsigned)((t0 + sl) & (page - 1)) + (unsigned)(g * page)) * 16u;
#pragma unroll
          for (int s = 0; s < KS; ++s) k[t2][s] = *reinterpret_cast<const u32x4 *>(p + (size_t)s * (4 * 16) * page);
        }
      };
      auto load_v = [&](int l, int pa, int pb, u32x4 (&v)[DT][M::VT]) {
        const int t0 = tile_of(l) * TILE;
#pragma unroll
        for (int t2 = 0; t2 < M::VT; ++t2) {
          const int sl = M::val_slot(t2, g);
          const char *p = vh + (unsigned long long)(unsigned)(sl < 16 ? pa : pb) * page_bytes + ((unsigned)(((t0 + sl) & (page - 1)) / E) * D + m) * 16u;
#pragma unroll
          for (int d = 0; d < DT; ++d) v[d][t2] = *reinterpret_cast<const u32x4 *>(p + d * 256);
        }
      };

      int l = (int)l0 + wid;
      u32x4 kf[2][KS];
      int pa = 0, pb = 0, na = 0, nb = 0;
      if (l < l1) {
        pages_of(l, pa, pb);
        load_k(l, pa, pb, kf);
        if (l + NW < l1) pages_of(l + NW, na, nb);
      }
      for (; l < l1; l += NW) {
        const int t0 = tile_of(l) * TILE;
        u32x4 vf[DT][M::VT];
        load_v(l, pa, pb, vf);
        f32x4 s[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) s[r][0] = s[r][1] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][t2] = M::qk(kf[t2][k], qf[r][k], s[r][t2]);
        pa = na;
        pb = nb;
        if (l + NW < l1) {
          load_k(l + NW, pa, pb, kf);
          if (l + 2 * NW < l1) pages_of(l + 2 * NW, na, nb);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) s[r][t2] = s[r][t2] * a.c2;

        // Tiles that every row of the unit sees whole need no mask.
        const bool plain = t0 + TILE <= sq.len &&
                           (a.window <= 0 || t0 + TILE <= a.sinks || (long long)sq.len + sq.m - 1 - t0 < a.window);
        unsigned vis[R];  // the row's view of this lane's slots, bit 4 t2 + i
#pragma unroll
        for (int r = 0; r < R; ++r) vis[r] = 0u;
        if (!plain) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const int pos_r = sq.len + dep[r], lo = (a.window > 0) ? pos_r - a.window + 1 : 0;
            const int head = par ? sq.len : pos_r + 1;  // slots that window and sinks alone decide
            unsigned see = slots32(t0, lo, head) | slots32(t0, 0, min(a.sinks, head));
            if (par) see |= anc32(&s_anc[(node[r] - i0) * words], words, t0 - sq.len);
            vis[r] = M::lane_bits(see, g);
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[r][t2][i] = ((vis[r] >> (4 * t2 + i)) & 1u) ? s[r][t2][i] : -INFINITY;
          }
          if (t0 + TILE > end_all)  // slots behind the sequence hold anything
#pragma unroll
            for (int t2 = 0; t2 < M::VT; ++t2)
#pragma unroll
              for (int d = 0; d < DT; ++d) vf[d][t2] = M::cut(vf[d][t2], end_all - t0 - M::val_slot(t2, g));
        }

        typename M::P pw[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float mx = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                           fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
          mx = fmaxf(rm[r], xor_max(mx));
          if (__any(mx > rm[r])) {  // a new maximum in some row: all sums so far to the new scale
            const float f = (rm[r] == -INFINITY) ? 0.0f : fast_exp2(rm[r] - mx);
            rl[r] *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[r][d] = o[r][d] * f;
            rm[r] = mx;
          }
          const float mu = (mx == -INFINITY) ? 0.0f : mx;
          float sum = 0.0f;
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[r][t2][i] = fast_exp2(s[r][t2][i] - mu);
            sum += (s[r][t2][0] + s[r][t2][1]) + (s[r][t2][2] + s[r][t2][3]);
          }
          rl[r] += sum;
          pw[r] = M::weights(s[r]);
        }

        // A value that is not finite must reach the rows that see it and no others, and a
        // zero weight does not keep it away (0 * inf): such values are taken out of the
        // product, and what they are to each row follows from products of flags.
        bool odd = false;
        if (!plain) {
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int t2 = 0; t2 < M::VT; ++t2) odd |= M::non_finite(vf[d][t2]);
        }
        if (!plain && __any(odd)) {
          typename M::P sees[R];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            f32x4 one[2];
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
              for (int i = 0; i < 4; ++i) one[t2][i] = ((vis[r] >> (4 * t2 + i)) & 1u) ? 1.0f : 0.0f;
            sees[r] = M::weights(one);
          }
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            u32x4 fn[M::VT], fp[M::VT], fm[M::VT];
#pragma unroll
            for (int t2 = 0; t2 < M::VT; ++t2) {
              fn[t2] = M::flags(vf[d][t2], [](float x) { return !(x == x); });
              fp[t2] = M::flags(vf[d][t2], [](float x) { return x == INFINITY; });
              fm[t2] = M::flags(vf[d][t2], [](float x) { return x == -INFINITY; });
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const f32x4 z = {0, 0, 0, 0};
              const f32x4 cn = M::pv(fn, sees[r], z), cp = M::pv(fp, sees[r], z), cm = M::pv(fm, sees[r], z);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                o[r][d][i] += (cn[i] > 0.0f || (cp[i] > 0.0f && cm[i] > 0.0f)) ? NAN
                              : cp[i] > 0.0f ? INFINITY : cm[i] > 0.0f ? -INFINITY : 0.0f;
            }
          }
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int t2 = 0; t2 < M::VT; ++t2) {
              const u32x4 ok = M::flags(vf[d][t2], [](float x) { return x - x == 0.0f; });
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const unsigned keep = (sizeof(T) == 2) ? ((ok[j] & 0xffffu ? 0xffffu : 0u) | (ok[j] >> 16 ? 0xffff0000u : 0u))
                                                       : (ok[j] ? 0xffffffffu : 0u);
                vf[d][t2][j] &= keep;
              }
            }
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < R; ++r) o[r][d] = M::pv(vf[d], pw[r], o[r][d]);
      }
    }

    // ---- the four waves joined: rows' maxima and sums, then the output tiles
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float l_row = xor_sum(rl[r]);
      if (g == 0) {
        s_m[wid * RT + 16 * r + m] = rm[r];
        s_l[wid * RT + 16 * r + m] = l_row;
      }
#pragma unroll
      for (int d = 0; d < DT; ++d)
        *reinterpret_cast<f32x4 *>(&s_o[(wid * RT + 16 * r + m) * PADD + 16 * d + 4 * g]) = o[r][d];
    }
    __syncthreads();
    const unsigned slot = 2 * w + (l0 == 0 ? 1u : 0u);
    for (int x = tid; x < RT * (D / 4); x += NT) {
      const int row = x / (D / 4), c4 = x - row * (D / 4);
      float mt = -INFINITY;
#pragma unroll
      for (int k = 0; k < NW; ++k) mt = fmaxf(mt, s_m[k * RT + row]);
      f32x4 acc = {0, 0, 0, 0};
      float ls = 0.0f;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float mk = s_m[k * RT + row];
        if (mk == -INFINITY && s_l[k * RT + row] == 0.0f) continue;  // a wave without a tile
        const float f = fast_exp2(mk - mt);
        ls += f * s_l[k * RT + row];
        acc += *reinterpret_cast<const f32x4 *>(&s_o[(k * RT + row) * PADD + 4 * c4]) * f;
      }
      const int rg = rt * RT + row, i = rg / a.group, hh = rg - i * a.group;
      if (whole) {
        if (i >= a.N) continue;
        float inv = 1.0f / ls;
        if (code != 0) inv = NAN;
        f32x4 y = acc * inv;
        if (code == 0 && i >= sq.m) y = f32x4{0, 0, 0, 0};
        M::store4(a.out + ((((size_t)b * a.N + i) * a.Hq + h * a.group + hh) * D + 4 * c4) * ESZ, y[0], y[1], y[2], y[3]);
      } else {
        *reinterpret_cast<f32x4 *>(&a.part_o[((size_t)slot * RT + row) * D + 4 * c4]) = acc;
        if (c4 == 0) a.part_ml[(size_t)slot * RT + row] = make_float2(mt, ls);
      }
    }
    if (tid == 0 && l0 == 0) {
      const unsigned last = (pos + (unsigned)sp.tiles - 1) / share;
      a.desc[unit] = make_uint4(w, last - w + 1, (unsigned)(code ? 0x80000000u : 0u) | (unsigned)max(0, sq.ok ? sq.m : 0), 0u);
    }
    pos += (unsigned)l1 - l0;
    off += (unsigned)l1 - l0;
  }
}

// Units that several workgroups streamed: one wave a row, its partial tiles in the order of
// the slots.
template <typename T, int D, int R>
__global__ __launch_bounds__(NT) void k_attn_join(const AttnArgs a) {
  typedef Mma<T> M;
  constexpr int RT = 16 * R, ESZ = (int)sizeof(T), PL = D / 4;  // lanes that hold a row
  const int lane = lane_id(), wid = threadIdx.x / WAVE;
  const int unit = blockIdx.x / (RT / NW), row = (blockIdx.x % (RT / NW)) * NW + wid;
  const uint4 ds = a.desc[unit];
  const int n = (int)ds.y;
  if (n <= 1) return;
  const int rt = unit % a.n_rt, bh = unit / a.n_rt, h = bh % a.Hkv, b = bh / a.Hkv;
  const int rg = rt * RT + row, i = rg / a.group, hh = rg - i * a.group;
  if (i >= a.N) return;
  char *out = a.out + (((size_t)b * a.N + i) * a.Hq + h * a.group + hh) * (size_t)D * ESZ;
  auto slot_of = [&](int k) { return 2 * (ds.x + (unsigned)k) + (k == 0 ? 1u : 0u); };
  float mt = -INFINITY;
  for (int k = lane; k < n; k += WAVE) mt = fmaxf(mt, a.part_ml[(size_t)slot_of(k) * RT + row].x);
#pragma unroll
  for (int o = 32; o; o >>= 1) mt = fmaxf(mt, __shfl_xor(mt, o));
  // Lanes in groups of PL take the partials in turn (PL = 16, 32 or 64: 4, 2 or 1 of them).
  constexpr int NG = WAVE / PL;
  const int c4 = lane % PL, grp = lane / PL;
  f32x4 acc = {0, 0, 0, 0};
  float ls = 0.0f;
#pragma unroll 4
  for (int k = grp; k < n; k += NG) {
    const size_t s = (size_t)slot_of(k) * RT + row;
    const float2 ml = a.part_ml[s];
    const f32x4 x = *reinterpret_cast<const f32x4 *>(&a.part_o[s * D + 4 * c4]);
    const float f = (ml.x == -INFINITY && ml.y == 0.0f) ? 0.0f : fast_exp2(ml.x - mt);
    const bool none = ml.x == -INFINITY && ml.y == 0.0f;
    ls += none ? 0.0f : f * ml.y;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += none ? 0.0f : f * x[j];
  }
#pragma unroll
  for (int o = PL; o < WAVE; o <<= 1) {
    ls += __shfl_xor(ls, o);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], o);
  }
  if (grp != 0) return;
  float inv = 1.0f / ls;
  f32x4 y = acc * inv;
  if ((int)(ds.z & 0x7fffffffu) <= i) y = f32x4{0, 0, 0, 0};
  if (ds.z >> 31) y = f32x4{NAN, NAN, NAN, NAN};
  M::store4(out + c4 * 4 * ESZ, y[0], y[1], y[2], y[3]);
}

}  // namespace sv

// ======================================================================== host side

namespace {

using namespace sv;
using sv_host::align256;

struct AttnPlan {
  int R, RT, n_rt, occ;
  unsigned grid;
  long long units;
  size_t part_o, part_ml, desc, total;
};

// Row tiles a wave holds: as many as the rows need, up to what its registers take.
int rows_R(long long rows, int D, int esz) {
  const int most = (esz == 2) ? (D == 256 ? 2 : 4) : (D == 64 ? 4 : D == 128 ? 2 : 1);
  const int need = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  return need < most ? need : most;
}

bool pow2_page(int32_t page) { return page >= 16 && page <= 256 && (page & (page - 1)) == 0; }

template <typename T, int D, int R>
constexpr int occ_of() { return attn_occ<T, D, R>(); }

int plan_occ(int D, int esz, int R) {
  if (esz == 2) {
    if (D == 64) return R == 1 ? occ_of<uint16_t, 64, 1>() : R == 2 ? occ_of<uint16_t, 64, 2>() : occ_of<uint16_t, 64, 4>();
    if (D == 128) return R == 1 ? occ_of<uint16_t, 128, 1>() : R == 2 ? occ_of<uint16_t, 128, 2>() : occ_of<uint16_t, 128, 4>();
    return R == 1 ? occ_of<uint16_t, 256, 1>() : occ_of<uint16_t, 256, 2>();
  }
  if (D == 64) return R == 1 ? occ_of<float, 64, 1>() : R == 2 ? occ_of<float, 64, 2>() : occ_of<float, 64, 4>();
  if (D == 128) return R == 1 ? occ_of<float, 128, 1>() : occ_of<float, 128, 2>();
  return occ_of<float, 256, 1>();
}

bool attn_shape_ok(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page, int32_t W) {
  return B >= 1 && N >= 1 && N <= SV_CACHE_MAX_NEW && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 &&
         (D == 64 || D == 128 || D == 256) && pow2_page(page) && W >= 1 && (long long)W * page <= 0x7fffffffLL - 4096;
}

bool attn_plan(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page, int32_t W, int esz, AttnPlan &p) {
  const long long rows = (long long)N * (Hq / Hkv);
  p.R = rows_R(rows, D, esz);
  p.RT = 16 * p.R;
  const long long n_rt = (rows + p.RT - 1) / p.RT;
  p.units = (long long)B * Hkv * n_rt;
  const long long most = ((long long)W * page + TILE - 1) / TILE + 1;  // tiles of a unit
  if (p.units * most > 0x7fffffffLL || p.units * p.RT > 0x7fffffffLL) return false;
  p.n_rt = (int)n_rt;
  p.occ = plan_occ(D, esz, p.R);
  long long grid = 256LL * p.occ;  // one resident set of the device's 256 CUs
  const long long need = (p.units * most + 3) / 4;
  if (need < grid) grid = need;
  p.grid = (unsigned)((grid + LANES - 1) / LANES * LANES);
  size_t o = 0;
  p.part_o = o; o = align256(o + (size_t)2 * p.grid * p.RT * D * 4);
  p.part_ml = o; o = align256(o + (size_t)2 * p.grid * p.RT * 8);
  p.desc = o; o = align256(o + (size_t)p.units * 16);
  p.total = o;
  return true;
}

template <typename T, int D, int R>
void attn_go(sv_host::Launcher &L, AttnArgs &a, const AttnPlan &p) {
  void *args[] = {&a};
  L.go((const void *)&k_attn<T, D, R>, p.grid, args);
  L.go((const void *)&k_attn_join<T, D, R>, (unsigned)(p.units * (p.RT / NW)), args);
}

sv_status attn_run(const void *q, int64_t q_sb, int64_t q_sn, const void *k_pages, const void *v_pages, sv_dtype dt,
                   const int32_t *table, const int32_t *cache_len, const int32_t *n_new, const int32_t *parent, int32_t B,
                   int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page, int32_t P, int32_t W, float scale,
                   int32_t window, int32_t sinks, void *out, int32_t *status, void *ws, size_t ws_bytes, void *stream,
                   void *const *ev, int32_t nev, int32_t *nl) {
  if (nl) *nl = 0;
  if (dt != SV_F32 && dt != SV_BF16) return SV_ERR_DTYPE;
  const int esz = dt == SV_BF16 ? 2 : 4;
  if (!attn_shape_ok(B, N, Hq, Hkv, D, page, W) || P < 1) return SV_ERR_SHAPE;
  if (!isfinite(scale) || window < 0 || sinks < 0 || (sinks > 0 && window == 0)) return SV_ERR_PARAM;
  AttnPlan p;
  if (!attn_plan(B, N, Hq, Hkv, D, page, W, esz, p)) return SV_ERR_SHAPE;
  if (!q || !k_pages || !v_pages || !table || !cache_len || !out || !status || !ws) return SV_ERR_NULL;
  if (((uintptr_t)q | (uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)out | (uintptr_t)(q_sb * esz) | (uintptr_t)(q_sn * esz)) & 15)
    return SV_ERR_ALIGN;
  if (ws_bytes < p.total || ((uintptr_t)ws & 255)) return SV_ERR_WORKSPACE;
  char *base = static_cast<char *>(ws);
  AttnArgs a = {};
  a.q = static_cast<const char *>(q);
  a.k_pages = static_cast<const char *>(k_pages);
  a.v_pages = static_cast<const char *>(v_pages);
  a.q_sb = q_sb * esz;
  a.q_sn = q_sn * esz;
  a.page_table = table;
  a.cache_len = cache_len;
  a.n_new = n_new;
  a.parent = parent;
  a.B = B;
  a.N = N;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.page_shift = __builtin_ctz((unsigned)page);
  a.P = P;
  a.W = W;
  a.c2 = (float)((double)scale * LOG2E);
  a.window = window;
  a.sinks = sinks;
  a.out = static_cast<char *>(out);
  a.row_status = status;
  a.n_rt = p.n_rt;
  a.grid = p.grid;
  a.part_o = (float *)(base + p.part_o);
  a.part_ml = (float2 *)(base + p.part_ml);
  a.desc = (uint4 *)(base + p.desc);
  sv_host::Launcher L{(hipStream_t)stream, ev, nev};
  if (esz == 2) {
    if (D == 64) p.R == 1 ? attn_go<uint16_t, 64, 1>(L, a, p) : p.R == 2 ? attn_go<uint16_t, 64, 2>(L, a, p) : attn_go<uint16_t, 64, 4>(L, a, p);
    else if (D == 128) p.R == 1 ? attn_go<uint16_t, 128, 1>(L, a, p) : p.R == 2 ? attn_go<uint16_t, 128, 2>(L, a, p) : attn_go<uint16_t, 128, 4>(L, a, p);
    else p.R == 1 ? attn_go<uint16_t, 256, 1>(L, a, p) : attn_go<uint16_t, 256, 2>(L, a, p);
  } else {
    if (D == 64) p.R == 1 ? attn_go<float, 64, 1>(L, a, p) : p.R == 2 ? attn_go<float, 64, 2>(L, a, p) : attn_go<float, 64, 4>(L, a, p);
    else if (D == 128) p.R == 1 ? attn_go<float, 128, 1>(L, a, p) : attn_go<float, 128, 2>(L, a, p);
    else attn_go<float, 256, 1>(L, a, p);
  }
  if (nl) *nl = L.n;
  return L.e == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

}  // namespace

extern "C" {

size_t sv_attention_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                                    int32_t table_width, sv_dtype dtype) {
  AttnPlan p;
  if ((dtype != SV_F32 && dtype != SV_BF16) || !attn_shape_ok(B, N, Hq, Hkv, D, page_size, table_width) ||
      !attn_plan(B, N, Hq, Hkv, D, page_size, table_width, dtype == SV_BF16 ? 2 : 4, p))
    return 256;
  return p.total;
}

sv_status spec_paged_attention(const void *q, int64_t q_stride_b, int64_t q_stride_n, const void *k_pages,
                               const void *v_pages, sv_dtype dtype, const int32_t *page_table,
                               const int32_t *cache_len, const int32_t *n_new, const int32_t *parent, int32_t B,
                               int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                               int32_t table_width, float scale, int32_t window, int32_t sinks, void *out,
                               int32_t *row_status, void *workspace, size_t workspace_bytes, void *stream) {
  return attn_run(q, q_stride_b, q_stride_n, k_pages, v_pages, dtype, page_table, cache_len, n_new, parent, B, N, Hq, Hkv, D,
                  page_size, num_pages, table_width, scale, window, sinks, out, row_status, workspace, workspace_bytes,
                  stream, nullptr, 0, nullptr);
}

sv_status spec_paged_attention_timed(const void *q, int64_t q_stride_b, int64_t q_stride_n, const void *k_pages,
                                     const void *v_pages, sv_dtype dtype, const int32_t *page_table,
                                     const int32_t *cache_len, const int32_t *n_new, const int32_t *parent, int32_t B,
                                     int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                                     int32_t num_pages, int32_t table_width, float scale, int32_t window, int32_t sinks,
                                     void *out, int32_t *row_status, void *workspace, size_t workspace_bytes,
                                     void *stream, void *const *events, int32_t n_events, int32_t *n_launched) {
  return attn_run(q, q_stride_b, q_stride_n, k_pages, v_pages, dtype, page_table, cache_len, n_new, parent, B, N, Hq, Hkv, D,
                  page_size, num_pages, table_width, scale, window, sinks, out, row_status, workspace, workspace_bytes,
                  stream, events, n_events, n_launched);
}

const char *sv_attention_launch_plan(void) { return "k_attn;k_attn_join"; }

}  // extern "C"
