// spec_attention.hip -- attention of a round's new tokens over a paged key-value cache.
//
// For node i of sequence b and query head h: out = softmax(scale q.k) v over the slots the
// node sees (include/spec_cache.h).  All query rows of one key head, row r = node * group +
// head in group, read the same keys and values, so a unit of work is (sequence, key head,
// row tile) and streams the sequence's slots once, 32 at a time:
//   S^T = K Q^T   keys as the matrix instruction's A operand, query rows as its columns
//   O^T += V^T P^T
// With rows as columns a lane owns one query row of each 16-row tile, in both products:
// the row's running maximum and sum live in that lane's registers, rescaling is one factor
// a lane, and the weights leave the first product in exactly the lanes and order in which
// the second one takes them (the order of the slots in a score tile is chosen for that).
//
// Two kernels, by the rows of a unit (attn_plan):
//   k_attn       up to 32 rows: bound by the cache's bytes.  The cache's layout puts the 16
//                bytes a lane multiplies together, so keys and values go from HBM to the lanes
//                that use them with no staging; each of the four waves takes every fourth tile,
//                and they join through LDS at the end.
//   k_attn_wide  more rows: the waves own rows instead, and share each tile through LDS, so
//                that the L2 and L1 are read once for 64 or 128 rows.
// The tiles of all units are laid end to end, in rounds of what a workgroup takes at a time,
// and cut into equal shares, one a workgroup,
// whatever the lengths of the sequences (a share may end in the middle of one unit and go on
// with the next); units that several workgroups streamed are joined by k_attn_join.  Sums run
// in a fixed order: same call, same bits.

#include "sv_common.h"

#include "spec_cache.h"

namespace sv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int TILE = 32;  // slots a wave takes at a time

struct AttnArgs {
  const char *q, *k_pages, *v_pages;
  long long q_sb, q_sn;  // bytes
  const int32_t *page_table, *cache_len, *n_new, *parent, *prior;
  int B, N, Hq, Hkv, group, page_shift, P, W;
  float c2;        // |scale| log2 e: weights are powers of two
  unsigned flip;   // the sign bits of q, for a negative scale
  float slack;     // 8 / c2: see Rows::soften
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
  bool ok;  // not refused before, and lengths fit; the pages and the tree are checked elsewhere
};

// The code of an earlier call that refused the sequence, or 0.
SVD int prior_of(const AttnArgs &a, int b) { return a.prior ? min(a.prior[b], 0) : 0; }

SVD Seq seq_of(const AttnArgs &a, int b) {
  Seq s;
  s.len = a.cache_len[b];
  s.m = a.n_new ? a.n_new[b] : a.N;
  s.ok = prior_of(a, b) == 0 && s.len >= 0 && s.m >= 0 && s.m <= a.N && (long long)s.len + s.m <= ((long long)a.W << a.page_shift);
  if (!s.ok) s.len = s.m = 0;
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
// Work is counted in rounds of ROUND tiles, what a workgroup takes at a time; a unit begins with
// a round of its own.
template <int ROUND>
SVD unsigned rounds_of(const Span &p) { return (unsigned)(p.tiles + ROUND - 1) / ROUND; }
// The parts that a unit of r rounds is cut into, at most `most` rounds each, and a head's row
// tiles together (most = 1: its rounds).
SVD unsigned parts_of(unsigned r, unsigned most) { return (r + most - 1) / most; }
template <int RT, int ROUND>
SVD unsigned head_parts(const AttnArgs &a, const Seq &s, unsigned most) {
  unsigned t = 0;
  for (int rt = 0; rt < a.n_rt; ++rt) t += parts_of(rounds_of<ROUND>(span_of<RT>(a, s, rt)), most);
  return t;
}

// Over the four lanes of a column (lane % 16 equal): the swaps exchange halves of lane rows
// between two registers, which leaves both operands of each step in every lane.
SVD float col_max(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned v = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
SVD float col_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}
// Page ids by scalar loads: they do not queue behind the keys and values in flight.  (No
// kernel here writes the table.)
typedef const __attribute__((address_space(4))) int32_t *TablePtr;
SVD int page_at(TablePtr t, int i) { return t[i]; }

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

// Score tile t2 (0, 1) of a tile holds its slots 16 t2 + m, m the row: 16 lanes read 256 bytes
// of keys together (in pieces of 64 a tile took a fifth longer).  Lane group g then has the
// scores of slots 16 t2 + 4 g + i, i < 4.

// bf16: a 16-byte unit is 8 elements, one operand of a 16x16x32 instruction.
template <>
struct Mma<uint16_t> {
  static constexpr int E = 8, VT = 1;  // elements a unit; value units a lane needs per 16 d
  SVD static int val_slot(int, int g) { return 8 * g; }           // first slot of the lane's unit
  // A score tile's sums while they grow, and the scores.
  typedef f32x4 Dot;
  SVD static void qk(u32x4 k, u32x4 q, Dot &c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k), __builtin_bit_cast(bf16x8, q), c, 0, 0, 0);
  }
  SVD static f32x4 score(const Dot &c) { return c; }
  struct P {
    bf16x8 w;
  };
  // The weights are rounded to bf16 (by at most 2^-8 relative each, as the inputs themselves
  // were), and the sum they are divided by is that of the rounded weights, in f32: an error that
  // the weights share cancels, and a row that sees one slot gets its value exactly.  The sum is
  // one more product, with ones.  A lane of the second product wants
  // slots 8 g .. 8 g + 7, a value unit: with the two score tiles' pairs of weights by lane group
  // as a0 a1 a2 a3 and b0 b1 b2 b3, the swaps make a0 a2 b0 b2 and a1 a3 b1 b3 of them.
  SVD static P weights(const f32x4 (&s)[2]) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned x = __builtin_bit_cast(unsigned, bf16x2{(__bf16)s[0][2 * j], (__bf16)s[0][2 * j + 1]});
      const unsigned y = __builtin_bit_cast(unsigned, bf16x2{(__bf16)s[1][2 * j], (__bf16)s[1][2 * j + 1]});
      const auto h = __builtin_amdgcn_permlane32_swap(x, y, false, false);
      const auto q = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
      w[j] = q[0];
      w[2 + j] = q[1];
    }
    return P{__builtin_bit_cast(bf16x8, w)};
  }
  SVD static f32x4 pv(const u32x4 (&v)[1], const P &p, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v[0]), p.w, c, 0, 0, 0);
  }
  // A row's sum of weights: all of it in every element.
  typedef f32x4 Sum;
  SVD static Sum add(const P &p, const f32x4 (&)[2], Sum c) {
    const u32x4 ones[1] = {u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}};
    return pv(ones, p, c);
  }
  SVD static float total(Sum c) { return c[0]; }
  SVD static bool non_finite(u32x4 v) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) bad |= (v[j] & 0x7f800000u) == 0x7f800000u || (v[j] & 0x7f80u) == 0x7f80u;
    return bad;
  }
  // The unit with elements that are not finite set to zero.
  SVD static u32x4 finite(u32x4 v) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] &= ((v[j] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) | ((v[j] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
    return v;
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
// of a step contracts over element j of every lane group's unit); the lane's value units are
// slots 16 t2 + 4 g .. + 3, as its scores are.
template <>
struct Mma<float> {
  static constexpr int E = 4, VT = 2;
  SVD static int val_slot(int t2, int g) { return 16 * t2 + 4 * g; }
  // Four sums, one for each element of a unit: a single one, which every instruction lengthens
  // by four products, gathers more rounding errors, and the weights carry them (350 slots, D =
  // 256, against 64 bits: 1.2e-6, with four 4.1e-7; one token of 16 sequences of 4096 slots: D =
  // 128 93, with four 96 us, D = 256 184, with four 198 us).
  struct Dot {
    f32x4 c[4];
  };
  SVD static void qk(u32x4 k, u32x4 q, Dot &s) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s.c[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[j]), __uint_as_float(q[j]), s.c[j], 0, 0, 0);
  }
  SVD static f32x4 score(const Dot &s) { return (s.c[0] + s.c[1]) + (s.c[2] + s.c[3]); }
  struct P {
    f32x4 w[2];
  };
  SVD static P weights(const f32x4 (&s)[2]) { return P{{s[0], s[1]}}; }
  // A row's sum of weights: a part of it in each of its four lanes.
  typedef float Sum;
  SVD static Sum add(const P &, const f32x4 (&s)[2], Sum c) {
    return c + (((s[0][0] + s[0][1]) + (s[0][2] + s[0][3])) + ((s[1][0] + s[1][1]) + (s[1][2] + s[1][3])));
  }
  SVD static float total(Sum c) { return col_sum(c); }
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
  SVD static u32x4 finite(u32x4 v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (v[j] & 0x7f800000u) == 0x7f800000u ? 0u : v[j];
    return v;
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

// ---------------------------------------------------------------- a workgroup's share

// One unit's part of a share, and what the whole workgroup knows about it.
struct Segment {
  Seq sq;
  Span sp;
  int b, h, rt, l0, l1;  // the segment is the unit's tiles [l0, l1)
  TablePtr table;
  const int32_t *par;
  int words;   // of a node's bit string
  bool masks;  // some tile of the segment is not seen whole by every row

  SVD int tile(int l) const { return (l < sp.n_sink ? l : l - sp.n_sink + sp.first) * TILE; }
  SVD int end() const { return sq.len + sq.m; }
  // Every row of the unit sees the whole tile.
  SVD bool plain(const AttnArgs &a, int t0) const {
    return t0 + TILE <= sq.len && (a.window <= 0 || t0 + TILE <= a.sinks || (long long)sq.len + sq.m - 1 - t0 < a.window);
  }
  // The pages of a tile's two halves (a page has at least 16 slots).  A half that no row sees
  // may have no page any more (behind the sequence, or left of the window): the other half's
  // page stands in for it.
  SVD void pages(const AttnArgs &a, int t0, int &pa, int &pb) const {
    const int t1 = t0 + TILE / 2;
    const bool ha = t0 < a.sinks || t1 > sp.from;
    const bool hb = t1 < end() && (t1 < a.sinks || t1 + TILE / 2 > sp.from);
    const int ia = t0 >> a.page_shift, ib = t1 >> a.page_shift;
    pa = page_at(table, ha ? ia : ib);
    pb = (hb && ib != ia) ? page_at(table, ib) : pa;
    // Tiles are fetched before the sequence's pages have been checked: a page of no pool is
    // page 0 here (and the sequence's rows become NaN).
    pa = (unsigned)pa < (unsigned)a.P ? pa : 0;
    pb = (unsigned)pb < (unsigned)a.P ? pb : 0;
  }
  // The slots of a tile that a row sees, as bits.
  SVD unsigned sees(const AttnArgs &a, int t0, int dep, const unsigned *anc) const {
    const int pos = sq.len + dep, lo = (a.window > 0) ? max(0, pos - a.window + 1) : 0;
    const int head = par ? sq.len : pos + 1;  // slots that window and sinks alone decide
    unsigned see = slots32(t0, lo, head) | slots32(t0, 0, min(a.sinks, head));
    if (par) see |= anc32(anc, words, t0 - sq.len);
    return see;
  }
};

// LDS of either kernel besides its tiles: the tree, sized by the call (books_bytes), and what
// the prologue needs.
struct SharedBooks {
  uint16_t *par;   // [N] parents (node 0's is not kept)
  uint16_t *dep;   // [nodes of a row tile] their depths
  unsigned *anc;   // [nodes of a row tile][words] the nodes each of them sees
  unsigned *w, *at, *tries;  // [NW], [2], [4]
  int *bad;
};
SV_HD int tile_nodes(int RT, int N, int group) {
  const int n = (RT - 1) / group + 2;  // a tile may begin and end inside a node's heads
  return n < N ? n : N;
}
SV_HD unsigned books_bytes(int RT, int N, int group, bool tree) {
  const unsigned n = tree ? (unsigned)tile_nodes(RT, N, group) : 0u;
  return (NW + 12) * 4 + n * ((N + 31) / 32) * 4 + ((n + (tree ? (unsigned)N : 0u) + 1) / 2) * 4;
}
SVD SharedBooks books_at(unsigned *p, int RT, int N, int group) {
  const int n = tile_nodes(RT, N, group);
  SharedBooks s;
  s.w = p;
  s.at = p + NW;
  s.bad = reinterpret_cast<int *>(p + NW + 2);
  s.tries = p + NW + 4;
  s.anc = p + NW + 12;
  s.dep = reinterpret_cast<uint16_t *>(s.anc + n * ((N + 31) / 32));
  s.par = s.dep + n;
  return s;
}

// The code of a sequence: the same test in every workgroup that streams a part of it, so that
// all its rows agree.
SVD int seq_code(const AttnArgs &a, const Seq &sq, int b, const SharedBooks &s) {
  const int tid = threadIdx.x, page = 1 << a.page_shift;
  const int32_t *table = a.page_table + (size_t)b * a.W;
  if (!sq.ok) {
    const int prior = prior_of(a, b);
    return prior != 0 ? prior : SV_ROW_BAD_LENGTH;
  }
  if (sq.m == 0) return 0;
  int bad = 0;
  if (a.parent)
    for (int i = tid; i < sq.m; i += NT) {
      const int p = a.parent[(size_t)b * a.N + i];
      s.par[i] = (uint16_t)p;
      if (i == 0 ? p != -1 : (p < 0 || p >= i)) bad = 2;
    }
  // pages of the sinks, then from the window on
  const int first = (a.window > 0) ? max(0, sq.len - a.window + 1) : 0;
  const int p0 = first >> a.page_shift;
  const int ps = min((min(a.sinks, first) + page - 1) >> a.page_shift, p0);
  const int np = ((sq.len + sq.m + page - 1) >> a.page_shift) - p0 + ps;
  for (int i = tid; i < np; i += NT)
    if ((unsigned)table[i < ps ? i : i - ps + p0] >= (unsigned)a.P) bad |= 1;
  if (tid == 0) *s.bad = 0;
  __syncthreads();
  if (bad) atomicOr(s.bad, bad);
  __syncthreads();
  const int x = *s.bad;
  return (x & 2) ? SV_ROW_BAD_TREE : (x & 1) ? SV_ROW_BAD_PAGE : 0;
}

// Depths of the row tile's nodes and the nodes each sees, window and sinks included.
SVD void tree_books(const AttnArgs &a, const Segment &g, const SharedBooks &s) {
  const int tid = threadIdx.x, i0 = g.sp.i0, n = g.sp.i1 - i0 + 1;
  for (int i = tid; i < n * g.words; i += NT) s.anc[i] = 0u;
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    // up from the node, then down in depth again where the window cuts ancestors off
    unsigned *anc = s.anc + i * g.words;
    int dep = 0, j = i0 + i;
    for (;; j = s.par[j], ++dep) {
      anc[j >> 5] |= 1u << (j & 31);
      if (j == 0) break;
    }
    s.dep[i] = (uint16_t)dep;
    if (a.window > 0 && dep >= a.window)
      for (int d = dep, k = i0 + i;; k = s.par[k], --d) {  // d: the depth of k
        if (dep - d >= a.window && g.sq.len + d >= a.sinks) anc[k >> 5] &= ~(1u << (k & 31));
        if (d == 0) break;
      }
  }
  __syncthreads();
}

// Where a row of a segment goes: to the output if the segment is the whole unit, else to the
// segment's partial tile.
template <typename T, int D>
struct RowSink {
  enum { SKIP, OUT, ZERO, PART } kind;
  char *p;
  float inv;
  // Elements 4 c4 .. 4 c4 + 3 for c4 = first, first + step, ...: acc[0], acc[1], ...
  template <int n>
  SVD void put(int first, int step, const f32x4 (&acc)[n]) const {
    if (kind == PART) {
#pragma unroll
      for (int k = 0; k < n; ++k) reinterpret_cast<f32x4 *>(p)[first + k * step] = acc[k];
    } else if (kind != SKIP) {
#pragma unroll
      for (int k = 0; k < n; ++k) {
        f32x4 y = acc[k] * inv;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (kind == ZERO) ? 0.0f : y[i];
        Mma<T>::store4(p + (first + k * step) * 4 * sizeof(T), y[0], y[1], y[2], y[3]);
      }
    }
  }
};

// The least rounds of a part: a part's sums are written and read once more when its unit is
// joined, and should be no more than half of the keys and values they come from.
template <typename T, int RT, int ROUND>
constexpr unsigned least_part() {
  constexpr int n = RT * 4 / (ROUND * TILE * (int)sizeof(T));
  return n > 1 ? n : 1;
}

// Walks the workgroup's share, a segment at a time: begin(segment) sends for the first tiles,
// and while they come the sequence is checked and its tree laid out; run(segment, code, sink)
// then computes the rows' sums over the segment's slots and puts every row of the tile into
// sink(row, reference, sum of weights).  begin is called for every segment, also one whose rows
// are no new tokens (its tile 0 is then some page's, and not used): what it leaves in registers
// would have to be kept from segment to segment otherwise.
template <typename T, int D, int RT, int ROUND, bool WIDE, typename Begin, typename Run>
SVD void attn_share(const AttnArgs &a, const SharedBooks &s, Begin begin, Run run) {
  constexpr int ESZ = (int)sizeof(T);
  const int tid = threadIdx.x;
  // The parts' size.  Where a few rounds more than an equal share cut the units into no more
  // parts than there are workgroups, every workgroup gets one part: one that goes on with a
  // second unit begins anew there (in k_attn_wide about 6 us, 3 rounds' time: 32
  // sequences with window and sinks took 59 us with shares that run on, 50 so).  Otherwise parts are
  // single rounds and shares of them as equal as can be (units of 257 to 16001 slots, one a
  // workgroup: 392 us, so 343).
  constexpr unsigned LEAST = least_part<T, RT, ROUND>();
  const bool aligned = (unsigned)a.B * (unsigned)(a.Hkv * a.n_rt) <= a.grid && ((long long)a.W << a.page_shift) < (1 << 27);
  unsigned v = 0, ex = 0, total = 0;
  auto scan = [&](unsigned most) {  // of every sequence's parts; for the first NT (all of them, mostly) v and ex stay
    total = 0;
    for (int b0 = (a.B - 1) / NT * NT; b0 >= 0; b0 -= NT) {
      v = (b0 + tid < a.B) ? head_parts<RT, ROUND>(a, seq_of(a, b0 + tid), most) * (unsigned)a.Hkv : 0u;
      unsigned tot;
      ex = block_excl_scan(v, s.w, tot);
      total += tot;
    }
  };
  scan(1u);
  unsigned share = (total + a.grid - 1) / a.grid, most = 1;  // rounds a share, rounds a part
  if (aligned && share > 1u) {
    constexpr int TRY = 4;
    const unsigned tries = WIDE ? TRY : min(1u + share / 16, (unsigned)TRY);
    unsigned n[TRY];
#pragma unroll
    for (int k = 0; k < TRY; ++k) n[k] = 0;
    for (int b = tid; b < a.B; b += NT) {
      const Seq sq = seq_of(a, b);
#pragma unroll
      for (int k = 0; k < TRY; ++k) n[k] += head_parts<RT, ROUND>(a, sq, max(share + k, LEAST)) * (unsigned)a.Hkv;
    }
    if (tid < TRY) s.tries[tid] = 0u;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TRY; ++k) {
      const unsigned t = scan_add_u(n[k]);
      if (lane_id() == WAVE - 1) atomicAdd(&s.tries[k], t);
    }
    __syncthreads();
#pragma unroll
    for (int k = TRY - 1; k >= 0; --k)
      if (k < (int)tries && s.tries[k] <= a.grid) most = max(share + k, LEAST);
    if (most > 1u) {
      scan(most);
      share = 1;
    }
  } else if (aligned && LEAST > 1) {
    most = LEAST;
    scan(most);
  }
  // Consecutive shares on one XCD (block p runs on XCD p % LANES), as many on each: the row
  // tiles of a key head read the same keys and values through that XCD's L2.
  const unsigned shares = (total + share - 1) / share, per_xcd = (shares + LANES - 1) / LANES;
  const unsigned w = (blockIdx.x % LANES) * per_xcd + blockIdx.x / LANES;
  if (blockIdx.x / LANES >= per_xcd || w >= shares) return;
  unsigned pos = w * share;
  const unsigned pos_end = min(total, pos + share);
  if (a.B <= NT) {
    if (pos >= ex && pos < ex + v) {
      s.at[0] = (unsigned)tid;
      s.at[1] = pos - ex;
    }
  } else {
    unsigned seen = 0;
    for (int b0 = 0; seen <= pos; b0 += NT) {
      v = (b0 + tid < a.B) ? head_parts<RT, ROUND>(a, seq_of(a, b0 + tid), most) * (unsigned)a.Hkv : 0u;
      unsigned tot;
      ex = seen + block_excl_scan(v, s.w, tot);
      if (pos >= ex && pos < ex + v) {
        s.at[0] = (unsigned)(b0 + tid);
        s.at[1] = pos - ex;
      }
      seen += tot;
    }
  }
  __syncthreads();
  Segment g;
  g.b = __builtin_amdgcn_readfirstlane((int)s.at[0]);
  unsigned off = (unsigned)__builtin_amdgcn_readfirstlane((int)s.at[1]);  // parts of the sequence before pos
  g.sq = seq_of(a, g.b);
  int code = 0, code_b = -1;           // the code of sequence code_b
  int books_b = -1, books_rt = -1;     // the row tile whose books are in LDS
  while (pos < pos_end) {
    const unsigned per_head = head_parts<RT, ROUND>(a, g.sq, most);
    if (off >= per_head * (unsigned)a.Hkv) {
      off -= per_head * (unsigned)a.Hkv;
      g.sq = seq_of(a, ++g.b);
      continue;
    }
    g.h = (int)(off / per_head);
    unsigned r0 = off - (unsigned)g.h * per_head;
    g.rt = 0;
    g.sp = span_of<RT>(a, g.sq, 0);
    unsigned rounds = rounds_of<ROUND>(g.sp), parts = parts_of(rounds, most);
    while (r0 >= parts) {
      r0 -= parts;
      g.sp = span_of<RT>(a, g.sq, ++g.rt);
      rounds = rounds_of<ROUND>(g.sp);
      parts = parts_of(rounds, most);
    }
    const unsigned r1 = min(parts, r0 + (pos_end - pos));
    // parts of a unit differ by a round at most (parts <= grid and rounds < 2^22 where they are not the same)
    g.l0 = (int)((parts == rounds ? r0 : r0 * rounds / parts) * ROUND);
    g.l1 = min(g.sp.tiles, (int)((parts == rounds ? r1 : r1 * rounds / parts) * ROUND));
    g.table = (TablePtr)(a.page_table + (size_t)g.b * a.W);
    g.par = a.parent ? a.parent + (size_t)g.b * a.N : nullptr;
    g.words = (g.sq.m + 31) >> 5;
    g.masks = a.window > 0 || g.tile(g.l1 - 1) + TILE > g.sq.len;
    const bool whole = r0 == 0 && r1 == parts;

    __syncthreads();  // the previous segment is done with the LDS
    begin(g);
    if (code_b != g.b) {
      code = seq_code(a, g.sq, g.b, s);
      code_b = g.b;
    }
    if (tid == 0 && g.h == 0 && g.rt == 0 && g.l0 == 0) a.row_status[g.b] = code;
    if (tid == 0 && g.l0 == 0) {
      const unsigned last = (pos + parts - 1) / share;
      a.desc[(g.b * a.Hkv + g.h) * a.n_rt + g.rt] =
          make_uint4(w, last - w + 1, (code ? 0x80000000u : 0u) | (unsigned)(g.sq.ok ? g.sq.m : 0), 0u);
    }
    if (code == 0 && g.par && g.masks && g.sp.i0 <= g.sp.i1 && (books_b != g.b || books_rt != g.rt)) {
      tree_books(a, g, s);  // the same for every key head
      books_b = g.b;
      books_rt = g.rt;
    }

    const unsigned slot = 2 * w + (g.l0 == 0 ? 1u : 0u);
    auto sink = [&](int row, float mt, float ls) {
      RowSink<T, D> to;
      const int rg = g.rt * RT + row, i = rg / a.group, hh = rg - i * a.group;
      if (whole) {
        to.kind = i >= a.N ? to.SKIP : (code == 0 && i >= g.sq.m) ? to.ZERO : to.OUT;
        to.p = a.out + (((size_t)g.b * a.N + i) * a.Hq + g.h * a.group + hh) * D * ESZ;
        to.inv = code != 0 ? NAN : 1.0f / ls;
      } else {
        to.kind = to.PART;
        to.p = reinterpret_cast<char *>(a.part_o + ((size_t)slot * RT + row) * D);
        to.inv = 1.0f;
        a.part_ml[(size_t)slot * RT + row] = make_float2(mt, ls);  // by every lane that asks: the same
      }
      return to;
    };
    run(g, code, sink);
    pos += r1 - r0;
    off += r1 - r0;
  }
}

// A wave's rows over one tile of scores: masks, running maximum and sum, weights.
template <typename T, int D, int R>
struct Rows {
  typedef Mma<T> M;
  static constexpr int KS = D / (4 * M::E), DT = D / 16;
  f32x4 o[R][DT];
  float rm[R];          // the largest score that ref stands for
  typename M::Sum rl[R];  // sums of weights
  float ref[R], lim[R];  // see soften
  u32x4 q[R][KS];
  int node[R], dep[R];  // clamped to the segment's nodes

  SVD void clear() {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rm[r] = lim[r] = -INFINITY;
      rl[r] = typename M::Sum{};
      ref[r] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[r][d] = f32x4{0, 0, 0, 0};
    }
  }
  // Rows row0 + 16 r + m of the unit; rows that are no new token's get zeros.
  SVD void load(const AttnArgs &a, const Segment &sg, int row0, int m, int g) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = row0 + 16 * r + m, i = row / a.group, hh = row - i * a.group;
      const bool in = i < sg.sq.m;
      node[r] = min(i, sg.sp.i1);
      const char *qp = a.q + (long long)sg.b * a.q_sb + (long long)(in ? i : 0) * a.q_sn + (size_t)(sg.h * a.group + hh) * D * sizeof(T);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const u32x4 x = *reinterpret_cast<const u32x4 *>(qp + (4 * k + g) * 16);
        q[r][k] = in ? x ^ a.flip : u32x4{0, 0, 0, 0};
      }
    }
  }
  SVD void depths(const Segment &sg, const SharedBooks &s) {
#pragma unroll
    for (int r = 0; r < R; ++r) dep[r] = (sg.par && sg.masks) ? (int)s.dep[node[r] - sg.sp.i0] : node[r];
  }
  // The query rows are waited for here, not in a loop that counts what is on its way.
  SVD void arrived() {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < KS; ++k) asm volatile("" : "+v"(q[r][k]));
  }
  SVD unsigned view(const AttnArgs &a, const Segment &sg, const SharedBooks &s, int t0, int r, int g) const {
    const unsigned see = sg.sees(a, t0, dep[r], &s.anc[(node[r] - sg.sp.i0) * sg.words]);
    return ((see >> (4 * g)) & 0xfu) | (((see >> (16 + 4 * g)) & 0xfu) << 4);  // bit 4 t2 + i
  }
  SVD void mask(const AttnArgs &a, const Segment &sg, const SharedBooks &s, int t0, int g, f32x4 (&sc)[R][2]) const {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const unsigned vis = view(a, sg, s, t0, r, g);
#pragma unroll
      for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[r][t2][i] = ((vis >> (4 * t2 + i)) & 1u) ? sc[r][t2][i] : -INFINITY;
    }
  }
  // Scores to weights 2^(c2 (score - ref)).  ref follows the row's maximum loosely: it moves only
  // when a score passes it by a factor of 2^8, so that after the first tiles no sum has to be
  // rescaled and the four lanes of a row need not compare notes (weights up to 2^8 keep their
  // relative rounding, and the quotient of the sums is the same).  One test for all of a lane's
  // rows, so that what follows is one stretch of code (16 trees of 32 nodes: 2 % off a test each).
  // The difference is taken first: c2 score - c2 ref in one instruction has the rounding of c2 ref
  // in it, which for scores around 10^9 is more than 2^7, and the weights were infinite or none.
  SVD void soften(const AttnArgs &a, f32x4 (&sc)[R][2], typename M::P (&p)[R]) {
    float top[R];
    bool past = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const f32x4 x = sc[r][0], y = sc[r][1];
      top[r] = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
      past |= top[r] > lim[r];
    }
    if (__any(past)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float mx = fmaxf(rm[r], col_max(top[r]));
        const float f = (rm[r] == -INFINITY) ? 0.0f : fast_exp2((rm[r] - mx) * a.c2);
        rl[r] = rl[r] * f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[r][d] = o[r][d] * f;
        rm[r] = mx;
        ref[r] = (mx == -INFINITY) ? 0.0f : mx;
        lim[r] = mx + a.slack;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[r][t2][i] = fast_exp2((sc[r][t2][i] - ref[r]) * a.c2);
      p[r] = M::weights(sc[r]);
      rl[r] = M::add(p[r], sc[r], rl[r]);
    }
  }
  // The score that a row's sums are relative to (-inf: nothing seen so far).
  SVD float scale(int r) const { return rm[r]; }
  // What values that are not finite are to each row that sees them (they are left out of the
  // products, where a weight of zero would not keep them from the other rows): flags of the
  // values times flags of the view, both 0 or 1, count the sightings.
  SVD void odd_values(int r, int d, const u32x4 (&v)[M::VT], unsigned vis) {
    f32x4 one[2];
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
      for (int i = 0; i < 4; ++i) one[t2][i] = ((vis >> (4 * t2 + i)) & 1u) ? 1.0f : 0.0f;
    const typename M::P see = M::weights(one);
    u32x4 fn[M::VT], fp[M::VT], fm[M::VT];
#pragma unroll
    for (int t2 = 0; t2 < M::VT; ++t2) {
      fn[t2] = M::flags(v[t2], [](float x) { return !(x == x); });
      fp[t2] = M::flags(v[t2], [](float x) { return x == INFINITY; });
      fm[t2] = M::flags(v[t2], [](float x) { return x == -INFINITY; });
    }
    const f32x4 z = {0, 0, 0, 0};
    const f32x4 cn = M::pv(fn, see, z), cp = M::pv(fp, see, z), cm = M::pv(fm, see, z);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[r][d][i] += (cn[i] > 0.0f || (cp[i] > 0.0f && cm[i] > 0.0f)) ? NAN : cp[i] > 0.0f ? INFINITY : cm[i] > 0.0f ? -INFINITY : 0.0f;
  }
};

// ---------------------------------------------------------------- few rows

// Workgroups resident on a CU, which is also how many the grid has per CU.
template <typename T, int D, int R>
constexpr int attn_occ() { return (R * D * (int)sizeof(T) <= 128) ? 3 : (D * (int)sizeof(T) <= 256 ) ? 2 : (D * (int)sizeof(T) <= 512 && R == 1) ? 2 : 1; }

template <typename T, int D, int R>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(attn_occ<T, D, R>()))) void k_attn(const AttnArgs a) {
  typedef Mma<T> M;
  constexpr int RT = 16 * R, E = M::E, ESZ = (int)sizeof(T);
  constexpr int KS = D / (4 * E);  // key units a lane holds of a 16-slot score tile
  constexpr int DT = D / 16;       // 16-wide tiles of the output's d
  constexpr int PADD = D + 4;      // rows of the LDS join tile, padded against bank conflicts
  extern __shared__ unsigned s_books[];
  const SharedBooks s = books_at(s_books, RT, a.N, a.group);
  __shared__ float s_o[NW * RT * PADD];
  __shared__ float s_m[NW * RT], s_l[NW * RT];

  const int tid = threadIdx.x, lane = lane_id(), wid = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int m = lane & 15, g = lane >> 4;
  const int page = 1 << a.page_shift;
  const unsigned long long page_bytes = (unsigned long long)a.Hkv * page * D * ESZ;
  const unsigned head_bytes = (unsigned)page * D * ESZ;

  Rows<T, D, R> rows;
  u32x4 kf[2][KS], vf[DT][M::VT];
  // `last`: there is no such tile; one unit stands in for all of them, so that the loop's waits
  // can count loads instead of draining them.
  auto load_k = [&](const Segment &sg, int t0, int pa, int pb, bool last) {
    const char *kh = a.k_pages + (size_t)sg.h * head_bytes;
    const size_t step = last ? 0 : (size_t)(4 * 16) * page;
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2) {
      const int sl = 16 * t2 + m;
      const char *p = kh + (unsigned long long)(unsigned)(sl < 16 ? pa : pb) * page_bytes + ((unsigned)((t0 + sl) & (page - 1)) + (unsigned)(g * page)) * 16u;
#pragma unroll
      for (int k4 = 0; k4 < KS; ++k4) kf[t2][k4] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + k4 * step));
    }
  };
  auto load_v = [&](const Segment &sg, int t0, int pa, int pb) {
    const char *vh = a.v_pages + (size_t)sg.h * head_bytes;
#pragma unroll
    for (int t2 = 0; t2 < M::VT; ++t2) {
      const int sl = M::val_slot(t2, g);
      const char *p = vh + (unsigned long long)(unsigned)(sl < 16 ? pa : pb) * page_bytes + ((unsigned)(((t0 + sl) & (page - 1)) / E) * D + m) * 16u;
#pragma unroll
      for (int d = 0; d < DT; ++d) vf[d][t2] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + d * 256));
    }
  };
  auto cut_v = [&](const Segment &sg, int t0) {  // slots behind the sequence hold anything
    if (t0 + TILE > sg.end())
#pragma unroll
      for (int t2 = 0; t2 < M::VT; ++t2)
#pragma unroll
        for (int d = 0; d < DT; ++d) vf[d][t2] = M::cut(vf[d][t2], sg.end() - t0 - M::val_slot(t2, g));
  };
  auto begin = [&](const Segment &sg) {
    const int t0 = sg.tile(min(sg.l0 + wid, sg.l1 - 1));
    int pa, pb;
    sg.pages(a, t0, pa, pb);
    load_k(sg, t0, pa, pb, false);
    load_v(sg, t0, pa, pb);
    rows.load(a, sg, sg.rt * RT, m, g);
  };

  attn_share<T, D, RT, NW, false>(a, s, begin, [&](const Segment &sg, int code, auto sink) {
    rows.clear();
    int l = sg.l0 + wid;
    if (sg.sp.i0 <= sg.sp.i1 && code == 0 && l < sg.l1) {
      rows.depths(sg, s);
      bool odd_any = false;
      for (;;) {
        const bool last = l + NW >= sg.l1;
        const int t0 = sg.tile(l), tn = sg.tile(last ? l : l + NW);
        int pa, pb;
        sg.pages(a, tn, pa, pb);
        f32x4 sc[R][2];
        if constexpr (E == 8) {
          typename M::Dot dot[R][2] = {};
#pragma unroll
          for (int k4 = 0; k4 < KS; ++k4)
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
              for (int r = 0; r < R; ++r) M::qk(kf[t2][k4], rows.q[r][k4], dot[r][t2]);
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) sc[r][t2] = M::score(dot[r][t2]);
        } else {  // four sums a score: a score tile at a time, so that they fit the registers
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {
              typename M::Dot dot = {};
#pragma unroll
              for (int k4 = 0; k4 < KS; ++k4) M::qk(kf[t2][k4], rows.q[r][k4], dot);
              sc[r][t2] = M::score(dot);
              __builtin_amdgcn_sched_barrier(0);
            }
        }
        load_k(sg, tn, pa, pb, last);
        if (!sg.plain(a, t0)) {
          rows.mask(a, sg, s, t0, g, sc);
          cut_v(sg, t0);
          bool odd = false;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int t2 = 0; t2 < M::VT; ++t2) odd |= M::non_finite(vf[d][t2]);
          if (__any(odd)) {
            odd_any = true;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int t2 = 0; t2 < M::VT; ++t2) vf[d][t2] = M::finite(vf[d][t2]);
          }
        }
        typename M::P pw[R];
        rows.soften(a, sc, pw);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < R; ++r) rows.o[r][d] = M::pv(vf[d], pw[r], rows.o[r][d]);
        if (last) break;
        l += NW;
        load_v(sg, tn, pa, pb);
      }
      if (odd_any)
        for (l = sg.l0 + wid; l < sg.l1; l += NW) {
          const int t0 = sg.tile(l);
          if (sg.plain(a, t0)) continue;
          int pa, pb;
          sg.pages(a, t0, pa, pb);
          load_v(sg, t0, pa, pb);
          cut_v(sg, t0);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const unsigned vis = rows.view(a, sg, s, t0, r, g);
#pragma unroll
            for (int d = 0; d < DT; ++d) rows.odd_values(r, d, vf[d], vis);
          }
        }
    }

    // the four waves joined: rows' maxima and sums, then the output tiles
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float l_row = M::total(rows.rl[r]);
      if (g == 0) {
        s_m[wid * RT + 16 * r + m] = rows.scale(r);
        s_l[wid * RT + 16 * r + m] = l_row;
      }
#pragma unroll
      for (int d = 0; d < DT; ++d)
        *reinterpret_cast<f32x4 *>(&s_o[(wid * RT + 16 * r + m) * PADD + 16 * d + 4 * g]) = rows.o[r][d];
    }
    __syncthreads();
    for (int x = tid; x < RT * (D / 4); x += NT) {
      const int row = x / (D / 4), c4 = x - row * (D / 4);
      float mt = -INFINITY;
#pragma unroll
      for (int k = 0; k < NW; ++k) mt = fmaxf(mt, s_m[k * RT + row]);
      f32x4 acc = {0, 0, 0, 0};
      float ls = 0.0f;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float mk = s_m[k * RT + row], lk = s_l[k * RT + row];
        if (mk == -INFINITY && lk == 0.0f) continue;  // a wave that saw nothing
        const float f = fast_exp2((mk - mt) * a.c2);
        ls += f * lk;
        acc += *reinterpret_cast<const f32x4 *>(&s_o[(k * RT + row) * PADD + 4 * c4]) * f;
      }
      const f32x4 one[1] = {acc};
      sink(row, mt, ls).put(c4, 0, one);
    }
  });
}

// ---------------------------------------------------------------- many rows

// A tile's keys and values lie in LDS in the order in which the lanes read them, 16 lanes
// 256 bytes: keys [unit of d][slot], values [unit of slots][d].  They come there straight from
// memory, without registers in between, a stage of ST tiles at a time: while the waves work on
// one stage the next is on its way, and one barrier hands a stage over and frees the other.
// (16 trees of 32 nodes: 92 us; with the next tile alone in flight, in registers, 110.)  The
// two stages are variables of their own, so that the compiler sees that reads of one do not
// wait for the other; four of one tile each, one more in flight, made the code twice as long,
// and a workgroup spends its first microseconds fetching code.
typedef __attribute__((address_space(3))) void *LdsPtr;
typedef const __attribute__((address_space(1))) void *GlobalPtr;

template <typename T, int D, int R>
constexpr int wide_occ() { return (R * D * (int)sizeof(T) <= 512) ? 2 : 1; }
// Tiles of a stage: as many as let two workgroups' stages fit a CU's LDS (two f32 heads of 256
// fill it alone).
template <typename T, int D>
constexpr int wide_stage() { return D * (int)sizeof(T) <= 256 ? 2 : 1; }

// Waits until none of the wave's memory operations is on its way, then for the other waves; no
// memory access moves across.
SVD void hand_over() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x70);  // vmcnt 0, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <typename T, int D, int R>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(wide_occ<T, D, R>()))) void k_attn_wide(const AttnArgs a) {
  typedef Mma<T> M;
  constexpr int RT = 16 * R * NW, E = M::E, ESZ = (int)sizeof(T);
  constexpr int KS = D / (4 * E), DT = D / 16;
  constexpr int UNITS = TILE * D / E;                 // 16-byte units of a tile's keys, and of its values
  constexpr int PW = UNITS / NT;                      // of each, 64-unit pieces that a wave fetches
  constexpr int ST = wide_stage<T, D>();
  extern __shared__ unsigned s_books[];
  const SharedBooks s = books_at(s_books, RT, a.N, a.group);
  __shared__ u32x4 s_a[ST][2 * UNITS], s_b[ST][2 * UNITS];
  __shared__ int s_odd;

  const int tid = threadIdx.x, lane = lane_id(), wid = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int m = lane & 15, g = lane >> 4;
  const int page = 1 << a.page_shift;
  const unsigned long long page_bytes = (unsigned long long)a.Hkv * page * D * ESZ;
  const unsigned head_bytes = (unsigned)page * D * ESZ;

  Rows<T, D, R> rows;
  auto fetch = [&](const Segment &sg, int l, u32x4 *buf) {
    const char *kh = a.k_pages + (size_t)sg.h * head_bytes, *vh = a.v_pages + (size_t)sg.h * head_bytes;
    const int t0 = sg.tile(l);
    int pa, pb;
    sg.pages(a, t0, pa, pb);
    const int sl = lane % TILE;
    const char *kp = kh + (unsigned long long)(unsigned)(sl < 16 ? pa : pb) * page_bytes +
                     (size_t)((2 * wid + lane / TILE) * page + ((t0 + sl) & (page - 1))) * 16;
#pragma unroll
    for (int j = 0; j < PW; ++j)
      __builtin_amdgcn_global_load_lds((GlobalPtr)(kp + (size_t)j * (2 * NW * 16) * page), (LdsPtr)(buf + (j * NW + wid) * WAVE), 16, 0, 2);
#pragma unroll
    for (int j = 0; j < PW; ++j) {
      const int x = (j * NW + wid) * WAVE, vs = x / D * E;  // D units a value unit's slots: a piece lies in one of them
      const char *vp = vh + (unsigned long long)(unsigned)(vs < 16 ? pa : pb) * page_bytes +
                       (size_t)(((t0 + vs) & (page - 1)) / E * D + x % D + lane) * 16;
      __builtin_amdgcn_global_load_lds((GlobalPtr)vp, (LdsPtr)(buf + UNITS + x), 16, 0, 2);
    }
  };
  auto fetch_stage = [&](const Segment &sg, int l, u32x4 (&st)[ST][2 * UNITS]) {
#pragma unroll 1
    for (int k = 0; k < ST; ++k)
      if (l + k < sg.l1) fetch(sg, l + k, st[k]);
  };
  auto begin = [&](const Segment &sg) {
    rows.load(a, sg, sg.rt * RT + wid * 16 * R, m, g);
    if (tid == 0) s_odd = 0;
    fetch_stage(sg, sg.l0, s_a);
  };

  attn_share<T, D, RT, ST, true>(a, s, begin, [&](const Segment &sg, int code, auto sink) {
    rows.clear();
    if (sg.sp.i0 > sg.sp.i1 || code != 0) {
      hand_over();  // what begin sent for has come before the buffers are used again
    } else {
      rows.depths(sg, s);
      rows.arrived();
      // Slots behind the sequence hold anything, and values that are not finite are left out of
      // the products where not every row sees them.
      auto clean = [&](int t0, u32x4 *vb) {
        bool odd = false;
#pragma unroll
        for (int j = 0; j < PW; ++j) {
          u32x4 v = M::cut(vb[tid + j * NT], sg.end() - t0 - (tid + j * NT) / D * E);
          odd |= M::non_finite(v);
          vb[tid + j * NT] = M::finite(v);
        }
        if (odd) s_odd = 1;
        __syncthreads();
      };
      auto work = [&](int l, u32x4 *buf) {
        const int t0 = sg.tile(l);
        const bool plain = sg.plain(a, t0);
        if (!plain) clean(t0, buf + UNITS);
        typename M::Dot dot[R][2] = {};
#pragma unroll
        for (int k4 = 0; k4 < KS; ++k4)
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) {
            const u32x4 k = buf[(4 * k4 + g) * TILE + 16 * t2 + m];
#pragma unroll
            for (int r = 0; r < R; ++r) M::qk(k, rows.q[r][k4], dot[r][t2]);
          }
        f32x4 sc[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) sc[r][t2] = M::score(dot[r][t2]);
        if (!plain) rows.mask(a, sg, s, t0, g, sc);
        typename M::P pw[R];
        rows.soften(a, sc, pw);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          u32x4 v[M::VT];
#pragma unroll
          for (int t2 = 0; t2 < M::VT; ++t2) v[t2] = buf[UNITS + M::val_slot(t2, g) / E * D + 16 * d + m];
#pragma unroll
          for (int r = 0; r < R; ++r) rows.o[r][d] = M::pv(v, pw[r], rows.o[r][d]);
        }
      };
      auto stage = [&](int l, u32x4 (&now)[ST][2 * UNITS], u32x4 (&next)[ST][2 * UNITS]) {
        hand_over();
        fetch_stage(sg, l + ST, next);
#pragma unroll 1
        for (int k = 0; k < ST; ++k)
          if (l + k < sg.l1) work(l + k, now[k]);
      };

      for (int l = sg.l0; l < sg.l1; l += 2 * ST) {
        stage(l, s_a, s_b);
        if (l + ST < sg.l1) stage(l + ST, s_b, s_a);
      }
      __syncthreads();
      if (s_odd)
        for (int l = sg.l0; l < sg.l1; ++l) {
          const int t0 = sg.tile(l);
          if (sg.plain(a, t0)) continue;
          fetch(sg, l, s_a[0]);
          hand_over();
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const unsigned vis = rows.view(a, sg, s, t0, r, g);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              u32x4 v[M::VT];
#pragma unroll
              for (int t2 = 0; t2 < M::VT; ++t2)
                v[t2] = M::cut(s_a[0][UNITS + M::val_slot(t2, g) / E * D + 16 * d + m], sg.end() - t0 - M::val_slot(t2, g));
              rows.odd_values(r, d, v, vis);
            }
          }
          __syncthreads();
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sink(wid * 16 * R + 16 * r + m, rows.scale(r), M::total(rows.rl[r])).put(g, 4, rows.o[r]);
    }
  });
}

// Units that several workgroups streamed: one wave a row, its partial tiles in the order of
// the slots.
template <typename T, int D, int RT>
__global__ __launch_bounds__(NT) void k_attn_join(const AttnArgs a) {
  typedef Mma<T> M;
  constexpr int ESZ = (int)sizeof(T), PL = D / 4;  // lanes that hold a row
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
    const bool none = ml.x == -INFINITY && ml.y == 0.0f;  // it saw nothing of the row
    const float f = fast_exp2((ml.x - mt) * a.c2);
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

template <int N>
struct Int {
  static constexpr int value = N;
};

using sv_host::align256;

struct AttnPlan {
  bool wide;
  int R, RT, n_rt;
  unsigned grid;
  long long units;
  size_t part_o, part_ml, desc, total;
};

bool pow2_page(int32_t page) { return page >= 16 && page <= 256 && (page & (page - 1)) == 0; }

template <typename T, int D, int R>
void attn_go(sv_host::Launcher &L, AttnArgs &a, const AttnPlan &p) {
  void *args[] = {&a};
  L.lds = books_bytes(p.RT, a.N, a.group, a.parent != nullptr);
  if (p.wide) {
    L.go((const void *)&k_attn_wide<T, D, R>, p.grid, args);
    L.lds = 0;
    L.go((const void *)&k_attn_join<T, D, 16 * R * NW>, (unsigned)(p.units * (p.RT / NW)), args);
  } else if constexpr (D <= 128 || R == 1) {
    L.go((const void *)&k_attn<T, D, R>, p.grid, args);
    L.lds = 0;
    L.go((const void *)&k_attn_join<T, D, 16 * R>, (unsigned)(p.units * (p.RT / NW)), args);
  }
}

// The kernel for a head size and type: f is called with the constants.
template <typename F>
auto attn_pick(int esz, int D, int R, F f) {
  typedef uint16_t h;
  if (esz == 2) {
    if (D == 64) return R == 1 ? f(h{}, Int<64>{}, Int<1>{}) : f(h{}, Int<64>{}, Int<2>{});
    if (D == 128) return R == 1 ? f(h{}, Int<128>{}, Int<1>{}) : f(h{}, Int<128>{}, Int<2>{});
    return R == 1 ? f(h{}, Int<256>{}, Int<1>{}) : f(h{}, Int<256>{}, Int<2>{});
  }
  if (D == 64) return R == 1 ? f(0.0f, Int<64>{}, Int<1>{}) : f(0.0f, Int<64>{}, Int<2>{});
  if (D == 128) return R == 1 ? f(0.0f, Int<128>{}, Int<1>{}) : f(0.0f, Int<128>{}, Int<2>{});
  return f(0.0f, Int<256>{}, Int<1>{});
}

bool attn_shape_ok(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page, int32_t W) {
  return B >= 1 && N >= 1 && N <= SV_CACHE_MAX_NEW && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 &&
         (D == 64 || D == 128 || D == 256) && pow2_page(page) && W >= 1 && (long long)W * page <= 0x7fffffffLL - 4096;
}

// Up to 16 rows of a key head, or 32 up to D = 128: one wave holds them in its registers; more go to
// the kernel whose waves share them, with one row tile a wave up to 64 rows, else two.  Calls in us,
// 16 sequences of 1000 to 4000 slots and 8 key heads, the rule's choice first:
//   20 rows, k_attn with two row tiles against k_attn_wide with one: bf16 D = 64 27 / 32, D = 128
//   46 / 45 (64 sequences 141 / 143); f32 D = 64 49 / 72, D = 128 91 / 122
//   128 rows, two row tiles a wave against one: bf16 D = 64 48 / 55, D = 128 65 / 82, D = 256
//   141 / 145; f32 D = 64 131 / 125 (256 rows 226 / 246), D = 128 237 / 224 (256 rows 463 / 434)
// The rule looks at rows alone.  One row tile a wave would be faster for f32 at D = 128 (two need
// 101 registers more than there are) and where little is to be read (2 sequences of up to 1000
// slots, 128 rows: bf16 D = 128 24 / 20, D = 256 40 / 30).
bool attn_plan(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page, int32_t W, int esz, AttnPlan &p) {
  const long long rows = (long long)N * (Hq / Hkv);
  const bool two = D <= 128;  // the registers take two row tiles of k_attn
  p.wide = rows > (two ? 32 : 16);
  p.R = p.wide ? (rows <= 64 || D * esz == 1024 ? 1 : 2) : (rows <= 16 ? 1 : 2);
  p.RT = 16 * p.R * (p.wide ? NW : 1);
  const long long n_rt = (rows + p.RT - 1) / p.RT;
  const long long most = ((long long)W * page + TILE - 1) / TILE + 1;  // tiles of a unit
  const long long heads = (long long)B * Hkv, limit = 0x7fffffffLL;
  if (heads > limit || n_rt > limit / heads) return false;
  p.units = heads * n_rt;
  // the join has a wave a row, and a launch fewer than 2^32 threads
  if (most > limit / p.units || p.RT > 0xffffffffLL / WAVE / p.units) return false;
  p.n_rt = (int)n_rt;
  const int occ = attn_pick(esz, D, p.R, [&](auto t, auto d, auto r) {
    typedef decltype(t) T;
    return p.wide ? wide_occ<T, decltype(d)::value, decltype(r)::value>() : attn_occ<T, decltype(d)::value, decltype(r)::value>();
  });
  // One resident set of the device's 256 CUs (trees of near 1024 nodes: their books leave room for
  // one workgroup a CU of k_attn_wide, and the set comes in two turns; none waits for another).
  long long grid = 256LL * occ;
  const long long round = p.wide ? (D * esz <= 256 ? 2 : 1) : NW;  // tiles of a round, the least share
  const long long need = p.units * ((most + round - 1) / round);
  if (need < grid) grid = need;
  p.grid = (unsigned)((grid + LANES - 1) / LANES * LANES);
  size_t o = 0;
  p.part_o = o; o = align256(o + (size_t)2 * p.grid * p.RT * D * 4);
  p.part_ml = o; o = align256(o + (size_t)2 * p.grid * p.RT * 8);
  p.desc = o; o = align256(o + (size_t)p.units * 16);
  p.total = o;
  return true;
}

sv_status attn_run(const void *q, int64_t q_sb, int64_t q_sn, const void *k_pages, const void *v_pages, sv_dtype dt,
                   const int32_t *table, const int32_t *cache_len, const int32_t *n_new, const int32_t *parent,
                   const int32_t *prior, int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page, int32_t P,
                   int32_t W, float scale, int32_t window, int32_t sinks, void *out, int32_t *status, void *ws,
                   size_t ws_bytes, void *stream, void *const *ev, int32_t nev, int32_t *nl) {
  if (nl) *nl = 0;
  if (dt != SV_F32 && dt != SV_BF16) return SV_ERR_DTYPE;
  const int esz = dt == SV_BF16 ? 2 : 4;
  if (!attn_shape_ok(B, N, Hq, Hkv, D, page, W) || P < 1) return SV_ERR_SHAPE;
  if (!isfinite(scale) || window < 0 || sinks < 0 || (sinks > 0 && window == 0)) return SV_ERR_PARAM;
  AttnPlan p;
  if (!attn_plan(B, N, Hq, Hkv, D, page, W, esz, p)) return SV_ERR_SHAPE;
  if (!q || !k_pages || !v_pages || !table || !cache_len || !out || !status || !ws) return SV_ERR_NULL;
  if (((uintptr_t)q | (uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)out | ((uintptr_t)q_sb * esz) | ((uintptr_t)q_sn * esz)) & 15)
    return SV_ERR_ALIGN;
  if (ws_bytes < p.total || ((uintptr_t)ws & 255)) return SV_ERR_WORKSPACE;
  // several workgroups read prior, and one writes the status
  if (prior && (uintptr_t)prior < (uintptr_t)(status + B) && (uintptr_t)status < (uintptr_t)(prior + B)) return SV_ERR_PARAM;
  char *base = static_cast<char *>(ws);
  AttnArgs a = {};
  a.q = static_cast<const char *>(q);
  a.k_pages = static_cast<const char *>(k_pages);
  a.v_pages = static_cast<const char *>(v_pages);
  a.q_sb = (long long)((unsigned long long)q_sb * esz);
  a.q_sn = (long long)((unsigned long long)q_sn * esz);
  a.page_table = table;
  a.cache_len = cache_len;
  a.n_new = n_new;
  a.parent = parent;
  a.prior = prior;
  a.B = B;
  a.N = N;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.page_shift = __builtin_ctz((unsigned)page);
  a.P = P;
  a.W = W;
  // A scale of zero becomes one too small for any finite score to matter (2^-149 times 2^128), so
  // that 0 times -inf need not be met; the largest one stays finite for the same reason.
  a.c2 = (float)fmin(fmax(fabs((double)scale) * LOG2E, (double)__FLT_DENORM_MIN__), (double)__FLT_MAX__);
  a.flip = scale < 0.0f ? (esz == 2 ? 0x80008000u : 0x80000000u) : 0u;
  a.slack = fminf(8.0f / a.c2, 1e30f);
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
  attn_pick(esz, D, p.R, [&](auto t, auto d, auto r) {
    attn_go<decltype(t), decltype(d)::value, decltype(r)::value>(L, a, p);
    return 0;
  });
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
  return attn_run(q, q_stride_b, q_stride_n, k_pages, v_pages, dtype, page_table, cache_len, n_new, parent, nullptr, B, N, Hq, Hkv, D,
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
  return attn_run(q, q_stride_b, q_stride_n, k_pages, v_pages, dtype, page_table, cache_len, n_new, parent, nullptr, B, N, Hq, Hkv, D,
                  page_size, num_pages, table_width, scale, window, sinks, out, row_status, workspace, workspace_bytes,
                  stream, events, n_events, n_launched);
}

sv_status spec_paged_attention_after(const void *q, int64_t q_stride_b, int64_t q_stride_n, const void *k_pages,
                                     const void *v_pages, sv_dtype dtype, const int32_t *page_table,
                                     const int32_t *cache_len, const int32_t *n_new, const int32_t *parent,
                                     const int32_t *prior, int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                     int32_t page_size, int32_t num_pages, int32_t table_width, float scale, int32_t window,
                                     int32_t sinks, void *out, int32_t *row_status, void *workspace,
                                     size_t workspace_bytes, void *stream, void *const *events, int32_t n_events,
                                     int32_t *n_launched) {
  return attn_run(q, q_stride_b, q_stride_n, k_pages, v_pages, dtype, page_table, cache_len, n_new, parent, prior, B, N, Hq, Hkv, D,
                  page_size, num_pages, table_width, scale, window, sinks, out, row_status, workspace, workspace_bytes,
                  stream, events, n_events, n_launched);
}

const char *sv_attention_launch_plan(int32_t N, int32_t Hq, int32_t Hkv, int32_t D, sv_dtype dtype) {
  AttnPlan p;
  if ((dtype != SV_F32 && dtype != SV_BF16) || !attn_shape_ok(1, N, Hq, Hkv, D, 16, 1) ||
      !attn_plan(1, N, Hq, Hkv, D, 16, 1, dtype == SV_BF16 ? 2 : 4, p))
    return "";
  return p.wide ? "k_attn_wide;k_attn_join" : "k_attn;k_attn_join";
}

}  // extern "C"
