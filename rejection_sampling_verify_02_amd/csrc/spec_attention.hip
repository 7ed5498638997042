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

#include "sv_attention.h"

namespace sv {

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

}  // namespace sv

// ======================================================================== host side

namespace {

using namespace sv;

using namespace sv_host;

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
  const int occ = attn_pick(esz, D, p.R, [&](auto t, auto d, auto r) {
    typedef decltype(t) T;
    return p.wide ? wide_occ<T, decltype(d)::value, decltype(r)::value>() : attn_occ<T, decltype(d)::value, decltype(r)::value>();
  });
  return attn_cut(B, rows, Hkv, D, page, W, occ, p.wide ? (D * esz <= 256 ? 2 : 1) : NW, p);
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
  AttnArgs a = {};
  a.k_pages = static_cast<const char *>(k_pages);
  a.v_pages = static_cast<const char *>(v_pages);
  attn_fill(a, p, q, q_sb, q_sn, esz, table, cache_len, n_new, parent, prior, B, N, Hq, Hkv, page, P, W, scale, window, sinks, out,
            status, ws);
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
