// spec_attention4.hip -- attention of a round's new tokens over a paged cache in 4 bits
// (include/spec_cache.h): the method, the work's cut and the rows' softmax of spec_attention.hip,
// with keys and values that come as codes and become bf16 operands on their way to the matrix
// cores (v_cvt_scalef32_pk_bf16_fp4, two codes an instruction, the block's power of two included).
// What a code stands for is a bf16 number, so nothing is rounded there.
//
//   k_attn4       up to 32 rows.  A lane's 16 bytes of keys are a whole block of one slot, 32
//                 elements: step k of the first product contracts over elements 8 k .. 8 k + 7 of
//                 four blocks, and the queries are laid out to match.  A lane's codes of values
//                 are D / 16 neighbours d of eight slots, all of one block: a conversion gives two
//                 neighbours of one slot, and a byte permutation makes pairs of slots of them, the
//                 second product's operand.  Row tile j of the output then holds d = D / 16 m + j,
//                 m the row of the matrix instruction.  Each wave has its tiles sent to LDS, where
//                 they wait without registers.  Bound by the cache's bytes: 64 sequences of 257 to
//                 16001 slots, 8 key heads of 128: 104 us, 5.4 TB/s; its loads alone take 98.  (With
//                 the codes in registers, one tile ahead, and shares of equal length: 135.)  The
//                 keys could go into the scaled matrix instruction as they are, the queries as two
//                 8-bit parts; but that one's sums are only good to 2^-12 of their terms.  With 17
//                 to 32 rows, 64 chains of 5 over the same slots, 158 us, twice its bytes' time:
//                 256 registers, and 13 more in scratch memory.
//   k_attn4_wide  more rows.  The waves share each tile through LDS as bf16, converted once by one
//                 of them.  16 trees of 32 nodes, 4 heads a key head: 94 us; the products alone
//                 would be 37.  The rest is what a wave does between them, weights and conversions,
//                 with one other wave on its SIMD to fill in: all its registers are taken.  (Two
//                 tiles at a time, one's weights beside the other's products, spills in the loop:
//                 166 to 193 us a call for 100.)

#include "sv_attention.h"

#include <type_traits>

#include "sv_fp4.h"

namespace sv {

struct Attn4Args : AttnArgs {
  const char *k_scales, *v_scales;
};

// Step k of lane group g takes unit (8 elements) k of the group's own block: half blocks at
// D = 64, and blocks g, then g + 4, at D = 256.
template <int D>
struct UnitsWithin {
  static constexpr int KH = D / 32 < 4 ? D / 32 : 4;
  SVD static int at(int k, int g) { return k / KH * (4 * KH) + KH * g + k % KH; }
};

// Waits until at most N of the wave's memory operations are on their way.
template <int N>
SVD void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0xf70);
  asm volatile("" ::: "memory");
}

// A tile's codes and scales on their way from memory to LDS, with no registers in between: a wave's
// loads put 16 bytes (scales: 4) of lane after lane one behind the other.  Written as assembly
// because the compiler, where it sees them, has every read of LDS wait for all of them; their
// order and wait_loads see to that here.  They return nothing in registers.
// In LDS: keys, a load being what 64 lanes multiply in a step; values, in the pool's order; then
// scales [block][slot], of keys and of values.
template <int D>
struct Fetch {
  static constexpr int KL = D / 64, SL = D <= 128 ? 1 : 2, LOADS = 2 * KL + SL;  // of keys (of values as many), of scales
  static constexpr int VALUES = KL * 1024, SCALES = 2 * KL * 1024, VSCALES = SCALES + D, BYTES = SCALES + SL * 256;
  const char *kh, *vh;   // the head in page 0
  const char *sh[SL];    // of the lane's scales: its pool, block and slot of a half tile

  // 16 bytes a lane, from a place that all lanes know and one of its own
  SVD static void line(const char *at, unsigned own, unsigned lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(own), "s"(at), "{m0}"(lds) : "memory");
  }
  SVD static void line(const char *own, unsigned lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(own), "{m0}"(lds) : "memory");
  }
  SVD static void word(const char *own, unsigned lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(own), "{m0}"(lds) : "memory");
  }

  SVD void head(const Attn4Args &a, int h, int lane) {
    const unsigned page = 1u << a.page_shift, codes = page * D / 2, scales = page * D / F4_BLOCK;
    kh = a.k_pages + (size_t)h * codes;
    vh = a.v_pages + (size_t)h * codes;
#pragma unroll
    for (int j = 0; j < SL; ++j) {
      const int x = (SL == 2 ? j * 64 + lane : lane) % (D / 2);  // D / 4 words of keys' scales, as many of values'; at D = 64 all of it twice
      const char *pool = x < D / 4 ? a.k_scales : a.v_scales;
      sh[j] = pool + (size_t)h * scales + (x % (D / 4) / 8 * page + x % 4 * 4);
    }
  }
  // The tile at slot t0, its halves in pages pa and pb, to `lds`.
  SVD void send(const Attn4Args &a, int t0, int pa, int pb, unsigned lds, int lane) const {
    const unsigned page = 1u << a.page_shift;
    const unsigned long long page_codes = (unsigned long long)a.Hkv * (page * D / 2), page_scales = (unsigned long long)a.Hkv * (page * D / F4_BLOCK);
    const unsigned ta = (unsigned)t0 & (page - 1), tb = (unsigned)(t0 + 16) & (page - 1);
    const unsigned long long ca = (unsigned)pa * page_codes, cb = (unsigned)pb * page_codes;
    if constexpr (D == 64) {
      const bool kb = lane & 16, vb = lane & 32;
      line(kh + (kb ? cb : ca) + ((unsigned)(lane / 32) * page + (kb ? tb : ta) + (unsigned)(lane & 15)) * 16u, lds);
      line(vh + (vb ? cb : ca) + ((vb ? tb : ta) / 8 * 16 + (unsigned)(lane & 31)) * 16u, lds + VALUES);
    } else {
      const unsigned own = (unsigned)(lane / 16 * page + lane % 16) * 16u;
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int t2 = i / (KL / 2), b = i % (KL / 2);
        line(kh + (t2 ? cb : ca) + (4 * b * page + (t2 ? tb : ta)) * 16u, own, lds + i * 1024);
      }
      constexpr int S = 512 / D, PER = 4 * S;  // slots of a unit, and of a load
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const bool hb = i * PER >= 16;
        line(vh + (hb ? cb : ca) + ((hb ? tb : ta) + i * PER % 16) / S * 256u, (unsigned)lane * 16u, lds + VALUES + i * 1024);
      }
    }
    const unsigned long long sa = (unsigned)pa * page_scales + ta, sb = (unsigned)pb * page_scales + tb;
#pragma unroll
    for (int j = 0; j < SL; ++j) word(sh[j] + (lane & 4 ? sb : sa), lds + SCALES + j * 256);
  }
};

// A lane's codes of a 32-slot tile, and their scales: of keys slots 16 t2 + m, of values slots
// 8 g .. 8 g + 7.
template <int D>
struct Codes {
  static constexpr int KS = D / 32, KB = D <= 128 ? 1 : 2;  // steps; blocks of a key that a lane holds (half of one at D = 64)
  static constexpr int S = 512 / D, VU = 8 / S, DPL = D / 16, B = D / 32;  // slots and units of values, elements and bytes a slot
  unsigned k[2][KS], ks[2][KB];
  u32x4 v[VU];
  u32x2 vs;

  // pa, pb: the pages of the tile's halves; `kh`, `ksh`: the head in page 0.
  SVD void load_k(const char *kh, const char *ksh, unsigned long long page_codes, unsigned long long page_scales, int page, int t0, int pa,
                  int pb, int m, int g) {
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2) {
      const unsigned p = (unsigned)(t2 == 0 ? pa : pb), t = (unsigned)((t0 + 16 * t2 + m) & (page - 1));
      const char *c = kh + p * page_codes, *sc = ksh + p * page_scales;
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const unsigned u = D == 64 ? (unsigned)g / 2 : (unsigned)(g + 4 * b), at = u * (unsigned)page + t;
        ks[t2][b] = __builtin_nontemporal_load(reinterpret_cast<const unsigned char *>(sc + at));
        if constexpr (D == 64) {
          const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(c + at * 16u + (g & 1) * 8));
          k[t2][0] = w.x;
          k[t2][1] = w.y;
        } else {
          const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(c + at * 16u));
#pragma unroll
          for (int j = 0; j < 4; ++j) k[t2][4 * b + j] = w[j];
        }
      }
    }
  }
  SVD void load_v(const char *vh, const char *vsh, unsigned long long page_codes, unsigned long long page_scales, int page, int t0, int pa,
                  int pb, int m, int g) {
    const unsigned p = (unsigned)(g < 2 ? pa : pb), t = (unsigned)((t0 + 8 * g) & (page - 1));
    const char *c = vh + p * page_codes + (t / S * 16 + m) * 16u;
#pragma unroll
    for (int u = 0; u < VU; ++u) v[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(c + u * 256));
    vs = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(vsh + p * page_scales + (unsigned)(m * DPL / F4_BLOCK * page) + t));
  }
  // The same, of a tile that Fetch put into LDS.
  SVD void read_k(const char *t, int m, int g) {
    typedef Fetch<D> F;
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const int u = D == 64 ? g / 2 : g + 4 * b;
        ks[t2][b] = *reinterpret_cast<const unsigned char *>(t + F::SCALES + u * 32 + 16 * t2 + m);
        if constexpr (D == 64) {
          const u32x2 w = *reinterpret_cast<const u32x2 *>(t + (u * 32 + 16 * t2 + m) * 16 + (g & 1) * 8);
          k[t2][0] = w.x;
          k[t2][1] = w.y;
        } else {
          const u32x4 w = *reinterpret_cast<const u32x4 *>(t + ((t2 * KB + b) * 64 + 16 * g + m) * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) k[t2][4 * b + j] = w[j];
        }
      }
  }
  SVD void read_v(const char *t, int m, int g) {
    typedef Fetch<D> F;
#pragma unroll
    for (int u = 0; u < VU; ++u) v[u] = *reinterpret_cast<const u32x4 *>(t + F::VALUES + ((g * VU + u) * 16 + m) * 16);
    vs = *reinterpret_cast<const u32x2 *>(t + F::VSCALES + m * DPL / F4_BLOCK * 32 + 8 * g);
  }
  // Step k4's operand of score tile t2.
  SVD u32x4 key(int t2, int k4) const { return f4_unit(k[t2][k4], f4_factor(ks[t2][D == 64 ? 0 : k4 / 4])); }
  SVD void factors(float (&f)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = f4_factor(vs[e / 4], e % 4);
  }
  // Elements 2 i and 2 i + 1 of the lane's D / 16, of its eight slots: the operands of output
  // tiles 2 i and 2 i + 1.
  SVD void values(int i, const float (&f)[8], u32x4 &lo, u32x4 &hi) const {
    unsigned w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = e % S * B + i;  // byte in the unit
      const unsigned x = v[e / S][at / 4];
      w[e] = at % 4 == 0 ? f4_pair<0>(x, f[e]) : at % 4 == 1 ? f4_pair<1>(x, f[e]) : at % 4 == 2 ? f4_pair<2>(x, f[e]) : f4_pair<3>(x, f[e]);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      lo[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x05040100u);
      hi[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x07060302u);
    }
  }
  // Whether a block among the first n of the lane's eight slots is not finite.
  SVD bool odd(int n) const {
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) bad |= e < n && ((vs[e / 4] >> (8 * (e % 4))) & 255u) == F4_NAN;
    return bad;
  }
};

// A lane's part of a row, output tiles o[j][i] with d = D / 16 (4 g + i) + j, as pieces of four
// neighbours, the first at d = D / 16 * 4 g.
template <int D>
SVD void row_pieces(const f32x4 (&o)[D / 16], f32x4 (&out)[D / 16]) {
  constexpr int Q = D / 64;  // pieces of the D / 16 elements of an i
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < Q; ++q) out[i * Q + q] = f32x4{o[4 * q][i], o[4 * q + 1][i], o[4 * q + 2][i], o[4 * q + 3][i]};
}

// The least rounds of a part (least_part, with 17/32 of a byte an element).
template <int RT, int ROUND>
constexpr unsigned least_part4() {
  constexpr int n = RT * 4 * 32 / (ROUND * TILE * 17);
  return n > 1 ? n : 1;
}

// Workgroups of a CU, and tiles of LDS that a wave has: 70 KB of a CU on their way at D = 64 and
// 128, where more is slower (D = 128, the 64 sequences below: 105 us so, 108 with three tiles, 111
// with three workgroups as well).
template <int D, int R>
constexpr int attn4_occ() { return D > 64 ? 2 : R == 1 ? 4 : 3; }
template <int D>
constexpr int attn4_stages() { return D == 64 ? 3 : 2; }
// What the start of a unit costs a workgroup, in rounds: it waits for the unit's page ids, then its
// first tiles, and joins at the end.  Without it the workgroup with ten short sequences was the
// last one by 25 of 130 us.
constexpr unsigned ATTN4_LEAD = 5;

template <int D, int R>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(attn4_occ<D, R>()))) void k_attn4(const Attn4Args a) {
  typedef uint16_t T;
  typedef Mma<T> M;
  constexpr int RT = 16 * R, KS = D / 32, DT = D / 16, Q = D / 64;
  constexpr int PADD = D + 4;  // rows of the LDS join tile, padded against bank conflicts
  constexpr int ST = attn4_stages<D>();
  typedef Fetch<D> F;
  extern __shared__ unsigned s_books[];
  const SharedBooks s = books_at(s_books, RT, a.N, a.group);
  constexpr int RING = NW * ST * F::BYTES, JOIN = NW * RT * PADD * 4;
  __shared__ __attribute__((aligned(16))) char s_buf[RING > JOIN ? RING : JOIN];  // tiles on their way, and the join behind them
  float *const s_o = reinterpret_cast<float *>(s_buf);
  __shared__ float s_m[NW * RT], s_l[NW * RT];

  const int tid = threadIdx.x, lane = lane_id(), wid = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int m = lane & 15, g = lane >> 4;
  const char *const ring = s_buf + wid * (ST * F::BYTES);
  const unsigned ring_at = (unsigned)(uintptr_t)(__attribute__((address_space(3))) const char *)ring;

  Rows<T, D, R, UnitsWithin<D>> rows;
  F fetch;
  auto send = [&](const Segment &sg, int l, int slot) {
    const int t0 = sg.tile(l);
    int pa, pb;
    sg.pages(a, t0, pa, pb);
    pa = __builtin_amdgcn_readfirstlane(pa);
    pb = __builtin_amdgcn_readfirstlane(pb);
    fetch.send(a, t0, pa, pb, ring_at + slot * F::BYTES, lane);
  };
  auto begin = [&](const Segment &sg) {
    rows.load(a, sg, sg.rt * RT, m, g);
    fetch.head(a, __builtin_amdgcn_readfirstlane(sg.h), lane);
#pragma unroll
    for (int k = 0; k < ST; ++k)
      if (sg.l0 + wid + k * NW < sg.l1) send(sg, sg.l0 + wid + k * NW, k);
  };

  attn_share<T, D, RT, NW, false, least_part4<RT, NW>(), ATTN4_LEAD>(a, s, begin, [&](const Segment &sg, int code, auto sink) {
    rows.clear();
    int l = sg.l0 + wid;
    if (sg.sp.i0 <= sg.sp.i1 && code == 0 && l < sg.l1) {
      rows.depths(sg, s);
      bool odd_any = false;
      int slot = 0;
      auto work = [&](auto plain) {  // whether every row sees the whole tile: the rest of the code is kept apart from theirs
        const int t0 = sg.tile(l);
        const char *tile = ring + slot * F::BYTES;
        // what may still be on its way: the tiles behind this one
        if (l + (ST - 1) * NW < sg.l1) wait_loads<(ST - 1) * F::LOADS>();
        else if (ST > 2 && l + NW < sg.l1) wait_loads<F::LOADS>();
        else wait_loads<0>();
        Codes<D> c;
        c.read_k(tile, m, g);
        f32x4 sc[R][2];
        {
          typename M::Dot dot[R][2] = {};
#pragma unroll
          for (int k4 = 0; k4 < KS; ++k4)
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {
              const u32x4 k = c.key(t2, k4);
#pragma unroll
              for (int r = 0; r < R; ++r) M::qk(k, rows.q[r][k4], dot[r][t2]);
            }
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) sc[r][t2] = M::score(dot[r][t2]);
        }
        c.read_v(tile, m, g);
        const int n = sg.end() - t0 - 8 * g;  // slots behind the sequence hold anything
        bool odd = false;
        if constexpr (!plain) {
          rows.mask(a, sg, s, t0, g, sc);
          odd = __any(c.odd(n));
          odd_any |= odd;
        }
        typename M::P pw[R];
        rows.soften(a, sc, pw);
        float f[8];
        c.factors(f);
#pragma unroll
        for (int i = 0; i < DT / 2; ++i) {
          u32x4 v[2];
          c.values(i, f, v[0], v[1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if constexpr (!plain) {
              v[j] = M::cut(v[j], n);
              if (odd) v[j] = M::finite(v[j]);
            }
            const u32x4 one[1] = {v[j]};
#pragma unroll
            for (int r = 0; r < R; ++r) rows.o[r][2 * i + j] = M::pv(one, pw[r], rows.o[r][2 * i + j]);
          }
        }
        if (l + ST * NW < sg.l1) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the tile has been read
          send(sg, l + ST * NW, slot);
        }
        slot = slot + 1 == ST ? 0 : slot + 1;
        l += NW;
      };
      while (l < sg.l1) {
        while (l < sg.l1 && sg.plain(a, sg.tile(l))) work(std::true_type{});
        while (l < sg.l1 && !sg.plain(a, sg.tile(l))) work(std::false_type{});
      }
      if (odd_any)
        for (l = sg.l0 + wid; l < sg.l1; l += NW) {
          const int t0 = sg.tile(l);
          if (sg.plain(a, t0)) continue;
          send(sg, l, 0);
          wait_loads<0>();
          Codes<D> c;
          c.read_v(ring, m, g);
          float f[8];
          c.factors(f);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const unsigned vis = rows.view(a, sg, s, t0, r, g);
#pragma unroll
            for (int i = 0; i < DT / 2; ++i) {
              u32x4 v[2];
              c.values(i, f, v[0], v[1]);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const u32x4 one[1] = {M::cut(v[j], sg.end() - t0 - 8 * g)};
                rows.odd_values(r, 2 * i + j, one, vis);
              }
            }
          }
        }
    }

    wait_loads<0>();  // of a sequence that is refused, too
    __syncthreads();

    // the four waves joined: rows' maxima and sums, then the output tiles
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float l_row = M::total(rows.rl[r]);
      if (g == 0) {
        s_m[wid * RT + 16 * r + m] = rows.scale(r);
        s_l[wid * RT + 16 * r + m] = l_row;
      }
      f32x4 piece[DT];
      row_pieces<D>(rows.o[r], piece);
#pragma unroll
      for (int x = 0; x < DT; ++x) *reinterpret_cast<f32x4 *>(&s_o[(wid * RT + 16 * r + m) * PADD + 4 * (g * 4 * Q + x)]) = piece[x];
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
        const float fk = fast_exp2((mk - mt) * a.c2);
        ls += fk * lk;
        acc += *reinterpret_cast<const f32x4 *>(&s_o[(k * RT + row) * PADD + 4 * c4]) * fk;
      }
      const f32x4 one[1] = {acc};
      sink(row, mt, ls).put(c4, 0, one);
    }
  });
}

// ---------------------------------------------------------------- many rows

// Tiles of a stage and workgroups of a CU: as for bf16 pages, whose tiles the stages hold.
template <int D>
constexpr int wide4_stage() { return D <= 128 ? 2 : 1; }
// What the start of a unit costs, in rounds of a stage (64 sequences of 100 to 4000 slots, 32 nodes
// each: 195 us without, 158 so).
constexpr unsigned WIDE4_LEAD = 3;
template <int D, int R>
constexpr int wide4_occ() { return R * D <= 256 ? 2 : 1; }

// A stage's codes come into registers a stage ahead of their conversion, which is a stage ahead of
// their use: wave w converts half (keys or values) of tile w / 2, at D = 256 a quarter of one tile.
// In LDS a tile is keys [unit of d][slot], values [unit of slots][d'] with d' = 16 j + m for
// d = D / 16 m + j, so that neither side has bank conflicts.
template <int D, int R>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(wide4_occ<D, R>()))) void k_attn4_wide(const Attn4Args a) {
  typedef uint16_t T;
  typedef Mma<T> M;
  constexpr int RT = 16 * R * NW, KS = D / 32, DT = D / 16, Q = D / 64;
  constexpr int UNITS = TILE * D / 8;  // 16-byte units of a tile's keys, and of its values
  constexpr int PW = UNITS / NT;
  constexpr int ST = wide4_stage<D>();
  extern __shared__ unsigned s_books[];
  const SharedBooks s = books_at(s_books, RT, a.N, a.group);
  __shared__ u32x4 s_t[2][ST][2 * UNITS];
  __shared__ int s_odd;

  const int tid = threadIdx.x, lane = lane_id(), wid = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int m = lane & 15, g = lane >> 4;
  const int page = 1 << a.page_shift;
  const unsigned head_codes = (unsigned)page * D / 2, head_scales = (unsigned)page * D / F4_BLOCK;
  const unsigned long long page_codes = (unsigned long long)a.Hkv * head_codes, page_scales = (unsigned long long)a.Hkv * head_scales;
  // the wave's tile of a stage, and its part of it
  const int my_tile = ST == 2 ? wid / 2 : 0;
  const bool my_keys = ST == 2 ? wid % 2 == 0 : wid < 2;
  const int my_half = wid % 2;  // of the keys' slots or the values' elements, at D = 256

  Rows<T, D, R> rows;
  Codes<D> c;
  auto send = [&](const Segment &sg, int l) {  // the codes of stage l's tiles
    if (l + my_tile >= sg.l1) return;
    const int t0 = sg.tile(l + my_tile);
    int pa, pb;
    sg.pages(a, t0, pa, pb);
    if (my_keys)
      c.load_k(a.k_pages + (size_t)sg.h * head_codes, a.k_scales + (size_t)sg.h * head_scales, page_codes, page_scales, page, t0, pa, pb, m, g);
    else
      c.load_v(a.v_pages + (size_t)sg.h * head_codes, a.v_scales + (size_t)sg.h * head_scales, page_codes, page_scales, page, t0, pa, pb, m, g);
  };
  auto convert = [&](const Segment &sg, int l, u32x4 (&st)[ST][2 * UNITS]) {
    if (l + my_tile >= sg.l1) return;
    u32x4 *buf = st[my_tile];
    if (my_keys) {
#pragma unroll
      for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
        for (int k4 = 0; k4 < KS; ++k4)
          if (ST == 2 || t2 == my_half) buf[UnitsWithin<D>::at(k4, g) * TILE + 16 * t2 + m] = c.key(t2, k4);
    } else {
      float f[8];
      c.factors(f);
#pragma unroll
      for (int i = 0; i < DT / 2; ++i)
        if (ST == 2 || i / (DT / 4) == my_half) {
          u32x4 lo, hi;
          c.values(i, f, lo, hi);
          buf[UNITS + g * D + 32 * i + m] = lo;
          buf[UNITS + g * D + 32 * i + 16 + m] = hi;
        }
    }
  };
  auto begin = [&](const Segment &sg) {
    rows.load(a, sg, sg.rt * RT + wid * 16 * R, m, g);
    if (tid == 0) s_odd = 0;
    send(sg, sg.l0);
  };

  attn_share<T, D, RT, ST, true, least_part4<RT, ST>(), WIDE4_LEAD>(a, s, begin, [&](const Segment &sg, int code, auto sink) {
    rows.clear();
    if (sg.sp.i0 <= sg.sp.i1 && code == 0) {
      rows.depths(sg, s);
      rows.arrived();
      convert(sg, sg.l0, s_t[0]);
      send(sg, sg.l0 + ST);
      // Slots behind the sequence hold anything, and values that are not finite are left out of
      // the products where not every row sees them.
      auto clean = [&](int t0, u32x4 *vb) {
        bool odd = false;
#pragma unroll
        for (int j = 0; j < PW; ++j) {
          u32x4 v = M::cut(vb[tid + j * NT], sg.end() - t0 - (tid + j * NT) / D * 8);
          odd |= M::non_finite(v);
          vb[tid + j * NT] = M::finite(v);
        }
        if (odd) s_odd = 1;
        __syncthreads();
      };
      auto scores = [&](const u32x4 *buf, f32x4 (&sc)[R][2]) {
        typename M::Dot dot[R][2] = {};
#pragma unroll
        for (int k4 = 0; k4 < KS; ++k4)
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) {
            const u32x4 k = buf[(4 * k4 + g) * TILE + 16 * t2 + m];
#pragma unroll
            for (int r = 0; r < R; ++r) M::qk(k, rows.q[r][k4], dot[r][t2]);
          }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) sc[r][t2] = M::score(dot[r][t2]);
      };
      auto add = [&](const u32x4 *buf, const typename M::P (&pw)[R]) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const u32x4 v[1] = {buf[UNITS + g * D + 16 * d + m]};
#pragma unroll
          for (int r = 0; r < R; ++r) rows.o[r][d] = M::pv(v, pw[r], rows.o[r][d]);
        }
      };
      auto work = [&](int l, u32x4 *buf) {
        const int t0 = sg.tile(l);
        const bool plain = sg.plain(a, t0);
        if (!plain) clean(t0, buf + UNITS);
        f32x4 sc[R][2];
        scores(buf, sc);
        if (!plain) rows.mask(a, sg, s, t0, g, sc);
        typename M::P pw[R];
        rows.soften(a, sc, pw);
        add(buf, pw);
      };
      for (int l = sg.l0, at = 0; l < sg.l1; l += ST, at ^= 1) {
        __syncthreads();  // this stage is whole, and nobody reads the other buffer any more
        convert(sg, l + ST, s_t[at ^ 1]);
        send(sg, l + 2 * ST);
#pragma unroll 1
        for (int k = 0; k < ST; ++k)
          if (l + k < sg.l1) work(l + k, s_t[at][k]);
      }
      __syncthreads();
      if (s_odd)
        for (int l = sg.l0; l < sg.l1; ++l) {
          const int t0 = sg.tile(l);
          if (sg.plain(a, t0)) continue;
          if (my_tile == 0) {
            send(sg, l);
            convert(sg, l, s_t[0]);
          }
          __syncthreads();
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const unsigned vis = rows.view(a, sg, s, t0, r, g);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              const u32x4 v[1] = {M::cut(s_t[0][0][UNITS + g * D + 16 * d + m], sg.end() - t0 - 8 * g)};
              rows.odd_values(r, d, v, vis);
            }
          }
          __syncthreads();
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f32x4 piece[DT];
      row_pieces<D>(rows.o[r], piece);
      sink(wid * 16 * R + 16 * r + m, rows.scale(r), M::total(rows.rl[r])).put(g * 4 * Q, 1, piece);
    }
  });
}

}  // namespace sv

// ======================================================================== host side

namespace {

using namespace sv;
using namespace sv_host;

// The kernel for a head size: f is called with the constants.
template <typename F>
auto attn4_pick(int D, int R, F f) {
  if (D == 64) return R == 1 ? f(Int<64>{}, Int<1>{}) : f(Int<64>{}, Int<2>{});
  if (D == 128) return R == 1 ? f(Int<128>{}, Int<1>{}) : f(Int<128>{}, Int<2>{});
  return R == 1 ? f(Int<256>{}, Int<1>{}) : f(Int<256>{}, Int<2>{});
}

template <int D, int R>
void attn4_go(Launcher &L, Attn4Args &a, const AttnPlan &p) {
  void *args[] = {&a};
  AttnArgs shared = a;
  void *join_args[] = {&shared};
  L.lds = books_bytes(p.RT, a.N, a.group, a.parent != nullptr);
  if (p.wide) {
    L.go((const void *)&k_attn4_wide<D, R>, p.grid, args);
    L.lds = 0;
    L.go((const void *)&k_attn_join<uint16_t, D, 16 * R * NW>, (unsigned)(p.units * (p.RT / NW)), join_args);
  } else if constexpr (D <= 128 || R == 1) {
    L.go((const void *)&k_attn4<D, R>, p.grid, args);
    L.lds = 0;
    L.go((const void *)&k_attn_join<uint16_t, D, 16 * R>, (unsigned)(p.units * (p.RT / NW)), join_args);
  }
}

// Rows as for bf16 pages: one wave holds up to 16 of a key head in its registers, 32 up to D = 128;
// more go to the kernel whose waves share them.
bool attn4_plan(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page, int32_t W, AttnPlan &p) {
  const long long rows = (long long)N * (Hq / Hkv);
  p.wide = rows > (D <= 128 ? 32 : 16);
  p.R = p.wide ? (rows <= 64 ? 1 : 2) : (rows <= 16 ? 1 : 2);
  p.RT = 16 * p.R * (p.wide ? NW : 1);
  const int occ = attn4_pick(D, p.R, [&](auto d, auto r) {
    return p.wide ? wide4_occ<decltype(d)::value, decltype(r)::value>() : attn4_occ<decltype(d)::value, decltype(r)::value>();
  });
  return attn_cut(B, rows, Hkv, D, page, W, occ, p.wide ? (D <= 128 ? 2 : 1) : NW, p);
}

}  // namespace

extern "C" {

size_t sv_attention4_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                                     int32_t table_width) {
  AttnPlan p;
  if (!attn_shape_ok(B, N, Hq, Hkv, D, page_size, table_width) || !attn4_plan(B, N, Hq, Hkv, D, page_size, table_width, p)) return 256;
  return p.total;
}

sv_status spec_paged_attention4(const void *q, int64_t q_stride_b, int64_t q_stride_n, const void *k_codes, const void *k_scales,
                                const void *v_codes, const void *v_scales, const int32_t *page_table, const int32_t *cache_len,
                                const int32_t *n_new, const int32_t *parent, const int32_t *prior, int32_t B, int32_t N,
                                int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages, int32_t table_width,
                                float scale, int32_t window, int32_t sinks, void *out, int32_t *row_status, void *workspace,
                                size_t workspace_bytes, void *stream, void *const *events, int32_t n_events,
                                int32_t *n_launched) {
  if (n_launched) *n_launched = 0;
  if (!attn_shape_ok(B, N, Hq, Hkv, D, page_size, table_width) || num_pages < 1) return SV_ERR_SHAPE;
  if (!isfinite(scale) || window < 0 || sinks < 0 || (sinks > 0 && window == 0)) return SV_ERR_PARAM;
  AttnPlan p;
  if (!attn4_plan(B, N, Hq, Hkv, D, page_size, table_width, p)) return SV_ERR_SHAPE;
  if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !page_table || !cache_len || !out || !row_status || !workspace) return SV_ERR_NULL;
  if ((((uintptr_t)q | (uintptr_t)k_codes | (uintptr_t)v_codes | (uintptr_t)out | ((uintptr_t)q_stride_b * 2) | ((uintptr_t)q_stride_n * 2)) & 15) ||
      (((uintptr_t)k_scales | (uintptr_t)v_scales) & 7))
    return SV_ERR_ALIGN;
  if (workspace_bytes < p.total || ((uintptr_t)workspace & 255)) return SV_ERR_WORKSPACE;
  // several workgroups read prior, and one writes the status
  if (overlap(prior, row_status, B) || codes_on_inputs(row_status, B, N, table_width, page_table, cache_len, n_new, parent, nullptr)) return SV_ERR_PARAM;
  Attn4Args a = {};
  a.k_pages = static_cast<const char *>(k_codes);
  a.k_scales = static_cast<const char *>(k_scales);
  a.v_pages = static_cast<const char *>(v_codes);
  a.v_scales = static_cast<const char *>(v_scales);
  attn_fill(a, p, q, q_stride_b, q_stride_n, 2, page_table, cache_len, n_new, parent, prior, B, N, Hq, Hkv, page_size, num_pages,
            table_width, scale, window, sinks, out, row_status, workspace);
  Launcher L{(hipStream_t)stream, events, n_events};
  attn4_pick(D, p.R, [&](auto d, auto r) {
    attn4_go<decltype(d)::value, decltype(r)::value>(L, a, p);
    return 0;
  });
  if (n_launched) *n_launched = L.n;
  return L.e == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

const char *sv_attention4_launch_plan(int32_t N, int32_t Hq, int32_t Hkv, int32_t D) {
  AttnPlan p;
  if (!attn_shape_ok(1, N, Hq, Hkv, D, 16, 1) || !attn4_plan(1, N, Hq, Hkv, D, 16, 1, p)) return "";
  return p.wide ? "k_attn4_wide;k_attn_join" : "k_attn4;k_attn_join";
}

}  // extern "C"
