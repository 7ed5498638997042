// spec_rotary.hip -- positions on the way into the cache: queries and keys rotated, keys and
// values written to their slots, in the cache's type or in 4 bits (include/spec_cache.h), and
// entries read back.
//
// Pair j of a head, (x, y), becomes factor * (x cos t - y sin t, y cos t + x sin t) with
// t = position * inv_freq[j].  What a call has to move is its inputs once and its outputs once;
// the angles are one for each token and pair, whatever the heads, so a workgroup takes a few
// tokens, computes their cosines and sines once into LDS and streams the heads past them.
//
// Bound by bytes where there are many tokens: 8 prompts of up to 999, 32 query and 8 key heads of
// 128 in bf16, 36 us for 140 MB read and written (3.9 TB/s; a copy reaches 4.8), into 4 bits 39 us.
// A token each of 64 sequences takes 7 us, short chains into 4 bits 11: latency.  Queries have
// workgroups apart from keys and values, each with the next piece's loads on their way while it
// turns this one's (together and one piece at a time: 54 us into 4 bits).

#include "sv_fp4.h"

namespace sv {

struct RotaryArgs {
  const char *q, *k, *v;
  long long q_sb, q_sn, k_sb, k_sn, v_sb, v_sn;  // bytes
  char *k_pages, *k_scales, *v_pages, *v_scales, *q_out;
  const float *inv_freq;
  const int32_t *page_table, *cache_len, *n_new, *parent, *positions, *prior;
  int N, Hq, R, interleaved;
  double factor;
  int chunks, parts, q_parts, q_part, kv_part;  // workgroups of a sequence: chunks of tokens times parts of the heads
  int32_t *row_status;
  Pool pool;
};

// Tokens of a workgroup: whole units of values (8 slots of bf16, 4 of f32), so that a unit has
// one writer.
constexpr int ROT_TOKENS = 8;
constexpr int F4_LDS = 4096;  // floats of turned keys on their way to 4 bits

// cos t and sin t of t = n * f, in 64 bits: the product of a whole number and a float, rounded
// once; a quarter turn's multiple taken off in two parts (the first exactly, in the fused
// subtraction; below 2^31 * 2^8 turns what the two parts leave out is under 2^-60); and the
// Taylor series on [-pi/4, pi/4], whose next terms are under 2^-54.
SVD void turn_of(int n, float f, double factor, double &c, double &s) {
  const double t = (double)n * (double)f;
  const double k = rint(t * 0.63661977236758134308);
  double r = fma(-k, 1.57079632679489655800, t);
  r = fma(-k, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double p = -1.0 / 1307674368000.0;
  p = fma(p, z, 1.0 / 6227020800.0);
  p = fma(p, z, -1.0 / 39916800.0);
  p = fma(p, z, 1.0 / 362880.0);
  p = fma(p, z, -1.0 / 5040.0);
  p = fma(p, z, 1.0 / 120.0);
  p = fma(p, z, -1.0 / 6.0);
  const double sn = fma(p * z, r, r);
  double h = 1.0 / 20922789888000.0;
  h = fma(h, z, -1.0 / 87178291200.0);
  h = fma(h, z, 1.0 / 479001600.0);
  h = fma(h, z, -1.0 / 3628800.0);
  h = fma(h, z, 1.0 / 40320.0);
  h = fma(h, z, -1.0 / 720.0);
  h = fma(h, z, 1.0 / 24.0);
  h = fma(h, z, -0.5);
  const double cs = fma(h, z, 1.0);
  // k mod 4 quarter turns
  const int m = (int)(k - 4.0 * floor(k * 0.25));
  const double a = (m & 1) ? sn : cs, b = (m & 1) ? cs : sn;
  c = ((m == 1 || m == 2) ? -a : a) * factor;
  s = ((m >= 2) ? -b : b) * factor;
}

template <typename T>
struct Unit {  // 16 bytes of elements
  static constexpr int E = 16 / (int)sizeof(T);
  float x[E];
  SVD void load(const char *p) { Fmt<T>::unpack(*reinterpret_cast<const u32x4 *>(p), x); }
  SVD u32x4 pack() const {
    u32x4 w;
    if constexpr (E == 8) {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __builtin_bit_cast(unsigned, bf16x2{(__bf16)x[2 * j], (__bf16)x[2 * j + 1]});
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(x[j]);
    }
    return w;
  }
};

// A thread's place in a space of t, h < H, y < I, and on to NT places further without dividing.
struct Walk {
  int t, h, y, H, I, dh, dy;
  SVD Walk(int x, int H_, int I_) : H(H_), I(I_), dh(NT / I_), dy(NT % I_) {
    h = x / I;
    y = x - h * I;
    t = h / H;
    h -= t * H;
  }
  SVD void on() {
    y += dy;
    h += dh;
    if (y >= I) {
      y -= I;
      ++h;
    }
    while (h >= H) {
      h -= H;
      ++t;
    }
  }
};

// E units of E elements turned: element j of unit i becomes element i of unit j.
template <typename T>
SVD void transpose(u32x4 (&w)[Unit<T>::E]) {
  constexpr int E = Unit<T>::E;
  u32x4 r[E];
  if constexpr (E == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = u32x4{w[0][i], w[1][i], w[2][i], w[3][i]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)  // words i: elements 2 i and 2 i + 1
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[2 * i][j] = __builtin_amdgcn_perm(w[2 * j + 1][i], w[2 * j][i], 0x05040100u);
        r[2 * i + 1][j] = __builtin_amdgcn_perm(w[2 * j + 1][i], w[2 * j][i], 0x07060302u);
      }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) w[i] = r[i];
}

// A double as a float32, or where it goes on to be a bf16 number as one that is rounded as the double
// would be (to float32 and on to bf16 one in 10^5 went the other way): the double's upper word, with its
// last bit set for what is cut off, is exact in float32 and far from a bf16 number's last bit.
template <typename T>
SVD float narrowed(double x) {
  if constexpr (sizeof(T) == 4) return (float)x;
  else return (float)__hiloint2double(__double2hiint(x) | (int)min((unsigned)__double2loint(x), 1u), 0);
}

// x and y of a pair turned, to become Ts.
template <typename T>
SVD void turned(float &x, float &y, const double2 cs) {
  const double a = x, b = y;
  x = narrowed<T>(fma(a, cs.x, -(b * cs.y)));
  y = narrowed<T>(fma(b, cs.x, a * cs.y));
}

// Where pair j's cosine and sine lie among a token's in LDS: a gap behind every four, so that lanes
// that read neighbouring units' pairs meet in no bank.
SV_HD int cs_at(int j) { return j + (j >> 2); }
SV_HD int cs_row(int pairs) { return cs_at(pairs) + 1; }

// Element d of a head at p, turned, to become a To: for heads whose pairs do not lie unit against unit.
template <typename T, typename To>
SVD float turned_one(const char *p, int d, int R, const double2 *cs) {  // cs: of the token
  const T *x = reinterpret_cast<const T *>(p);
  float a = Fmt<T>::at(x, d);
  if (d >= R) return a;
  const int h = R / 2;
  const bool second = d >= h;
  float b = Fmt<T>::at(x, second ? d - h : d + h);
  if (second) {
    turned<To>(b, a, cs[cs_at(d - h)]);
  } else {
    turned<To>(a, b, cs[cs_at(d)]);
  }
  return a;
}

// The code of a sequence (the same test in every workgroup of it), and its parents in LDS.
SVD int rotary_code(const RotaryArgs &a, int b, int len, int m, uint16_t *s_par) {
  const int sh = a.pool.page_shift, tid = threadIdx.x;
  const int prior = a.prior ? min(a.prior[b], 0) : 0;
  if (prior != 0) return prior;
  if (len < 0 || m < 0 || m > a.N || (long long)len + m > ((long long)a.pool.W << sh)) return SV_ROW_BAD_LENGTH;
  if (m == 0) return 0;
  bool bad = false;
  if (a.parent) {
    for (int i = tid; i < m; i += NT) {
      const int p = a.parent[(size_t)b * a.N + i];
      s_par[i] = (uint16_t)p;
      bad |= i == 0 ? p != -1 : (p < 0 || p >= i);
    }
    if (__syncthreads_or(bad)) return SV_ROW_BAD_TREE;
  }
  const int32_t *table = a.page_table + (size_t)b * a.pool.W;
  const int p0 = len >> sh, p1 = (len + m - 1) >> sh;
  for (int i = p0 + tid; i <= p1; i += NT) bad |= (unsigned)table[i] >= (unsigned)a.pool.P;
  return __syncthreads_or(bad) ? SV_ROW_BAD_PAGE : 0;
}

// T: the inputs' type; F4: the cache is in 4 bits; PAIRS: pairs lie unit against unit (neighbours
// interleaved, or halves of whole units), so that a thread turns 16 bytes and their partners.
template <typename T, bool F4, bool PAIRS>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(4))) void k_append_rotary(const RotaryArgs a) {
  constexpr int E = Unit<T>::E, ESZ = (int)sizeof(T);
  extern __shared__ double2 s_cs[];  // [tokens][cs_row], then the parents
  const int tid = threadIdx.x;
  const int part = (int)(blockIdx.x % (unsigned)a.parts);
  const unsigned bc = blockIdx.x / (unsigned)a.parts;
  const int chunk = (int)(bc % (unsigned)a.chunks), b = (int)(bc / (unsigned)a.chunks);
  const int m = a.n_new ? a.n_new[b] : a.N;
  int len = a.cache_len[b];
  const int sh = a.pool.page_shift, page = 1 << sh, D = (int)a.pool.D, Hkv = (int)a.pool.Hkv, H2 = a.R / 2, CS = cs_row(H2), U = D / E;
  uint16_t *s_par = reinterpret_cast<uint16_t *>(s_cs + ROT_TOKENS * CS);
  const int32_t *table = a.page_table + (size_t)b * a.pool.W;
  // The workgroup's tokens: those whose slots are in the chunk'th eight from the sequence's first on.
  auto first_token = [&](int l) { return max(0, chunk * ROT_TOKENS - (l & (ROT_TOKENS - 1))); };
  auto last_token = [&](int l) { return min(a.N, (chunk + 1) * ROT_TOKENS - (l & (ROT_TOKENS - 1))); };
  int i0 = first_token(len), i1 = last_token(len);
  // The part's heads of the queries, and of the keys and values.
  const int q0 = part < a.q_parts ? min(a.Hq, part * a.q_part) : a.Hq, q1 = q0 + min(a.Hq - q0, a.q_part);
  const int h0 = part < a.q_parts ? Hkv : min(Hkv, (part - a.q_parts) * a.kv_part), h1 = min(Hkv, h0 + a.kv_part);

  // Queries, and the keys of a cache of the inputs' type, in jobs: 16 bytes and, where the head's
  // halves are turned against each other, their partners, of up to NB tokens.  A job's loads are on
  // their way while the one before it is turned, the first one's while the sequence is checked.
  constexpr int NB = 2;
  const int HU = PAIRS && !a.interleaved ? H2 / E : 0;  // units of a half
  const int items = U - HU, n_q = q1 - q0, n_heads = n_q + (F4 ? 0 : h1 - h0);
  struct Job {
    const char *p;
    long long stride;
    int h, y, t0;
  };
  auto job_at = [&](const Walk &w) {
    Job o;
    o.t0 = w.t * NB;
    o.h = w.h;
    o.y = w.y;
    const bool q = o.h < n_q;
    o.stride = q ? a.q_sn : a.k_sn;
    o.p = (q ? a.q + (long long)b * a.q_sb + (size_t)(q0 + o.h) * D * ESZ : a.k + (long long)b * a.k_sb + (size_t)(h0 + o.h - n_q) * D * ESZ) +
          (long long)(i0 + o.t0) * o.stride;
    return o;
  };
  auto load = [&](const Job &o, int n, u32x4 (&lw)[NB], u32x4 (&lv)[NB]) {
#pragma unroll
    for (int t = 0; t < NB; ++t)
      if (t == 0 || o.t0 + t < n) {
        lw[t] = *reinterpret_cast<const u32x4 *>(o.p + t * o.stride + (o.y < HU ? o.y : o.y + HU) * 16);
        if (o.y < HU) lv[t] = *reinterpret_cast<const u32x4 *>(o.p + t * o.stride + (o.y + HU) * 16);
      }
  };
  u32x4 lw[NB], lv[NB];
  Job job = {};
  Walk walk(tid, max(n_heads, 1), items);
  const int jobs = i0 < i1 ? n_heads * items * ((i1 - i0 + NB - 1) / NB) : 0;
  if constexpr (PAIRS)
    if (tid < jobs) {  // (rows of tokens are there whatever the sequence's length says)
      job = job_at(walk);
      load(job, i1 - i0, lw, lv);
    }

  const int code = rotary_code(a, b, len, m, s_par);
  if (chunk == 0 && part == 0 && tid == 0) a.row_status[b] = code;
  if (code != 0) {
    len = 0;
    i0 = first_token(0);
    i1 = last_token(0);
  }
  if (i0 >= i1) return;
  const int live = code != 0 ? i0 : min(max(m, i0), i1);  // tokens from here on are not new
  if (live < i1) {  // queries of no token: zero, or NaN for a sequence with a code
    const unsigned fill = code == 0 ? 0u : ESZ == 2 ? 0x7fc07fc0u : 0x7fc00000u;
    for (int i = live; i < i1; ++i)
      for (int x = tid; x < n_q * U; x += NT)
        *reinterpret_cast<u32x4 *>(a.q_out + (((size_t)b * a.N + i) * a.Hq + q0) * D * ESZ + (size_t)x * 16) = u32x4{fill, fill, fill, fill};
  }
  if (live <= i0) return;
  const int nt = live - i0;

  for (int x = tid; x < nt * H2; x += NT) {
    const int t = x / H2, j = x - t * H2, i = i0 + t;
    int pos = len + i;
    if (a.positions) {
      pos = a.positions[(size_t)b * a.N + i];
    } else if (a.parent) {
      pos = len;
      for (int n = i; n > 0; n = s_par[n]) ++pos;
    }
    double2 cs;
    turn_of(pos, a.inv_freq[j], a.factor, cs.x, cs.y);
    s_cs[t * CS + cs_at(j)] = cs;
  }
  __syncthreads();

  // The workgroup's slots lie in one page (8 slots from a multiple of 8 on).
  const size_t ph0 = (size_t)table[(len + i0) >> sh] * Hkv;
  const int at0 = (len + i0) & (page - 1);  // the first slot in it

  char *qo = a.q_out + (((size_t)b * a.N + i0) * a.Hq + q0) * D * ESZ;
  const size_t hb = head_bytes<T>(a.pool);  // of a cache of the inputs' type
  char *ko = a.k_pages + (ph0 + h0) * hb + (size_t)at0 * 16;
  auto put = [&](int t, int h, int u, u32x4 w) {
    char *o = h < n_q ? qo + ((size_t)t * a.Hq + h) * D * ESZ + u * 16 : ko + (size_t)(h - n_q) * hb + ((size_t)u * page + t) * 16;
    *reinterpret_cast<u32x4 *>(o) = w;
  };
  if constexpr (PAIRS) {
    for (int j = tid; j < jobs; j += NT) {
      u32x4 nw[NB], nv[NB];
      Job after = job;
      if (j + NT < jobs) {
        walk.on();
        after = job_at(walk);
        load(after, nt, nw, nv);
      }
#pragma unroll
      for (int t = 0; t < NB; ++t)
        if (job.t0 + t < nt) {
          const double2 *cs = s_cs + (job.t0 + t) * CS;
          Unit<T> w, v;
          Fmt<T>::unpack(lw[t], w.x);
          if (job.y < HU) {
            Fmt<T>::unpack(lv[t], v.x);
#pragma unroll
            for (int e = 0; e < E; ++e) turned<T>(w.x[e], v.x[e], cs[cs_at(job.y * E + e)]);
            put(job.t0 + t, job.h, job.y + HU, v.pack());
          } else if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
              if (job.y * E + 2 * e < a.R) turned<T>(w.x[2 * e], w.x[2 * e + 1], cs[cs_at(job.y * (E / 2) + e)]);
          }
          put(job.t0 + t, job.h, job.y < HU ? job.y : job.y + HU, w.pack());
        }
      job = after;
#pragma unroll
      for (int t = 0; t < NB; ++t) {
        lw[t] = nw[t];
        lv[t] = nv[t];
      }
    }
  } else {
    for (int x = tid; x < n_heads * U * nt; x += NT) {
      const int t = x / (n_heads * U), hy = x - t * (n_heads * U), h = hy / U, y = hy - h * U;
      const char *p = h < n_q ? a.q + (long long)b * a.q_sb + (long long)(i0 + t) * a.q_sn + (size_t)(q0 + h) * D * ESZ
                              : a.k + (long long)b * a.k_sb + (long long)(i0 + t) * a.k_sn + (size_t)(h0 + h - n_q) * D * ESZ;
      Unit<T> w;
#pragma unroll
      for (int e = 0; e < E; ++e) w.x[e] = turned_one<T, T>(p, y * E + e, a.R, s_cs + t * CS);
      put(t, h, y, w.pack());
    }
  }
  if constexpr (!F4) {
    // values: a whole unit of slots, E tokens, is turned in registers; of others single elements
    const int s0 = len + i0, s1 = len + live;
    for (int x = tid; x < (h1 - h0) * U; x += NT) {
      const int h = x / U, u = x - h * U;
      for (int f = s0 / E * E; f < s1; f += E) {
        const char *vs = a.v + (long long)b * a.v_sb + (long long)(f - len) * a.v_sn + ((size_t)(h0 + h) * D + u * E) * ESZ;
        char *out = a.v_pages + (ph0 + h0 + h) * hb + ((size_t)((f & (page - 1)) / E) * D + u * E) * 16;
        u32x4 w[E];
#pragma unroll
        for (int j = 0; j < E; ++j) w[j] = *reinterpret_cast<const u32x4 *>(vs + (long long)(min(max(f + j, s0), s1 - 1) - f) * a.v_sn);
        if (f >= s0 && f + E <= s1) {
          transpose<T>(w);
#pragma unroll
          for (int j = 0; j < E; ++j) *reinterpret_cast<u32x4 *>(out + j * 16) = w[j];
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (f + j >= s0 && f + j < s1) {
              T e[E];
              __builtin_memcpy(e, &w[j], 16);
#pragma unroll
              for (int d = 0; d < E; ++d) reinterpret_cast<T *>(out + d * 16)[j] = e[d];
            }
        }
      }
    }
  } else {
    // 4 bits: a thread codes 8 elements of a token, a word; the four threads of a block share its
    // largest.  Word w of unit u (8 elements) of the token in slot at.
    auto code8 = [&](const float (&f)[8], unsigned &byte) {
      unsigned w;
      byte = f4_encode8(f, w);
      return w;
    };
    // keys: turned into LDS, some heads at a time, since a block's elements come from different threads
    const int group = F4_LDS / (ROT_TOKENS * D);
    float *s_k = reinterpret_cast<float *>(s_cs + ROT_TOKENS * CS + (a.parent ? (a.N * 2 + 15) / 16 : 0));
    for (int g0 = h0; g0 < h1; g0 += group) {
      const int gn = min(group, h1 - g0);
      if (g0 > h0) __syncthreads();
      const char *ks = a.k + (long long)b * a.k_sb + (long long)i0 * a.k_sn + (size_t)g0 * D * ESZ;
      Walk from(tid, gn, items);
      for (int x = tid; x < nt * gn * items; x += NT, from.on()) {
        const int t = from.t, h = from.h, y = from.y;
        const char *p = ks + (long long)t * a.k_sn + (size_t)h * D * ESZ;
        const double2 *cs = s_cs + t * CS;
        float *o = s_k + (size_t)(t * gn + h) * D;
        auto keep = [&](int u, const Unit<T> &w) {
          *reinterpret_cast<float4 *>(o + u * 8) = make_float4(w.x[0], w.x[1], w.x[2], w.x[3]);
          *reinterpret_cast<float4 *>(o + u * 8 + 4) = make_float4(w.x[4], w.x[5], w.x[6], w.x[7]);
        };
        Unit<T> w, v;
        if constexpr (!PAIRS) {
#pragma unroll
          for (int e = 0; e < E; ++e) w.x[e] = turned_one<T, float>(p, y * E + e, a.R, cs);
          keep(y, w);
        } else {
          const int u = y < HU ? y : y + HU;
          w.load(p + u * 16);
          if (y < HU) {
            v.load(p + (y + HU) * 16);
#pragma unroll
            for (int e = 0; e < E; ++e) turned<float>(w.x[e], v.x[e], cs[cs_at(y * E + e)]);
            keep(y + HU, v);
          } else if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
              if (u * E + 2 * e < a.R) turned<float>(w.x[2 * e], w.x[2 * e + 1], cs[cs_at(u * (E / 2) + e)]);
          }
          keep(u, w);
        }
      }
      __syncthreads();
      Walk at(tid, gn, U);
      for (int x = tid; x < nt * gn * U; x += NT, at.on()) {
        const int t = at.t, h = at.h, u = at.y;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = s_k[(size_t)(t * gn + h) * D + u * 8 + e];
        unsigned byte;
        const unsigned w = code8(f, byte);
        const size_t ph = ph0 + g0 + h;
        *reinterpret_cast<unsigned *>(a.k_pages + ph * f4_codes(a.pool) + f4_key(a.pool, u / 4, at0 + t) + (u & 3) * 4) = w;
        if ((u & 3) == 0) a.k_scales[ph * f4_scales(a.pool) + f4_scale(a.pool, u / 4, at0 + t)] = (char)byte;
      }
    }
    // values: a thread's words of all tokens, in 16 bytes where eight slots are written
    const bool full = nt == ROT_TOKENS && at0 % ROT_TOKENS == 0;
    for (int x = tid; x < (h1 - h0) * U; x += NT) {
      const int h = x / U, u = x - h * U;
      const char *vs = a.v + (long long)b * a.v_sb + (long long)i0 * a.v_sn + ((size_t)(h0 + h) * D + u * 8) * ESZ;
      const size_t ph = ph0 + h0 + h;
      char *o = a.v_pages + ph * f4_codes(a.pool);
      char *sc = a.v_scales + ph * f4_scales(a.pool) + f4_scale(a.pool, u / 4, at0);
      u32x4 in[ROT_TOKENS];
#pragma unroll
      for (int t = 0; t < ROT_TOKENS; ++t)
        if (t < nt) in[t] = *reinterpret_cast<const u32x4 *>(vs + (long long)t * a.v_sn);
      unsigned w[ROT_TOKENS], bytes[2] = {0, 0};
#pragma unroll
      for (int t = 0; t < ROT_TOKENS; ++t)
        if (t < nt) {
          float f[8];
          Fmt<T>::unpack(in[t], f);
          unsigned byte;
          w[t] = code8(f, byte);
          bytes[t / 4] |= byte << (8 * (t & 3));
        }
      if (full) {
        if ((u & 3) == 0) *reinterpret_cast<uint2 *>(sc) = make_uint2(bytes[0], bytes[1]);
        if (D == 128) {
          *reinterpret_cast<u32x4 *>(o + f4_value(a.pool, at0, u)) = u32x4{w[0], w[1], w[2], w[3]};
          *reinterpret_cast<u32x4 *>(o + f4_value(a.pool, at0 + 4, u)) = u32x4{w[4], w[5], w[6], w[7]};
        } else if (D == 64) {
          u32x4 lo, hi;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            lo[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x05040100u);
            hi[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x07060302u);
          }
          *reinterpret_cast<u32x4 *>(o + f4_value(a.pool, at0, 2 * u)) = lo;
          *reinterpret_cast<u32x4 *>(o + f4_value(a.pool, at0, 2 * u + 1)) = hi;
        } else {
#pragma unroll
          for (int t = 0; t < ROT_TOKENS; ++t) *reinterpret_cast<unsigned *>(o + f4_value(a.pool, at0 + t, u / 2) + (u & 1) * 4) = w[t];
        }
      } else {
#pragma unroll
        for (int t = 0; t < ROT_TOKENS; ++t)
          if (t < nt) {
            if ((u & 3) == 0) sc[t] = (char)(bytes[t / 4] >> (8 * (t & 3)));
            if (D == 64) {
              *reinterpret_cast<uint16_t *>(o + f4_value(a.pool, at0 + t, 2 * u)) = (uint16_t)w[t];
              *reinterpret_cast<uint16_t *>(o + f4_value(a.pool, at0 + t, 2 * u + 1)) = (uint16_t)(w[t] >> 16);
            } else if (D == 128) {
              *reinterpret_cast<unsigned *>(o + f4_value(a.pool, at0 + t, u)) = w[t];
            } else {
              *reinterpret_cast<unsigned *>(o + f4_value(a.pool, at0 + t, u / 2) + (u & 1) * 4) = w[t];
            }
          }
      }
    }
  }
}

// ---------------------------------------------------------------- entries read back

struct ReadArgs {
  const char *k_pages, *k_scales, *v_pages, *v_scales;
  const int32_t *page_table, *first, *count;
  int N, chunks;
  char *k, *v;
  int32_t *row_status;
  Pool pool;
};

constexpr int READ_TOKENS = 8;

template <typename T, bool F4>
__global__ __launch_bounds__(NT) void k_cache_read(const ReadArgs a) {
  constexpr int E = Unit<T>::E, ESZ = (int)sizeof(T);
  const int tid = threadIdx.x;
  const int chunk = (int)(blockIdx.x % (unsigned)a.chunks), b = (int)(blockIdx.x / (unsigned)a.chunks);
  const int sh = a.pool.page_shift, page = 1 << sh, D = (int)a.pool.D, Hkv = (int)a.pool.Hkv;
  const int first = a.first[b], m = a.count ? a.count[b] : a.N;
  const int32_t *table = a.page_table + (size_t)b * a.pool.W;
  int code = 0;
  if (first < 0 || m < 0 || m > a.N || (long long)first + m > ((long long)a.pool.W << sh)) {
    code = SV_ROW_BAD_LENGTH;
  } else if (m > 0) {
    bool bad = false;
    for (int i = (first >> sh) + tid; i <= (first + m - 1) >> sh; i += NT) bad |= (unsigned)table[i] >= (unsigned)a.pool.P;
    if (__syncthreads_or(bad)) code = SV_ROW_BAD_PAGE;
  }
  if (chunk == 0 && tid == 0) a.row_status[b] = code;
  const int i0 = chunk * READ_TOKENS, i1 = min(a.N, i0 + READ_TOKENS);
  const unsigned fill = code == 0 ? 0u : ESZ == 2 ? 0x7fc07fc0u : 0x7fc00000u;
  const int U = D / E, row = Hkv * U;
  for (int x = tid; x < (i1 - i0) * row; x += NT) {
    const int i = i0 + x / row, h = x % row / U, u = x % U;
    u32x4 kw = {fill, fill, fill, fill}, vw = kw;
    if (code == 0 && i < m) {
      const int s = first + i, at = s & (page - 1);
      const size_t ph = (size_t)table[s >> sh] * Hkv + h;
      if constexpr (F4) {
        const size_t sc = ph * f4_scales(a.pool) + f4_scale(a.pool, u / 4, at), co = ph * f4_codes(a.pool);
        kw = f4_unit(*reinterpret_cast<const unsigned *>(a.k_pages + co + f4_key(a.pool, u / 4, at) + (u % 4) * 4),
                     f4_factor((unsigned char)a.k_scales[sc]));
        const int B = D / 32;  // 8 elements are two pieces, one, or half a one
        unsigned w;
        if (B == 2)
          w = *reinterpret_cast<const uint16_t *>(a.v_pages + co + f4_value(a.pool, at, 2 * u)) |
              (unsigned)*reinterpret_cast<const uint16_t *>(a.v_pages + co + f4_value(a.pool, at, 2 * u + 1)) << 16;
        else
          w = *reinterpret_cast<const unsigned *>(a.v_pages + co + f4_value(a.pool, at, u * 4 / B) + u * 4 % B);
        vw = f4_unit(w, f4_factor((unsigned char)a.v_scales[sc]));
      } else {
        const size_t hb = head_bytes<T>(a.pool);
        kw = *reinterpret_cast<const u32x4 *>(a.k_pages + ph * hb + ((size_t)u * page + at) * 16);
        const T *vp = reinterpret_cast<const T *>(a.v_pages + ph * hb + ((size_t)(at / E) * D + u * E) * 16) + at % E;
        T e[E];
#pragma unroll
        for (int j = 0; j < E; ++j) e[j] = vp[j * E];
        __builtin_memcpy(&vw, e, 16);
      }
    }
    const size_t o = (((size_t)b * a.N + i) * Hkv + h) * D * ESZ + (size_t)u * 16;
    *reinterpret_cast<u32x4 *>(a.k + o) = kw;
    *reinterpret_cast<u32x4 *>(a.v + o) = vw;
  }
}

}  // namespace sv

// ======================================================================== host side

namespace {

using namespace sv;
using namespace sv_host;

bool f4_dim(int32_t D) { return D == 64 || D == 128 || D == 256; }

}  // namespace

extern "C" {

sv_status spec_cache_append_rotary(const void *q, int64_t q_stride_b, int64_t q_stride_n, const void *k, int64_t k_stride_b,
                                   int64_t k_stride_n, const void *v, int64_t v_stride_b, int64_t v_stride_n, sv_dtype dtype,
                                   void *k_pages, void *k_scales, void *v_pages, void *v_scales, const sv_rotary *rotary,
                                   const int32_t *page_table, const int32_t *cache_len, const int32_t *n_new,
                                   const int32_t *parent, const int32_t *positions, const int32_t *prior, int32_t B, int32_t N,
                                   int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                                   int32_t table_width, void *q_out, int32_t *row_status, void *stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  const bool f4 = k_scales || v_scales;
  if (f4 && dtype != SV_BF16) return SV_ERR_DTYPE;
  const int esz = dtype == SV_BF16 ? 2 : 4, E = 16 / esz;
  if (B < 1 || N < 1 || N > SV_CACHE_MAX_NEW || Hq < 0 || (Hq == 0) != (q == nullptr) || !pool_ok(Hkv, D, page_size, num_pages, table_width) ||
      (f4 && !f4_dim(D)))
    return SV_ERR_SHAPE;
  const int R = rotary ? rotary->rot_dim : 0;
  if (R < 0 || R > D || R % 2) return SV_ERR_SHAPE;
  if (rotary && !(fabsf(rotary->factor) <= __FLT_MAX__)) return SV_ERR_PARAM;
  RotaryArgs a = {};
  a.chunks = (N + ROT_TOKENS - 2) / ROT_TOKENS + 1;  // the first may begin anywhere in a chunk
  // Parts of the heads, queries apart from keys and values, so that small calls use more of the card
  // and the steps of a workgroup are few (each part computes the tokens' angles anew).
  const long long wgs = (long long)B * a.chunks;
  const int want = (int)(wgs >= 512 ? 1 : (512 + wgs - 1) / wgs);
  auto parts = [&](int heads) { return heads < want ? heads : want; };
  a.q_parts = parts(Hq < 8 ? Hq : 8);
  const int kv_parts = parts(Hkv < 8 ? Hkv : 8);
  a.parts = a.q_parts + kv_parts;
  if (wgs > MAX_WGS / a.parts) return SV_ERR_SHAPE;
  a.q_part = a.q_parts ? (Hq - 1) / a.q_parts + 1 : 0;
  a.kv_part = (Hkv - 1) / kv_parts + 1;
  if (!k || !v || !k_pages || !v_pages || (f4 && (!k_scales || !v_scales)) || !page_table || !cache_len || !row_status ||
      (q && !q_out) || (R && !rotary->inv_freq))
    return SV_ERR_NULL;
  a.q = static_cast<const char *>(q);
  a.k = static_cast<const char *>(k);
  a.v = static_cast<const char *>(v);
  const int64_t strides[6] = {q_stride_b, q_stride_n, k_stride_b, k_stride_n, v_stride_b, v_stride_n};
  long long *to[6] = {&a.q_sb, &a.q_sn, &a.k_sb, &a.k_sn, &a.v_sb, &a.v_sn};
  uintptr_t bits = (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)q_out;
  for (int i = 0; i < 6; ++i) {
    *to[i] = (long long)((unsigned long long)strides[i] * esz);
    if (i > 1 || q) bits |= (uintptr_t)*to[i];
  }
  if ((bits & 15) || (((uintptr_t)k_scales | (uintptr_t)v_scales) & 7) || (R && ((uintptr_t)rotary->inv_freq & 3))) return SV_ERR_ALIGN;
  if (overlap(prior, row_status, B)) return SV_ERR_PARAM;
  if (q) {  // a pair's elements are read and written by different threads, keys and values by other workgroups
    const uintptr_t head = (uintptr_t)D * esz, o0 = (uintptr_t)q_out, o1 = o0 + (uintptr_t)B * N * Hq * head;
    auto meets = [&](const void *x, int heads, long long sb, long long sn) {
      const uintptr_t x0 = (uintptr_t)x, x1 = x0 + (uintptr_t)(B - 1) * (uintptr_t)sb + (uintptr_t)(N - 1) * (uintptr_t)sn + (uintptr_t)heads * head;
      return x0 < o1 && o0 < x1;
    };
    if (meets(q, Hq, a.q_sb, a.q_sn) || meets(k, Hkv, a.k_sb, a.k_sn) || meets(v, Hkv, a.v_sb, a.v_sn)) return SV_ERR_PARAM;
  }
  if (codes_on_inputs(row_status, B, N, table_width, page_table, cache_len, n_new, parent, positions)) return SV_ERR_PARAM;
  a.k_pages = static_cast<char *>(k_pages);
  a.k_scales = static_cast<char *>(k_scales);
  a.v_pages = static_cast<char *>(v_pages);
  a.v_scales = static_cast<char *>(v_scales);
  a.q_out = static_cast<char *>(q_out);
  a.page_table = page_table;
  a.cache_len = cache_len;
  a.n_new = n_new;
  a.parent = parent;
  a.positions = positions;
  a.prior = prior;
  a.N = N;
  a.Hq = Hq;
  a.R = R;
  if (R) {
    a.inv_freq = rotary->inv_freq;
    a.interleaved = rotary->interleaved != 0;
    a.factor = rotary->factor;
  }
  a.row_status = row_status;
  a.pool = pool_of(Hkv, D, page_size, num_pages, table_width);
  const bool pairs = a.interleaved || (R / 2) % E == 0;
  unsigned lds = ROT_TOKENS * cs_row(R / 2) * 16 + (parent ? ((unsigned)N * 2 + 15) / 16 * 16 : 0u);
  if (f4) lds += (a.kv_part < F4_LDS / (ROT_TOKENS * D) ? (unsigned)a.kv_part * ROT_TOKENS * D : F4_LDS) * 4;
  const void *fn = f4 ? (pairs ? (const void *)&k_append_rotary<uint16_t, true, true> : (const void *)&k_append_rotary<uint16_t, true, false>)
                 : esz == 2 ? (pairs ? (const void *)&k_append_rotary<uint16_t, false, true> : (const void *)&k_append_rotary<uint16_t, false, false>)
                            : (pairs ? (const void *)&k_append_rotary<float, false, true> : (const void *)&k_append_rotary<float, false, false>);
  return launch(fn, a, wgs * a.parts, NT, stream, lds);
}

sv_status spec_cache_read(const void *k_pages, const void *k_scales, const void *v_pages, const void *v_scales, sv_dtype dtype,
                          const int32_t *page_table, const int32_t *first, const int32_t *count, int32_t B, int32_t N,
                          int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages, int32_t table_width, void *k, void *v,
                          int32_t *row_status, void *stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  const bool f4 = k_scales || v_scales;
  if (f4 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (B < 1 || N < 1 || !pool_ok(Hkv, D, page_size, num_pages, table_width) || (f4 && !f4_dim(D)) ||
      (long long)N > ((long long)table_width * page_size) || (long long)READ_TOKENS * Hkv * D > 0x7fffffffLL)
    return SV_ERR_SHAPE;
  ReadArgs a = {};
  a.chunks = (N + READ_TOKENS - 1) / READ_TOKENS;
  if (B > MAX_WGS / a.chunks) return SV_ERR_SHAPE;
  if (!k_pages || !v_pages || (f4 && (!k_scales || !v_scales)) || !page_table || !first || !k || !v || !row_status) return SV_ERR_NULL;
  if ((((uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)k | (uintptr_t)v) & 15) || (((uintptr_t)k_scales | (uintptr_t)v_scales) & 7))
    return SV_ERR_ALIGN;
  if (codes_on_inputs(row_status, B, 1, table_width, page_table, first, count, nullptr, nullptr)) return SV_ERR_PARAM;
  a.k_pages = static_cast<const char *>(k_pages);
  a.k_scales = static_cast<const char *>(k_scales);
  a.v_pages = static_cast<const char *>(v_pages);
  a.v_scales = static_cast<const char *>(v_scales);
  a.page_table = page_table;
  a.first = first;
  a.count = count;
  a.N = N;
  a.k = static_cast<char *>(k);
  a.v = static_cast<char *>(v);
  a.row_status = row_status;
  a.pool = pool_of(Hkv, D, page_size, num_pages, table_width);
  const void *fn = f4 ? (const void *)&k_cache_read<uint16_t, true>
                      : dtype == SV_BF16 ? (const void *)&k_cache_read<uint16_t, false> : (const void *)&k_cache_read<float, false>;
  return launch(fn, a, (long long)B * a.chunks, NT, stream);
}

}  // extern "C"
