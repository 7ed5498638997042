// spec_filter.hip -- sampling and filtered logits under temperature, top-k, min-p and top-p
// (include/spec_filter.h).
//
// Each of the three cuts keeps the logits at or above some value, so a row's policy comes down to
// one threshold, found by weighted selection: the largest value t with W(z >= t) >= a target,
// where W counts tokens (top-k) or adds their weights (top-p).  Weights are 2^x for
// x = z log2(e) / T.  They are fixed-point numbers relative to a power of two near the row's
// largest, so that sums do not depend on their order, and they are taken in 64 bits to
// 5 * 10^-11: a vocabulary of 10^5 tokens of probability 10^-6 leaves cumulative weights no room for
// float32's rounding.  Bins add up weights as they are, each token's to a unit of 2^-35 of its own
// octave; where weights of different octaves meet, the unit goes by the row's total, which is put
// between 2^59 and 2^61 units: cutting off what is smaller costs a sum over 2^24 tokens, the largest of
// them or all, 2^-35 of itself at most (a unit that went by the vocabulary's size and the row's largest:
// 2 * 10^-9 at 2^18 tokens, 2 * 10^-5 at 2^24, and thresholds with hundreds of tokens too many).
//
//   k_filter_scan    a chunk of a row a workgroup, one read of the logits: the chunk's largest, and
//                    counts and weights by quarter octave of the weight (the same ones for every
//                    chunk)
//   k_filter_plan    a row a workgroup: adds up the row's bins and finds the bin in which the first
//                    threshold lies
//   k_filter_gather  a chunk a workgroup again: puts what its chunk has in that bin on the row's list
//   k_filter_pick    a row a workgroup: selects on the list, looks for more where a further
//                    threshold needs it, and draws: the chunk whose cumulative kept weight passes u
//                    times the total, and the token in it
//   k_filter_write   the row again, with -inf below the threshold
//
// Bound by the weights: 26 vector instructions and a place in LDS for a logit.  320 rows of 128256
// in bf16, top-p 0.9: scan 43 us (its bytes 12), plan 10, gather 21, pick 14, write 28 (the
// row read and written; a copy takes 34).  64 rows drawn from: 13, 8, 8, 13.

#include "sv_common.h"

#include "spec_filter.h"

namespace sv {

typedef unsigned long long w64;

constexpr int FC = 8192;        // logits of a chunk, counted from the 16-byte block that the row begins in
constexpr int BINS = 128;       // quarter octaves of weight kept apart; the last takes all that is smaller
constexpr int LIST = 8192;      // tokens of the list of k_filter_pick
constexpr int FPT = FC / NT;    // logits of a thread of k_filter_scan

enum { F_ODD = 1, F_FINITE = 2, F_FAR = 4 };  // a chunk's flags: NaN or +inf, some finite logit, weights out of range

// A chunk's bin j holds its tokens in quarter octave q - j: their number from bit 50 up, and below
// it the sum of their weights relative to the octave that the bin lies in, in units of 2^-35 (8192
// tokens of at most 2.02: 14 and 50 bits).
constexpr int W_BITS = 35, W_COUNT = 50;
struct ChunkSum {
  int q;           // the quarter octave of the largest
  unsigned top;    // the largest finite logit's key
  unsigned flags, pad;
  w64 bin[BINS];
};

// What k_filter_plan found out about a row.
struct RowPlan {
  w64 mass[BINS];        // the row's bins: weights in units of 2^-F of the octave of q, and numbers
  unsigned count[BINS];
  w64 above;             // of the first step: what lies above its range
  double target;         // and what it looks for
  int q, F, step, bin, jt;  // the largest's quarter octave; its octave's units; the step, its bin, the lowest threshold's bin
  unsigned flags, tau, lo, hi, list_lo, list_hi;  // thresholds so far, the step's range, the list's
  float zmax;
  int by_k, by_m, cuts, whole;
};

struct FilterArgs {
  const void *logits;
  const float *u;
  int rows, V, chunks, F0;  // F0: 2^F0 units of the largest's octave, V times, fit 62 bits
  sv_policy policy;
  ChunkSum *sums;          // [rows][chunks]
  RowPlan *plans;          // [rows]
  w64 *over;               // [rows][chunks] draw: a chunk's weight in the bins above the lowest threshold's
  unsigned *n_list;        // [rows]
  uint2 *list;             // [rows][cap] keys and places (in blocks) of tokens
  int cap;
  uint2 *cut;              // [rows] filter: the threshold's key and the one token kept (-1: all above; -2: a code)
  int32_t *tokens, *row_status;
  void *out;
};

struct Policy {
  double c64;  // 64 log2(e) / T
  float t, p, m;
  int k;
  bool ok;
};
SVD Policy policy_of(const FilterArgs &a, int row) {
  const sv_policy &s = a.policy;
  Policy r;
  r.t = s.temperatures ? s.temperatures[row] : s.temperature;
  r.k = s.top_ks ? s.top_ks[row] : s.top_k;
  r.p = s.top_ps ? s.top_ps[row] : s.top_p;
  r.m = s.min_ps ? s.min_ps[row] : s.min_p;
  r.ok = r.t >= 0.0f && r.t < INFINITY && r.p > 0.0f && r.p <= 1.0f && r.m >= 0.0f && r.m <= 1.0f;
  r.c64 = r.ok && r.t > 0.0f ? 64.0 * 1.4426950408889634074 / (double)r.t : 0.0;
  return r;
}

// 2^d for d > -1000: the Taylor series of 2^f on [-1/2, 1/2], whose next term is under 10^-14.
SVD double pow2(double d) {
  const double k = rint(d), f = (d - k) * 0.69314718055994530942;
  double p = 1.0 / 39916800.0;
  p = fma(p, f, 1.0 / 3628800.0);
  p = fma(p, f, 1.0 / 362880.0);
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  p = fma(p, f, 1.0);
  return ldexp(p, (int)k);
}

// Weights of a row.  64 x = z * c64 = k + r with k whole, |r| <= 1/2 (adding 1.5 * 2^52 leaves k in
// the sum's low word; |64 x| is below 2^30): 2^x = 2^(k / 64) * 2^(r / 64), the first from 64 powers
// in LDS and k's upper bits, the second from three terms of its series (the fourth is under
// 4 * 10^-11, and always positive).  A token's quarter octave is k >> 4, its octave k >> 6.
struct Weight {
  int q;    // quarter octave
  w64 m;    // 2^x relative to the octave, or to `rest` where that is higher, in units of 2^-35
};
SVD void powers(double *tab) {  // [64], before a barrier
  if (threadIdx.x < 64) tab[threadIdx.x] = pow2(W_BITS + (double)threadIdx.x / 64.0);
}
SVD int k64(double z, double c64, double &y) {
  y = fma(z, c64, 6755399441055744.0);
  return (int)(unsigned)__double_as_longlong(y);
}
SVD int quarter_of(double z, double c64) {
  double y;
  return k64(z, c64, y) >> 4;
}
SVD Weight weight_of(double z, double c64, const double *tab, int rest) {
  constexpr double L = 0.69314718055994530942 / 64.0;
  double y;
  const int k = k64(z, c64, y);
  const double r = fma(z, c64, 6755399441055744.0 - y), t = tab[k & 63];
  const double e = fma(fma(L * L * L / 6.0, r, L * L / 2.0), r, L), v = fma(t * r, e, t);
  Weight w;
  w.q = k >> 4;
  const int down = max(min((k >> 6) - rest, 0), -100);
  const double x = __hiloint2double(__double2hiint(v) + (down << 20), __double2loint(v)) + 4503599627370496.0;  // its ulp is one unit
  w.m = (w64)__double_as_longlong(x) & 0xfffffffffffffull;
  return w;
}
// Logits below this are taken as this, so that |64 x| stays below 2^30 (as a float32, not below
// -10^9 / c64).
SVD float lowest_of(double c64) { return fmaxf((float)(-0.999e9 / c64), -__FLT_MAX__); }
SVD int octave_of(int q) { return q >> 2; }
SVD w64 shifted(w64 m, int left) { return left >= 0 ? m << left : left > -64 ? m >> -left : 0ull; }

// Logits in an order of whole numbers, and back: bf16 in 16 bits.  -0 is taken as 0 (they are equal).
template <typename T>
struct Key {
  static constexpr int SHIFT = sizeof(T) == 2 ? 16 : 0;
  SVD static unsigned of(float z) { return f2key(z + 0.0f) >> SHIFT; }
  SVD static float value(unsigned k) { return key2f(SHIFT ? (k << 16) | ((k & 0x8000u) ? 0u : 0xffffu) : k); }
  SVD static unsigned lowest() { return of(-__FLT_MAX__) & (SHIFT ? 0xffffu : 0xffffffffu); }
};

// A row as 16-byte blocks: block i holds elements i E - lead .. of the row, those outside it masked.
template <typename T>
struct RowBlocks {
  static constexpr int E = Fmt<T>::VEC;
  const u32x4 *p;
  int lead, n, V;
  SVD RowBlocks(const void *logits, int row, int V_) : V(V_) {
    const T *r = static_cast<const T *>(logits) + (size_t)row * V_;
    lead = (int)(((uintptr_t)r & 15u) / sizeof(T));
    p = reinterpret_cast<const u32x4 *>((uintptr_t)r & ~(uintptr_t)15);
    n = (lead + V_ + E - 1) / E;
  }
  SVD u32x4 load(int i) const { return p[min(i, n - 1)]; }
  SVD int index(int i, int e) const { return i * E + e - lead; }
  // Elements of block i; outside the row -inf.
  SVD void unpack(u32x4 w, int i, float (&z)[E]) const {
    Fmt<T>::unpack(w, z);
    if (i == 0 || i >= n - 1)
#pragma unroll
      for (int e = 0; e < E; ++e) z[e] = (unsigned)index(i, e) < (unsigned)V ? z[e] : -INFINITY;
  }
};

// ---------------------------------------------------------------- scan

constexpr int COPIES = 16;  // of a workgroup's bins, so that a wave's lanes seldom add to one place

template <typename T>
__global__ __launch_bounds__(NT) void k_filter_scan(const FilterArgs a) {
  constexpr int E = Fmt<T>::VEC, NV = FPT / E;
  __shared__ w64 s_bin[BINS * COPIES];
  __shared__ double s_tab[64];
  __shared__ unsigned s_top[NW], s_flags[NW];
  const int tid = threadIdx.x, lane = lane_id(), wid = tid / WAVE;
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), c = (int)(blockIdx.x % (unsigned)a.chunks);
  const RowBlocks<T> r(a.logits, row, a.V);
  const Policy pol = policy_of(a, row);
  u32x4 w[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) w[k] = r.load(c * (FC / E) + k * NT + tid);
  for (int i = tid; i < BINS * COPIES; i += NT) s_bin[i] = 0;
  powers(s_tab);
  float z[NV][E];
  float top = -INFINITY;
  int most = (int)0x80000000;  // of the bits as whole numbers: from +inf up they are not finite
  unsigned least = 0;          // likewise for negative ones: beyond -inf
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    r.unpack(w[k], c * (FC / E) + k * NT + tid, z[k]);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      top = fmaxf(top, z[k][e]);
      most = max(most, __float_as_int(z[k][e]));
      least = max(least, __float_as_uint(z[k][e]));
    }
  }
  const bool odd = most >= 0x7f800000 || least > 0xff800000u;
  top = wave_max(top);
  // out of range: 64 x too large, or temperatures at which even the lowest float32 weighs something (a
  // chunk all far below zero says nothing of its row: k_filter_plan looks at the row's largest)
  const unsigned far = (double)top * pol.c64 < 0.99e9 && pol.c64 > 4e-30 ? 0u : (unsigned)F_FAR;
  const unsigned fl = wave_or((odd ? (unsigned)F_ODD : 0u) | (top > -INFINITY ? F_FINITE | far : 0u));
  if (lane == 0) {
    s_top[wid] = f2key(top);
    s_flags[wid] = fl;
  }
  __syncthreads();
  unsigned tk = 0, flags = 0;
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    tk = max(tk, s_top[k]);
    flags |= s_flags[k];
  }
  ChunkSum *out = a.sums + (size_t)row * a.chunks + c;
  const bool weigh = pol.c64 != 0.0 && flags == F_FINITE;
  // Logits so low that they weigh nothing are taken higher (-inf among them: they add nothing to the
  // last bin but their number, which then only makes it look fuller).
  const float low = lowest_of(pol.c64);
  const int q = weigh ? quarter_of((double)fmaxf(key2f(tk), low), pol.c64) : 0;
  if (weigh) {
    const int rest = octave_of(q - (BINS - 1));
    w64 *mine = s_bin + (lane & (COPIES - 1));
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const Weight x = weight_of((double)fmaxf(z[k][e], low), pol.c64, s_tab, rest);
        atomicAdd(&mine[min(q - x.q, BINS - 1) * COPIES], x.m | (1ull << W_COUNT));
      }
    __syncthreads();
  }
  if (tid < BINS) {
    w64 m = 0;
#pragma unroll
    for (int k = 0; k < COPIES; ++k) m += s_bin[tid * COPIES + (k + tid) % COPIES];
    out->bin[tid] = m;
  }
  if (tid == 0) {
    out->q = q;
    out->top = tk;
    out->flags = flags;
    if (c == 0) a.n_list[row] = 0;
  }
}

// ---------------------------------------------------------------- rows

enum { ALL, COUNT, REST, MASS, DRAWN, END };
// Steps of a row.  ALL: a far row's bins.  COUNT: selection by number.  REST: the kept weight of
// tau's bin.  MASS: selection by weight.  DRAWN: the chunks' kept weight of tau's bin.

struct RowShared {
  w64 mass[BINS];
  unsigned count[BINS];
  double tab[64];
  unsigned flags, top;
  int q;
};

// The smallest key in [lo, hi] of which pred holds, pred(hi) taken to; by every wave alike.
template <typename F>
SVD unsigned first_key(unsigned lo, unsigned hi, F pred) {
  while (lo < hi) {
    const unsigned n = hi - lo, step = n / (WAVE - 1) + (n % (WAVE - 1) != 0 ? 1u : 0u);  // lo + 63 step >= hi
    const unsigned long long off = (unsigned long long)step * (unsigned)lane_id();
    const unsigned k = off < n ? lo + (unsigned)off : hi;
    const unsigned long long yes = __ballot(k == hi || pred(k));
    const int f = __ffsll(yes) - 1;
    hi = (unsigned)__builtin_amdgcn_readlane((int)k, f);
    if (f == 0) break;
    lo = (unsigned)__builtin_amdgcn_readlane((int)k, f - 1) + 1u;
  }
  return hi;
}

SVD w64 wave_incl(w64 v) {
#define STEP(C, R) v += ((w64)dpp_u<C, R>((unsigned)(v >> 32), 0u) << 32) | dpp_u<C, R>((unsigned)v, 0u);
  SV_SCAN_STEPS(STEP)
#undef STEP
  return v;
}
SVD w64 wave_total64(w64 v) {
  v = wave_incl(v);
  const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)v, WAVE - 1), hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(v >> 32), WAVE - 1);
  return ((w64)hi << 32) | lo;
}

// A row as both kernels see it once its chunks have been added up.
template <typename T>
struct Row {
  typedef Key<T> K;
  RowShared &s;
  Policy pol;
  int F, F0, Q, O, rest;
  unsigned flags, top_key;
  float zmax;
  bool far;
  double off, least, inv64;
  // Lane l has bins 2 l and 2 l + 1, and what lies in front of them, in units of 2^-F of the octave O.
  w64 m0, m1, pm, kept;
  unsigned c0, c1, pc, n_all;
  // the cuts: kept are keys from tau on; the lowest bin that a threshold can lie in; whether everything
  // from it up fits a list
  bool by_k, by_m, by_p, cuts, whole;
  unsigned tau;
  int jt;

  SVD Row(RowShared &sh, const FilterArgs &a, int row) : s(sh), pol(policy_of(a, row)), F(a.F0), F0(a.F0) {}
  // Rows out of range (F_FAR) are taken relative to their largest logit, and their bins are counted one
  // token at a time; differences so large that their weight is nothing are cut off.
  SVD void set(unsigned fl, float z, int q) {
    flags = fl;
    zmax = z;
    top_key = K::of(z);
    far = fl & F_FAR;
    Q = far ? 0 : q;
    O = octave_of(Q);
    rest = octave_of(Q - (BINS - 1));
    off = far ? (double)z : 0.0;
    inv64 = 1.0 / pol.c64;  // for guesses
    least = far ? -1e9 / pol.c64 : (double)lowest_of(pol.c64);
    by_p = pol.p < 1.0f;
  }
  SVD double arg(float z) const { return fmax((double)z - off, least); }
  SVD int bin_of(float z) const { return min(Q - quarter_of(arg(z), pol.c64), BINS - 1); }
  SVD Weight plain_weight(float z) const { return weight_of(arg(z), pol.c64, s.tab, rest); }
  SVD w64 in_units(const Weight &w) const { return shifted(w.m, F - W_BITS - (O - max(octave_of(w.q), rest))); }
  // The weight of a chunk's bin, of quarter octave q: as the row's weights are, and as its bin j adds them up.
  SVD w64 mass_of_chunk(int q, w64 x) const { return shifted(x & ((1ull << W_COUNT) - 1ull), F - W_BITS - (O - octave_of(q))); }
  SVD w64 mass_for_bin(int q, int j, w64 x) const { return shifted(x & ((1ull << W_COUNT) - 1ull), octave_of(q) - octave_of(Q - j)); }
  // The first key of bin j, tried near where it has to be.
  SVD unsigned first_of(int j) const {
    if (j >= BINS - 1) return K::lowest();
    auto in = [&](unsigned k) { return Q - quarter_of(arg(K::value(k)), pol.c64) <= j; };
    return near_key(K::of((float)((double)((Q - j) * 16) * inv64 + off)), in);
  }
  template <typename P>
  SVD unsigned near_key(unsigned g, P in) const {
    const unsigned lo = max(g, K::lowest() + 32u) - 32u, hi = min(lo + 63u, top_key);
    const unsigned long long b = __ballot(in(min(lo + (unsigned)lane_id(), hi)));
    if (lo < hi && b != 0 && !(b & 1)) return lo + (unsigned)__ffsll(b) - 1u;
    return first_key(K::lowest(), top_key, in);
  }
  SVD unsigned upper_of(int j) const { return j == 0 ? top_key : first_of(j - 1) - 1u; }
  SVD static w64 lane64(w64 v, int l) {
    return ((w64)(unsigned)__builtin_amdgcn_readlane((int)(unsigned)(v >> 32), l) << 32) | (unsigned)__builtin_amdgcn_readlane((int)(unsigned)v, l);
  }
  SVD unsigned count_in_front(int j) const { return (unsigned)__builtin_amdgcn_readlane((int)(pc + ((j & 1) ? c0 : 0u)), j >> 1); }
  SVD w64 mass_in_front(int j) const { return lane64(pm + ((j & 1) ? m0 : 0ull), j >> 1); }
  // The first bin up to and with which there are n tokens, or a weight of w; the last if none.
  SVD int bin_by_count(unsigned n) const {
    const unsigned long long b0 = __ballot(pc + c0 >= n), b1 = __ballot(pc + c0 + c1 >= n);
    return b1 == 0 ? BINS - 1 : 2 * (__ffsll(b1) - 1) + ((b0 >> (__ffsll(b1) - 1)) & 1 ? 0 : 1);
  }
  SVD int bin_by_mass(double w) const {
    const unsigned long long b0 = __ballot((double)(pm + m0) >= w), b1 = __ballot((double)(pm + m0 + m1) >= w);
    return b1 == 0 ? BINS - 1 : 2 * (__ffsll(b1) - 1) + ((b0 >> (__ffsll(b1) - 1)) & 1 ? 0 : 1);
  }
  SVD int bits_down(int j) const { return W_BITS + O - octave_of(Q - j); }  // of bin j's own units below the octave O
  // `own`: the bins are in units of their own, and F is yet to be chosen.
  SVD void prefixes(bool own) {
    const int lane = lane_id();
    m0 = s.mass[2 * lane];
    m1 = s.mass[2 * lane + 1];
    c0 = s.count[2 * lane];
    c1 = s.count[2 * lane + 1];
    if (own) {
      // the total in units of 2^(30 - F0), more than it is by 64 at most; F puts it below 2^61 units
      const int d0 = bits_down(2 * lane), d1 = bits_down(2 * lane + 1);
      const unsigned part = (unsigned)((shifted(m0, F0 - d0) + shifted(m1, F0 - d1)) >> 30);
      F = F0 - 1 + __clz(__builtin_amdgcn_readlane((int)scan_add_u(part), WAVE - 1) + WAVE);
      m0 = shifted(m0, F - d0);
      m1 = shifted(m1, F - d1);
    }
    const w64 im = wave_incl(m0 + m1);
    const unsigned ic = scan_add_u(c0 + c1);
    pm = im - m0 - m1;
    pc = ic - c0 - c1;
    n_all = (unsigned)__builtin_amdgcn_readlane((int)ic, WAVE - 1);
    kept = lane64(im, WAVE - 1);
  }
  // Once the bins are known: the cuts.  Returns the first step.
  SVD int plan() {
    prefixes(true);
    tau = K::lowest();
    jt = BINS - 1;
    by_k = pol.k > 0 && (unsigned)pol.k < n_all;
    if (pol.m > 0.0f) {
      const double xm = arg(zmax) * pol.c64;
      tau = near_key(K::of(fminf((float)((double)zmax + 64.0 * (double)log2f(pol.m) / pol.c64), zmax)), [&](unsigned k) {
        const double d = (arg(K::value(k)) * pol.c64 - xm) * (1.0 / 64.0);
        return d > -200.0 && pow2(d) >= (double)pol.m;
      });
      jt = bin_of(K::value(tau));
    }
    by_m = tau > K::lowest();
    if (by_k) {
      const int j = bin_by_count((unsigned)pol.k);
      if (j > jt) by_k = false;  // min-p cuts off more
      else jt = j;
    } else if (by_p && !by_m) {
      jt = bin_by_mass((double)pol.p * (double)kept);
    }
    cuts = by_k || by_m || by_p;
    whole = count_in_front(jt) + s.count[jt] <= (unsigned)LIST;
    return by_k ? COUNT : by_m ? (by_p ? REST : DRAWN) : by_p ? MASS : DRAWN;
  }
  // Where a step looks.
  SVD void begin(int step, int &bin, w64 &above, double &target, unsigned &lo, unsigned &hi) {
    if (step == COUNT) {
      bin = bin_by_count((unsigned)pol.k);
      above = count_in_front(bin);
      target = (double)pol.k;
      lo = first_of(bin);
    } else if (step == MASS) {
      target = (double)pol.p * (double)kept;
      bin = min(bin_by_mass(target), by_k || by_m ? jt : BINS - 1);
      above = mass_in_front(bin);
      lo = max(tau, first_of(bin));
    } else if (step == REST || step == DRAWN) {
      bin = jt;
      lo = tau;
    }
    hi = step == ALL || (step == DRAWN && far) ? top_key : upper_of(bin);
  }
};

// ---------------------------------------------------------------- plan

constexpr int PLAN_NT = 512;

template <typename T, bool DRAW>
__global__ __launch_bounds__(PLAN_NT) void k_filter_plan(const FilterArgs a) {
  typedef Key<T> K;
  constexpr int E = Fmt<T>::VEC, STEP = PLAN_NT / BINS, AHEAD = 8;
  __shared__ RowShared s;
  __shared__ int s_first;
  const int tid = threadIdx.x;
  const int row = blockIdx.x;
  const ChunkSum *sums = a.sums + (size_t)row * a.chunks;
  // thread: one bin of every fourth chunk, eight of them on their way together
  const int b = tid % BINS;
  w64 x[AHEAD];
  int q[AHEAD];
  auto load = [&](int c0) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = min(c0 + k * STEP, a.chunks - 1);
      x[k] = sums[i].bin[b];
      q[k] = sums[i].q - b;
    }
  };
  load(tid / BINS);
  Row<T> R(s, a, row);
  RowPlan &p = a.plans[row];
  const float u = DRAW && a.u ? a.u[row] : NAN;

  if (tid < BINS) {
    s.mass[tid] = 0;
    s.count[tid] = 0;
  }
  if (tid == 0) {
    s.flags = s.top = 0;
    s.q = (int)0x80000000;
    s_first = 0x7fffffff;
  }
  __syncthreads();
  for (int i = tid; i < a.chunks; i += PLAN_NT) {
    const unsigned f = sums[i].flags, top = sums[i].top;
    const int qi = sums[i].q;
    if (f) atomicOr(&s.flags, f);
    if (f & F_FINITE) {
      atomicMax(&s.top, top);
      atomicMax(&s.q, qi);
    }
  }
  __syncthreads();
  // A row with a larger logit than this has none that weighs something among those that the scan took
  // higher, 3 * 10^5 octaves below.
  const float zmax = key2f(s.top);
  R.set(s.flags | ((double)zmax * R.pol.c64 < -0.98e9 ? (unsigned)F_FAR : 0u), zmax, s.q);
  int code = 0;
  if (!R.pol.ok) code = SV_ROW_BAD_POLICY;
  else if ((R.flags & F_ODD) || !(R.flags & F_FINITE)) code = SV_ROW_BAD_LOGITS;
  else if (DRAW && R.pol.t > 0.0f && !(u >= 0.0f && u < 1.0f)) code = SV_ROW_BAD_UNIFORM;
  if (tid == 0) {
    a.row_status[row] = code;
    p.list_lo = 1;
    p.list_hi = 0;
    p.step = END;  // unless there is more to do
    if (code != 0) {
      if (DRAW) a.tokens[row] = -1;
      else a.cut[row] = make_uint2(0u, (unsigned)-2);
    }
  }
  if (code != 0) return;
  if (R.pol.t == 0.0f) {  // greedy: the first of the largest, in the first chunk that has it
    const RowBlocks<T> r(a.logits, row, a.V);
    for (int i = tid; i < a.chunks; i += PLAN_NT)
      if ((sums[i].flags & F_FINITE) && key2f(sums[i].top) == R.zmax) atomicMin(&s_first, i);
    __syncthreads();
    const int c = s_first;
    __syncthreads();
    if (tid == 0) s_first = 0x7fffffff;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < FC / E; k += PLAN_NT) {
      const int i = c * (FC / E) + k + tid;
      float z[E];
      r.unpack(r.load(i), i, z);
#pragma unroll
      for (int e = E - 1; e >= 0; --e)
        if (z[e] == R.zmax) atomicMin(&s_first, r.index(i, e));
    }
    __syncthreads();
    if (tid == 0) {
      if (DRAW) a.tokens[row] = s_first;
      else a.cut[row] = make_uint2(R.top_key, (unsigned)s_first);
    }
    return;
  }
  int step = ALL, bin = 0;
  w64 above = 0;
  double target = 0.0;
  unsigned lo = K::lowest(), hi = R.top_key, list_lo = 1, list_hi = 0;
  if (!R.far) {
    for (int c0 = tid / BINS;;) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (c0 + k * STEP < a.chunks && x[k] != 0) {
          const int j = min(R.Q - q[k], BINS - 1);
          atomicAdd(&s.mass[j], R.mass_for_bin(q[k], j, x[k]));
          atomicAdd(&s.count[j], (unsigned)(x[k] >> W_COUNT));
        }
      c0 += AHEAD * STEP;
      if (c0 >= a.chunks) break;
      load(c0);
    }
    __syncthreads();
    step = R.plan();
    if (step != DRAWN || (DRAW && R.cuts)) {
      R.begin(step, bin, above, target, lo, hi);
      // all that is to come, if it fits; else this step's range, if that does
      if (R.whole) {
        list_lo = R.first_of(R.jt);
        list_hi = R.top_key;
      } else if (s.count[bin] <= (unsigned)LIST) {
        list_lo = lo;
        list_hi = hi;
      }
    }
  }
  for (int i = tid; i < BINS; i += PLAN_NT) {
    p.mass[i] = shifted(s.mass[i], R.F - R.bits_down(i));
    p.count[i] = s.count[i];
  }
  if (tid == 0) {
    p.above = above;
    p.target = target;
    p.q = R.Q;
    p.F = R.F;
    p.step = step;
    p.bin = bin;
    p.jt = R.far ? 0 : R.jt;
    p.flags = R.flags;
    p.tau = R.far ? K::lowest() : R.tau;
    p.lo = lo;
    p.hi = hi;
    p.list_lo = list_lo;
    p.list_hi = list_hi;
    p.zmax = R.zmax;
    p.by_k = !R.far && R.by_k;
    p.by_m = !R.far && R.by_m;
    p.cuts = !R.far && R.cuts;
    p.whole = !R.far && R.whole;
  }
}

// ---------------------------------------------------------------- gather

// As many workgroups as the scan had look through the row's chunks at once (one a row, in
// k_filter_pick, 64 rows: 11 of its 35 us).  Their places on the row's list are given out a workgroup
// at a time (a wave at a time, 320 rows: 28 us for 21).
template <typename T, bool DRAW>
__global__ __launch_bounds__(NT) void k_filter_gather(const FilterArgs a) {
  typedef Key<T> K;
  constexpr int E = Fmt<T>::VEC, NV = FPT / E;
  __shared__ w64 s_over[NW];
  __shared__ int s_n[NW], s_at;
  const int tid = threadIdx.x, lane = lane_id(), wid = tid / WAVE;
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), c = (int)(blockIdx.x % (unsigned)a.chunks);
  const RowPlan &p = a.plans[row];
  const unsigned list_lo = p.list_lo, list_hi = p.list_hi;
  const bool some = list_lo <= list_hi;
  const RowBlocks<T> r(a.logits, row, a.V);
  u32x4 w[NV];
  if (some) {
#pragma unroll
    for (int k = 0; k < NV; ++k) w[k] = r.load(c * (FC / E) + k * NT + tid);
  }
  const int step = p.step;
  if (step == END) return;
  if (DRAW && step != ALL) {  // the chunk's weight in the bins above the lowest threshold's
    const ChunkSum &cs = a.sums[(size_t)row * a.chunks + c];
    w64 over = 0;
    if (tid < BINS) {
      const w64 x = cs.bin[tid];
      const int q = cs.q - tid, Q = p.q;
      if (!p.cuts || Q - q < p.jt) over = shifted(x & ((1ull << W_COUNT) - 1ull), p.F - W_BITS - (octave_of(Q) - octave_of(q)));
    }
    over = wave_total64(over);
    if (lane == 0) s_over[wid] = over;
    __syncthreads();
    if (tid == 0) a.over[(size_t)row * a.chunks + c] = s_over[0] + s_over[1];
  }
  if (!some) return;
  const float z_lo = K::value(list_lo), z_hi = K::value(list_hi);
  float z[NV][E];
  int n = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    r.unpack(w[k], c * (FC / E) + k * NT + tid, z[k]);
#pragma unroll
    for (int e = 0; e < E; ++e) n += __popcll(__ballot(z[k][e] >= z_lo && z[k][e] <= z_hi));
  }
  if (lane == 0) s_n[wid] = n;
  __syncthreads();
  if (tid == 0) {  // one addition a workgroup
    int all = 0;
#pragma unroll
    for (int v = 0; v < NW; ++v) all += s_n[v];
    s_at = all ? (int)atomicAdd(&a.n_list[row], (unsigned)all) : 0;
  }
  __syncthreads();
  if (n == 0) return;
  int o = s_at;
#pragma unroll
  for (int v = 0; v < NW; ++v) o += v < wid ? s_n[v] : 0;
  o = __builtin_amdgcn_readfirstlane(o);
  uint2 *list = a.list + (size_t)row * a.cap;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = z[k][e] >= z_lo && z[k][e] <= z_hi;
      const unsigned long long b = __ballot(in);
      const int at = o + __builtin_amdgcn_mbcnt_hi((unsigned)(b >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)b, 0u));
      if (in && at < a.cap) list[at] = make_uint2(K::of(z[k][e]), (unsigned)((c * (FC / E) + k * NT + tid) * E + e));
      o += __popcll(b);
    }
}

// ---------------------------------------------------------------- pick

constexpr int PICK_NT = 512;  // threads; two workgroups and their lists fit a CU

struct PickShared {
  RowShared row;
  w64 hist[256], total, above;
  w64 wave[PICK_NT / WAVE];
  unsigned list_key[LIST];
  int list_at[LIST];
  int n_list, found;
  unsigned key;
};

// A row is one workgroup's, and its steps follow one another: what bounds it is latency.  Each step
// looks at the tokens with keys of a range: those that k_filter_gather put on the list, or, where a
// later threshold lies elsewhere or a bin holds more than a list, those that a pass over the row
// finds.
template <typename T, bool DRAW>
__global__ __launch_bounds__(PICK_NT) __attribute__((amdgpu_waves_per_eu(4))) void k_filter_pick(const FilterArgs a) {
  typedef Key<T> K;
  constexpr int E = Fmt<T>::VEC, PW = PICK_NT / WAVE;
  __shared__ PickShared s;
  extern __shared__ w64 s_chunk[];  // [chunks] kept weight
  const int tid = threadIdx.x, lane = lane_id(), wid = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int row = blockIdx.x;
  const RowPlan &p = a.plans[row];
  int step = p.step;
  if (step == END) return;
  const RowBlocks<T> r(a.logits, row, a.V);
  const ChunkSum *sums = a.sums + (size_t)row * a.chunks;
  Row<T> R(s.row, a, row);
  R.set(p.flags, p.zmax, p.q);
  int bin = p.bin;
  w64 above = p.above;
  double target = p.target;
  unsigned lo = p.lo, hi = p.hi, list_lo = p.list_lo, list_hi = p.list_hi;  // the list has all tokens of its keys
  R.tau = p.tau;
  R.jt = p.jt;
  R.by_k = p.by_k;
  R.by_m = p.by_m;
  R.cuts = p.cuts;
  R.whole = p.whole;
  const int over_jt = R.jt;  // the bin that a.over goes by
  unsigned here = ~0u;       // the tokens of this step's range, at most
  unsigned least = 0;        // no token below this key is kept, and what is kept fits the list
  if (tid < BINS) {
    s.row.mass[tid] = p.mass[tid];
    s.row.count[tid] = p.count[tid];
  }
  if (list_lo <= list_hi) {
    const int n = min((int)a.n_list[row], a.cap);
    const uint2 *list = a.list + (size_t)row * a.cap;
    for (int i = tid; i < n; i += PICK_NT) {
      const uint2 x = list[i];
      s.list_key[i] = x.x;
      s.list_at[i] = (int)x.y;
    }
    if (tid == 0) s.n_list = n;
  }
  powers(s.row.tab);
  __syncthreads();
  R.F = __builtin_amdgcn_readfirstlane(p.F);
  R.prefixes(false);
  bool begin = R.far || step == DRAWN;  // of a step: the gather has begun the others
  for (;;) {
    if (begin) {
      begin = false;
      if (step == DRAWN && !DRAW) step = END;
      if (step == DRAWN) {
        const bool ready = !R.far && R.jt == over_jt;
        for (int c = tid; c < a.chunks; c += PICK_NT) s_chunk[c] = ready ? a.over[(size_t)row * a.chunks + c] : 0ull;
        if (!R.cuts && !R.far) step = END;  // the bins are enough
      }
      if (step == END) break;
      R.begin(step, bin, above, target, lo, hi);
      here = ~0u;
    }
    if (here == ~0u && !R.far) here = s.row.count[bin];
    const unsigned span = hi - lo;
    const int bits = 32 - __clz((int)(span | 1u)), sh = bits > 8 ? bits - 8 : 0;
    for (int i = tid; i < 256; i += PICK_NT) s.hist[i] = 0;
    if (tid == 0) s.total = 0;

    w64 part = 0;
    auto take = [&](unsigned k, int at) {  // a token's key, and its place in the row
      if (k < lo || k > hi) return;
      if (step == COUNT) {
        atomicAdd(&s.hist[(k - lo) >> sh], 1ull);
      } else {
        const Weight x = R.plain_weight(K::value(k));
        const w64 w = R.in_units(x);
        if (step == MASS) {
          atomicAdd(&s.hist[(k - lo) >> sh], w);
        } else if (step == REST) {
          part += w;
        } else if (step == DRAWN) {
          atomicAdd(&s_chunk[at / FC], w);
        } else {
          const int j = min(R.Q - x.q, BINS - 1);
          atomicAdd(&s.row.mass[j], x.m);
          atomicAdd(&s.row.count[j], 1u);
        }
      }
    };
    bool direct = false;
    if (lo < list_lo || hi > list_hi) {  // gather
      // all that is to come, if it fits; else this step's range, without a list where that does not fit
      const unsigned g_lo = R.whole && step != ALL ? max(R.first_of(R.jt), least) : lo, g_hi = R.whole && step != ALL ? R.top_key : hi;
      direct = step == ALL || (!R.whole && here > (unsigned)LIST);
      const float z_lo = K::value(g_lo), z_hi = K::value(g_hi);
      __syncthreads();
      if (tid == 0) s.n_list = 0;
      __syncthreads();
      auto add = [&](const u32x4 &w, int i) {
        float z[E];
        r.unpack(w, i, z);
        unsigned long long b[E];
        int n = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          b[e] = __ballot(z[e] >= z_lo && z[e] <= z_hi);
          n += __popcll(b[e]);
        }
        if (n == 0) return;
        int o = 0;
        if (lane == 0) o = atomicAdd(&s.n_list, n);
        o = __builtin_amdgcn_readfirstlane(o);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int at = o + __builtin_amdgcn_mbcnt_hi((unsigned)(b[e] >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)b[e], 0u));
          if (((b[e] >> lane) & 1) && at < LIST) {
            s.list_key[at] = K::of(z[e]);
            s.list_at[at] = i * E + e;
          }
          o += __popcll(b[e]);
        }
      };
      constexpr int AHEAD = 8;
      for (int i0 = tid; i0 - tid < r.n; i0 += AHEAD * PICK_NT) {
        u32x4 w[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) w[k] = r.load(i0 + k * PICK_NT);
        if (!direct) {
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) add(w[k], i0 + k * PICK_NT);
          continue;
        }
#pragma unroll 1
        for (int k = 0; k < AHEAD; ++k) {  // one stretch of code for all of them, w[0] being the next
          const int i = i0 + k * PICK_NT;
          float z[E];
          r.unpack(w[0], i, z);
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (z[e] >= z_lo && z[e] <= z_hi) take(K::of(z[e]), i * E + e);
#pragma unroll
          for (int j = 0; j + 1 < AHEAD; ++j) w[j] = w[j + 1];
        }
      }
      list_lo = direct ? 1u : g_lo;
      list_hi = direct ? 0u : g_hi;
    }
    __syncthreads();
    if (!direct)
      for (int i = tid, n = min(s.n_list, LIST); i < n; i += PICK_NT) take(s.list_key[i], s.list_at[i]);
    if (part) atomicAdd(&s.total, part);
    __syncthreads();

    if (step == ALL) {
      step = R.plan();
      begin = true;
    } else if (step == REST) {
      R.kept = s.total + R.mass_in_front(R.jt);
      __syncthreads();
      step = R.by_p ? MASS : DRAWN;
      begin = true;
    } else if (step == DRAWN) {
      break;
    } else {
      // The largest key t of the range with above + W(keys in [t, hi]) >= target, by eight bits of the
      // key at a time: lane l owns bins 255 - 4 l down to 252 - 4 l.
      if (wid == 0) {
        w64 h[4], t = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          h[q] = s.hist[255 - 4 * lane - q];
          t += h[q];
        }
        w64 run = above + wave_incl(t) - t;
        int pick = -1, some = -1;
        w64 over = 0, upto = 0, below_some = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (h[q] != 0) {
            some = 255 - 4 * lane - q;
            below_some = run;
          }
          if (pick < 0 && h[q] != 0 && (double)(run + h[q]) >= target) {
            pick = 255 - 4 * lane - q;
            over = run;
            upto = run + h[q];
          }
          run += h[q];
        }
        const unsigned long long b = __ballot(pick >= 0), any = __ballot(some >= 0);
        const int l = b != 0 ? __ffsll(b) - 1 : any != 0 ? 63 - __clzll((long long)any) : 63;
        if (lane == l) {  // where the target is all there is, up to its rounding: the lowest
          s.key = (unsigned)(b != 0 ? pick : max(some, 0));
          s.above = b != 0 ? over : below_some;
          s.total = b != 0 ? upto : run;
        }
      }
      __syncthreads();
      const unsigned pick = s.key;
      above = s.above;
      const w64 upto = s.total;
      if (step == COUNT) here = (unsigned)s.hist[pick];
      __syncthreads();
      lo += pick << sh;
      if (hi - lo >= 1u << sh) hi = lo + ((1u << sh) - 1u);
      if (sh == 0) {
        begin = true;
        if (step == COUNT) {
          R.tau = max(R.tau, lo);
          R.jt = R.bin_of(K::value(R.tau));
          if (!R.whole && upto <= (unsigned)LIST) {  // of the tokens from tau up
            R.whole = true;
            least = R.tau;
          }
          step = R.by_p ? REST : DRAWN;
        } else {
          R.tau = lo;
          R.jt = bin;
          R.kept = upto;
          step = DRAWN;
        }
      }
    }
  }
  if (!DRAW) {
    if (tid == 0) a.cut[row] = make_uint2(R.tau, (unsigned)-1);
    return;
  }

  // ---- the chunks' kept weights: bins above tau's from the scan, where the gather went by another
  __syncthreads();
  if (!R.far && R.jt != over_jt)
    for (int i = tid; i < a.chunks * BINS; i += PICK_NT) {
      const ChunkSum &cs = sums[i / BINS];
      const w64 x = cs.bin[i % BINS];
      const int q = cs.q - i % BINS;
      if (x == 0 || (R.cuts && min(R.Q - q, BINS - 1) >= R.jt)) continue;
      const w64 m = R.mass_of_chunk(q, x);
      if (m) atomicAdd(&s_chunk[i / BINS], m);
    }
  __syncthreads();
  const float u = a.u[row];
  if (wid == 0) {  // the first chunk whose cumulative weight passes the target
    w64 total = 0;
    for (int c0 = 0; c0 < a.chunks; c0 += WAVE) total += wave_total64(c0 + lane < a.chunks ? s_chunk[c0 + lane] : 0ull);
    const double t = (double)u * (double)total;
    w64 run = 0, before = 0, fb = 0;
    int pick = -1, fallback = 0;
    for (int c0 = 0; c0 < a.chunks && pick < 0; c0 += WAVE) {
      const w64 w = c0 + lane < a.chunks ? s_chunk[c0 + lane] : 0ull, inc = wave_incl(w);
      const unsigned long long b = __ballot(w != 0 && (double)(run + inc) > t), some = __ballot(w != 0);
      if (b != 0) {
        const int l = __ffsll(b) - 1;
        pick = c0 + l;
        before = run + R.lane64(inc - w, l);
      } else if (some != 0) {
        const int l = 63 - __clzll((long long)some);
        fallback = c0 + l;
        fb = run + R.lane64(inc - w, l);
      }
      run += R.lane64(inc, WAVE - 1);
    }
    if (lane == 0) {
      s.n_list = pick >= 0 ? pick : fallback;
      s.above = pick >= 0 ? before : fb;
      s.total = total;
      s.found = -1;
    }
  }
  __syncthreads();
  const int c = s.n_list;
  const double goal = (double)u * (double)s.total;
  w64 base = s.above;
  // ---- the token: the chunk's kept weights in index order
  constexpr int TURNS = FC / E / PICK_NT;
  u32x4 raw[TURNS];
#pragma unroll
  for (int k = 0; k < TURNS; ++k) raw[k] = r.load((c * TURNS + k) * PICK_NT + tid);
#pragma unroll
  for (int k = 0; k < TURNS; ++k) {
    const int i = (c * TURNS + k) * PICK_NT + tid;
    w64 w[E], sum = 0;
    float z[E];
    r.unpack(raw[k], i, z);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      w[e] = i < r.n && z[e] > -INFINITY && K::of(z[e]) >= R.tau ? R.in_units(R.plain_weight(z[e])) : 0ull;
      sum += w[e];
    }
    const w64 inc = wave_incl(sum);
    if (lane == WAVE - 1) s.wave[wid] = inc;
    if (tid == 0) s.key = 0x7fffffffu;
    __syncthreads();
    w64 run = base, all = 0;
    for (int v = 0; v < PW; ++v) {
      if (v < wid) run += s.wave[v];
      all += s.wave[v];
    }
    run += inc - sum;
    int last = -1, pick = -1;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      run += w[e];
      if (w[e] != 0) {
        last = r.index(i, e);
        if (pick < 0 && (double)run > goal) pick = last;
      }
    }
    if (pick >= 0) atomicMin(&s.key, (unsigned)pick);
    if (last >= 0) atomicMax(&s.found, last);  // in case rounding leaves none
    base += all;
    __syncthreads();
    if (s.key != 0x7fffffffu) break;
    __syncthreads();
  }
  if (tid == 0) a.tokens[row] = s.key != 0x7fffffffu ? (int)s.key : s.found;
}

// ---------------------------------------------------------------- write

template <typename T>
__global__ __launch_bounds__(NT) void k_filter_write(const FilterArgs a) {
  typedef Key<T> K;
  constexpr int E = Fmt<T>::VEC, NV = FPT / E;
  const int tid = threadIdx.x;
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), c = (int)(blockIdx.x % (unsigned)a.chunks);
  const RowBlocks<T> r(a.logits, row, a.V);
  T *out = static_cast<T *>(a.out) + (size_t)row * a.V;
  const uint2 cut = a.cut[row];
  const int only = (int)cut.y;
  constexpr T MINUS = sizeof(T) == 2 ? (T)0xff80u : (T)(-__builtin_inff());
  const bool same = (((uintptr_t)out ^ ((uintptr_t)r.p + (uintptr_t)r.lead * sizeof(T))) & 15) == 0;  // blocks of both coincide
  u32x4 w[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) w[k] = r.load(c * (FC / E) + k * NT + tid);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = c * (FC / E) + k * NT + tid;
    if (i >= r.n) break;
    float z[E];
    Fmt<T>::unpack(w[k], z);
    T e_[E];
    __builtin_memcpy(e_, &w[k], 16);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool keep = only >= 0 ? r.index(i, e) == only : K::of(z[e]) >= cut.x;
      if (only == -2) {
        if constexpr (sizeof(T) == 2) e_[e] = (T)0x7fc0u;
        else e_[e] = (T)NAN;
      } else if (!keep) {
        e_[e] = MINUS;
      }
    }
    if (same && i > 0 && i < r.n - 1) {
      u32x4 o;
      __builtin_memcpy(&o, e_, 16);
      *reinterpret_cast<u32x4 *>(out + r.index(i, 0)) = o;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((unsigned)r.index(i, e) < (unsigned)a.V) out[r.index(i, e)] = e_[e];
    }
  }
}

}  // namespace sv

// ======================================================================== host side

namespace {

using namespace sv;
using sv_host::align256;
using sv_host::Launcher;

struct FilterPlan {
  int chunks, cap;
  size_t sums, plans, over, n_list, list, cut, total;
};
bool filter_plan(int32_t rows, int32_t V, int esz, FilterPlan &p) {
  if (rows < 1 || V < 1 || V > SV_FILTER_MAX_V) return false;
  const int E = 16 / esz;
  p.chunks = (int)(((long long)V + E - 1 + FC - 1) / FC);  // a row may begin anywhere in a block
  if ((long long)rows * p.chunks > 0xffffffffLL / NT || rows > 0xffffffffLL / PICK_NT) return false;
  size_t o = 0;
  p.sums = o; o = align256(o + (size_t)rows * p.chunks * sizeof(ChunkSum));
  p.plans = o; o = align256(o + (size_t)rows * sizeof(RowPlan));
  p.over = o; o = align256(o + (size_t)rows * p.chunks * 8);
  p.n_list = o; o = align256(o + (size_t)rows * 4);
  p.cap = V < LIST ? V : LIST;
  p.list = o; o = align256(o + (size_t)rows * p.cap * 8);
  p.cut = o; o = align256(o + (size_t)rows * 8);
  p.total = o;
  return true;
}

sv_status filter_run(bool draw, const void *logits, sv_dtype dt, const float *u, int32_t rows, int32_t V, const sv_policy *pol,
                     int32_t *tokens, void *out, int32_t *status, void *ws, size_t ws_bytes, void *stream, void *const *ev,
                     int32_t nev, int32_t *nl) {
  if (nl) *nl = 0;
  if (dt != SV_F32 && dt != SV_BF16) return SV_ERR_DTYPE;
  const int esz = dt == SV_BF16 ? 2 : 4;
  FilterPlan p;
  if (!filter_plan(rows, V, esz, p)) return SV_ERR_SHAPE;
  if (!pol) return SV_ERR_NULL;
  if (!pol->temperatures && !(pol->temperature >= 0.0f && pol->temperature <= __FLT_MAX__)) return SV_ERR_TEMPERATURE;
  if ((!pol->top_ps && !(pol->top_p > 0.0f && pol->top_p <= 1.0f)) || (!pol->min_ps && !(pol->min_p >= 0.0f && pol->min_p <= 1.0f)))
    return SV_ERR_PARAM;
  const bool greedy = !pol->temperatures && pol->temperature == 0.0f;
  if (!logits || !status || !ws || (draw ? !tokens || (!u && !greedy) : !out)) return SV_ERR_NULL;
  if (((uintptr_t)logits | (uintptr_t)out) & (unsigned)(esz - 1)) return SV_ERR_ALIGN;
  const uintptr_t in = (uintptr_t)logits, to = (uintptr_t)out, size = (uintptr_t)rows * (uintptr_t)V * esz;
  if (!draw && in != to && in < to + size && to < in + size) return SV_ERR_PARAM;
  if (ws_bytes < p.total || ((uintptr_t)ws & 255)) return SV_ERR_WORKSPACE;
  // Several kernels read the logits and what is set for each row, and write for each row while others
  // still read: what is written lies apart from all that is read, and from what else is written (rows
  // over logits have been looked at above).
  struct Range {
    const void *p;
    uintptr_t n;
  };
  const uintptr_t ints = (uintptr_t)rows * 4;
  const Range read[] = {{logits, size}, {u, ints}, {pol->temperatures, ints}, {pol->top_ks, ints}, {pol->top_ps, ints}, {pol->min_ps, ints}};
  const Range written[] = {{status, ints}, {tokens, ints}, {out, size}};
  auto meet = [](const Range &x, const Range &y) {
    return x.p && y.p && (uintptr_t)x.p < (uintptr_t)y.p + y.n && (uintptr_t)y.p < (uintptr_t)x.p + x.n;
  };
  for (const Range &w : written)
    for (const Range &r : read)
      if (meet(w, r) && !(&w == &written[2] && &r == &read[0])) return SV_ERR_PARAM;
  if (meet(written[0], written[1]) || meet(written[0], written[2])) return SV_ERR_PARAM;
  char *base = static_cast<char *>(ws);
  FilterArgs a = {};
  a.logits = logits;
  a.u = u;
  a.rows = rows;
  a.V = V;
  a.chunks = p.chunks;
  // a row's weights are at most 2.02 each
  int bits = 0;
  while ((1LL << bits) < V) ++bits;
  a.F0 = 60 - bits;
  a.policy = *pol;
  a.sums = (ChunkSum *)(base + p.sums);
  a.plans = (RowPlan *)(base + p.plans);
  a.over = (w64 *)(base + p.over);
  a.n_list = (unsigned *)(base + p.n_list);
  a.list = (uint2 *)(base + p.list);
  a.cap = p.cap;
  a.cut = (uint2 *)(base + p.cut);
  a.tokens = tokens;
  a.row_status = status;
  a.out = out;
  void *args[] = {&a};
  Launcher L{(hipStream_t)stream, ev, nev};
  const unsigned grid = (unsigned)((long long)rows * p.chunks);
  L.go(esz == 2 ? (const void *)&k_filter_scan<uint16_t> : (const void *)&k_filter_scan<float>, grid, args);
  auto go = [&](const void *h, const void *f, unsigned n) { L.go(esz == 2 ? h : f, n, args); };
  L.block = PLAN_NT;
  if (draw) go((const void *)&k_filter_plan<uint16_t, true>, (const void *)&k_filter_plan<float, true>, (unsigned)rows);
  else go((const void *)&k_filter_plan<uint16_t, false>, (const void *)&k_filter_plan<float, false>, (unsigned)rows);
  L.block = NT;
  if (draw) go((const void *)&k_filter_gather<uint16_t, true>, (const void *)&k_filter_gather<float, true>, grid);
  else go((const void *)&k_filter_gather<uint16_t, false>, (const void *)&k_filter_gather<float, false>, grid);
  L.block = PICK_NT;
  L.lds = draw ? (unsigned)p.chunks * 8 : 0;
  if (draw) go((const void *)&k_filter_pick<uint16_t, true>, (const void *)&k_filter_pick<float, true>, (unsigned)rows);
  else go((const void *)&k_filter_pick<uint16_t, false>, (const void *)&k_filter_pick<float, false>, (unsigned)rows);
  if (!draw) {
    L.block = NT;
    L.lds = 0;
    go((const void *)&k_filter_write<uint16_t>, (const void *)&k_filter_write<float>, grid);
  }
  if (nl) *nl = L.n;
  return L.e == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

}  // namespace

extern "C" {

size_t sv_filter_workspace_bytes(int32_t rows, int32_t V, sv_dtype dtype) {
  FilterPlan p;
  if ((dtype != SV_F32 && dtype != SV_BF16) || !filter_plan(rows, V, dtype == SV_BF16 ? 2 : 4, p)) return 256;
  return p.total;
}

sv_status spec_sample_filtered(const void *logits, sv_dtype dtype, const float *u, int32_t B, int32_t V, const sv_policy *policy,
                               int32_t *tokens, int32_t *row_status, void *workspace, size_t workspace_bytes, void *stream,
                               void *const *events, int32_t n_events, int32_t *n_launched) {
  return filter_run(true, logits, dtype, u, B, V, policy, tokens, nullptr, row_status, workspace, workspace_bytes, stream, events, n_events,
                    n_launched);
}

sv_status spec_filter_logits(const void *logits, sv_dtype dtype, int32_t rows, int32_t V, const sv_policy *policy, void *out,
                             int32_t *row_status, void *workspace, size_t workspace_bytes, void *stream, void *const *events,
                             int32_t n_events, int32_t *n_launched) {
  return filter_run(false, logits, dtype, nullptr, rows, V, policy, nullptr, out, row_status, workspace, workspace_bytes, stream, events,
                    n_events, n_launched);
}

const char *sv_filter_launch_plan(int32_t draw) { return draw ? "k_filter_scan;k_filter_plan;k_filter_gather;k_filter_pick" : "k_filter_scan;k_filter_plan;k_filter_gather;k_filter_pick;k_filter_write"; }

}  // extern "C"
