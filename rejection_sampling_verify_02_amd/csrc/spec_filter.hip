// spec_filter.hip -- sampling and filtered logits under temperature, top-k, min-p and top-p
// (include/spec_filter.h).
//
// Each of the three cuts keeps the logits at or above some value, so a row's policy comes down to
// one threshold, found by weighted selection: the largest value t with W(z >= t) >= a target,
// where W counts tokens (top-k) or adds their weights (top-p).  Weights are 2^x for
// x = z log2(e) / T.  They are fixed-point numbers of 64 bits relative to a power of two near the
// row's largest, so that sums do not depend on their order, and they are computed to about 1e-13
// in 64 bits: a vocabulary of 10^5 tokens of probability 10^-6 leaves cumulative weights no room
// for float32's rounding.
//
//   k_filter_scan    a chunk of a row a workgroup, one read of the logits: the chunk's largest, and
//                    counts and weights by octave of the weight (ceil(x), the same for every chunk)
//   k_filter_pick    a row a workgroup: adds the chunks' octaves, finds the octaves in which the
//                    thresholds lie, and selects inside them.  Where all tokens from the lowest of
//                    these octaves up fit a list, they are gathered into LDS in one pass over the
//                    row (which comes from the L2 now) and everything else happens there; otherwise
//                    each step is a pass over the row.  Then the draw: the chunk whose cumulative
//                    kept weight passes u times the total, and the token in it.
//   k_filter_write   the row again, with -inf below the threshold

#include "sv_common.h"

#include "spec_filter.h"

namespace sv {

typedef unsigned long long w64;

constexpr int FC = 8192;        // logits of a chunk, counted from the 16-byte block that the row begins in
constexpr int OCT = 32;         // octaves of weight kept apart; the last takes all that is smaller
constexpr int PICK_NT = 1024;   // threads of k_filter_pick
constexpr int LIST = 8192;      // tokens of its list
constexpr int FPT = FC / NT;    // logits of a thread of k_filter_scan

enum { F_ODD = 1, F_FINITE = 2, F_FAR = 4 };  // a chunk's flags: NaN or +inf, some finite logit, weights out of range

struct ChunkSum {
  double x;        // a whole number, at least every z log2(e) / T of the chunk's finite logits
  unsigned top;    // the largest finite logit's key
  unsigned flags;
  w64 mass[OCT];   // relative to 2^x: octave j holds weights in (2^(x - j - 1), 2^(x - j)]
  unsigned count[OCT];
};

struct FilterArgs {
  const void *logits;
  const float *u;
  int rows, V, chunks, F;  // F: bits of the fixed point behind the binary point
  sv_policy policy;
  ChunkSum *sums;          // [rows][chunks]
  uint2 *cut;              // [rows] filter: the threshold's key and the one token kept (-1: all above; -2: a code)
  int32_t *tokens, *row_status;
  void *out;
};

struct Policy {
  double c2;   // log2(e) / T
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
  r.c2 = r.ok && r.t > 0.0f ? 1.4426950408889634074 / (double)r.t : 0.0;
  return r;
}

// 2^d for d at most about 0, d > -1000: the Taylor series of 2^f on [-1/2, 1/2], whose next term
// is under 10^-14.
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
// 2^d with F bits behind the binary point (F at most 50): adding 2^52 leaves the rounded whole number in the
// mantissa.
SVD w64 mass_of(double d, int F) {
  if (d < -64.0) return 0;
  return (w64)__double_as_longlong(ldexp(pow2(d), F) + 4503599627370496.0) & 0xfffffffffffffull;
}

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

constexpr int COPIES = 16;  // of a workgroup's octaves, so that a wave's lanes seldom add to one place

template <typename T>
__global__ __launch_bounds__(NT) void k_filter_scan(const FilterArgs a) {
  constexpr int E = Fmt<T>::VEC, NV = FPT / E;
  __shared__ w64 s_mass[OCT * COPIES];
  __shared__ unsigned s_count[OCT * COPIES];
  __shared__ unsigned s_top[NW], s_flags[NW];
  const int tid = threadIdx.x, lane = lane_id(), wid = tid / WAVE;
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), c = (int)(blockIdx.x % (unsigned)a.chunks);
  const RowBlocks<T> r(a.logits, row, a.V);
  const Policy pol = policy_of(a, row);
  float z[NV][E];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = c * (FC / E) + k * NT + tid;
    r.unpack(r.load(i), i, z[k]);
    if (i >= r.n)
#pragma unroll
      for (int e = 0; e < E; ++e) z[k][e] = -INFINITY;
  }
  for (int i = tid; i < OCT * COPIES; i += NT) {
    s_mass[i] = 0;
    s_count[i] = 0;
  }
  float top = -INFINITY, low = INFINITY;
  bool odd = false;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = z[k][e];
      odd |= !(x < INFINITY);
      top = fmaxf(top, x);
      low = x > -INFINITY ? fminf(low, x) : low;
    }
  top = wave_max(top);
  low = -wave_max(-low);
  const unsigned far = (fabs((double)top * pol.c2) < 1e12 && fabs((double)low * pol.c2) < 1e12) ? 0u : (unsigned)F_FAR;
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
  double X = 0.0;
  if (pol.c2 != 0.0 && flags == F_FINITE) {
    X = ceil((double)key2f(tk) * pol.c2);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float v = z[k][e];
        if (v == -INFINITY) continue;
        const double x = (double)v * pol.c2;
        const int j = min((int)(X - ceil(x)), OCT - 1), at = j * COPIES + (lane & (COPIES - 1));
        atomicAdd(&s_mass[at], mass_of(x - X, a.F));
        atomicAdd(&s_count[at], 1u);
      }
    __syncthreads();
    if (tid < OCT) {
      w64 m = 0;
      unsigned n = 0;
      for (int k = 0; k < COPIES; ++k) {
        m += s_mass[tid * COPIES + (k + tid) % COPIES];
        n += s_count[tid * COPIES + (k + tid) % COPIES];
      }
      out->mass[tid] = m;
      out->count[tid] = n;
    }
  } else if (tid < OCT) {
    out->mass[tid] = 0;
    out->count[tid] = 0;
  }
  if (tid == 0) {
    out->x = X;
    out->top = tk;
    out->flags = flags;
  }
}

// ---------------------------------------------------------------- pick

constexpr int PICK_W = PICK_NT / WAVE;

struct PickShared {
  w64 mass[OCT], hist[256], total;
  unsigned count[OCT], cnt[256];
  w64 wave[PICK_W];
  unsigned list_key[LIST];
  int list_at[LIST];
  int n_list, found;
  unsigned key[2];
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

SVD w64 shfl_up64(w64 v, int d) {
  const unsigned lo = __shfl_up((unsigned)v, d), hi = __shfl_up((unsigned)(v >> 32), d);
  return ((w64)hi << 32) | lo;
}
SVD w64 wave_incl(w64 v) {
#pragma unroll
  for (int d = 1; d < WAVE; d <<= 1) {
    const w64 y = shfl_up64(v, d);
    if (lane_id() >= d) v += y;
  }
  return v;
}
SVD w64 wave_total64(w64 v) {
  v = wave_incl(v);
  const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)v, WAVE - 1), hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(v >> 32), WAVE - 1);
  return ((w64)hi << 32) | lo;
}

template <typename T, bool DRAW>
__global__ __launch_bounds__(PICK_NT) void k_filter_pick(const FilterArgs a) {
  typedef Key<T> K;
  constexpr int E = Fmt<T>::VEC;
  __shared__ PickShared s;
  extern __shared__ w64 s_chunk[];  // [chunks] kept weight
  const int tid = threadIdx.x, lane = lane_id(), wid = tid / WAVE;
  const int row = blockIdx.x;
  const RowBlocks<T> r(a.logits, row, a.V);
  const Policy pol = policy_of(a, row);
  const ChunkSum *sums = a.sums + (size_t)row * a.chunks;

  // ---- the chunks put together
  double X = -INFINITY;
  unsigned tk = 0, flags = 0;
  for (int c = tid; c < a.chunks; c += PICK_NT) {
    const unsigned f = sums[c].flags;
    flags |= f;
    if (f & F_FINITE) {
      X = fmax(X, sums[c].x);
      tk = max(tk, sums[c].top);
    }
  }
  if (tid < OCT) {
    s.mass[tid] = 0;
    s.count[tid] = 0;
  }
  if (tid == 0) {
    s.key[0] = s.key[1] = 0;
    s.total = 0;
    s.n_list = 0;
    s.found = 0x7fffffff;
  }
  __syncthreads();
  if (flags) atomicOr(&s.key[0], flags);
  if (tk) atomicMax(&s.key[1], tk);
  // whole numbers below 2^41: their order is that of the bits, offset to be positive
  if (X > -INFINITY) atomicMax(&s.total, (w64)(long long)(X + 4398046511104.0));
  __syncthreads();
  flags = s.key[0];
  const float zmax = key2f(s.key[1]);
  X = (double)(long long)s.total - 4398046511104.0;
  int code = 0;
  float u = 0.0f;
  if (!pol.ok) code = SV_ROW_BAD_POLICY;
  else if ((flags & F_ODD) || !(flags & F_FINITE)) code = SV_ROW_BAD_LOGITS;
  else if (DRAW && pol.t > 0.0f) {
    u = a.u ? a.u[row] : NAN;
    if (!(u >= 0.0f && u < 1.0f)) code = SV_ROW_BAD_UNIFORM;
  }
  if (tid == 0) a.row_status[row] = code;
  if (code != 0) {
    if (tid == 0) {
      if (DRAW) a.tokens[row] = -1;
      else a.cut[row] = make_uint2(0u, (unsigned)-2);
    }
    return;
  }
  const unsigned top_key = K::of(zmax);
  __syncthreads();

  // ---- the row, block by block, or the list: f(key, logit, index in blocks)
  auto over_row = [&](auto f) {
    constexpr int AHEAD = 4;
    for (int i0 = tid; i0 < r.n; i0 += AHEAD * PICK_NT) {
      u32x4 w[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) w[k] = r.load(i0 + k * PICK_NT);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int i = i0 + k * PICK_NT;
        if (i >= r.n) break;
        float z[E];
        r.unpack(w[k], i, z);
#pragma unroll
        for (int e = 0; e < E; ++e) f(K::of(z[e]), z[e], i * E + e);
      }
    }
  };

  if (pol.t == 0.0f) {  // greedy: the first of the largest
    int best = 0x7fffffff;
    over_row([&](unsigned key, float, int at) {
      if (key == top_key) best = min(best, at - r.lead);
    });
    if (best != 0x7fffffff) atomicMin(&s.found, best);
    __syncthreads();
    if (tid == 0) {
      if (DRAW) a.tokens[row] = s.found;
      else a.cut[row] = make_uint2(top_key, (unsigned)s.found);
    }
    return;
  }

  // x of a logit, and its weight relative to 2^X.  Rows whose x pass 2^40 are taken relative to
  // their largest logit, and counted here.
  const bool far = flags & F_FAR;
  const double off = far ? (double)zmax : 0.0;
  if (far) X = 0.0;
  auto x_of = [&](float z) { return ((double)z - off) * pol.c2; };
  auto weight = [&](float z) { return mass_of(x_of(z) - X, a.F); };
  auto octave = [&](float z) {
    const double d = X - ceil(x_of(z));
    return d < OCT - 1 ? (int)d : OCT - 1;
  };
  if (!far) {
    for (int i = tid; i < a.chunks * OCT; i += PICK_NT) {
      const ChunkSum &cs = sums[i / OCT];
      const unsigned n = cs.count[i % OCT];
      if (!(cs.flags & F_FINITE) || n == 0) continue;
      const double sh = X - cs.x;
      const int up = sh < 64.0 ? (int)sh : 64, j = min(i % OCT + up, OCT - 1);
      atomicAdd(&s.mass[j], up < 64 ? cs.mass[i % OCT] >> up : 0ull);
      atomicAdd(&s.count[j], n);
    }
  } else {
    over_row([&](unsigned, float z, int) {
      if (z == -INFINITY) return;
      atomicAdd(&s.mass[octave(z)], weight(z));
      atomicAdd(&s.count[octave(z)], 1u);
    });
  }
  __syncthreads();
  // The keys of octave j: those from first(j) on that are below first(j - 1).
  auto first_of = [&](int j) {
    if (j >= OCT - 1) return K::lowest();
    return first_key(K::lowest(), top_key, [&](unsigned k) { return X - ceil(x_of(K::value(k))) <= (double)j; });
  };

  // ---- the lowest octave that a threshold can lie in
  unsigned n_all = 0;
  w64 w_all = 0;
  for (int j = 0; j < OCT; ++j) {
    n_all += s.count[j];
    w_all += s.mass[j];
  }
  const bool by_k = pol.k > 0 && (unsigned)pol.k < n_all, by_p = pol.p < 1.0f;
  unsigned tau = K::lowest();  // kept: keys from tau on
  int jt = OCT - 1;            // tau's octave
  if (pol.m > 0.0f) {
    const double xm = x_of(zmax);
    tau = first_key(K::lowest(), top_key, [&](unsigned k) {
      const double d = x_of(K::value(k)) - xm;
      return d > -200.0 && pow2(d) >= (double)pol.m;
    });
    jt = octave(K::value(tau));
  }
  const bool by_m = tau > K::lowest();
  if (by_k) {
    unsigned n = 0;
    int j = 0;
    for (; j < OCT - 1; ++j) {
      n += s.count[j];
      if (n >= (unsigned)pol.k) break;
    }
    jt = min(jt, j);
  }
  if (by_p && !by_k && !by_m) {
    w64 w = 0;
    int j = 0;
    for (; j < OCT - 1; ++j) {
      w += s.mass[j];
      if ((double)w >= (double)pol.p * (double)w_all) break;
    }
    jt = j;
  }
  unsigned n_up = 0;
  for (int j = 0; j <= jt; ++j) n_up += s.count[j];
  const unsigned low = first_of(jt);  // everything from here on is n_up tokens
  const bool cuts = by_k || by_p || by_m;
  const bool listed = cuts && n_up <= (unsigned)LIST;
  if (listed) {
    over_row([&](unsigned key, float z, int at) {
      const bool in = key >= low && z > -INFINITY;
      const unsigned long long b = __ballot(in);
      if (b == 0) return;
      // lanes that have left the loop are not in the ballot: the first that is in it takes the places
      int base = 0;
      const int lead = __ffsll(b) - 1;
      if (lane == lead) base = atomicAdd(&s.n_list, __popcll(b));
      base = __builtin_amdgcn_readlane(base, lead);
      if (in) {
        const int o = base + __popcll(b & ((1ull << lane) - 1ull));
        if (o < LIST) {
          s.list_key[o] = key;
          s.list_at[o] = at;
        }
      }
    });
    __syncthreads();
  }
  const int n_list = listed ? min(s.n_list, LIST) : 0;
  // f(key, logit, place) for tokens with keys from lo to hi
  auto visit = [&](unsigned lo, unsigned hi, auto f) {
    if (listed) {
      for (int i = tid; i < n_list; i += PICK_NT) {
        const unsigned k = s.list_key[i];
        if (k >= lo && k <= hi) f(k, K::value(k), s.list_at[i]);
      }
    } else {
      over_row([&](unsigned k, float z, int at) {
        if (k >= lo && k <= hi && z > -INFINITY) f(k, z, at);
      });
    }
  };
  // The largest key t in [lo, hi] with above + W(lo.. >= t) >= target, by eight bits of the key at
  // a time; W counts or adds weights.  Returns W of what lies above t's octave and at or above t too.
  auto select = [&](unsigned lo, unsigned hi, w64 above, double target, bool counts, w64 &at_least) {
    for (;;) {
      const unsigned span = hi - lo;
      const int bits = 32 - __clz((int)(span | 1u)), sh = bits > 8 ? bits - 8 : 0;
      for (int i = tid; i < 256; i += PICK_NT) s.hist[i] = 0;
      __syncthreads();
      visit(lo, hi, [&](unsigned k, float z, int) { atomicAdd(&s.hist[(k - lo) >> sh], counts ? 1ull : weight(z)); });
      __syncthreads();
      if (wid == 0) {  // lane l owns bins 255 - 4 l down to 252 - 4 l
        w64 h[4], t = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          h[q] = s.hist[255 - 4 * lane - q];
          t += h[q];
        }
        w64 run = above + wave_incl(t) - t;
        int bin = -1, some = -1;
        w64 over = 0, upto = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (h[q] != 0) some = 255 - 4 * lane - q;
          if (bin < 0 && h[q] != 0 && (double)(run + h[q]) >= target) {
            bin = 255 - 4 * lane - q;
            over = run;
            upto = run + h[q];
          }
          run += h[q];
        }
        const unsigned long long b = __ballot(bin >= 0), any = __ballot(some >= 0);
        if (b != 0) {
          if (lane == __ffsll(b) - 1) {
            s.key[0] = (unsigned)bin;
            s.hist[0] = over;
            s.total = upto;
          }
        } else {  // the target is all there is, up to its rounding: the lowest
          const int l = any ? 63 - __clzll((long long)any) : 63;
          if (lane == l) {
            s.key[0] = (unsigned)max(some, 0);
            s.hist[0] = run - (some >= 0 ? s.hist[some] : 0ull);
            s.total = run;
          }
        }
      }
      __syncthreads();
      const unsigned bin = s.key[0];
      above = s.hist[0];
      at_least = s.total;
      __syncthreads();
      lo += bin << sh;
      if (hi - lo >= 1u << sh) hi = lo + ((1u << sh) - 1u);
      if (sh == 0) return lo;
    }
  };
  auto upper_of = [&](int j) { return j == 0 ? top_key : first_of(j - 1) - 1u; };

  // ---- the thresholds
  if (by_k) {
    w64 above = 0;
    int j = 0;
    for (; j < OCT - 1; ++j) {
      if (above + s.count[j] >= (w64)pol.k) break;
      above += s.count[j];
    }
    w64 n;
    const unsigned t = select(first_of(j), upper_of(j), above, (double)pol.k, true, n);
    tau = max(tau, t);
  }
  // the weight of what is kept so far
  w64 kept = w_all;
  if (by_k || by_m) {
    jt = octave(K::value(tau));
    kept = 0;
    for (int j = 0; j < jt; ++j) kept += s.mass[j];
    if (tid == 0) s.total = 0;
    __syncthreads();
    w64 part = 0;
    visit(tau, upper_of(jt), [&](unsigned, float z, int) { part += weight(z); });
    part = wave_total64(part);
    if (lane == 0 && part) atomicAdd(&s.total, part);
    __syncthreads();
    kept += s.total;
    __syncthreads();
  }
  if (by_p) {
    const double target = (double)pol.p * (double)kept;
    w64 above = 0;
    int j = 0;
    const int last = (by_k || by_m) ? jt : OCT - 1;
    for (; j < last; ++j) {
      if ((double)(above + s.mass[j]) >= target) break;
      above += s.mass[j];
    }
    tau = select(max(tau, first_of(j)), upper_of(j), above, target, false, kept);
    jt = j;
  }
  if (!DRAW) {
    if (tid == 0) a.cut[row] = make_uint2(tau, (unsigned)-1);
    return;
  }

  // ---- the chunks' kept weights: octaves above tau's from the scan, tau's own token by token
  for (int c = tid; c < a.chunks; c += PICK_NT) s_chunk[c] = 0;
  __syncthreads();
  if (!far) {
    for (int i = tid; i < a.chunks * OCT; i += PICK_NT) {
      const ChunkSum &cs = sums[i / OCT];
      if (!(cs.flags & F_FINITE)) continue;
      const double sh = X - cs.x;
      const int up = sh < 64.0 ? (int)sh : 64;
      const int j = min(i % OCT + up, OCT - 1);
      if (up < 64 && (cuts ? j < jt : true)) {
        const w64 w = cs.mass[i % OCT] >> up;
        if (w) atomicAdd(&s_chunk[i / OCT], w);
      }
    }
  }
  if (far || cuts) {
    const unsigned hi = far ? top_key : upper_of(jt);
    // a wave's blocks lie in one chunk: their sum is added once
    if (listed && !far) {
      visit(tau, hi, [&](unsigned, float z, int at) { atomicAdd(&s_chunk[at / FC], weight(z)); });
    } else {
      constexpr int STEP = FC / E;  // blocks of a chunk: a whole number of the workgroup's strides, or the reverse
      for (int i0 = 0; i0 < r.n; i0 += PICK_NT) {
        const int i = i0 + tid;
        w64 part = 0;
        if (i < r.n) {
          float z[E];
          r.unpack(r.load(i), i, z);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const unsigned k = K::of(z[e]);
            if (k >= tau && k <= hi && z[e] > -INFINITY) part += weight(z[e]);
          }
        }
        if (__any(part != 0)) {
          part = wave_total64(part);
          if (lane == 0) atomicAdd(&s_chunk[(i0 + wid * WAVE) / STEP], part);
        }
      }
    }
  }
  __syncthreads();
  if (wid == 0) {  // the first chunk whose cumulative weight passes the target
    w64 total = 0;
    for (int c0 = 0; c0 < a.chunks; c0 += WAVE) total += wave_total64(c0 + lane < a.chunks ? s_chunk[c0 + lane] : 0ull);
    const double target = (double)u * (double)total;
    w64 run = 0, before = 0;
    int pick = -1, fallback = 0;
    w64 fb = 0;
    for (int c0 = 0; c0 < a.chunks && pick < 0; c0 += WAVE) {
      const w64 w = c0 + lane < a.chunks ? s_chunk[c0 + lane] : 0ull, inc = wave_incl(w);
      const unsigned long long b = __ballot(w != 0 && (double)(run + inc) > target), some = __ballot(w != 0);
      auto at = [&](w64 v, int l) {
        return ((w64)(unsigned)__builtin_amdgcn_readlane((int)(unsigned)(v >> 32), l) << 32) | (unsigned)__builtin_amdgcn_readlane((int)(unsigned)v, l);
      };
      if (b != 0) {
        const int l = __ffsll(b) - 1;
        pick = c0 + l;
        before = run + at(inc - w, l);
      } else if (some != 0) {
        const int l = 63 - __clzll((long long)some);
        fallback = c0 + l;
        fb = run + at(inc - w, l);
      }
      run += at(inc, WAVE - 1);
    }
    if (lane == 0) {
      s.n_list = pick >= 0 ? pick : fallback;
      s.hist[0] = pick >= 0 ? before : fb;
      s.total = total;
    }
  }
  __syncthreads();
  const int c = s.n_list;
  const double target = (double)u * (double)s.total;
  w64 base = s.hist[0];
  if (tid == 0) s.found = -1;
  // ---- the token: the chunk's kept weights in index order
  constexpr int STEP = FC / E;
  for (int k = 0; k < STEP; k += PICK_NT) {
    const int i = c * STEP + k + tid;
    w64 w[E], sum = 0;
    const bool in = k + tid < STEP && i < r.n;
    float z[E];
    if (in) r.unpack(r.load(i), i, z);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      w[e] = in && z[e] > -INFINITY && K::of(z[e]) >= tau ? weight(z[e]) : 0ull;
      sum += w[e];
    }
    const w64 inc = wave_incl(sum);
    if (lane == WAVE - 1) s.wave[wid] = inc;
    if (tid == 0) s.key[0] = 0x7fffffffu;
    __syncthreads();
    w64 run = base, all = 0;
    for (int v = 0; v < PICK_W; ++v) {
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
        if (pick < 0 && (double)run > target) pick = last;
      }
    }
    if (pick >= 0) atomicMin(&s.key[0], (unsigned)pick);
    if (last >= 0) atomicMax(&s.found, last);  // in case rounding leaves none
    base += all;
    __syncthreads();
    if (s.key[0] != 0x7fffffffu) break;
    __syncthreads();
  }
  if (tid == 0) a.tokens[row] = s.key[0] != 0x7fffffffu ? (int)s.key[0] : s.found;
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
  int chunks;
  size_t sums, cut, total;
};
bool filter_plan(int32_t rows, int32_t V, int esz, FilterPlan &p) {
  if (rows < 1 || V < 1 || V > SV_FILTER_MAX_V) return false;
  const int E = 16 / esz;
  p.chunks = (int)(((long long)V + E - 1 + FC - 1) / FC);  // a row may begin anywhere in a block
  if ((long long)rows * p.chunks > 0xffffffffLL / NT || rows > 0xffffffffLL / PICK_NT) return false;
  size_t o = 0;
  p.sums = o; o = align256(o + (size_t)rows * p.chunks * sizeof(ChunkSum));
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
  char *base = static_cast<char *>(ws);
  FilterArgs a = {};
  a.logits = logits;
  a.u = u;
  a.rows = rows;
  a.V = V;
  a.chunks = p.chunks;
  // a row's weights are at most 1 each: their sum fits 62 bits
  int bits = 0;
  while ((1LL << bits) < V) ++bits;
  a.F = 62 - bits < 50 ? 62 - bits : 50;
  a.policy = *pol;
  a.sums = (ChunkSum *)(base + p.sums);
  a.cut = (uint2 *)(base + p.cut);
  a.tokens = tokens;
  a.row_status = status;
  a.out = out;
  void *args[] = {&a};
  Launcher L{(hipStream_t)stream, ev, nev};
  const unsigned grid = (unsigned)((long long)rows * p.chunks);
  L.go(esz == 2 ? (const void *)&k_filter_scan<uint16_t> : (const void *)&k_filter_scan<float>, grid, args);
  L.block = PICK_NT;
  L.lds = draw ? (unsigned)p.chunks * 8 : 0;
  if (draw) L.go(esz == 2 ? (const void *)&k_filter_pick<uint16_t, true> : (const void *)&k_filter_pick<float, true>, (unsigned)rows, args);
  else L.go(esz == 2 ? (const void *)&k_filter_pick<uint16_t, false> : (const void *)&k_filter_pick<float, false>, (unsigned)rows, args);
  if (!draw) {
    L.block = NT;
    L.lds = 0;
    L.go(esz == 2 ? (const void *)&k_filter_write<uint16_t> : (const void *)&k_filter_write<float>, grid, args);
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

const char *sv_filter_launch_plan(int32_t draw) { return draw ? "k_filter_scan;k_filter_pick" : "k_filter_scan;k_filter_pick;k_filter_write"; }

}  // extern "C"
