// sv_fp4.h -- the cache in 4 bits (include/spec_cache.h): blocks of 32 elements as codes and a
// power of two, where they lie in a pool, and the conversions of gfx950 between codes and numbers.
#pragma once

#include "sv_cache.h"

namespace sv {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int F4_BLOCK = 32;     // elements that share a scale
constexpr int F4_NAN = 255;      // the scale byte of a block that is not finite
constexpr int F4_MIN = -120, F4_MAX = 125;  // exponents of a scale

// Bytes of one head of one page: codes, and scales.
SVD size_t f4_codes(const Pool &p) { return ((size_t)p.D << p.page_shift) / 2; }
SVD size_t f4_scales(const Pool &p) { return ((size_t)p.D << p.page_shift) / F4_BLOCK; }

// In one head of one page: the 16 bytes of block u of slot t's key, its scale's byte (values'
// scales lie alike), and the D / 32 bytes of piece m (elements D / 16 * m ..) of slot t's value.
SVD unsigned f4_key(const Pool &p, int u, int t) { return (unsigned)((u << p.page_shift) + t) * 16u; }
SVD unsigned f4_scale(const Pool &p, int u, int t) { return (unsigned)((u << p.page_shift) + t); }
SVD unsigned f4_value(const Pool &p, int t, int m) {
  const int S = 512 / (int)p.D, B = (int)p.D / 32;
  return (unsigned)((t / S * 16 + m) * 16 + (t % S) * B);
}

// What a scale byte stands for, as the conversions want it: they read the exponent alone, and with
// that of byte 255 they give NaN whatever the code.  So a byte of a word need not be cut out.
SVD float f4_factor(unsigned byte) { return __uint_as_float(byte << 23); }
SVD float f4_factor(unsigned word, int i) { return __uint_as_float(i == 3 ? word >> 1 : word << (23 - 8 * i)); }

// Eight elements of a block, the other three threads of the quad having the rest: their codes in a
// word, and the block's scale byte.  The conversion rounds x / scale to the nearest code, ties to
// the even one.
SVD unsigned f4_encode8(const float (&x)[8], unsigned &w) {
  float top = 0.0f;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    odd |= !(fabsf(x[i]) < INFINITY);
    top = fmaxf(top, fabsf(x[i]));
  }
  unsigned u = odd ? 0x7f800000u : __float_as_uint(top);
  u = max(u, (unsigned)__builtin_amdgcn_update_dpp(0, (int)u, 0xb1, 0xf, 0xf, false));  // quad_perm 1 0 3 2
  u = max(u, (unsigned)__builtin_amdgcn_update_dpp(0, (int)u, 0x4e, 0xf, 0xf, false));  // quad_perm 2 3 0 1
  // top = m 2^E with m in [1/2, 1): 6 = 3/4 * 2^3
  int e = (int)(u >> 23) - 126 - ((u & 0x7fffffu) <= 0x400000u ? 3 : 2);
  e = min(max(e, F4_MIN), F4_MAX);
  const float scale = __uint_as_float((unsigned)(e + 127) << 23), most = 6.0f * scale;
  auto y = [&](int i) { return fminf(fmaxf(x[i], -most), most); };
  unsigned c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y(0), y(1), scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y(2), y(3), scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y(4), y(5), scale, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y(6), y(7), scale, 3);
  const bool none = u >= 0x7f800000u;
  w = none ? 0u : c;
  return none ? F4_NAN : (unsigned)(e + 127);
}

// Codes 2 I and 2 I + 1 of a word as two bf16 numbers, times a power of two.
template <int I>
SVD unsigned f4_pair(unsigned w, float factor) {
  return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, factor, I));
}
// All eight.
SVD u32x4 f4_unit(unsigned w, float factor) {
  return u32x4{f4_pair<0>(w, factor), f4_pair<1>(w, factor), f4_pair<2>(w, factor), f4_pair<3>(w, factor)};
}

}  // namespace sv
