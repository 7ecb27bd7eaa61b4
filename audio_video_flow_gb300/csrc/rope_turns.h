// Frequencies of the rotary positions: turns per position of every rotated
// pair in 64-bit fixed point (2^64 = one turn), on the host.
//
// A position of 2^31 multiplies an error of the frequency by 2^31, so the table
// is computed from numbers of 128 bits and is right to its last bits: within
// 2 units of 2^-64 for every configuration h3_rope accepts, 2^-32 of a turn at
// the farthest position (a double's rounding would be 2^-24 there, at a base
// of 2^40 or on a YaRN ramp with alpha next to beta more).  The frequencies of
// an axis are a geometric series whose ratio is one double root corrected by
// one Newton step: a long double pow per frequency costs more than the launch.
// Plain C++ without CUDA.
#ifndef H3_ROPE_TURNS_H_
#define H3_ROPE_TURNS_H_

#include <cmath>
#include <cstdint>
#include <cstring>

#include "h3.h"

namespace h3 {

typedef unsigned __int128 u128;

// A number >= 0 as m 2^e with 2^127 <= m < 2^128, or m = 0.  The operations
// truncate: each product is within 2^-124 of its value, relatively.
struct Wide {
  u128 m;
  int e;
};
inline int wide_leading_zeros(u128 m) {
  const uint64_t hi = (uint64_t)(m >> 64);
  return hi ? __builtin_clzll(hi) : 64 + __builtin_clzll((uint64_t)m);
}
inline Wide wide_normal(u128 m, int e) {
  if (m == 0) return {0, 0};
  const int z = wide_leading_zeros(m);
  return {m << z, e - z};
}
inline Wide wide(double x) {   // exactly, x >= 0
  if (!(x > 0.0)) return {0, 0};
  int e;
  const uint64_t m = (uint64_t)std::ldexp(std::frexp(x, &e), 53);
  return wide_normal(m, e - 53);
}
inline Wide wide_mul(const Wide& a, const Wide& b) {
  const uint64_t al = (uint64_t)a.m, ah = (uint64_t)(a.m >> 64), bl = (uint64_t)b.m, bh = (uint64_t)(b.m >> 64);
  // in [2^126, 2^128) (or 0), less at most 3 for what is not carried up
  const u128 m = (u128)ah * bh + (uint64_t)((u128)al * bh >> 64) + (uint64_t)((u128)ah * bl >> 64);
  return (uint64_t)(m >> 64) >> 63 ? Wide{m, a.e + b.e + 128} : Wide{m << 1, a.e + b.e + 127};
}
inline bool wide_less(const Wide& a, const Wide& b) {
  if (a.m == 0 || b.m == 0) return b.m != 0;
  return a.e != b.e ? a.e < b.e : a.m < b.m;
}
inline Wide wide_add(const Wide& a, const Wide& b) {
  if (wide_less(a, b)) return wide_add(b, a);
  if (b.m == 0) return a;
  const int d = a.e - b.e;
  const u128 m = a.m + (d < 128 ? b.m >> d : 0);
  return m < a.m ? Wide{m >> 1 | (u128)1 << 127, a.e + 1} : Wide{m, a.e};
}
inline Wide wide_sub(const Wide& a, const Wide& b) {   // a >= b
  if (b.m == 0) return a;
  const int d = a.e - b.e;
  return wide_normal(a.m - (d < 128 ? b.m >> d : 0), a.e);
}
// 1 / a for a > 0: a double's reciprocal and two Newton steps, r += r (1 - a r).
inline Wide wide_inverse(const Wide& a) {
  const Wide one = {(u128)1 << 127, -127};
  const Wide scaled = {a.m, -128};   // in [1/2, 1)
  Wide r = wide(1.0 / std::ldexp((double)(uint64_t)(a.m >> 64), -64));
  for (int k = 0; k < 2; ++k) {
    const Wide p = wide_mul(scaled, r);
    r = wide_less(one, p) ? wide_sub(r, wide_mul(r, wide_sub(p, one))) : wide_add(r, wide_mul(r, wide_sub(one, p)));
  }
  r.e -= a.e + 128;
  return r;
}
// b^(-1/n) for b >= 1: a double's root r, and one Newton step on r^n b = 1.
inline Wide wide_inverse_root(float b, int n) {
  const Wide one = {(u128)1 << 127, -127};
  const Wide r = wide(std::pow((double)b, -1.0 / n));
  Wide power = wide((double)b), square = r;
  for (int k = n; k > 0; k >>= 1) {
    if (k & 1) power = wide_mul(power, square);
    square = wide_mul(square, square);
  }
  const bool above = wide_less(one, power);
  const Wide off = wide_mul(above ? wide_sub(power, one) : wide_sub(one, power), wide(1.0 / n));
  return above ? wide_sub(r, wide_mul(r, off)) : wide_add(r, wide_mul(r, off));
}
// to 64-bit fixed point, to nearest (0 <= a < 1/4)
inline uint64_t wide_fixed64(const Wide& a) {
  const int shift = -a.e - 64;   // a 2^64 = m 2^-shift, shift >= 66
  if (a.m == 0 || shift > 128) return 0;
  return (uint64_t)(((a.m >> (shift - 1)) + 1) >> 1);
}

// turns[a * n_freqs + f] of a valid configuration.
inline void rope_turns(const h3_rope_config& c, uint64_t* turns) {
  // 1 / (2 pi)
  const Wide inv_two_pi = {((u128)0xA2F9836E4E441529ull << 64) | 0xFC2757D1F534DDC0ull, -130};
  const Wide one = {(u128)1 << 127, -127};
  const int F = c.n_freqs;
  bool done[2] = {false, false};
  int at[2] = {0, 0};
  for (int a = 0; a < c.n_axes; ++a) {
    const int scaled = c.scaling != H3_ROPE_SCALE_NONE && ((c.scaled_axes >> a) & 1);
    if (done[scaled]) {   // the axes of one kind share their frequencies
      std::memcpy(turns + a * F, turns + at[scaled] * F, (size_t)F * sizeof(uint64_t));
      continue;
    }
    done[scaled] = true;
    at[scaled] = a;
    const int scaling = scaled ? c.scaling : H3_ROPE_SCALE_NONE;
    Wide ratio = F > 1 ? wide_inverse_root(c.theta, F) : one;
    if (scaling == H3_ROPE_SCALE_NTK) ratio = wide_mul(ratio, wide_inverse_root(c.factor, F - 1));
    Wide w = inv_two_pi;
    Wide inv_s = one, change = {0, 0}, alpha = {0, 0}, beta = {0, 0}, inv_ramp = one, trained = one;
    if (scaling == H3_ROPE_SCALE_LINEAR || scaling == H3_ROPE_SCALE_YARN) inv_s = wide_inverse(wide((double)c.factor));
    if (scaling == H3_ROPE_SCALE_LINEAR) w = wide_mul(w, inv_s);
    if (scaling == H3_ROPE_SCALE_YARN) {
      change = c.factor > 1.0f ? wide_sub(one, inv_s) : Wide{0, 0};
      alpha = wide((double)c.alpha);
      beta = wide((double)c.beta);
      inv_ramp = wide_inverse(wide_sub(beta, alpha));
      trained = wide((double)c.trained_length);
    }
    for (int f = 0; f < F; ++f) {
      Wide t = w;
      if (scaling == H3_ROPE_SCALE_YARN) {
        // turns over the trained length, and by them the share kept: g + (1 - g) / s
        const Wide n = wide_mul(trained, w);
        if (!wide_less(alpha, n)) {
          t = wide_mul(w, inv_s);
        } else if (wide_less(n, beta)) {
          const Wide g = wide_mul(wide_sub(n, alpha), inv_ramp);
          t = wide_mul(w, wide_add(inv_s, wide_mul(g, change)));
        }
      }
      turns[a * F + f] = wide_fixed64(t);
      w = wide_mul(w, ratio);
    }
  }
}

}  // namespace h3

#endif  // H3_ROPE_TURNS_H_
