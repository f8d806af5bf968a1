// rotary.h — the angles of rotary positions, for kv_append.cu and kv_append_fp8.cu.
//
// Pair i of a head turns by t = p base^(-2i/R) at position p.  In turns,
// t / 2pi = p f with f = base^(-2i/R) / 2pi computed on the host in double and
// passed as two floats f_hi + f_lo.  p is split into a multiple of 2^16 and the
// rest, both exact floats; fma gives what the rounded products with f_hi leave
// over, whole turns drop out of every term exactly, and sincospi needs no further
// range reduction.  Errors in turns: f's double products 2^-49 p f, f_lo's rounding
// 2^-50 p f, and the roundings of the sums, 2^-26 each: 2^-23 below position 2^24.
// From there on the product p f_lo has whole turns as well: 2^-18 up to 2^31.  (The
// fp32 product p base^(-2i/R) would be off by 2^-25 p.)
#pragma once
#include <cmath>

#include "decode_ops.h"

namespace pgs {
namespace {

constexpr int kMaxPairs = 64;  // head_dim <= 128

struct RotaryRates { float hi[kMaxPairs], lo[kMaxPairs]; };

__device__ __forceinline__ float part_turn(float x) { return x - rintf(x); }

__device__ __forceinline__ void pair_angle(const RotaryRates& r, int i, int pos, float* cs, float* sn) {
  const float hi = (float)(pos & ~0xffff), lo = (float)(pos & 0xffff);
  const float f = r.hi[i], a = hi * f, b = lo * f;
  const float rest = part_turn(fmaf(hi, f, -a)) + fmaf(lo, f, -b) + (float)pos * r.lo[i];
  const float t = part_turn(part_turn(a) + part_turn(b)) + rest;
  sincospif(2.0f * t, sn, cs);
}

// The same with what the sums' roundings leave, for which sine and cosine are corrected: off by 2^-25 of a turn below
// position 2^24, by 2^-32 below 2^16, less than sine and cosine are.
__device__ __forceinline__ float rest_of_sum(float x, float y, float sum) {
  const float z = __fsub_rn(sum, x);
  return __fadd_rn(__fsub_rn(x, __fsub_rn(sum, z)), __fsub_rn(y, z));
}
__device__ __forceinline__ void pair_angle_fine(const RotaryRates& r, int i, int pos, float* cs, float* sn) {
  const float hi = (float)(pos & ~0xffff), lo = (float)(pos & 0xffff);
  const float f = r.hi[i], a = hi * f, b = lo * f, a1 = part_turn(a), b1 = part_turn(b), ab = a1 + b1, ab1 = part_turn(ab);
  const float rest = part_turn(fmaf(hi, f, -a)) + fmaf(lo, f, -b) + fmaf((float)pos, r.lo[i], rest_of_sum(a1, b1, ab));
  const float t = ab1 + rest;
  const float more = 6.28318531f * rest_of_sum(ab1, rest, t);
  float s, c;
  sincospif(2.0f * t, &s, &c);
  *cs = fmaf(-s, more, c), *sn = fmaf(c, more, s);
}

// base^(-2i/R) / 2pi, at most six products each
inline void set_rates(RotaryRates* r, double base, int dims) {
  double f[kMaxPairs] = {1.0 / 6.283185307179586476925};
  const int pairs = dims / 2;
  for (int n = 1; n < pairs; n *= 2) {
    const double step = std::pow(base, -2.0 * n / dims);
    for (int i = n; i < pairs && i < 2 * n; ++i) f[i] = f[i - n] * step;
  }
  for (int i = 0; i < pairs; ++i) r->hi[i] = (float)f[i], r->lo[i] = (float)(f[i] - (double)r->hi[i]);
}

}  // namespace
}  // namespace pgs
