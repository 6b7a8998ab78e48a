// weight.cuh -- exp((x - max) / T) as a whole number, right to about 2^-40 of itself.
//
// With d = x - max, y = d log2(e) / T and N = round(256 y): w = 2^(N >> 8) 2^((N & 255) / 256) 2^r, |r| <= 2^-9.
// The middle factor comes from a table of 46-bit fractions; z = r ln 2 and the end of the series
// 2^r - 1 = z + z^2/2 + z^3/6 + z^4/24 are taken to 2^-40 by carrying what each 32-bit product rounds off;
// then one whole-number product.  About 40 instructions and no 64-bit floating point, whose rate
// on this GPU is a sixtieth of the 32-bit rate.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace pkv {

constexpr int kWeightBits = 46;  // of the table

struct Powers {
  uint64_t v[256];
};
// 2^(j / 256) 2^46, from the square roots of 2, sqrt(2), ... (Newton's method)
constexpr Powers make_powers() {
  double root[8] = {};
  double of = 2.0;
  for (int k = 0; k < 8; ++k) {
    double x = 1.5;
    for (int n = 0; n < 60; ++n) x = 0.5 * (x + of / x);
    root[k] = x;  // 2^(1 / 2^(k + 1))
    of = x;
  }
  Powers p{};
  for (int j = 0; j < 256; ++j) {
    double x = 1.0;
    for (int k = 0; k < 8; ++k)
      if (j >> (7 - k) & 1) x *= root[k];
    p.v[j] = static_cast<uint64_t>(x * 70368744177664.0 + 0.5);
  }
  return p;
}
__device__ const Powers kPowers = make_powers();

// Bits that weights are shifted down by, so that a row's sum stays below 2^63.
inline int weight_shift(int vocab) {
  int bits = 0;
  while ((int64_t(1) << bits) < vocab) ++bits;
  return bits + kWeightBits > 62 ? bits + kWeightBits - 62 : 0;
}

// floor(share * mass) and ceil(share * mass), exactly, for a share in [0, 1) (below 2^-40 it is cut off to
// a multiple of 2^-64).
__device__ __forceinline__ uint64_t fraction64(float share) {
  const uint32_t u = __float_as_uint(share) & 0x7fffffffu;  // (-0 is 0)
  const int e = static_cast<int>(u >> 23) - 127 - 23;  // share = m 2^e
  const uint64_t m = (u & 0x7fffffu) | 0x800000u;
  const int up = 64 + e;
  return (u >> 23) == 0 || up <= -24 ? 0 : up >= 0 ? m << up : m >> -up;
}
__device__ __forceinline__ uint64_t part_of(uint64_t mass, float share) { return __umul64hi(mass, fraction64(share)); }
__device__ __forceinline__ uint64_t part_of_up(uint64_t mass, float share) {
  const uint64_t f = fraction64(share);
  return __umul64hi(mass, f) + (mass * f != 0 ? 1 : 0);
}

struct Weight {
  float top, ch, cl;  // the largest logit; log2(e) / T in two parts
  float unit;         // a weight of 1 as a whole number
  int shift;

  __device__ __forceinline__ Weight(float top_, float temperature, int shift_) : top(top_), shift(shift_) {
    unit = __int_as_float((127 + kWeightBits - shift) << 23);
    constexpr float kHigh = 1.44269502162933349609375f, kLow = 1.925963033500e-8f;  // log2(e)
    ch = kHigh / temperature;
    if (!(ch < 1e30f)) {  // (a temperature next to zero: only the largest logit has a weight)
      ch = 1e30f;
      cl = 0.f;
    } else {  // (the remainder is exact)
      cl = (fmaf(-ch, temperature, kHigh) + kLow) / temperature;
    }
  }

  __device__ __forceinline__ uint64_t of(float x, const uint64_t* table) const {
    // d = dh + dl exactly
    const float dh = x - top, minus = dh - x;
    const float dl = (x - (dh - minus)) - (top + minus);
    const float yh = dh * ch;
    if (!(yh > -64.f)) return 0;
    const float yl = fmaf(dl, ch, fmaf(dh, cl, fmaf(dh, ch, -yh)));
    const float t = fmaf(yh, 256.f, 12582912.f);
    const int n = __float_as_int(t) - 0x4b400000;
    const float r = fmaf(t - 12582912.f, -1.f / 256.f, yh);
    constexpr float kLnH = 0.693147182464599609375f, kLnL = -1.904654299957767878541e-9f;
    const float zh = r * kLnH;
    const float zl = fmaf(yl, kLnH, fmaf(r, kLnL, fmaf(r, kLnH, -zh)));
    const float rest = fmaf(zh * zh, fmaf(zh, fmaf(zh, 1.f / 24.f, 1.f / 6.f), 0.5f), zl);
    constexpr float kUnit = 1099511627776.f;  // 2^40
    const int z = __float2int_rn(zh * kUnit) + __float2int_rn(rest * kUnit);
    const uint64_t p = table[n & 255];
    const int64_t more = static_cast<int64_t>(static_cast<int32_t>((p + 32768) >> 16)) * z;  // 2^30 times 2^40
    const uint64_t m = p + static_cast<uint64_t>(more >> 24);
    const int down = shift - (n >> 8);
    return down >= 64 ? 0 : down == 0 ? m : (m + (uint64_t(1) << (down - 1))) >> down;
  }

  // The least whole weight that is `share` or more.
  __device__ __forceinline__ uint64_t part_up(float share) const {
    return share >= 1.f ? uint64_t(1) << (kWeightBits - shift) : part_of_up(uint64_t(1) << (kWeightBits - shift), share);
  }

  // Two weights in fp32, parts of 1, of d = x - max (of what is no candidate: anything).
  __device__ __forceinline__ Two rounded(Two d) const {
    const Two minus_yh = mul2(d, two(-ch)), yl = fma2(d, two(cl), fma2(d, two(ch), minus_yh));
    const float2 y = both(minus_yh);
    const Two m = two(ex2_approx(-y.x), ex2_approx(-y.y));
    return fma2(mul2(m, two(0.6931472f)), yl, m);
  }

  // log(w / mass) of logit x with weight w.  Few units of weight say little: then it is (x - max) / T - log(mass of the largest's weight).
  __device__ __forceinline__ float log_share(float x, float temperature, uint64_t w, uint64_t mass) const {
    const float all = __ull2float_rn(mass);
    if (w < (1u << 24)) return (x - top) / temperature - logf(all / unit);
    return w > mass - w ? log1pf(-(__ull2float_rn(mass - w) / all)) : logf(__ull2float_rn(w) / all);
  }
};

}  // namespace pkv
