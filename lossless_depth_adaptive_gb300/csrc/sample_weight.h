// The weight of a logit as an integer (host and device, so that a test can compile it by itself).
#pragma once

#include <math.h>
#include <stdint.h>
#include <string.h>

#ifdef __CUDACC__
#define DEX_WEIGHT_FN __host__ __device__ __forceinline__
#else
#define DEX_WEIGHT_FN inline
#endif

namespace dex {

constexpr int kWeightBits = 43;
constexpr int kWeightTable = 33;

// Products and sums that are not contracted into one rounding.
DEX_WEIGHT_FN float mul_rn(float x, float y) {
#ifdef __CUDA_ARCH__
  return __fmul_rn(x, y);
#else
  return x * y;
#endif
}
DEX_WEIGHT_FN float sub_rn(float x, float y) {
#ifdef __CUDA_ARCH__
  return __fsub_rn(x, y);
#else
  return x - y;
#endif
}
DEX_WEIGHT_FN float fma_rn(float x, float y, float z) {
#ifdef __CUDA_ARCH__
  return __fmaf_rn(x, y, z);
#else
  return fmaf(x, y, z);
#endif
}
DEX_WEIGHT_FN int32_t float_bits(float x) {
#ifdef __CUDA_ARCH__
  return __float_as_int(x);
#else
  int32_t i;
  memcpy(&i, &x, 4);
  return i;
#endif
}

// Entry j of weight_of's table.
DEX_WEIGHT_FN double weight_table_entry(int j) { return exp2((j - 16) * 0.03125); }

DEX_WEIGHT_FN float exp2_fast(float x) {   // to 2^-22 of it
#ifdef __CUDA_ARCH__
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
#else
  return exp2f(x);
#endif
}

// A number as the sum of two floats.
struct Pair {
  float hi, lo;
};
DEX_WEIGHT_FN Pair pair_of(double x) {
  Pair p;
  p.hi = static_cast<float>(x);
  p.lo = p.hi <= 3.402823466e38f ? static_cast<float>(x - p.hi) : 0.0f;
  return p;
}

// From here on temperatures and logits are scaled down before weight_of, as octaves_per_unit would lose its lower part below the
// normal floats and the difference of two logits that matter could overflow.  (A power of two: no rounding but of what is far too
// small to matter.)
constexpr float kHot = 0x1p100f, kHotScale = 0x1p-40f;

// log2(e) / temperature, to 2^-46 of it and more (0 < temperature < kHot; infinite where that is).
DEX_WEIGHT_FN Pair octaves_per_unit(float temperature) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299112661746e-8f;
  Pair c;
  c.hi = kLog2e / temperature;
  c.lo = c.hi <= 3.402823466e38f ? (fmaf(-c.hi, temperature, kLog2e) + kLog2eLow) / temperature : 0.0f;
  return c;
}

// (x - top) c, that is how many octaves x lies below top, as a pair: the difference, its rounding error and the products' ones.
// scale: a power of two that x and top are multiplied by.  (x == top where c is infinite, and infinities: NaN)
DEX_WEIGHT_FN Pair octaves_of(float x, float top, Pair c, float scale = 1.0f) {
  const float most = mul_rn(top, scale);
  const float d = fma_rn(x, scale, -most);
  const float b = fma_rn(-x, scale, d);              // the part of -most that is in d
  const float dl = fma_rn(x, scale, -sub_rn(d, b)) - (most + b);
  Pair y;
  y.hi = mul_rn(d, c.hi);
  y.lo = fmaf(d, c.hi, -y.hi) + fmaf(d, c.lo, mul_rn(dl, c.hi));
  return y;
}

constexpr float kLn2 = 0.693147182464599609375f, kLn2Low = -1.904654323148236e-9f;

// The log of 2^y / (mass 2^-43), for what is at most half of it: ln 2 y and the log of the mass have one sign, so nothing cancels; 2^-22 of
// the result with a log good to one unit in the last place.  (An integer weight would not do: at 20 nats below the largest it has some 15
// bits left, at 29 one.)
DEX_WEIGHT_FN float log_share(Pair y, uint64_t mass) {
  const float m = static_cast<float>(mass), rest = static_cast<float>(static_cast<int64_t>(mass - static_cast<uint64_t>(m)));
  const float t = mul_rn(y.hi, kLn2);
  const float tl = fmaf(y.hi, kLn2, -t) + fmaf(y.hi, kLn2Low, mul_rn(y.lo, kLn2));
  return sub_rn(t, logf(mul_rn(m, 0x1p-43f))) + (tl - rest / m);
}

// w = 2^((x - top) c), c = log2(e) / temperature, in units of 2^-43; 0 below half a unit.  To within two units:
// below 2^-22 of the largest by a float's own 22 bits, before that
// differences, products and the exponential are pairs of floats (46 bits and more): y = (x - top) c = n + j/32 + f with
// 2^(j/32) from a table of pairs (j from -16 to 16) and 2^f = 1 + t + t^2/2 + ..., t = f ln 2 below 2^-6.5, of which the
// first two terms need their low parts.
DEX_WEIGHT_FN uint64_t weight_of(float x, float top, Pair c, const Pair* table, float scale = 1.0f) {
  if (x == top) return uint64_t(1) << kWeightBits;   // also where c is infinite
  const Pair o = octaves_of(x, top, c, scale);
  const float y = o.hi, yl = o.lo;
  if (!(y >= -45.0f)) return 0;                      // also NaN: infinities
  if (y < -22.0f) {
    const float w = mul_rn(exp2_fast(y), 8796093022208.0f);   // in units, below 2^21
    return static_cast<uint64_t>(static_cast<uint32_t>(fmaf(w, mul_rn(yl, 0.693147182f), w) + 0.5f));
  }
  const float n = rintf(y);
  const float r = sub_rn(y, n);                      // exact, at most 1/2
  const float j = rintf(mul_rn(r, 32.0f));
  const float f = fmaf(j, -0.03125f, r);             // exact
  const float th = mul_rn(f, kLn2);
  const float rest_t = fmaf(f, kLn2, -th) + fmaf(f, kLn2Low, mul_rn(yl, kLn2));
  const float t = th + rest_t;                       // f may be smaller than yl
  const float back = sub_rn(t, th);
  const float tl = sub_rn(th, sub_rn(t, back)) + sub_rn(rest_t, back);
  const float s = mul_rn(t, t);
  const float sl = fmaf(t, t, -s) + mul_rn(t + t, tl);
  const float q = mul_rn(mul_rn(s, t), fmaf(t, fmaf(t, 1.0f / 120.0f, 1.0f / 24.0f), 1.0f / 6.0f));
  const float e = fmaf(0.5f, s, t);
  const float el = fmaf(0.5f, s, -sub_rn(e, t)) + (tl + fmaf(0.5f, sl, q));   // q is up to 2^-22
  const Pair p = table[static_cast<int>(j) + 16];
  const float pe = mul_rn(p.hi, e);
  const float pl = fmaf(p.hi, e, -pe) + fmaf(p.hi, el, fmaf(p.lo, e, p.lo));
  const float w0 = p.hi + pe;
  const float w1 = sub_rn(pe, sub_rn(w0, p.hi)) + pl;
  const float w = w0 + w1, wl = sub_rn(w1, sub_rn(w, w0));
  // w lies in [0.69, 1.43]: 22 bits behind the point, then 21 of what is left, by adding numbers whose last place is 1
  const float m1 = fmaf(w, 4194304.0f, 8388608.0f);
  const float rest = fmaf(w, 4194304.0f, -sub_rn(m1, 8388608.0f)) + mul_rn(wl, 4194304.0f);
  const float m2 = fmaf(rest, 2097152.0f, 12582912.0f);
  const int64_t full = (static_cast<int64_t>(float_bits(m1) - 0x4B000000) << 21) + (float_bits(m2) - 0x4B400000);
  const int down = -static_cast<int>(n);             // 0 .. 22
  return static_cast<uint64_t>(full + ((int64_t(1) << down) >> 1)) >> down;
}

// The same as a float, roughly: off by at most 2^-22 (the exponential) + 2^-24 (the last sum) + 2^-24 |y| ln 2 (what the
// difference loses) of itself, 2^-18 for y above -45; below that it counts for nothing.  An eighth of the instructions.  c.hi has to be
// finite and temperatures below kHot; far: -128 / c.hi.
DEX_WEIGHT_FN float weight_near(float x, float top, Pair c, float far) {
  const float d = fmaxf(sub_rn(x, top), far);
  const float y = mul_rn(d, c.hi);
  const float yl = fmaf(d, c.lo, fmaf(d, c.hi, -y));
  const float w = exp2_fast(y);
  return fmaf(w, mul_rn(yl, 0.693147182f), w);
}
// A float in [0, 2^18] in units of 2^-43, rounded down.
DEX_WEIGHT_FN uint64_t in_units(float w) {
  if (w < 0x1p-11f) return static_cast<uint32_t>(mul_rn(w, 0x1p43f));   // most are
  const int32_t bits = float_bits(w), e = (bits >> 23) - (127 + 23 - kWeightBits);   // its last place is 2^e units
  const uint64_t m = static_cast<uint64_t>((bits & 0x7fffff) | 0x800000);
  return e >= 0 ? m << e : e > -24 ? m >> -e : 0;
}

// What a sum of such weights of tokens down to `octaves` below the largest may be off by, against the sum of weight_of: each by the
// above, and by three roundings where four of them were added as floats first, 2^-21 and 2^-24 ln 2 per octave in all (and some
// 2^-30 for what is of second order); and of the up to 2^18 tokens each by the unit that rounding down loses, the two
// that weight_of may be off by and the half below which it is nothing.
DEX_WEIGHT_FN uint64_t rough_slack(uint64_t sum, float octaves) {
  return static_cast<uint64_t>(static_cast<float>(sum) * (4.78e-7f + octaves * 4.2e-8f)) + (uint64_t(1) << 20);
}

}  // namespace dex
