// Softmax weights as integers.
//
// Whether the last token of a top-p set belongs to it is decided by comparing
// two sums of weights, and in a flat row that token's share is 1e-5 or less:
// float32 sums would decide one row in a hundred wrongly, and sums of floats
// depend on their order. Here a weight is round(2^F * 2^(s log2 e - K)) with
// K = floor(s_max log2 e): integers, so sums are exact in any order, and equal
// logits have equal weights.
//
// exp by table, after Tang, "Table-driven implementation of the exponential
// function in IEEE floating-point arithmetic" (1989), the steps taken in pairs
// of float32 and the end in integers:
//   y = s log2 e = k + j / 32 + r  (r exact, the rounding of y kept in yl)
//   2^y = 2^k T[j] e^z,  z = (r + yl) ln 2 = zh + zl, |z| < 0.011
//   e^z - 1 = zh + (zl + z^2 (1/2 + z (1/6 + z (1/24 + z / 120))))
// Largest error found 2^-35.8 of the weight, mean 2^-39 (20000 values of
// |s| < 512 against 60 digits).
#pragma once

#include "tv_common.cuh"

namespace tv {

constexpr int kWeightTable = 32;         // 2^(j / 32) times 2^44
__constant__ const unsigned long long c_weight_table[kWeightTable] = {
    17592186044416ull, 17977404757381ull, 18371058661769ull, 18773332464219ull,
    19184414915921ull, 19604498901178ull, 20033781527906ull, 20472464220127ull,
    20920752812471ull, 21378857646762ull, 21846993670708ull, 22325380538761ull,
    22814242715178ull, 23313809579344ull, 23824315533396ull, 24346000112214ull,
    24879108095804ull, 25423889624159ull, 25980600314626ull, 26549501381838ull,
    27130859760289ull, 27724948229574ull, 28332045542385ull, 28952436555301ull,
    29586412362452ull, 30234270432094ull, 30896314746195ull, 31572855943056ull,
    32264211463077ull, 32970705697691ull, 33692670141585ull, 34430443548229ull};

constexpr float kLog2e = 1.44269502f, kLog2eLow = 0x1.4ae0c0p-26f;     // together log2 e to 2^-50
constexpr float kLn2 = 0x1.62e430p-1f, kLn2Low = -0x1.05c610p-29f;
constexpr float kWeightSpan = 512.0f;    // |s - ref| for which the reduction holds its error

// What the weights of one row are relative to.
struct WeightScale {
  float ref;       // subtracted from s first: 0, or s_max where |s_max| >= kWeightSpan (then exact
                   // for every s whose weight is not 0)
  float s_max;
  int k;           // floor((s_max - ref) log2 e), to the reduction's rounding
  int bits;        // F
  bool tie;        // s_max is infinite or NaN: what equals it weighs 2^F, all else nothing
};

// rint(32 y) for |y| < 2^16: adding a number whose last bit stands for 2^-5
// leaves it in the sum's last bits.
constexpr float kSteps = 0x1.8p18f;
__device__ __forceinline__ int weight_steps(float y) { return __float_as_int(y + kSteps) - __float_as_int(kSteps); }

__device__ __forceinline__ WeightScale weight_scale(float s_max, int bits) {
  WeightScale w;
  w.s_max = s_max;
  w.bits = bits;
  w.tie = !(fabsf(s_max) < __int_as_float(0x7f800000));
  w.ref = fabsf(s_max) < kWeightSpan || w.tie ? 0.0f : s_max;
  w.k = w.tie ? 0 : weight_steps(__fmul_rn(s_max - w.ref, kLog2e)) >> 5;
  return w;
}

// F for sums of n weights (each at most 2^(F+1)) that stay below 2^64
inline int weight_bits(int n) {
  int log = 0;
  while ((1ll << log) < n) ++log;
  return 62 - log < 44 ? 62 - log : 44;
}

// Integers come out of floats by adding a number whose last bit stands for the
// unit wanted: conversion instructions run at a fraction of that rate.
// The table in shared memory: 32 entries of 4 bytes lie in 32 banks, so any
// lookup of a warp is one access (of 8 bytes, three to four).
struct WeightTable {
  uint32_t low[kWeightTable], high[kWeightTable];        // of 2^(j / 32) times 2^44
  float near[kWeightTable], rest[kWeightTable];          // the same in float32, and its rounding's share
};
__device__ __forceinline__ void fill_weight_table(WeightTable& table, int j) {
  const unsigned long long t = c_weight_table[j];
  const float f = __ull2float_rn(t);
  table.low[j] = static_cast<uint32_t>(t);
  table.high[j] = static_cast<uint32_t>(t >> 32);
  table.near[j] = f * 0x1p-44f;
  table.rest[j] = static_cast<float>(static_cast<long long>(t) - static_cast<long long>(f)) / f;
}

__device__ __forceinline__ uint64_t weight_of(float s, const WeightScale& w, const WeightTable& table) {
  if (w.tie) return (s == w.s_max || (s != s && w.s_max != w.s_max)) ? 1ull << w.bits : 0ull;
  s -= w.ref;
  const float yh = __fmul_rn(s, kLog2e);
  if (!(yh > static_cast<float>(w.k - 62))) return 0ull;               // (s = -inf too)
  const float yl = __fmaf_rn(s, kLog2eLow, __fmaf_rn(s, kLog2e, -yh));
  constexpr float kUpper = 3.0f, kLower = 0x1.8p-12f;    // last bits 2^-22, 2^-35
  const float steps = yh + kSteps;                       // 32 k + j
  const float r = yh - (steps - kSteps);
  const int n = __float_as_int(steps) - __float_as_int(kSteps);
  const float zh = __fmul_rn(r, kLn2);
  const float zl = __fmaf_rn(yl, kLn2, __fmaf_rn(r, kLn2Low, __fmaf_rn(r, kLn2, -zh)));
  const float z = zh + zl;
  const float q = __fmaf_rn(z * z, __fmaf_rn(z, __fmaf_rn(z, __fmaf_rn(z, 1.0f / 120, 1.0f / 24), 1.0f / 6), 0.5f), zl);
  const float upper = zh + kUpper;                       // zh in steps of 2^-22, what is left beside q
  const float lower = (q + (zh - (upper - kUpper))) + kLower;
  const int e = ((__float_as_int(upper) - __float_as_int(kUpper)) << 13) + (__float_as_int(lower) - __float_as_int(kLower));
  const uint64_t t = static_cast<uint64_t>(table.high[n & 31]) << 32 | table.low[n & 31];
  const int g = static_cast<int>(static_cast<uint32_t>(t >> 12) ^ 0x80000000u);   // T - 3/2 in steps of 2^-32
  const uint64_t m = t + static_cast<uint64_t>(768ll * e + ((static_cast<long long>(g) * e) >> 23));
  const int shift = w.k - (n >> 5) + 44 - w.bits;
  return shift <= 0 ? m : shift > 63 ? 0ull : ((m >> (shift - 1)) + 1) >> 1;
}

// The same in float32, for a scale without tie: w (1 + q), w = 2^(y - k) to a
// multiple of 1 / 32 in y and to its rounding, whose share is in q. Off by 2^-30 of
// it (z's and q's roundings, 2^-24 of |z| < 2^-6.5; z^5 / 120 left out).
struct CloseWeight {
  float w, q;
};
__device__ __forceinline__ CloseWeight close_weight(float s, const WeightScale& w, const WeightTable& table) {
  const float k = static_cast<float>(w.k);
  const float sx = fmaxf(s - w.ref, (k - 100.0f) * kLn2);                // (-inf: 2^-100)
  const float yh = __fmul_rn(sx, kLog2e);
  const float steps = yh + (kSteps - k);                 // 32 (y - k) in the last bits
  const float yl = __fmaf_rn(sx, kLog2eLow, __fmaf_rn(sx, kLog2e, -yh));
  const float z = __fmaf_rn(yh - (steps - (kSteps - k)), kLn2, yl * kLn2);
  const int n = __float_as_int(steps);
  const float q = __fmaf_rn(z * z, __fmaf_rn(z, __fmaf_rn(z, 1.0f / 24, 1.0f / 6), 0.5f), z) + table.rest[n & 31];
  return {__int_as_float(__float_as_int(table.near[n & 31]) + ((n & ~31) << 18)), q};
}

// The smallest integer >= p * z for 0 <= p < 1, and 1 at least: a prefix whose
// weights reach it has a share of p.
__device__ __forceinline__ uint64_t share_of(float p, uint64_t z) {
  if (!(p > 0.0f)) return 1ull;
  int e;
  const float m = frexpf(p, &e);                         // p = m 2^e, m in [0.5, 1), e <= 0
  const uint64_t mant = static_cast<uint64_t>(m * 0x1p24f);
  const uint64_t lo = mant * z, hi = __umul64hi(mant, z);
  const int shift = 24 - e;                              // p z = (hi, lo) / 2^shift
  if (shift >= 126) return 1ull;
  const unsigned __int128 v = (static_cast<unsigned __int128>(hi) << 64) | lo;
  const unsigned __int128 one = 1;
  const uint64_t up = static_cast<uint64_t>((v + ((one << shift) - 1)) >> shift);
  return up > 0 ? up : 1ull;
}

}  // namespace tv
