// The 8-bit formats of the paged KV cache: a row's scale, its codes, and back.
#pragma once

#include <cuda_fp8.h>

#include "tv_common.cuh"

namespace tv {

constexpr int kKvMaxBatch = 4096;

// What a row's codes are made from: its scale and the factor of its values.
struct KvRowScale {
  float scale;   // stored beside the codes; NaN when the row is not finite
  float mul;     // e4m3: 1 / scale; int8: 127 / largest magnitude; 0: all codes are 0
  float pre;     // int8: a power of two that keeps mul in range, applied first
};

// `top` = largest magnitude of the row's bf16 values as bits 14..0 of bf16.
// Magnitudes of finite bf16 values order as those integers do, infinities
// (0x7f80) and NaN (above it) come last.
template <int kFmt>
__device__ __forceinline__ KvRowScale kv_row_scale(uint32_t top) {
  KvRowScale r;
  const float a = __uint_as_float(top << 16);
  r.pre = 1.0f;
  if constexpr (kFmt == TV_KV_E4M3) {
    // a = 2^E * m, 1 <= m < 2: 448 = 1.75 * 2^8, so n = E - 8, one more when
    // m > 1.75 (bf16 significand bits above 0x60), and not below -100
    int n = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
    n = max(n, -100);
    r.scale = __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
    r.mul = __uint_as_float(static_cast<uint32_t>(127 - n) << 23);   // n <= 120: exact, as is x * mul
  } else {
    const float b = fmaxf(a, 7.888609052210118e-31f);                // 2^-100
    r.scale = __fdiv_rn(b, 127.0f);
    if (b > 1e30f) r.pre = 9.5367431640625e-07f;                     // 2^-20: keeps mul a normal number
    r.mul = __fdiv_rn(127.0f, b * r.pre);
  }
  if (top >= 0x7f80u) {
    r.scale = __uint_as_float(0x7fc00000u);
    r.mul = 0.0f;
  }
  return r;
}

// The int8 code of x in the low byte. The exact quotient Q = 127 x / a of two
// bf16 numbers is 127 X / (A 2^k) with X, A < 2^8, so unless it is a tie (an
// integer and a half) it lies at least |Q| / (254 X) > 2^-16 |Q| away from
// one. x * fl(127 / a) is within 2^-22 |Q| of it. So a product within
// 2^-18 |Q| of half an integer IS that number, and is set to it before it is
// rounded to even; every other one rounds as Q does.
__device__ __forceinline__ uint32_t kv_int8_code(float x, const KvRowScale& r) {
  const float magic = 12582912.0f;                                   // 1.5 * 2^23: rounds to an integer
  const float y = x * r.pre * r.mul;
  const float twice = __fadd_rn(__fadd_rn(2.0f * y, magic), -magic); // nearest half integer, doubled
  const float snapped = fabsf(2.0f * y - twice) <= 7.62939453125e-06f * fabsf(y) ? 0.5f * twice : y;
  return __float_as_uint(__fadd_rn(snapped, magic)) & 0xffu;
}

// Two values to two codes (first in the low byte).
template <int kFmt>
__device__ __forceinline__ uint32_t kv_encode2(float x, float y, const KvRowScale& r) {
  if constexpr (kFmt == TV_KV_E4M3) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x * r.mul, y * r.mul), __NV_SATFINITE, __NV_E4M3);
  } else {
    return kv_int8_code(x, r) | (kv_int8_code(y, r) << 8);
  }
}

// Two codes (low 16 bits) to the two float values they stand for before the scale.
template <int kFmt>
__device__ __forceinline__ float2 kv_decode2(uint32_t w) {
  if constexpr (kFmt == TV_KV_E4M3) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
    return __half22float2(__half2(h));
  } else {
    return make_float2(static_cast<float>(static_cast<int8_t>(w & 0xffu)),
                       static_cast<float>(static_cast<int8_t>((w >> 8) & 0xffu)));
  }
}

}  // namespace tv
