// The 8-bit formats of the paged KV cache: a row's scale, its codes, and back.
#pragma once

#include <cuda_fp8.h>

#include "tv_common.cuh"

namespace tv {

constexpr int kKvMaxBatch = 4096;

// What a row's codes are made from: its scale and the factors of its values.
struct KvRowScale {
  float scale;   // stored beside the codes; NaN when the row is not finite
  float mul;     // e4m3: 1 / scale, a power of two, so x * mul is x / scale exactly
  float div;     // int8: code = rint(x * mul / div)
};

// `top` = largest magnitude of the row's bf16 values as bits 14..0 of bf16.
// Magnitudes of finite bf16 values order as those integers do, infinities
// (0x7f80) and NaN (above it) come last.
template <int kFmt>
__device__ __forceinline__ KvRowScale kv_row_scale(uint32_t top) {
  KvRowScale r;
  const bool finite = top < 0x7f80u;
  const float a = __uint_as_float(top << 16);
  if constexpr (kFmt == TV_KV_E4M3) {
    // a = 2^E * m, 1 <= m < 2: 448 = 1.75 * 2^8, so n = E - 8, one more when
    // m > 1.75 (bf16 significand bits above 0x60), and not below -100
    int n = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
    n = max(n, -100);
    r.scale = __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
    r.mul = __uint_as_float(static_cast<uint32_t>(127 - n) << 23);   // n <= 120
    r.div = 1.0f;
  } else {
    const float b = fmaxf(a, 7.888609052210118e-31f);                // 2^-100
    r.scale = __fdiv_rn(b, 127.0f);
    // 127 x must not overflow: large rows are scaled down, exactly
    const float down = b > 1e30f ? 9.5367431640625e-07f : 1.0f;      // 2^-20
    r.mul = 127.0f * down;
    r.div = b * down;
  }
  if (!finite) {
    r.scale = __uint_as_float(0x7fc00000u);
    r.mul = 0.0f;
    r.div = 1.0f;
  }
  return r;
}

// Two values to two codes (first in the low byte). bf16 x 127 and the float32
// quotient: 127 x has 15 significant bits and the divisor 8, so a quotient
// that is not a tie lies at least 2^-9 of an integer step away from one and
// the quotient's own rounding cannot reach it; exact ties come out exact.
template <int kFmt>
__device__ __forceinline__ uint32_t kv_encode2(float x, float y, const KvRowScale& r) {
  if constexpr (kFmt == TV_KV_E4M3) {
    if (r.mul == 0.0f) return 0u;                                    // 0 * infinity is NaN
    return __nv_cvt_float2_to_fp8x2(make_float2(x * r.mul, y * r.mul), __NV_SATFINITE, __NV_E4M3);
  } else {
    if (r.mul == 0.0f) return 0u;
    const int a = __float2int_rn(__fdiv_rn(x * r.mul, r.div));
    const int b = __float2int_rn(__fdiv_rn(y * r.mul, r.div));
    return (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8);
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
