// The 8-bit formats of the paged KV cache: a row's scale, its codes, and back.
#pragma once

#include <cuda_fp8.h>

#include "tv_common.cuh"

namespace tv {

constexpr int kKvMaxBatch = 4096;

// What a row's codes are made from: its scale and the factors of its values.
struct KvRowScale {
  float scale;   // stored beside the codes; NaN when the row is not finite
  float mul;     // e4m3: 1 / scale; int8: 1 / largest magnitude; 0: all codes are 0
  float top;     // int8: the largest magnitude, at least 2^-100
};

// `top` = largest magnitude of the row's bf16 values as bits 14..0 of bf16.
// Magnitudes of finite bf16 values order as those integers do, infinities
// (0x7f80) and NaN (above it) come last.
template <int kFmt>
__device__ __forceinline__ KvRowScale kv_row_scale(uint32_t top) {
  KvRowScale r;
  if constexpr (kFmt == TV_KV_E4M3) {
    // a = 2^E * m, 1 <= m < 2: 448 = 1.75 * 2^8, so n = E - 8, one more when
    // m > 1.75 (bf16 significand bits above 0x60), and not below -100
    int n = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
    n = max(n, -100);
    r.scale = __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
    r.mul = __uint_as_float(static_cast<uint32_t>(127 - n) << 23);   // n <= 120: exact, as is x * mul
    r.top = 0.0f;
  } else {
    r.top = fmaxf(__uint_as_float(top << 16), 7.888609052210118e-31f);         // 2^-100
    r.scale = __fdiv_rn(r.top, 127.0f);
    r.mul = __frcp_rn(r.top);
  }
  if (top >= 0x7f80u) {
    r.scale = __uint_as_float(0x7fc00000u);
    r.mul = 0.0f;
  }
  return r;
}

// The int8 code of x in the low byte: 127 x / top to the nearest integer. The
// product 127 x is exact (15 bits), and one Newton step from the reciprocal
// leaves the quotient within 2^-24 of itself, exactly where it is a float32
// number - so exactly at ties, integers and a half. Any other quotient of two
// bf16 numbers, 127 X / (A 2^k) with X, A < 2^8, is 1 / (254 X) > 2^-16 of
// itself away from the nearest tie and rounds the way the exact one does.
__device__ __forceinline__ uint32_t kv_int8_code(float x, const KvRowScale& r) {
  const float n = 127.0f * x;
  const float q = n * r.mul;
  const float y = fmaf(fmaf(-q, r.top, n), r.mul, q);
  return __float_as_uint(__fadd_rn(y, 12582912.0f));                 // 1.5 * 2^23: rounds to an integer
}

// (x.x * f, x.y * f) in one instruction, each rounded as on its own.
__device__ __forceinline__ float2 mul_both(float2 x, float f) {
  float2 r;
  asm("{ .reg .b64 a, b;\n"
      "  mov.b64 a, {%2, %3};\n"
      "  mov.b64 b, {%4, %4};\n"
      "  mul.rn.f32x2 a, a, b;\n"
      "  mov.b64 {%0, %1}, a; }"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(f));
  return r;
}

// Four values (two bf16 pairs) to four codes. (Paired instructions take 3 % off
// an e4m3 append of 16 to 26 MB; the int8 codes are slower with them.)
template <int kFmt>
__device__ __forceinline__ uint32_t kv_encode4(uint32_t a, uint32_t b, const KvRowScale& r) {
  if constexpr (kFmt == TV_KV_E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(mul_both(make_float2(bf16_lo(a), bf16_hi(a)), r.mul), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(mul_both(make_float2(bf16_lo(b), bf16_hi(b)), r.mul), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  } else {
    KvRowScale s = r;
    float x[4] = {bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b)};
    if (r.top > 1e30f) {               // 127 x must not overflow: the quotient of both by 2^20, exactly
      s.top *= 9.5367431640625e-07f;
      s.mul *= 1048576.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] *= 9.5367431640625e-07f;
    }
    const uint32_t lo = __byte_perm(kv_int8_code(x[0], s), kv_int8_code(x[1], s), 0x0040);
    const uint32_t hi = __byte_perm(kv_int8_code(x[2], s), kv_int8_code(x[3], s), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
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
