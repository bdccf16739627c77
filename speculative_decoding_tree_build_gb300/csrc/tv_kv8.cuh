// The 8-bit formats of the paged KV cache: a row's scale, its codes, and back.
#pragma once

#include <cuda_fp8.h>

#include "tv_common.cuh"

namespace tv {

constexpr int kKvMaxBatch = 4096;

// What a row's codes are made from: its scale and the factors of its values.
struct KvRowScale {
  float scale;   // stored beside the codes; NaN when the row is not finite
  float mul;     // e4m3: 1 / scale; int8: 127 / largest magnitude; 0: all codes are 0
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
  } else {
    const float largest = fmaxf(__uint_as_float(top << 16), 7.888609052210118e-31f);     // 2^-100
    r.scale = __fdiv_rn(largest, 127.0f);
    r.mul = __fdiv_rn(127.0f, largest);
  }
  if (top >= 0x7f80u) {
    r.scale = __uint_as_float(0x7fc00000u);
    r.mul = 0.0f;
  }
  return r;
}

// The int8 code of x in the low byte: the exact quotient q = 127 x / top to the
// nearest integer, ties to even. mul is 127 / top within 2^-24 of itself, so x mul
// is within |q| 2^-24 < 2^-17 of q; the sum with 384, rounded once, lies in [256,
// 512), where float32 has steps of 2^-15. A q that ends in exactly a half, or an
// integer, is a step, so the sum lands on it. Any other q = 127 X 2^s / A (X, A <
// 2^8) lies at least 2^s / A = |q| / (127 X) from the nearest half, which is 1.543
// 10^-5 or more next to 0.5 and three times that next to 1.5; half a step and the
// error of x mul there are 1.529 10^-5, so it stays on its side. The second sum is
// exact up to its rounding to an integer.
__device__ __forceinline__ uint32_t kv_int8_code(float x, const KvRowScale& r) {
  return __float_as_uint(__fadd_rn(fmaf(x, r.mul, 384.0f), 12582912.0f - 384.0f));   // 1.5 * 2^23 + q
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

// Four values (two bf16 pairs) to four codes. (The paired product takes 3 % off an
// e4m3 append of 16 to 26 MB.)
template <int kFmt>
__device__ __forceinline__ uint32_t kv_encode4(uint32_t a, uint32_t b, const KvRowScale& r) {
  if constexpr (kFmt == TV_KV_E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(mul_both(make_float2(bf16_lo(a), bf16_hi(a)), r.mul), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(mul_both(make_float2(bf16_lo(b), bf16_hi(b)), r.mul), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  } else {
    const uint32_t lo = __byte_perm(kv_int8_code(bf16_lo(a), r), kv_int8_code(bf16_hi(a), r), 0x0040);
    const uint32_t hi = __byte_perm(kv_int8_code(bf16_lo(b), r), kv_int8_code(bf16_hi(b), r), 0x0040);
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
    // code + 128 = u in the last bits of 2^23 + u, then minus 2^23 + 128: exact, and 3 to 5 % off
    // a small int8 call against conversions
    const uint32_t u = w ^ 0x8080u;
    return make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - 8388736.0f,
                       __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - 8388736.0f);
  }
}

}  // namespace tv
