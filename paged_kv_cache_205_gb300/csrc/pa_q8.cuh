// pa_q8.cuh -- the 8-bit cache format: e4m3 values with one power-of-two
// scale for each page, kv head and K or V.
//
//   pool    [num_blocks][2][BT][8][64] e4m3 (index 0 = K, 1 = V)
//   scales  [num_blocks][2][8] fp32, a value is byte * scale
//
// scale = 2^e, e the smallest exponent >= kMinExp with
//   max |k| <= 316 * 2^e (over the page's keys before their rotation)
//   max |v| <= 448 * 2^e.
// e4m3 reaches 448; a rotation lengthens a component by at most sqrt(2) and
// 316 sqrt(2) < 448, so K's scale holds whatever the position, and it does
// not depend on the rotation's rounding.  A floating-point byte keeps its
// relative precision (half a step: 2^-4) over 15 binades below the largest
// value, so a scale finer than a power of two would buy range, not
// precision; a power of two multiplies exactly, and a page whose scale grows
// keeps its bytes' mantissas (only values that become subnormal round
// again).
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kMinExp = -117;                        // byte * scale stays a normal bf16
constexpr int kMaxExp = 120;                         // covers bf16's largest value
constexpr int kQ8HeadBytes = kD;                     // one token, one head: 64
constexpr int kQ8TokBytes = kHkv * kD;               // one token, all kv heads: 512
constexpr uint32_t kMantK = 30, kMantV = 96;         // 316 = (1 + 30/128) 2^8, 448 = (1 + 96/128) 2^8

// Largest finite magnitude of two packed bf16 and `top` (a bf16 pattern
// without its sign); infinities and NaN do not count.
__device__ __forceinline__ uint32_t q8_top(uint32_t pair, uint32_t top) {
  const uint32_t a = pair & 0x7fffu, b = (pair >> 16) & 0x7fffu;
  top = max(top, a < 0x7f80u ? a : 0u);
  return max(top, b < 0x7f80u ? b : 0u);
}

// The scale's exponent for the largest magnitude `top` (a bf16 pattern).
__device__ __forceinline__ int q8_exponent(uint32_t top, uint32_t mant) {
  return max(kMinExp, static_cast<int>(top >> 7) - 135 + ((top & 127u) > mant ? 1 : 0));
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The exponent of a stored scale, or a value below kMinExp when it is no
// power of two of the format's range.
__device__ __forceinline__ int q8_scale_exponent(float scale) {
  const int u = __float_as_int(scale);
  const int e = (u >> 23) - 127;
  return (u & 0x7fffff) == 0 && u > 0 && e >= kMinExp && e <= kMaxExp ? e : kMinExp - 1;
}

// Two fp32 to packed e4m3 (lo in the low byte), round to nearest even; what
// is not finite becomes NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  constexpr float kBig = 3.3e38f;
  const float nan = __int_as_float(0x7fffffff);
  lo = fabsf(lo) <= kBig ? lo : nan;
  hi = fabsf(hi) <= kBig ? hi : nan;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The same for values none of which is infinite (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_plain(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two packed e4m3 to two packed f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair) {
  uint32_t r;
  const uint16_t p = static_cast<uint16_t>(pair);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(p));
  return r;
}

// Four bf16 (two packed words) times `inv` to four packed e4m3.  The product
// with a power of two is exact in fp32, so each value rounds once.
__device__ __forceinline__ uint32_t bf16x4_to_e4m3x4(uint32_t w0, uint32_t w1, float inv) {
  const float2 a = bf16x2_to_float2(w0), b = bf16x2_to_float2(w1);
  return e4m3x2(a.x * inv, a.y * inv) | (e4m3x2(b.x * inv, b.y * inv) << 16);
}

// Four e4m3 bytes brought from scale to scale / ratio (ratio a power of two).
__device__ __forceinline__ uint32_t e4m3x4_rescale(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t h = e4m3x2_to_f16x2(w >> (16 * half));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    out |= e4m3x2(f.x * ratio, f.y * ratio) << (16 * half);
  }
  return out;
}

}  // namespace pa
