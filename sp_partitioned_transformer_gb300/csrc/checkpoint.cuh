// Activations held in 8 bits: e4m3 codes with one power-of-two scale for 32
// neighbouring values of a row.
//
//   value = code·2^(byte − 127),  byte = the smallest with max|v| ≤ 448·2^(byte − 127)
//
// (448: the largest e4m3 number.)  A power of two makes the division exact, so a
// value is rounded once, to its nearest code; a scale that fits the group exactly would
// only move which values fall among e4m3's subnormals.
// Infinities and NaN become the code NaN and do not enter the group's scale.
#pragma once

#include "common.cuh"

namespace tpmlp {

constexpr int CKPT_GROUP = 32;

// The largest finite |v| of a group as the float's bits (ordered like integers).
__device__ __forceinline__ uint32_t ckpt_abs(float v) {
  const uint32_t a = __float_as_uint(v) & 0x7fffffffu;
  return a < 0x7f800000u ? a : 0u;
}

// The group's scale byte: with |v| = m·2^k, 1 ≤ m < 2, 448 = 1.75·2^8: k − 8, one
// more where m > 1.75 (the addition then carries into the exponent).
__device__ __forceinline__ uint32_t ckpt_byte(uint32_t top) {
  const int e = static_cast<int>((top + 0x1fffffu) >> 23) - 8;
  return static_cast<uint32_t>(e > 0 ? e : 0);
}

// 2^(127 − byte), for the bytes that ckpt_byte gives (≤ 247).
__device__ __forceinline__ float ckpt_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^(byte − 127); 255 stands for NaN.
__device__ __forceinline__ float ckpt_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}

// Four values to four codes, the first in the lowest byte.  v·0 + v leaves a finite
// v alone and makes an infinity NaN, which the conversion would take for 448.
// NO_INF: the caller has looked for infinities.
template <bool NO_INF = false>
__device__ __forceinline__ uint32_t ckpt_encode4(const float* v, float inverse) {
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = v[i] * inverse;
    q[i] = NO_INF ? t : fmaf(t, 0.0f, t);
  }
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[1]), "f"(q[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[3]), "f"(q[2]));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The numbers of four codes, without their scale.
__device__ __forceinline__ void ckpt_numbers4(uint32_t codes, float2* v) {
  uint32_t a, b;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(static_cast<uint16_t>(codes)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(static_cast<uint16_t>(codes >> 16)));
  v[0] = __half22float2(*reinterpret_cast<const __half2*>(&a));
  v[1] = __half22float2(*reinterpret_cast<const __half2*>(&b));
}

__device__ __forceinline__ void ckpt_decode4(uint32_t codes, float scale, float* v) {
  float2 n[2];
  ckpt_numbers4(codes, n);
  v[0] = n[0].x * scale;
  v[1] = n[0].y * scale;
  v[2] = n[1].x * scale;
  v[3] = n[1].y * scale;
}

// A code may round the group's largest value up past the storage type's range: the
// restored value is then the type's largest.
template <int DT>
__device__ __forceinline__ float ckpt_largest() {
  return DT == DT_F16 ? 65504.0f : DT == DT_BF16 ? __uint_as_float(0x7f7f0000u) : __uint_as_float(0x7f7fffffu);
}
template <int DT>
__device__ __forceinline__ float ckpt_in_range(float v) {
  const float top = ckpt_largest<DT>();
  return v > top ? top : v < -top ? -top : v;
}
// The same for a value of a block's U, which may be packed from float32 beyond float16's range:
// only what can have rounded up past the end (to 2^16, or 2^128) is brought back, and an
// overflow of the type's stays one in Y.
template <int DT>
__device__ __forceinline__ float ckpt_back_in_range(float v) {
  const float next = DT == DT_F16 ? 65536.0f : __uint_as_float(0x7f800000u);
  return fabsf(v) == next ? copysignf(ckpt_largest<DT>(), v) : v;
}

// Whether a group with this byte may hold such values: 256·2^(byte − 127) lies past the
// type's largest.  (float16: 2^16; bf16 and float32: 2^128, an infinity.)
template <int DT>
__device__ __forceinline__ bool ckpt_near_end(uint32_t byte) {
  return byte >= (DT == DT_F16 ? 135u : 247u);
}

}  // namespace tpmlp
