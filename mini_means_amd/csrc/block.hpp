// Device building blocks of the block codes: scales, encoding, number types.
#pragma once

#include "common.hpp"

namespace emk {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kInfBits = 0x7F800000u;

// Eight consecutive values as fp32 (dt 0 fp32, 1 bf16, 4 fp16). VEC: p is
// 16-byte aligned and holds all eight; else only the first `cnt` are read.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* base, int64_t at, int cnt, float (&v)[8]) {
  if constexpr (DT == 0) {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (VEC) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p);
      const f32x4 b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < cnt ? p[i] : 0.0f;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    uint16_t h[8];
    if constexpr (VEC) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = i < cnt ? p[i] : (uint16_t)0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = half_to_f32(h[i], DT == 4);
  }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The largest |v[i]| of the lane as fp32 bits (their order is that of the
// values; infinities and NaN compare above every finite value).
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  return m;
}

__device__ __forceinline__ uint32_t amax8_finite(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = abs_bits(v[i]);
    m = max(m, b < kInfBits ? b : 0u);
  }
  return m;
}

// E8M0 byte (e + 127) of a block whose largest finite magnitude has the bits
// a: with a = 1.f 2^E and L = 1.g 2^EL, a <= L 2^e holds first at
// e = E - EL + (f > g). Subnormal a falls under the lower end of the range.
template <bool I8>
__device__ __forceinline__ uint32_t scale_byte(uint32_t a) {
  constexpr int EL = I8 ? 6 : 8;                             // 127, 448
  constexpr uint32_t G = I8 ? 0x7E0000u : 0x600000u;         // 1.984375, 1.75
  const int b = (int)(a >> 23) - EL + ((a & 0x7FFFFFu) > G ? 1 : 0);
  return a == 0 ? 127u : (uint32_t)max(b, 0);
}

// 2^-(byte - 127): at most 2^127 (byte 0), at least 2^-122 here.
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); byte 0 is the fp32 subnormal 2^-127, byte 255 NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Codes of four values. `odd`: some value of the block is not finite, so
// infinities are saturated by hand (a clamp alone would lose the NaN).
template <bool I8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv,
                                           bool odd) {
  float y[4] = {a * inv, b * inv, c * inv, d * inv};
  if constexpr (I8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float r = __builtin_rintf(y[i]);
      if (odd) r = r != r ? 0.0f : fminf(fmaxf(r, -127.0f), 127.0f);
      w |= ((uint32_t)(int)r & 0xFFu) << (8 * i);
    }
    return w;
  } else {
    if (odd) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[i] = y[i] != y[i] ? y[i] : fminf(fmaxf(y[i], -448.0f), 448.0f);
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
    return (uint32_t)w;
  }
}

template <bool I8>
__device__ __forceinline__ u32x2 codes8(const float (&v)[8], float inv, bool odd) {
  return u32x2{codes4<I8>(v[0], v[1], v[2], v[3], inv, odd),
               codes4<I8>(v[4], v[5], v[6], v[7], inv, odd)};
}

// The largest of m over the G consecutive lanes of a group (G a power of two).
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  return m;
}

// Two values rounded to a 16-bit type.
template <int OT>  // 1 bf16, 4 fp16
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (OT == 1)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}

}  // namespace emk
