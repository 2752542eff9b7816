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

// A vector at any address: one load or store instruction, as the hardware takes
// global accesses of any alignment.
template <typename V>
__device__ __forceinline__ V load_any(const void* p) {
  V v;
  __builtin_memcpy(&v, p, sizeof v);
  return v;
}

template <typename V>
__device__ __forceinline__ void store_any(void* p, V v) {
  __builtin_memcpy(p, &v, sizeof v);
}

// The cnt <= 8 values from base[at] on (dt 0 fp32, 1 bf16, 4 fp16) as fp32,
// zeros after them.
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t at, int cnt, float (&v)[8]) {
  if constexpr (DT == 0) {
    const float* p = static_cast<const float*>(base) + at;
    if (cnt >= 8) {
      const f32x4 a = load_any<f32x4>(p);
      const f32x4 b = load_any<f32x4>(p + 4);
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
    u32x4 w = {0u, 0u, 0u, 0u};
    if (cnt >= 8) {
      w = load_any<u32x4>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < cnt) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = half_to_f32((uint16_t)(w[i >> 1] >> (16 * (i & 1))), DT == 4);
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

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t m) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, CTRL, 0xF, 0xF, false);
}

// max of m over lanes l and l ^ 16, and over l and l ^ 32 (MAX: any maximum).
template <typename MAX>
__device__ __forceinline__ uint32_t max_xor16(uint32_t m, MAX mx) {
  const auto r = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  return mx(r[0], r[1]);
}

template <typename MAX>
__device__ __forceinline__ uint32_t max_xor32(uint32_t m, MAX mx) {
  const auto r = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  return mx(r[0], r[1]);
}

struct MaxU32 {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};

// The largest of m over the G consecutive lanes of a group (G a power of two):
// lane moves within rows of 16 (quad permutations and mirrors), then swaps of
// rows, all without an LDS round trip.
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
  if constexpr (G >= 2) m = max(m, dpp_u32<0xB1>(m));   // lane ^ 1
  if constexpr (G >= 4) m = max(m, dpp_u32<0x4E>(m));   // lane ^ 2
  if constexpr (G >= 8) m = max(m, dpp_u32<0x141>(m));  // mirror of 8: the other four
  if constexpr (G >= 16) m = max(m, dpp_u32<0x140>(m));  // mirror of 16: the other eight
  if constexpr (G >= 32) m = max_xor16(m, MaxU32());
  if constexpr (G >= 64) m = max_xor32(m, MaxU32());
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
