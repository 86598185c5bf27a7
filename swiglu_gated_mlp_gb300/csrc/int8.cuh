// The 8-bit integer format of tokens and of kept activations: a group of values
// x (a token's row, or a token's 128 columns of Gate or Up) is held as codes q
// and one fp32 scale s, x ~ q s, with
//   m = max(max |x|, 2^-100),   s = m / 127,   q = 127 x / m to the nearest.
// The floor keeps 127 / m finite; a group of zeros has codes 0. A group that
// holds an infinity or a NaN has the scale NaN, so that every value read back
// is NaN (its codes mean nothing).
#pragma once

#include <cstdint>

namespace swg {

constexpr int kKeepBlock = 128;  // columns of Gate or Up that share a scale

// Largest magnitude of three values; a NaN stays.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

struct QuantScale {
  float scale, inverse;  // s and 127 / m
};

// From the largest magnitude of a group (NaN or infinite: see above).
__device__ __forceinline__ QuantScale quant_scale(float largest) {
  const float m = largest < 7.888609052210118e-31f ? 7.888609052210118e-31f : largest;  // 2^-100
  QuantScale q;
  q.scale = largest <= 3.402823466e+38f ? __fdiv_rn(m, 127.0f) : __int_as_float(0x7fffffff);
  q.inverse = __fdiv_rn(127.0f, m);
  return q;
}

// 1.5 * 2^23: a sum with it is a whole number, rounded to even at halves, whose low
// byte is that of the integer. fmaf rounds the exact product once.
constexpr float kRoundMagic = 12582912.0f;

// Code of x in the low byte (the other bytes are not zero).
__device__ __forceinline__ uint32_t quant_code(float x, float inverse) {
  return __float_as_uint(fmaf(x, inverse, kRoundMagic));
}

// A scale as a power of two and a factor in [1, 2), s = power * factor: codes times the power are
// bf16 values exactly, and the factor goes elsewhere in the product. Zero, subnormal, infinite and
// NaN scales stay whole (factor 1).
struct ScaleParts {
  float power, factor;
};

__device__ __forceinline__ ScaleParts split_scale(float s) {
  const uint32_t bits = __float_as_uint(s), e = bits >> 23 & 0xffu;
  if (e == 0u || e == 0xffu) return ScaleParts{s, 1.0f};
  return ScaleParts{__uint_as_float(bits & 0xff800000u), __uint_as_float((bits & 0x007fffffu) | 0x3f800000u)};
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Four codes as fp32: with its sign bit flipped, byte q is the low byte of
// 2^23 + (q + 128), and taking 2^23 + 128 away is exact.
__device__ __forceinline__ void unpack_codes(uint32_t w, float (&v)[4]) {
  w ^= 0x80808080u;
  v[0] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)) - 8388736.0f;
  v[1] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441)) - 8388736.0f;
  v[2] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)) - 8388736.0f;
  v[3] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443)) - 8388736.0f;
}

}  // namespace swg
