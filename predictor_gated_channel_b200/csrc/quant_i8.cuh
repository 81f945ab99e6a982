// quant_i8.cuh -- device side of the row-wise 8-bit quantisation
// (quant_i8.cu), shared with the kernels that quantise on the fly.
#pragma once

#include "sfn_internal.cuh"

namespace sfn {

// Largest |x| of a 16-byte chunk, as float32 bits (their integer order is the
// order of the values; an infinity is 0x7f800000 and NaNs lie above it).
template <class Elt>
__device__ __forceinline__ uint32_t abs_bits_max(const uint4 &v) {
  float f[Elt::kVec];
  Elt::unpack(v, f);
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < Elt::kVec; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}

// What a row's elements are quantised with, from its amax bits.
struct QuantScale {
  float amax, inv, pre, scale;
  bool zero, guarded;
  __device__ __forceinline__ explicit QuantScale(uint32_t bits) {
    amax = __uint_as_float(bits);
    zero = bits == 0u || bits >= 0x7f800000u;
    // 127 x must not overflow: scale x and amax by an exact power of two
    pre = amax > 1e36f ? 0.00390625f : 1.f;
    scale = bits >= 0x7f800000u ? __int_as_float(0x7fc00000) : amax / 127.f;
    amax *= pre;
    guarded = amax < 1e-30f;  // 1 / amax could overflow
    inv = zero || guarded ? 0.f : 1.f / amax;
  }
  // rint(127 x / amax).  t * inv is within 3e-5 of the rounded quotient
  // (|t / amax| <= 127, two roundings of 2^-24 each), so rint agrees unless
  // it lies that close to half way between integers; those divide.
  __device__ __forceinline__ int operator()(float x) const {
    if (zero) return 0;
    const float t = 127.f * (x * pre);
    float r = t * inv;
    const float n = rintf(r);
    if (guarded || fabsf(fabsf(r - n) - 0.5f) < 1e-4f) return (int)rintf(t / amax);
    return (int)n;
  }
};

template <class Elt>
struct QuantOut;
template <>
struct QuantOut<EltBF16> {
  using type = uint2;  // 8 values
};
template <>
struct QuantOut<EltF32> {
  using type = uint32_t;  // 4 values
};

__device__ __forceinline__ uint32_t pack_i8x4(int a, int b, int c, int d) {
  return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8) | ((uint32_t)(c & 0xff) << 16) |
         ((uint32_t)d << 24);
}

template <class Elt>
__device__ __forceinline__ typename QuantOut<Elt>::type quantize_chunk(const uint4 &v,
                                                                       const QuantScale &qs);
template <>
__device__ __forceinline__ uint32_t quantize_chunk<EltF32>(const uint4 &v, const QuantScale &qs) {
  float f[4];
  EltF32::unpack(v, f);
  return pack_i8x4(qs(f[0]), qs(f[1]), qs(f[2]), qs(f[3]));
}
template <>
__device__ __forceinline__ uint2 quantize_chunk<EltBF16>(const uint4 &v, const QuantScale &qs) {
  float f[8];
  EltBF16::unpack(v, f);
  return make_uint2(pack_i8x4(qs(f[0]), qs(f[1]), qs(f[2]), qs(f[3])),
                    pack_i8x4(qs(f[4]), qs(f[5]), qs(f[6]), qs(f[7])));
}

}  // namespace sfn
