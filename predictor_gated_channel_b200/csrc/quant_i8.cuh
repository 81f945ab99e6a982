// quant_i8.cuh -- device side of the row-wise 8-bit quantisation
// (quant_i8.cu), shared with the kernels that quantise on the fly.
#pragma once

#include "sfn_internal.cuh"

namespace sfn {

// Largest |x| of a 16-byte chunk, as float32 bits (their integer order is the
// order of the values; an infinity is 0x7f800000 and NaNs lie above it).
template <class Elt>
__device__ __forceinline__ uint32_t abs_bits_max(const uint4 &v);
template <>
__device__ __forceinline__ uint32_t abs_bits_max<EltF32>(const uint4 &v) {
  return max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu),
             max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
}
template <>
__device__ __forceinline__ uint32_t abs_bits_max<EltBF16>(const uint4 &v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                              __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m << 16, m & 0xffff0000u);
}

// What a row's elements are quantised with, from its amax bits: x pre against
// amax (which is already times pre).  pre is 1, but a power of two for rows so small
// or so large that products with 127 or amax, or 127 / amax, would leave the range
// (an x that it makes a subnormal is far below amax / 254 and quantises to 0).
struct QuantScale {
  float amax, mult, scale, pre;
  bool zero, plain;  // plain: pre is 1
  __device__ __forceinline__ explicit QuantScale(uint32_t bits) {
    amax = __uint_as_float(bits);
    zero = bits == 0u || bits >= 0x7f800000u;
    scale = bits >= 0x7f800000u ? __int_as_float(0x7fc00000) : amax / 127.f;
    pre = amax < 1e-30f ? 0x1p100f : (amax > 1e30f ? 0x1p-100f : 1.f);
    amax *= pre;
    plain = !zero && pre == 1.f;
    mult = 127.f / amax;
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

// One value's integer, in the low bits of a float that adding 1.5 * 2^23
// rounded.  x mult is within 8e-6 of 127 x / amax (|x / amax| <= 1, one
// rounding of 2^-24), so that both round to the same integer unless it lies
// that close to half way between two; `near` then says so.
constexpr float kRound = 12582912.f;
constexpr float kNearHalf = 0.49998f;
__device__ __forceinline__ float quantize_fast(float x, float mult, float &near) {
  const float n = __fmaf_rn(x, mult, kRound);
  near = fmaxf(near, fabsf(__fmaf_rn(x, mult, -(n - kRound))));
  return n;
}

// Sets that right without a division: with n the candidate, n moves by one where
// the remainder e = 127 x - n amax has |e| > amax / 2, or where it is equal and n
// is odd.  (Exact halves are not rare in bf16: 0.26 % of normal values, some in
// nearly every row.)  Of a bf16 x the remainder is exact: 127 x and n amax have 15
// bits, and for n != 0 their exponents are close.  Of a float32 x the two products
// are taken in two parts each, exactly; the difference of the first parts is exact
// (they are within a factor of two, or n is 0), as is |e| - amax / 2 where it is
// small, and the second parts have 7 bits each.
template <class Elt>
__device__ __forceinline__ float quantize_settle(float x, float n, float amax) {
  const float k = n - kRound;
  float e, over;
  if (Elt::kBytes == 4) {
    // (named roundings: fused into the difference, a product would be taken whole)
    const float a = __fmul_rn(127.f, x), b = __fmul_rn(k, amax);
    const float rest = __fsub_rn(__fmaf_rn(127.f, x, -a), __fmaf_rn(k, amax, -b));
    e = __fsub_rn(a, b);
    over = __fadd_rn(__fmaf_rn(-0.5f, amax, fabsf(e)), e < 0.f ? -rest : rest);
  } else {
    e = __fmaf_rn(x, 127.f, -__fmul_rn(k, amax));
    over = __fmaf_rn(-0.5f, amax, fabsf(e));
  }
  // over > 0, or over == 0 and the integer is odd
  const bool move = __float_as_int(over) + (int)(__float_as_uint(n) & 1u) > 0;
  return move ? n + copysignf(1.f, e) : n;
}

// The integers of four values from the low bits of their floats.
__device__ __forceinline__ uint32_t pack_low_bytes(const float *n) {
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(n[j]);
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// A chunk of a row whose pre is not 1; not inlined, as it is rare.
template <class Elt>
__device__ __noinline__ typename QuantOut<Elt>::type quantize_scaled(uint4 v, float amax,
                                                                     float pre) {
  float f[Elt::kVec];
  Elt::unpack(v, f);
  typename QuantOut<Elt>::type out;
  uint32_t *w = reinterpret_cast<uint32_t *>(&out);
  const float mult = 127.f / amax;
  float near = 0.f;
#pragma unroll
  for (int i = 0; i < Elt::kVec; ++i) {
    f[i] *= pre;
    f[i] = quantize_settle<Elt>(f[i], quantize_fast(f[i], mult, near), amax);
  }
#pragma unroll
  for (int i = 0; i < Elt::kVec / 4; ++i) w[i] = pack_low_bytes(f + 4 * i);
  return out;
}

template <class Elt>
__device__ __forceinline__ typename QuantOut<Elt>::type quantize_chunk(const uint4 &v,
                                                                       const QuantScale &qs) {
  typename QuantOut<Elt>::type out = {};
  if (qs.plain) {
    float f[Elt::kVec], n[Elt::kVec];
    Elt::unpack(v, f);
    uint32_t *w = reinterpret_cast<uint32_t *>(&out);
    float near = 0.f;
#pragma unroll
    for (int i = 0; i < Elt::kVec; ++i) n[i] = quantize_fast(f[i], qs.mult, near);
    if (near > kNearHalf) {
#pragma unroll
      for (int i = 0; i < Elt::kVec; ++i) n[i] = quantize_settle<Elt>(f[i], n[i], qs.amax);
    }
#pragma unroll
    for (int i = 0; i < Elt::kVec / 4; ++i) w[i] = pack_low_bytes(n + 4 * i);
  } else if (!qs.zero) {
    out = quantize_scaled<Elt>(v, qs.amax, qs.pre);
  }
  return out;
}

}  // namespace sfn
