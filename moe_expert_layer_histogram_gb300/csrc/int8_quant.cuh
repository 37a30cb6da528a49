// int8_quant.cuh -- 8-bit codes of a row: s = amax / 127 and round(x / s) to even
// within +-127, both quotients rounded to nearest in fp32.
//
// With r = 1 / s rounded to nearest, q = x r, e = x - q s and q' = q + e r, each
// rounded once, q' is the correctly rounded quotient x / s (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990): one reciprocal a row and three operations an element.  Adding a number of
// 1.5 2^23's size rounds q' to a whole number, to even, whose code is in the sum's
// last bits.  Scales below 2^-100, whose remainders could underflow, divide.
#pragma once

#include <cmath>
#include <cstdint>

namespace moe {

// Four codes in a word to two words of two f16 each: a code with 128 added under the
// f16 1024's bits is 1152 + code.
__device__ __forceinline__ void i8_widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  lo = __byte_perm(w, 0x64646464u, 0x4140);
  hi = __byte_perm(w, 0x64646464u, 0x4342);
  asm("sub.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
  asm("sub.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
}

// The scale of a row from the bits of its largest magnitude (NaN where an infinity
// or NaN is in the row: their bits are above those of every number).
__device__ __forceinline__ float i8_scale(uint32_t amax) {
  return amax >= 0x7F800000u ? NAN : __fdiv_rn(__uint_as_float(amax), 127.0f);
}

struct I8Coder {
  // Low half of the sum's bits: 0x6480 + code, which as f16 is 1152 + code.
  static constexpr float kMagic = 12582912.0f + 25728.0f;
  float s, r;
  __device__ explicit I8Coder(float scale) : s(scale), r(scale >= 0x1p-100f ? 1.0f / scale : 0.0f) {}

  __device__ static uint32_t divided(float v, float s) {
    const float q = s > 0.0f ? fminf(fmaxf(__fdiv_rn(v, s), -127.0f), 127.0f) : 0.0f;
    return static_cast<uint32_t>(0x6480 + __float2int_rn(q));
  }

  // 0x6480 + code of eight values, two to a word.
  __device__ __forceinline__ void biased(const float (&v)[8], uint32_t (&w)[4]) const {
    uint32_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __fmul_rn(v[i], r), e = __fmaf_rn(-q, s, v[i]);
      t[i] = __float_as_uint(__fadd_rn(__fmaf_rn(e, r, q), kMagic));
    }
    if (!(r > 0.0f)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = divided(v[i], s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __byte_perm(t[2 * i], t[2 * i + 1], 0x5410);
  }

  // The codes as f16.
  __device__ __forceinline__ uint4 f16(const float (&v)[8]) const {
    uint32_t w[4];
    biased(v, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("sub.f16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(0x64806480u));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }

  // The codes as bytes.
  __device__ __forceinline__ uint2 bytes(const float (&v)[8]) const {
    uint32_t w[4];
    biased(v, w);
    // (the low byte of 0x6480 + code is code + 128)
    return make_uint2(__byte_perm(w[0], w[1], 0x6420) ^ 0x80808080u,
                      __byte_perm(w[2], w[3], 0x6420) ^ 0x80808080u);
  }
};

// silu(g) u, both clamped.
__device__ __forceinline__ float clamp_to(float v, float limit) {
  // (a NaN stays one; fminf and fmaxf would drop it)
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(-limit));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(limit));
  return v;
}

__device__ __forceinline__ float swiglu(float g, float u, float clamp) {
  g = clamp_to(g, clamp);
  u = clamp_to(u, clamp);
  // e^-g by the hardware's power of two, off by two ulp and |g| 2^-24 of itself,
  // and an approximate quotient of two ulp
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  return __fdividef(g, 1.0f + e) * u;
}

}  // namespace moe
