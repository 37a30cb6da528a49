// blockscale_quant.cuh -- e4m3 quantisation of a block of up to 128 values
// with one fp32 scale: s = amax / 448 and codes e4m3(x / s), both quotients
// rounded to nearest in fp32.
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

namespace moe {

constexpr uint32_t kInfBits = 0x7F800000u;

// The bits of |x|: ordered like the magnitudes, with NaN above infinity, so
// an integer maximum finds the largest magnitude and keeps a NaN.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// x / s without a divide per element: with r = RN(1 / s) and q = RN(x r), one
// Newton step on the residual, q - (q s - x) r, both steps fused.  For bf16 x
// and s = RN(amax / 448) with a bf16 amax (128 significands each; a test runs
// through all of them) this is RN(x / s) for every s in the fast range: the
// residual stays exact while s >= 2^-80, since any x whose residual would be
// subnormal is then below 2^-22 s, far under the smallest code.  For the
// fp32 values of the fused SwiGLU it is within an ulp.  The signs are
// arranged so that -0 stays -0.  Blocks of smaller scale take divides.
// amax == 0: s = 0 and zero codes; an infinity or NaN in the block: s = NaN
// and NaN codes.
struct BlockQuant {
  float scale, r;
  bool slow;
  __device__ __forceinline__ explicit BlockQuant(uint32_t amax_bits) {
    scale = amax_bits >= kInfBits ? __uint_as_float(0x7FC00000u)
                                  : __fdiv_rn(__uint_as_float(amax_bits), 448.0f);
    r = amax_bits == 0u ? 0.0f : __frcp_rn(scale);
    slow = scale < 0x1p-80f && amax_bits != 0u;
  }
  // codes of a pair, a's in the low byte
  __device__ __forceinline__ uint32_t code2(float a, float b) const {
    const float2 x = make_float2(a, b), s2 = make_float2(scale, scale), r2 = make_float2(r, r);
    const float2 q = __fmul2_rn(x, r2);
    const float2 e = __ffma2_rn(q, s2, make_float2(-a, -b));
    return __nv_cvt_float2_to_fp8x2(__ffma2_rn(make_float2(-e.x, -e.y), r2, q), __NV_SATFINITE,
                                    __NV_E4M3);
  }
  __device__ __forceinline__ uint32_t code2_slow(float a, float b) const {
    return __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)),
                                    __NV_SATFINITE, __NV_E4M3);
  }
  // four codes, element i in byte i
  __device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) const {
    if (slow) return code2_slow(a, b) | (code2_slow(c, d) << 16);
    return code2(a, b) | (code2(c, d) << 16);
  }
};

// 16 bf16 values (pairs in v) of a block that eight neighbouring lanes share:
// their codes and the block's scale.  Called by whole warps.
__device__ __forceinline__ uint4 quantize_16(const uint32_t (&v)[8], float& scale) {
  // the larger magnitude of each half-word, then of the two
  uint32_t m2 = v[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m2 = __vmaxu2(m2, v[i] & 0x7FFF7FFFu);
  uint32_t amax = max(m2 << 16, m2 & 0xFFFF0000u);
#pragma unroll
  for (int off = 4; off; off >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
  const BlockQuant bq(amax);
  scale = bq.scale;
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  uint32_t w[4];
  if (bq.slow) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = bq.code2_slow(lo(v[2 * i]), hi(v[2 * i])) |
             (bq.code2_slow(lo(v[2 * i + 1]), hi(v[2 * i + 1])) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = bq.code2(lo(v[2 * i]), hi(v[2 * i])) |
             (bq.code2(lo(v[2 * i + 1]), hi(v[2 * i + 1])) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace moe
