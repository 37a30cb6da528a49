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
  __device__ __forceinline__ float quotient(float x) const {
    if (slow) return __fdiv_rn(x, scale);
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(-__fmaf_rn(q, scale, -x), r, q);
  }
  // four codes, element i in byte i
  __device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) const {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(quotient(a), quotient(b)),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(quotient(c), quotient(d)),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
};

// 16 bf16 values (pairs in v) of a block that eight neighbouring lanes share:
// their codes and the block's scale.  Called by whole warps.
__device__ __forceinline__ uint4 quantize_16(const uint32_t (&v)[8], float& scale) {
  float f[16];
  uint32_t amax = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    amax = max(amax, max(abs_bits(f[2 * i]), abs_bits(f[2 * i + 1])));
  }
#pragma unroll
  for (int off = 4; off; off >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
  const BlockQuant bq(amax);
  scale = bq.scale;
  return make_uint4(bq.code4(f[0], f[1], f[2], f[3]), bq.code4(f[4], f[5], f[6], f[7]),
                    bq.code4(f[8], f[9], f[10], f[11]), bq.code4(f[12], f[13], f[14], f[15]));
}

}  // namespace moe
