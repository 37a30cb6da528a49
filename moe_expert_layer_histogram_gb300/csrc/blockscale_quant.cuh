// blockscale_quant.cuh -- e4m3 quantisation of a block of up to 128 values
// with one fp32 scale: s = amax / 448 and codes e4m3(x / s), both quotients
// rounded to nearest in fp32.
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

namespace moe {

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kFastBits = (127u - 71u) << 23;  // 2^-71: 448 times and more of it, s >= 2^-80

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
// s == 0 (amax 0, or an fp32 amax up to 2^-149 * 224, whose quotient rounds to
// 0): zero codes; an infinity or NaN in the block: s = NaN and NaN codes.
struct BlockQuant {
  float scale, r;
  bool slow;
  BlockQuant() = default;
  __device__ __forceinline__ explicit BlockQuant(uint32_t amax_bits) {
    scale = amax_bits >= kInfBits ? __uint_as_float(0x7FC00000u)
                                  : __fdiv_rn(__uint_as_float(amax_bits), 448.0f);
    r = scale == 0.0f ? 0.0f : __frcp_rn(scale);
    slow = scale < 0x1p-80f && scale != 0.0f;
  }
  // The same for a bf16 block with is_fast(amax), without a branch: the
  // scale by the Newton step of the codes (exact in the same way), r by the
  // approximate reciprocal and one step of its own.
  __device__ __forceinline__ static bool is_fast(uint32_t amax_bits) {
    return amax_bits - kFastBits < kInfBits - kFastBits || amax_bits == 0u;
  }
  __device__ __forceinline__ static BlockQuant of_bf16(uint32_t amax_bits) {
    BlockQuant b;
    const float a = __uint_as_float(amax_bits), q = a * (1.0f / 448.0f);
    b.scale = fmaf(-fmaf(q, 448.0f, -a), 1.0f / 448.0f, q);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b.scale));
    r = fmaf(-fmaf(r, b.scale, -1.0f), r, r);
    b.r = amax_bits == 0u ? 0.0f : r;
    b.slow = false;
    return b;
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

// N times 16 bf16 values (pairs in v[k]), each of a block that eight
// neighbouring lanes share: their codes and the blocks' scales.  Called by
// whole warps.  There is one branch for all of them, so that the N chains of
// shuffles and quotients overlap.
template <int N>
__device__ __forceinline__ void quantize_16(const uint32_t (&v)[N][8], uint4 (&codes)[N],
                                            float (&scale)[N]) {
  uint32_t amax[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    // the larger magnitude of each half-word, then of the two
    uint32_t m2 = v[k][0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m2 = __vmaxu2(m2, v[k][i] & 0x7FFF7FFFu);
    amax[k] = max(m2 << 16, m2 & 0xFFFF0000u);
  }
#pragma unroll
  for (int off = 4; off; off >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) amax[k] = max(amax[k], __shfl_xor_sync(0xFFFFFFFFu, amax[k], off));
  bool fast = true;
#pragma unroll
  for (int k = 0; k < N; ++k) fast &= BlockQuant::is_fast(amax[k]);
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  if (__all_sync(0xFFFFFFFFu, fast)) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const BlockQuant bq = BlockQuant::of_bf16(amax[k]);
      scale[k] = bq.scale;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = bq.code2(lo(v[k][2 * i]), hi(v[k][2 * i])) |
               (bq.code2(lo(v[k][2 * i + 1]), hi(v[k][2 * i + 1])) << 16);
      codes[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const BlockQuant bq(amax[k]);
    scale[k] = bq.scale;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = bq.code4(lo(v[k][2 * i]), hi(v[k][2 * i]), lo(v[k][2 * i + 1]), hi(v[k][2 * i + 1]));
    codes[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace moe
