// blockscale.cu -- products of e4m3 matrices with one fp32 scale per block of
// 128: activations carry a scale per row and 128 columns, weights one per
// 128 x 128 block.
//
//   quantise:  s = amax / 448 and codes e4m3(x / s) of each row's 128-column
//              blocks, both quotients rounded to fp32; an all-zero block has
//              s = 0 and zero codes, a block with an infinity or NaN s = NaN
//              and NaN codes (so every product with it is NaN).
//   product:   y[m][n] = sum_b sa[m][b] sw[n/128][b] sum_{k in b} a[m][k] w[n][k]
//              over the rows of each expert, fp32 sums, one rounding to bf16.
//   SwiGLU:    the same for gate and up rows, h = silu(gate) up in fp32,
//              quantised as above.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "moe.h"
#include "quant.cuh"

namespace moe {

namespace {

constexpr int kBlk = 128;

__host__ __device__ __forceinline__ int blocks_of(int n) { return (n + kBlk - 1) / kBlk; }

// ---------------------------------------------------------------- quantise
// One warp per (row, block); lane l holds columns 4l .. 4l+3.
__global__ void __launch_bounds__(256)
    blockscale_quantize_kernel(const __nv_bfloat16* __restrict__ x, int64_t ldx, int x_rows,
                               const int32_t* __restrict__ slots, int top_k, int rows, int cols,
                               uint8_t* __restrict__ codes, int64_t ld_codes,
                               float* __restrict__ scales, int64_t ld_scales) {
  const int kb = blocks_of(cols);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= static_cast<int64_t>(rows) * kb) return;
  const int r = static_cast<int>(unit / kb), b = static_cast<int>(unit % kb);
  const int src = slots ? slots[r] / top_k : r;
  const bool in = src >= 0 && src < x_rows;
  float v[4], amax = 0.0f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = b * kBlk + lane * 4 + i;
    v[i] = in && c < cols ? __bfloat162float(x[src * ldx + c]) : 0.0f;
    amax = fmaxf(amax, fabsf(v[i]));
    bad |= !(fabsf(v[i]) < INFINITY);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
  bad = __any_sync(0xFFFFFFFFu, bad);
  const float s = bad ? NAN : __fdiv_rn(amax, 448.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = b * kBlk + lane * 4 + i;
    if (c < cols)
      codes[r * ld_codes + c] = bad ? 0x7Fu : s == 0.0f ? 0u : float_to_e4m3(__fdiv_rn(v[i], s));
  }
  if (lane == 0) scales[b * ld_scales + r] = s;
}

// ---------------------------------------------------------------- product
struct ProductArgs {
  const uint8_t* a;        // [M, lda]
  int64_t lda;
  const float* a_scales;   // [ceil(K/128), ld_as]
  int64_t ld_as;
  const uint8_t* w;
  int64_t ldw;
  const float* w_scales;
  const int32_t* offsets;  // [E+1] or null (one expert, all rows)
  int E, M, N, K;
  int transpose_w;
  void* out;
  int64_t ldo;
};

__device__ __forceinline__ void expert_rows(const ProductArgs& p, int e, int& r0, int& r1) {
  r0 = p.offsets ? min(max(p.offsets[e], 0), p.M) : 0;
  r1 = p.offsets ? min(max(p.offsets[e + 1], r0), p.M) : p.M;
}

// One thread per output element.
__device__ __forceinline__ float product_dot(const ProductArgs& p, int e, int m, int n) {
  const int wr = p.transpose_w ? p.K : p.N, wc = p.transpose_w ? p.N : p.K;
  const uint8_t* w = p.w + static_cast<int64_t>(e) * wr * p.ldw;
  const float* ws = p.w_scales + static_cast<int64_t>(e) * blocks_of(wr) * blocks_of(wc);
  float acc = 0.0f;
  for (int b = 0; b < blocks_of(p.K); ++b) {
    float s = 0.0f;
    for (int k = b * kBlk; k < min(p.K, (b + 1) * kBlk); ++k) {
      const float av = e4m3_to_float(p.a[m * p.lda + k]);
      const float wv = e4m3_to_float(p.transpose_w ? w[k * p.ldw + n] : w[n * p.ldw + k]);
      s = fmaf(av, wv, s);
    }
    const float sw = p.transpose_w ? ws[b * blocks_of(wc) + n / kBlk]
                                   : ws[(n / kBlk) * blocks_of(wc) + b];
    acc = fmaf(p.a_scales[b * p.ld_as + m] * sw, s, acc);
  }
  return acc;
}

__global__ void __launch_bounds__(128) blockscale_matmul_kernel(const ProductArgs p) {
  int r0, r1;
  expert_rows(p, blockIdx.z, r0, r1);
  const int n = blockIdx.x * 128 + threadIdx.x;
  if (n >= p.N) return;
  for (int m = r0 + blockIdx.y; m < r1; m += gridDim.y)
    static_cast<__nv_bfloat16*>(p.out)[m * p.ldo + n] =
        __float2bfloat16_rn(product_dot(p, blockIdx.z, m, n));
}

// p.N = 2 I; one block per 128 columns of h.
__global__ void __launch_bounds__(128)
    blockscale_swiglu_kernel(const ProductArgs p, float clamp, float* h_scales, int64_t ld_hs) {
  __shared__ float s_max[4];
  int r0, r1;
  expert_rows(p, blockIdx.z, r0, r1);
  const int I = p.N / 2, n = blockIdx.x * 128 + threadIdx.x;
  for (int m = r0 + blockIdx.y; m < r1; m += gridDim.y) {
    const float g = fminf(fmaxf(product_dot(p, blockIdx.z, m, n), -clamp), clamp);
    const float u = fminf(fmaxf(product_dot(p, blockIdx.z, m, I + n), -clamp), clamp);
    const float h = g / (1.0f + expf(-g)) * u;
    float amax = fabsf(h);
    for (int off = 16; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    const bool bad = __syncthreads_or(!(fabsf(h) < INFINITY));
    amax = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const float s = bad ? NAN : __fdiv_rn(amax, 448.0f);
    static_cast<uint8_t*>(p.out)[m * p.ldo + n] =
        bad ? 0x7Fu : s == 0.0f ? 0u : float_to_e4m3(__fdiv_rn(h, s));
    if (threadIdx.x == 0) h_scales[blockIdx.x * ld_hs + m] = s;
    __syncthreads();
  }
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The operands of both products.  TMA wants 16-byte aligned bases and row
// strides; the scales and offsets are read as 32-bit words.
moe_status check_product(const ProductArgs& p) {
  if (p.M < 0 || p.N < 1 || p.K < 1 || p.E < 1 || (!p.offsets && p.E != 1))
    return MOE_ERR_INVALID_ARG;
  if (p.E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  if (p.lda < p.K || p.ld_as < p.M || p.ldw < (p.transpose_w ? p.N : p.K))
    return MOE_ERR_INVALID_ARG;
  if (p.M == 0) return MOE_OK;
  if (!p.a || !p.a_scales || !p.w || !p.w_scales || !p.out) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(p.a, 16) || p.lda % 16 || !aligned_to(p.w, 16) || p.ldw % 16 ||
      !aligned_to(p.a_scales, 4) || !aligned_to(p.w_scales, 4) || !aligned_to(p.offsets, 4))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_blockscale_quantize(const void* x, int64_t ldx, int x_rows, const int32_t* slots,
                                   int top_k, int rows, int cols, void* codes, int64_t ld_codes,
                                   float* scales, int64_t ld_scales, void* stream) {
  if (rows < 0 || cols < 1 || x_rows < 0 || ldx < cols || ld_codes < cols || ld_scales < rows)
    return MOE_ERR_INVALID_ARG;
  if (slots ? top_k < 1 : x_rows < rows) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if ((!x && x_rows > 0) || !codes || !scales || !aligned_to(x, 2) || !aligned_to(slots, 4) ||
      !aligned_to(scales, 4))
    return MOE_ERR_INVALID_ARG;
  const int64_t grid = (static_cast<int64_t>(rows) * blocks_of(cols) + 7) / 8;
  if (grid > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const cudaError_t e = launch_pdl(
      false, blockscale_quantize_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0,
      static_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(x), ldx, x_rows, slots,
      top_k, rows, cols, static_cast<uint8_t*>(codes), ld_codes, scales, ld_scales);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_blockscale_matmul(const void* a, int64_t lda, const float* a_scales, int64_t ld_as,
                                 const void* w, int64_t ldw, const float* w_scales,
                                 const int32_t* offsets, int E, int M, int N, int K,
                                 int transpose_w, void* out, int64_t ldo, void* stream) {
  const ProductArgs p{static_cast<const uint8_t*>(a), lda, a_scales, ld_as,
                      static_cast<const uint8_t*>(w), ldw, w_scales, offsets, E, M, N, K,
                      transpose_w != 0, out, ldo};
  const moe_status st = check_product(p);
  if (st != MOE_OK) return st;
  if (ldo < N || !aligned_to(out, 2)) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const cudaError_t e =
      launch_pdl(false, blockscale_matmul_kernel, dim3((N + 127) / 128, std::min(M, 256), E),
                 dim3(128), 0, static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_blockscale_swiglu(const void* a, int64_t lda, const float* a_scales, int64_t ld_as,
                                 const void* w13, int64_t ldw, const float* w13_scales,
                                 const int32_t* offsets, int E, int M, int I, int K,
                                 float clamp_limit, void* h, int64_t ldh, float* h_scales,
                                 int64_t ld_hs, void* stream) {
  if (I < 1 || I > (1 << 29)) return MOE_ERR_INVALID_ARG;
  if (I % kBlk) return MOE_ERR_UNSUPPORTED;
  const ProductArgs p{static_cast<const uint8_t*>(a), lda, a_scales, ld_as,
                      static_cast<const uint8_t*>(w13), ldw, w13_scales, offsets, E, M, 2 * I, K,
                      0, h, ldh};
  const moe_status st = check_product(p);
  if (st != MOE_OK) return st;
  if (ldh < I || ld_hs < M) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!h_scales || !aligned_to(h_scales, 4) || !aligned_to(h, 16) || ldh % 16)
    return MOE_ERR_INVALID_ARG;
  const float clamp =
      clamp_limit > 0.0f && std::isfinite(clamp_limit) ? clamp_limit : INFINITY;
  const cudaError_t e =
      launch_pdl(false, blockscale_swiglu_kernel, dim3(I / 128, std::min(M, 256), E), dim3(128), 0,
                 static_cast<cudaStream_t>(stream), p, clamp, h_scales, ld_hs);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
