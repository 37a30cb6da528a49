// balance.cu -- the router's step in training: top-k routing, the softmax
// weights, per-expert counts and the load-balance loss (forward), and the
// gradient of the logits from the loss and from the weights (backward).
//
// With p_t the softmax of token t's E logits and n the number of live tokens
// (unmasked, at least one logit above -inf):
//   counts_e = live slots routed to e,   f_e = counts_e E / (K n),
//   P_e = sum_t p_te / n,                loss = coef * sum_e f_e P_e.
// The counts are piecewise constant, so with g_e = d_loss coef f_e / n
//   d_logits_te = p_te (g_e - sum_j p_tj g_j)
//               + [e = id_tk] w_tk (dw_tk - sum_j w_tj dw_tj).
// Both passes read every logit once.  Dead tokens get ids -1, weights 0 and
// a zero gradient; no live token at all gives loss 0.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "moe.h"
#include "route_token.cuh"

namespace moe {

namespace {

constexpr unsigned kAllLanes = 0xFFFFFFFFu;
constexpr int kBalanceWarps = 8;
constexpr int kBalanceMaxBlocks = 304;  // two blocks per SM

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kAllLanes, v, off);
  return v;
}

// Tokens are dealt to the warps in turn; a warp keeps the column sums of its
// tokens' probabilities in registers (lane l holds experts l, l+32, ...), the
// block adds its warps' sums in warp order and writes one row of partials, so
// the sums do not depend on timing.
template <int MAXJ, typename T>
__global__ void __launch_bounds__(32 * kBalanceWarps)
    balance_forward_kernel(const T* __restrict__ logits, int64_t ld,
                           const uint8_t* __restrict__ mask, int tokens, int E, int K,
                           int32_t* __restrict__ ids, float* __restrict__ weights,
                           float* __restrict__ psum_out, int32_t* __restrict__ count_out) {
  __shared__ float s_sum[kBalanceWarps][MAXJ * 32];
  __shared__ int s_cnt[MAXJ * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < MAXJ * 32; e += blockDim.x) s_cnt[e] = 0;
  __syncthreads();
  float psum[MAXJ];
#pragma unroll
  for (int j = 0; j < MAXJ; ++j) psum[j] = 0.0f;
  for (int t = blockIdx.x * kBalanceWarps + warp; t < tokens; t += gridDim.x * kBalanceWarps) {
    const T* row = logits + static_cast<int64_t>(t) * ld;
    float x[MAXJ];
    uint32_t key[MAXJ];
#pragma unroll
    for (int j = 0; j < MAXJ; ++j) {
      const int e = lane + 32 * j;
      x[j] = e < E ? load_logit(row + e) : -INFINITY;
      // (a NaN's key may be 0, which marks an empty slot)
      key[j] = e < E ? max(logit_key(x[j]), 1u) : 0u;
    }
    float my_v = 0.0f;
    int my_i = 0;
    for (int k = 0; k < K; ++k) {
      uint32_t m = 0u;
#pragma unroll
      for (int j = 0; j < MAXJ; ++j) m = max(m, key[j]);
      const uint32_t wmax = __reduce_max_sync(kAllLanes, m);
      uint32_t idx = 0xFFFFFFFFu;
#pragma unroll
      for (int j = MAXJ - 1; j >= 0; --j)
        if (key[j] == wmax) idx = static_cast<uint32_t>(lane + 32 * j);
      const uint32_t widx = __reduce_min_sync(kAllLanes, idx);
      if (static_cast<int>(widx & 31u) == lane) {
#pragma unroll
        for (int j = 0; j < MAXJ; ++j)
          if (static_cast<uint32_t>(j) == (widx >> 5)) key[j] = 0u;
      }
      if (lane == k) {
        my_v = key_logit(wmax);
        my_i = static_cast<int>(widx);
      }
    }
    const float m = __shfl_sync(kAllLanes, my_v, 0);
    const bool live = (!mask || mask[t]) && m != -INFINITY;
    if (lane < K) {
      ids[static_cast<int64_t>(t) * K + lane] = live ? my_i : -1;
      if (live) atomicAdd(&s_cnt[my_i], 1);
    }
    const float ex = live && lane < K ? expf(my_v - m) : 0.0f;
    const float wsum = warp_sum(ex);
    if (lane < K) weights[static_cast<int64_t>(t) * K + lane] = live ? ex / wsum : 0.0f;
    if (!live) continue;
    float p[MAXJ], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < MAXJ; ++j) {
      p[j] = expf(x[j] - m);
      sum += p[j];
    }
    const float r = 1.0f / warp_sum(sum);
#pragma unroll
    for (int j = 0; j < MAXJ; ++j) psum[j] += p[j] * r;
  }
#pragma unroll
  for (int j = 0; j < MAXJ; ++j) s_sum[warp][lane + 32 * j] = psum[j];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kBalanceWarps; ++w) s += s_sum[w][e];
    psum_out[static_cast<int64_t>(blockIdx.x) * E + e] = s;
    count_out[static_cast<int64_t>(blockIdx.x) * E + e] = s_cnt[e];
  }
}

// One block: adds the partial rows in order, then the loss.
__global__ void __launch_bounds__(kMaxExperts)
    balance_finish_kernel(const float* __restrict__ psum, const int32_t* __restrict__ count,
                          int blocks, int E, int K, float coef, int32_t* __restrict__ counts,
                          float* __restrict__ mean_probs, float* __restrict__ loss) {
  __shared__ float s_dot[kMaxExperts / 32];
  __shared__ int s_slots[kMaxExperts / 32];
  const int e = threadIdx.x, warp = e >> 5, lane = e & 31;
  float p = 0.0f;
  int c = 0;
  if (e < E)
    for (int b = 0; b < blocks; ++b) {
      p += psum[static_cast<int64_t>(b) * E + e];
      c += count[static_cast<int64_t>(b) * E + e];
    }
  const int slots_w = __reduce_add_sync(kAllLanes, c);
  const float dot_w = warp_sum(static_cast<float>(c) * p);
  if (lane == 0) {
    s_slots[warp] = slots_w;
    s_dot[warp] = dot_w;
  }
  __syncthreads();
  int slots = 0;
  float dot = 0.0f;
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
    slots += s_slots[w];
    dot += s_dot[w];
  }
  const float n = static_cast<float>(slots / K);
  if (e < E) {
    counts[e] = c;
    if (mean_probs) mean_probs[e] = slots ? p / n : 0.0f;
  }
  if (e == 0) *loss = slots ? coef * (static_cast<float>(E) / static_cast<float>(K)) * (dot / n) / n : 0.0f;
}

template <int MAXJ, typename T>
__global__ void __launch_bounds__(32 * kBalanceWarps)
    balance_backward_kernel(const T* __restrict__ logits, int64_t ld,
                            int tokens, int E, int K, float coef,
                            const int32_t* __restrict__ ids, const float* __restrict__ weights,
                            const int32_t* __restrict__ counts, const float* __restrict__ d_loss,
                            const float* __restrict__ d_weights, T* __restrict__ d_logits,
                            int64_t ld_d) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // g_e of this lane's experts
  float g[MAXJ];
  int slots = 0;
#pragma unroll
  for (int j = 0; j < MAXJ; ++j) {
    const int e = lane + 32 * j;
    const int c = e < E ? counts[e] : 0;
    slots += c;
    g[j] = static_cast<float>(c);
  }
  slots = __reduce_add_sync(kAllLanes, slots);
  const float n = static_cast<float>(max(slots / K, 1));
  const float gs = d_loss ? *d_loss * coef * (static_cast<float>(E) / static_cast<float>(K)) / n / n : 0.0f;
#pragma unroll
  for (int j = 0; j < MAXJ; ++j) g[j] *= gs;
  for (int t = blockIdx.x * kBalanceWarps + warp; t < tokens; t += gridDim.x * kBalanceWarps) {
    const T* row = logits + static_cast<int64_t>(t) * ld;
    T* drow = d_logits + static_cast<int64_t>(t) * ld_d;
    float p[MAXJ], m = -INFINITY;
#pragma unroll
    for (int j = 0; j < MAXJ; ++j) {
      const int e = lane + 32 * j;
      p[j] = e < E ? load_logit(row + e) : -INFINITY;
      m = fmaxf(m, p[j]);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAllLanes, m, off));
    const int id = lane < K ? ids[static_cast<int64_t>(t) * K + lane] : -1;
    if (__shfl_sync(kAllLanes, id, 0) < 0) {  // a dead token
#pragma unroll
      for (int j = 0; j < MAXJ; ++j)
        if (lane + 32 * j < E) store_logit(drow + lane + 32 * j, 0.0f);
      continue;
    }
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < MAXJ; ++j) {
      p[j] = expf(p[j] - m);
      sum += p[j];
      dot += p[j] * g[j];
    }
    sum = warp_sum(sum);
    dot = warp_sum(dot) / sum;
    float wd = 0.0f;
    if (d_weights) {
      const float w = lane < K ? weights[static_cast<int64_t>(t) * K + lane] : 0.0f;
      const float dw = lane < K ? d_weights[static_cast<int64_t>(t) * K + lane] : 0.0f;
      wd = w * (dw - warp_sum(w * dw));
    }
    const float r = 1.0f / sum;
#pragma unroll
    for (int j = 0; j < MAXJ; ++j) p[j] = p[j] * r * (g[j] - dot);
    for (int k = 0; k < K; ++k) {
      const int e = __shfl_sync(kAllLanes, id, k);
      const float v = __shfl_sync(kAllLanes, wd, k);
#pragma unroll
      for (int j = 0; j < MAXJ; ++j)
        if (e == lane + 32 * j) p[j] += v;
    }
#pragma unroll
    for (int j = 0; j < MAXJ; ++j)
      if (lane + 32 * j < E) store_logit(drow + lane + 32 * j, p[j]);
  }
}

// One warp per token until every SM has two blocks, then several.
int balance_blocks(int T) {
  return std::max(1, std::min(kBalanceMaxBlocks, (T + kBalanceWarps - 1) / kBalanceWarps));
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

moe_status check_logits(const void* logits, int dtype, int64_t ld, int T, int E, int K) {
  if (T < 0 || E < 1 || K < 1 || K > E || ld < E) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || K > kMaxTopK || static_cast<int64_t>(T) * K > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!logits || !aligned_to(logits, dtype == MOE_DTYPE_F32 ? 4 : 2)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Calls f with the keys per lane that E needs (4 / 8 / 12 / 16) as a
// compile-time constant.
template <typename F>
cudaError_t by_keys(int E, F&& f) {
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 384) return f(std::integral_constant<int, 12>{});
  return f(std::integral_constant<int, 16>{});
}

template <typename T>
cudaError_t run_forward(const T* logits, int64_t ld, const uint8_t* mask, int tokens, int E, int K,
                        int32_t* ids, float* weights, float* psum, int32_t* count,
                        cudaStream_t s) {
  return by_keys(E, [&](auto maxj) {
    return launch_pdl(false, balance_forward_kernel<decltype(maxj)::value, T>,
                      dim3(balance_blocks(tokens)), dim3(32 * kBalanceWarps), 0, s, logits, ld,
                      mask, tokens, E, K, ids, weights, psum, count);
  });
}

template <typename T>
cudaError_t run_backward(const T* logits, int64_t ld, int tokens, int E, int K, float coef, const int32_t* ids, const float* weights,
                         const int32_t* counts, const float* d_loss, const float* d_weights,
                         T* d_logits, int64_t ld_d, cudaStream_t s) {
  return by_keys(E, [&](auto maxj) {
    return launch_pdl(false, balance_backward_kernel<decltype(maxj)::value, T>,
                      dim3(balance_blocks(tokens)), dim3(32 * kBalanceWarps), 0, s, logits, ld,
                      tokens, E, K, coef, ids, weights, counts, d_loss, d_weights, d_logits,
                      ld_d);
  });
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_workspace(int T, int E) {
  if (T < 0 || E < 1 || E > kMaxExperts) return 0;
  return static_cast<size_t>(balance_blocks(T)) * E * 8;
}

moe_status moe_balance_forward(const void* logits, int dtype, int64_t ld, const uint8_t* mask,
                               int T, int E, int K, float coef, int32_t* ids, float* weights,
                               int32_t* counts, float* mean_probs, float* loss, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const moe_status st = check_logits(logits, dtype, ld, T, E, K);
  if (st != MOE_OK) return st;
  if (!counts || !loss || !workspace || (T > 0 && (!ids || !weights))) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(counts, 4) ||
      !aligned_to(mean_probs, 4) || !aligned_to(loss, 4) || !aligned_to(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_balance_workspace(T, E)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = balance_blocks(T);
  float* psum = static_cast<float*>(workspace);
  int32_t* count = reinterpret_cast<int32_t*>(psum + static_cast<int64_t>(blocks) * E);
  cudaError_t e = dtype == MOE_DTYPE_F32
                      ? run_forward(static_cast<const float*>(logits), ld, mask, T, E, K, ids,
                                    weights, psum, count, s)
                      : run_forward(static_cast<const __nv_bfloat16*>(logits), ld, mask, T, E, K,
                                    ids, weights, psum, count, s);
  if (e == cudaSuccess)
    e = launch_pdl(false, balance_finish_kernel, dim3(1), dim3((E + 31) / 32 * 32), 0, s, psum,
                   count, blocks, E, K, coef, counts, mean_probs, loss);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_balance_backward(const void* logits, int dtype, int64_t ld, int T, int E, int K,
                                float coef, const int32_t* ids, const float* weights,
                                const int32_t* counts, const float* d_loss,
                                const float* d_weights, void* d_logits, int64_t ld_d,
                                void* stream) {
  const moe_status st = check_logits(logits, dtype, ld, T, E, K);
  if (st != MOE_OK) return st;
  if (ld_d < E) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!ids || !weights || !counts || !d_logits) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(counts, 4) ||
      !aligned_to(d_loss, 4) || !aligned_to(d_weights, 4) ||
      !aligned_to(d_logits, dtype == MOE_DTYPE_F32 ? 4 : 2))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == MOE_DTYPE_F32
          ? run_backward(static_cast<const float*>(logits), ld, T, E, K, coef, ids, weights,
                         counts, d_loss, d_weights, static_cast<float*>(d_logits), ld_d, s)
          : run_backward(static_cast<const __nv_bfloat16*>(logits), ld, T, E, K, coef, ids,
                         weights, counts, d_loss, d_weights,
                         static_cast<__nv_bfloat16*>(d_logits), ld_d, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
