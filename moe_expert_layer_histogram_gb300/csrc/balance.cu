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
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "moe.h"
#include "ptx.cuh"
#include "route_token.cuh"

namespace moe {

namespace {

constexpr unsigned kAllLanes = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kAllLanes, v, off);
  return v;
}

// A row of E logits over a warp: lane l holds experts 128 i + 4 l .. + 3 in
// x[4 i ..], so an aligned row (VEC) is one 16-byte (bf16: 8-byte) load per
// 128 experts.  Past E: `fill`.
template <int MAXI, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float fill,
                                         float (&x)[4 * MAXI]) {
#pragma unroll
  for (int i = 0; i < MAXI; ++i) {
    const int e = 128 * i + 4 * lane;
    if (VEC && e + 4 <= E) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(row + e));
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[4 * i + c] = e + c < E ? __ldg(row + e + c) : fill;
    }
  }
}
template <int MAXI, bool VEC>
__device__ __forceinline__ void load_row(const __nv_bfloat16* __restrict__ row, int E, int lane,
                                         float fill, float (&x)[4 * MAXI]) {
#pragma unroll
  for (int i = 0; i < MAXI; ++i) {
    const int e = 128 * i + 4 * lane;
    if (VEC && e + 4 <= E) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + e));
      x[4 * i] = __uint_as_float(v.x << 16);
      x[4 * i + 1] = __uint_as_float(v.x & 0xFFFF0000u);
      x[4 * i + 2] = __uint_as_float(v.y << 16);
      x[4 * i + 3] = __uint_as_float(v.y & 0xFFFF0000u);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[4 * i + c] = e + c < E ? __bfloat162float(row[e + c]) : fill;
    }
  }
}

template <int MAXI, bool VEC>
__device__ __forceinline__ void store_row(float* __restrict__ row, int E, int lane,
                                          const float (&x)[4 * MAXI]) {
#pragma unroll
  for (int i = 0; i < MAXI; ++i) {
    const int e = 128 * i + 4 * lane;
    if (VEC && e + 4 <= E) {
      *reinterpret_cast<float4*>(row + e) =
          make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (e + c < E) row[e + c] = x[4 * i + c];
    }
  }
}
template <int MAXI, bool VEC>
__device__ __forceinline__ void store_row(__nv_bfloat16* __restrict__ row, int E, int lane,
                                          const float (&x)[4 * MAXI]) {
#pragma unroll
  for (int i = 0; i < MAXI; ++i) {
    const int e = 128 * i + 4 * lane;
    if (VEC && e + 4 <= E) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(x[4 * i], x[4 * i + 1]),
                           hi = __floats2bfloat162_rn(x[4 * i + 2], x[4 * i + 3]);
      *reinterpret_cast<uint2*>(row + e) = make_uint2(reinterpret_cast<const uint32_t&>(lo),
                                                      reinterpret_cast<const uint32_t&>(hi));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (e + c < E) row[e + c] = __float2bfloat16_rn(x[4 * i + c]);
    }
  }
}

// The K largest logits, value descending and lower index first on ties
// (-0 == +0): lane k < K receives the k-th expert.
//
// Each logit becomes one 32-bit word: the top 23 bits of its order-preserving
// key, then 511 - e.  The words differ, so one redux.sync per round finds the
// winner and its index.  Every lane keeps its two largest words: a lane that
// wins moves the second up, and only a lane that wins a third time (one token
// in ten at K = 8) looks through its words again.  A bf16 logit's key has 16
// bits, so the words order as the logits do.  Of fp32 logits two may agree
// in 23 bits and not in the rest; if that happens within the first K + 1
// words (about one token in fifty of N(0,1) logits), the rounds are done again
// on full keys, with a second reduction for the index.
template <int MAXI, bool EXACT>
__device__ __forceinline__ int top_k(const float (&x)[4 * MAXI], int E, int K, int lane) {
  uint32_t word[4 * MAXI], first = 0u, second = 0u;
#pragma unroll
  for (int j = 0; j < 4 * MAXI; ++j) {
    const int e = 128 * (j >> 2) + 4 * lane + (j & 3);
    // the key: sign bit flipped, the other bits too where it was set (x + 0
    // turns -0 into +0 and any NaN into the positive one, which comes first)
    const int32_t b = __float_as_int(x[j] + 0.0f);
    const uint32_t key = static_cast<uint32_t>(b) ^ (static_cast<uint32_t>(b >> 31) | 0x80000000u);
    word[j] = e < E ? (key & 0xFFFFFE00u) | static_cast<uint32_t>(511 - e) : 0u;
    second = max(second, min(first, word[j]));
    first = max(first, word[j]);
  }
  uint32_t mine = 0u;
  const int rounds = EXACT ? K : min(K + 1, E);
  for (int k = 0; k < rounds; ++k) {
    const uint32_t w = __reduce_max_sync(kAllLanes, first);
    if (lane == k) mine = w;
    const bool won = first == w;
    first = won ? second : first;
    second = won ? 0u : second;
    if (__any_sync(kAllLanes, won && first == 0u)) {
      uint32_t next = 0u;
#pragma unroll
      for (int j = 0; j < 4 * MAXI; ++j) next = max(next, word[j] < w ? word[j] : 0u);
      if (won) first = next;
    }
  }
  if (!EXACT) {
    const uint32_t before = __shfl_up_sync(kAllLanes, mine, 1);
    const bool same = lane > 0 && lane < rounds && (before >> 9) == (mine >> 9);
    if (__any_sync(kAllLanes, same)) {
      uint32_t key[4 * MAXI];
#pragma unroll
      for (int j = 0; j < 4 * MAXI; ++j)
        // (x + 0 again: every NaN is the same positive one, the largest key)
        key[j] = 128 * (j >> 2) + 4 * lane + (j & 3) < E ? logit_key(x[j] + 0.0f) : 0u;
      int id = 0;
      for (int k = 0; k < K; ++k) {
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 4 * MAXI; ++j) m = max(m, key[j]);
        const uint32_t wmax = __reduce_max_sync(kAllLanes, m);
        uint32_t idx = 0xFFFFFFFFu;
#pragma unroll
        for (int j = 4 * MAXI - 1; j >= 0; --j)
          if (key[j] == wmax) idx = static_cast<uint32_t>(128 * (j >> 2) + 4 * lane + (j & 3));
        const uint32_t widx = __reduce_min_sync(kAllLanes, idx);
#pragma unroll
        for (int j = 0; j < 4 * MAXI; ++j)
          if (widx == static_cast<uint32_t>(128 * (j >> 2) + 4 * lane + (j & 3))) key[j] = 0u;
        if (lane == k) id = static_cast<int>(widx);
      }
      return id;
    }
  }
  return 511 - static_cast<int>(mine & 511u);
}

// exp of a difference d of at most 0, in one multiply and the hardware's power
// of two: off by its two ulp and by |d| 2^-24 of itself, the product's rounding
// (some ten ulp at d = -20, where the value is 2e-9 of the row's largest).
__device__ __forceinline__ float exp_diff(float d) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d * kLog2e));
  return r;
}

// The routing of the tokens that this warp takes in turn, and the sums of
// their probabilities (psum: this lane's experts) and slots (s_cnt, shared).
template <int MAXI, bool VEC, typename T>
__device__ __forceinline__ void route_tokens(const T* __restrict__ logits, int64_t ld,
                                             const uint8_t* __restrict__ mask, int tokens, int E,
                                             int K, int first, int step,
                                             int32_t* __restrict__ ids, float* __restrict__ weights,
                                             float (&psum)[4 * MAXI], int* s_cnt) {
  const int lane = threadIdx.x & 31;
  for (int t = first; t < tokens; t += step) {
    const T* row = logits + static_cast<int64_t>(t) * ld;
    const bool unmasked = !mask || mask[t];
    float x[4 * MAXI];
    load_row<MAXI, VEC>(row, E, lane, -INFINITY, x);
    const int id = top_k<MAXI, sizeof(T) == 2>(x, E, K, lane);
    const float v = lane < K ? to_f32(row[id]) : -INFINITY;
    const float m = __shfl_sync(kAllLanes, v, 0);
    const bool live = unmasked && m != -INFINITY;
    const float ex = live && lane < K ? expf(v - m) : 0.0f;
    const float wsum = warp_sum(ex);
    if (lane < K) {
      ids[static_cast<int64_t>(t) * K + lane] = live ? id : -1;
      weights[static_cast<int64_t>(t) * K + lane] = live ? ex / wsum : 0.0f;
      if (live) atomicAdd(&s_cnt[id], 1);
    }
    if (!live) continue;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 4 * MAXI; ++j) {
      x[j] = exp_diff(x[j] - m);  // past E: exp(-inf) = 0
      sum += x[j];
    }
    const float r = 1.0f / warp_sum(sum);
#pragma unroll
    for (int j = 0; j < 4 * MAXI; ++j) psum[j] = fmaf(x[j], r, psum[j]);
  }
}

// counts, mean probabilities and the loss from the sums of thread e = expert
// (all threads of a block of at most 1024 call it; p = c = 0 past E).
__device__ __forceinline__ void finish(int e, float p, int c, int E, int K, float coef,
                                       int32_t* __restrict__ counts,
                                       float* __restrict__ mean_probs, float* __restrict__ loss) {
  __shared__ float s_dot[32];
  __shared__ int s_slots[32];
  const int slots_w = __reduce_add_sync(kAllLanes, c);
  const float dot_w = warp_sum(static_cast<float>(c) * p);
  if ((threadIdx.x & 31) == 0) {
    s_slots[threadIdx.x >> 5] = slots_w;
    s_dot[threadIdx.x >> 5] = dot_w;
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
  if (e == 0)
    *loss = slots ? coef * (static_cast<float>(E) / static_cast<float>(K)) * (dot / n) / n : 0.0f;
}

// Tokens are dealt to the warps in turn; a warp keeps the column sums of its
// tokens' probabilities in registers, the block adds its warps' sums in warp
// order and writes one row of partials, so the sums do not depend on timing.
constexpr int kBalanceWarps = 32;

template <int MAXI, bool VEC, typename T>
__global__ void __launch_bounds__(32 * kBalanceWarps)
    balance_forward_kernel(const T* __restrict__ logits, int64_t ld,
                           const uint8_t* __restrict__ mask, int tokens, int E, int K,
                           int32_t* __restrict__ ids, float* __restrict__ weights,
                           float* __restrict__ psum_out, int32_t* __restrict__ count_out) {
  pdl_launch_dependents();
  extern __shared__ float s_sum[];  // [kBalanceWarps][MAXI * 128]
  __shared__ int s_cnt[MAXI * 128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < MAXI * 128; e += blockDim.x) s_cnt[e] = 0;
  __syncthreads();
  float psum[4 * MAXI];
#pragma unroll
  for (int j = 0; j < 4 * MAXI; ++j) psum[j] = 0.0f;
  route_tokens<MAXI, VEC>(logits, ld, mask, tokens, E, K, warp * gridDim.x + blockIdx.x,
                          gridDim.x * kBalanceWarps, ids, weights, psum, s_cnt);
#pragma unroll
  for (int i = 0; i < MAXI; ++i)
    *reinterpret_cast<float4*>(&s_sum[warp * MAXI * 128 + 128 * i + 4 * lane]) =
        make_float4(psum[4 * i], psum[4 * i + 1], psum[4 * i + 2], psum[4 * i + 3]);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.0f;
#pragma unroll 8
    for (int w = 0; w < kBalanceWarps; ++w) s += s_sum[w * MAXI * 128 + e];
    psum_out[static_cast<int64_t>(blockIdx.x) * E + e] = s;
    count_out[static_cast<int64_t>(blockIdx.x) * E + e] = s_cnt[e];
  }
}

// Few tokens: the whole forward in one cluster of up to eight CTAs, one warp
// per token; the CTAs' sums are joined in rank order through distributed
// shared memory, so there is no second launch and no workspace.  Against the
// kernels for many tokens: 64 tokens of 64 experts 4.9 us and 7.1, 256 5.7 and
// 7.3, 512 7.6 and 7.5, 512 of 384 experts 10.4 and 8.8 (with a launch less on
// the host), 1024 of 64 11.0 and 7.3.
constexpr int kSmallCluster = 8;
constexpr int kSmallTokens = 2 * kBalanceWarps * kSmallCluster;

__device__ __forceinline__ uint32_t cluster_word(const void* local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];"
               : "=r"(v)
               : "r"(mapa_shared(smem_u32(local), rank))
               : "memory");
  return v;
}

// A cluster of kFinishRanks blocks adds the partial rows: within a block,
// groups of threads take every so many-th row of their expert and are added in
// order, then the blocks' sums in rank order.  (One block alone read the 1.9 MB
// of a 32K-token batch's rows in about 30 us.)
constexpr int kFinishThreads = 1024;
constexpr int kFinishRanks = 8;

__global__ void __cluster_dims__(kFinishRanks, 1, 1) __launch_bounds__(kFinishThreads)
    balance_finish_kernel(const float* psum, const int32_t* count, int blocks, int E, int K,
                          float coef, int32_t* counts, float* mean_probs, float* loss) {
  __shared__ float s_p[kFinishThreads];
  __shared__ int s_c[kFinishThreads];
  pdl_wait();
  const int width = (E + 31) / 32 * 32, groups = kFinishThreads / width;
  const int e = threadIdx.x % width, grp = threadIdx.x / width;
  const uint32_t rank = cluster_ctarank();
  float p = 0.0f;
  int c = 0;
  if (e < E && grp < groups) {
#pragma unroll 8
    for (int b = rank * groups + grp; b < blocks; b += groups * kFinishRanks) {
      p += psum[static_cast<int64_t>(b) * E + e];
      c += count[static_cast<int64_t>(b) * E + e];
    }
  }
  s_p[threadIdx.x] = p;
  s_c[threadIdx.x] = c;
  __syncthreads();
  if (grp == 0) {
    for (int g = 1; g < groups; ++g) {
      p += s_p[g * width + e];
      c += s_c[g * width + e];
    }
    s_p[e] = p;
    s_c[e] = c;
  }
  __syncwarp();
  cluster_sync();
  if (rank == 0) {
    p = 0.0f;
    c = 0;
    if (grp == 0)
      for (uint32_t k = 0; k < kFinishRanks; ++k) {
        p += __uint_as_float(cluster_word(&s_p[e], k));
        c += static_cast<int>(cluster_word(&s_c[e], k));
      }
    finish(grp == 0 ? e : E, p, c, E, K, coef, counts, mean_probs, loss);
  }
  __syncwarp();
  cluster_sync();  // the other ranks' shared memory stays until it has been read
}

template <int MAXI, bool VEC, typename T>
__global__ void __launch_bounds__(32 * kBalanceWarps)
    balance_small_kernel(const T* __restrict__ logits, int64_t ld,
                         const uint8_t* __restrict__ mask, int tokens, int E, int K, float coef,
                         int32_t* __restrict__ ids, float* __restrict__ weights,
                         int32_t* __restrict__ counts, float* __restrict__ mean_probs,
                         float* __restrict__ loss) {
  extern __shared__ float s_sum[];  // [kBalanceWarps][MAXI * 128]
  __shared__ int s_cnt[MAXI * 128];
  __shared__ float s_total[MAXI * 128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), ranks = gridDim.x;
  for (int e = threadIdx.x; e < MAXI * 128; e += blockDim.x) s_cnt[e] = 0;
  __syncthreads();
  float psum[4 * MAXI];
#pragma unroll
  for (int j = 0; j < 4 * MAXI; ++j) psum[j] = 0.0f;
  // (neighbouring tokens in different CTAs: few tokens use all of them)
  route_tokens<MAXI, VEC>(logits, ld, mask, tokens, E, K, warp * ranks + rank,
                          kBalanceWarps * ranks, ids, weights, psum, s_cnt);
#pragma unroll
  for (int i = 0; i < MAXI; ++i)
    *reinterpret_cast<float4*>(&s_sum[warp * MAXI * 128 + 128 * i + 4 * lane]) =
        make_float4(psum[4 * i], psum[4 * i + 1], psum[4 * i + 2], psum[4 * i + 3]);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.0f;
    for (int w = 0; w < kBalanceWarps; ++w) s += s_sum[w * MAXI * 128 + e];
    s_total[e] = s;
  }
  __syncwarp();
  cluster_sync();
  if (rank == 0) {
    const int e = threadIdx.x;
    float p = 0.0f;
    int c = 0;
    if (e < E)
      for (uint32_t k = 0; k < ranks; ++k) {
        p += __uint_as_float(cluster_word(&s_total[e], k));
        c += static_cast<int>(cluster_word(&s_cnt[e], k));
      }
    finish(e, p, c, E, K, coef, counts, mean_probs, loss);
  }
  __syncwarp();
  cluster_sync();  // the other ranks' shared memory stays until it has been read
}

constexpr int kBackWarps = 8;

template <int MAXI, bool VEC, typename T>
__global__ void __launch_bounds__(32 * kBackWarps)
    balance_backward_kernel(const T* __restrict__ logits, int64_t ld, int tokens, int E, int K,
                            float coef, const int32_t* __restrict__ ids,
                            const float* __restrict__ weights, const int32_t* __restrict__ counts,
                            const float* __restrict__ d_loss, const float* __restrict__ d_weights,
                            T* __restrict__ d_logits, int64_t ld_d) {
  __shared__ float s_row[kBackWarps][MAXI * 128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // g_e of this lane's experts
  float g[4 * MAXI];
  int slots = 0;
#pragma unroll
  for (int j = 0; j < 4 * MAXI; ++j) {
    const int e = 128 * (j >> 2) + 4 * lane + (j & 3);
    const int c = e < E ? counts[e] : 0;
    slots += c;
    g[j] = static_cast<float>(c);
  }
  slots = __reduce_add_sync(kAllLanes, slots);
  const float n = static_cast<float>(max(slots / K, 1));
  const float gs =
      d_loss ? *d_loss * coef * (static_cast<float>(E) / static_cast<float>(K)) / n / n : 0.0f;
#pragma unroll
  for (int j = 0; j < 4 * MAXI; ++j) g[j] *= gs;
  float* mine = s_row[warp];
  for (int t = blockIdx.x * kBackWarps + warp; t < tokens; t += gridDim.x * kBackWarps) {
    const int id = lane < K ? ids[static_cast<int64_t>(t) * K + lane] : -1;
    float w = 0.0f, dw = 0.0f;
    if (d_weights && lane < K) {
      w = weights[static_cast<int64_t>(t) * K + lane];
      dw = d_weights[static_cast<int64_t>(t) * K + lane];
    }
    float p[4 * MAXI];
    load_row<MAXI, VEC>(logits + static_cast<int64_t>(t) * ld, E, lane, -INFINITY, p);
    T* drow = d_logits + static_cast<int64_t>(t) * ld_d;
    if (__shfl_sync(kAllLanes, id, 0) < 0) {  // a dead token
#pragma unroll
      for (int j = 0; j < 4 * MAXI; ++j) p[j] = 0.0f;
      store_row<MAXI, VEC>(drow, E, lane, p);
      continue;
    }
    uint32_t key = 0u;
#pragma unroll
    for (int j = 0; j < 4 * MAXI; ++j) key = max(key, logit_key(p[j]));
    const float m = key_logit(__reduce_max_sync(kAllLanes, key));
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < 4 * MAXI; ++j) {
      p[j] = exp_diff(p[j] - m);
      sum += p[j];
      dot = fmaf(p[j], g[j], dot);
    }
    sum = warp_sum(sum);
    const float r = 1.0f / sum;
    dot = warp_sum(dot) * r;
#pragma unroll
    for (int j = 0; j < 4 * MAXI; ++j) p[j] = p[j] * r * (g[j] - dot);
    if (d_weights) {
      // the K selected experts' part, added where the row lies in shared memory
      const float part = w * (dw - warp_sum(w * dw));
#pragma unroll
      for (int i = 0; i < MAXI; ++i)
        *reinterpret_cast<float4*>(mine + 128 * i + 4 * lane) =
            make_float4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
      __syncwarp();
      if (id >= 0 && id < E) mine[id] += part;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < MAXI; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(mine + 128 * i + 4 * lane);
        p[4 * i] = v.x, p[4 * i + 1] = v.y, p[4 * i + 2] = v.z, p[4 * i + 3] = v.w;
      }
    }
    store_row<MAXI, VEC>(drow, E, lane, p);
  }
}

// Forward: one block of 32 warps per SM (a row of partial sums each), a token
// per warp until there are more.  Backward: blocks of 8 warps, four to an SM.
constexpr int kBalanceBlocks = 152;
constexpr int kBackBlocks = 4 * 152;
// Most tokens: a warp's next token (the stride is that of all warps) stays in 32 bits.
constexpr int kBalanceMaxTokens = INT32_MAX - 65535;
static_assert(kBalanceBlocks * kBalanceWarps <= 65535 && kBackBlocks * kBackWarps <= 65535);

int balance_blocks(int T) {
  return std::max(1, std::min(kBalanceBlocks, (T + kBalanceWarps - 1) / kBalanceWarps));
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

moe_status check_logits(const void* logits, int dtype, int64_t ld, int T, int E, int K) {
  if (T < 0 || E < 1 || K < 1 || K > E || ld < E) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || K > kMaxTopK || T > kBalanceMaxTokens ||
      static_cast<int64_t>(T) * K > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!logits || !aligned_to(logits, dtype == MOE_DTYPE_F32 ? 4 : 2)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Calls f with the logits per lane that E needs (4 / 8 / 12 / 16, in fours)
// and whether rows are read in fours, as compile-time constants.
template <typename F>
cudaError_t by_shape(int E, bool vec, F&& f) {
  auto with = [&](auto maxi) {
    return vec ? f(maxi, std::true_type{}) : f(maxi, std::false_type{});
  };
  if (E <= 128) return with(std::integral_constant<int, 1>{});
  if (E <= 256) return with(std::integral_constant<int, 2>{});
  if (E <= 384) return with(std::integral_constant<int, 3>{});
  return with(std::integral_constant<int, 4>{});
}

// Rows that start on a whole group of four elements.
template <typename T>
bool rows_of_fours(const T* p, int64_t ld) {
  return aligned_to(p, 4 * sizeof(T)) && ld % 4 == 0;
}

template <typename T>
cudaError_t run_forward(const T* logits, int64_t ld, const uint8_t* mask, int tokens, int E, int K,
                        float coef, int32_t* ids, float* weights, int32_t* counts,
                        float* mean_probs, float* loss, void* workspace, cudaStream_t s) {
  return by_shape(E, rows_of_fours(logits, ld), [&](auto maxi, auto vec) {
    constexpr int kI = decltype(maxi)::value;
    constexpr bool kV = decltype(vec)::value;
    constexpr int smem = kBalanceWarps * kI * 128 * 4;
    if (tokens <= kSmallTokens) {
      auto k = balance_small_kernel<kI, kV, T>;
      static OncePerDevice prepared;
      const cudaError_t ready = prepared([&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      });
      if (ready != cudaSuccess) return ready;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      int ranks = 1;
      while (ranks < kSmallCluster && ranks < tokens) ranks *= 2;
      attr[0].val.clusterDim.x = ranks;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(ranks);
      cfg.blockDim = dim3(32 * kBalanceWarps);
      cfg.dynamicSmemBytes = smem;
      cfg.stream = s;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      return cudaLaunchKernelEx(&cfg, k, logits, ld, mask, tokens, E, K, coef, ids, weights, counts,
                                mean_probs, loss);
    }
    const int blocks = balance_blocks(tokens);
    float* psum = static_cast<float*>(workspace);
    int32_t* count = reinterpret_cast<int32_t*>(psum + static_cast<int64_t>(blocks) * E);
    auto k = balance_forward_kernel<kI, kV, T>;
    static OncePerDevice prepared;
    const cudaError_t ready = prepared([&] {
      return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (ready != cudaSuccess) return ready;
    cudaError_t e = launch_pdl(false, k, dim3(blocks), dim3(32 * kBalanceWarps), smem, s, logits,
                               ld, mask, tokens, E, K, ids, weights, psum, count);
    if (e == cudaSuccess)
      e = launch_pdl(true, balance_finish_kernel, dim3(kFinishRanks), dim3(kFinishThreads), 0, s,
                     psum, count, blocks, E, K, coef, counts, mean_probs, loss);
    return e;
  });
}

template <typename T>
cudaError_t run_backward(const T* logits, int64_t ld, int tokens, int E, int K, float coef,
                         const int32_t* ids, const float* weights, const int32_t* counts,
                         const float* d_loss, const float* d_weights, T* d_logits, int64_t ld_d,
                         cudaStream_t s) {
  return by_shape(E, rows_of_fours(logits, ld) && rows_of_fours(d_logits, ld_d),
                  [&](auto maxi, auto vec) {
    return launch_pdl(false,
                      balance_backward_kernel<decltype(maxi)::value, decltype(vec)::value, T>,
                      dim3(std::min(kBackBlocks, (tokens + kBackWarps - 1) / kBackWarps)),
                      dim3(32 * kBackWarps), 0, s, logits, ld, tokens, E, K, coef, ids, weights,
                      counts, d_loss, d_weights, d_logits, ld_d);
  });
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_workspace(int T, int E) {
  if (T < 0 || T > kBalanceMaxTokens || E < 1 || E > kMaxExperts) return 0;
  return T <= kSmallTokens ? 16 : static_cast<size_t>(balance_blocks(T)) * E * 8;
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
  const cudaError_t e =
      dtype == MOE_DTYPE_F32
          ? run_forward(static_cast<const float*>(logits), ld, mask, T, E, K, coef, ids, weights,
                        counts, mean_probs, loss, workspace, s)
          : run_forward(static_cast<const __nv_bfloat16*>(logits), ld, mask, T, E, K, coef, ids,
                        weights, counts, mean_probs, loss, workspace, s);
  return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
  return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
