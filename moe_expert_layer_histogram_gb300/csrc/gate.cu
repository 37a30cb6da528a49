// gate.cu -- the router's gate: scores, the choice of groups and experts, the
// routing weights, and the gradient of the logits.
//
// With s = sigmoid(l) or softmax(l) of a token's E logits and a bias b that
// only the choice sees (c = s + b; experts whose logit is -inf come last):
//   a group's score is its largest c, or the sum of its two largest;
//   the best `group_top` groups stay, the K largest c within them are chosen,
//   both with ties to the lower index;
//   w_k = scale s_k, or scale s_k / sum_j s_j over the chosen.
// The choice is piecewise constant, so with u_k = s_k / sum_j s_j
//   normalised:  d s_k = scale / sum_j s_j (dw_k - sum_j u_j dw_j)
//   else:        d s_k = scale dw_k
// and d l_e = s_e (1 - s_e) d s_e (sigmoid; 0 for experts that were not
// chosen) or s_e (d s_e - sum_j s_j d s_j) (softmax; for normalised weights
// the sum is 0, so there too only the chosen experts' logits have a gradient).
//
// Sigmoid and softmax rise with the logit, so without a bias the choice goes by
// the logits themselves.  With one, two choices may be nearer to each other than
// fp32 tells apart (9 gaps of about 0.01 at K = 8 and E = 384, and scores off by
// up to 4e-7: one token in a thousand); such a token is decided again in 64 bits.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
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
constexpr int kMaxGroups = 32;

struct GateArgs {
  int64_t ld;
  const float* bias;    // [E] or null
  const uint8_t* mask;  // [T] or null
  int T, E, K;
  int groups, size, group_top;  // size: experts per group
  int lanes, per;               // lanes per group (a power of two), experts per lane
  int softmax, top2, normalize;
  int vec;                      // rows in fours, experts per lane a multiple of four
  float scale;
  int32_t* ids;
  float* weights;
  int32_t* counts;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void set(float& d, float v) { d = v; }
__device__ __forceinline__ void set(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kAllLanes, v, off);
  return v;
}

// The largest of the warp's floats (any NaN: NaN).
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    const float o = __shfl_xor_sync(kAllLanes, v, off);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(o));
  }
  return v;
}

// 2^(d log2 e) in one multiply and the hardware's power of two: off by its two
// ulp and by |d| 2^-24 of itself.
__device__ __forceinline__ float exp_fast(float d) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d * kLog2e));
  return r;
}

// Keys that order as the numbers do, 0 for none; -0 is +0 and every NaN the same
// largest key.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  return logit_key(v);
}
__device__ __forceinline__ uint64_t order_key(double v) {
  if (v != v) return ~uint64_t{0};
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return b >> 63 ? ~b : b | (uint64_t{1} << 63);
}

// How far apart two choices that were worked out in fp32 have to be for their
// order to be certain; s the larger score, c the larger choice.  Sigmoid: the
// power is off by (2 + 1.5 |l|) 2^-24 of itself, which moves s by s (1 - s) of
// that (|l| s (1 - s) <= 0.23), sum and quotient by 2^-23 s: below 3 2^-23 in
// all, twice for two.  Softmax: sum and powers are off by at most 50 2^-24 of
// themselves beside |d| e^d <= 0.37.  Adding the bias: 2^-24 |c|.
__device__ __forceinline__ float doubt(bool softmax, float s, float c) {
  const float of_sum = 0x1p-22f * fabsf(c);
  return softmax ? 0x1p-17f * fabsf(s) + 0x1p-22f + of_sum : 0x1p-20f + of_sum;
}

// The lane's share of a row: `per` experts of its group from `base` on, n real.
struct Share {
  int group, base, n;
  bool in;  // the lane has a group
  __device__ Share(const GateArgs& p, int lane) {
    group = lane / p.lanes;
    const int at = (lane % p.lanes) * p.per;
    in = group < p.groups;
    base = group * p.size + at;
    n = in ? min(max(p.size - at, 0), p.per) : 0;
  }
};

template <int NL, typename T>
__device__ __forceinline__ void load_share(const T* __restrict__ row, const Share& sh, bool vec,
                                           float (&x)[NL]) {
#pragma unroll
  for (int j = 0; j < NL; j += 4) {
    if (vec && j + 4 <= sh.n) {
      if constexpr (sizeof(T) == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(row + sh.base + j));
        x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + sh.base + j));
        x[j] = __uint_as_float(v.x << 16);
        x[j + 1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[j + 2] = __uint_as_float(v.y << 16);
        x[j + 3] = __uint_as_float(v.y & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j + i] = j + i < sh.n ? to_f32(row[sh.base + j + i]) : -INFINITY;
    }
  }
}

// ---------------------------------------------------------------- 64 bits
// The choice of one token in 64 bits, by the whole warp: lane k < K receives the
// k-th expert.  Rare, so it reads the row again and keeps its values in local
// memory.
template <typename T>
__device__ __noinline__ int choose_exact(const T* __restrict__ row, const GateArgs& p) {
  constexpr int kMost = 32;
  const int lane = threadIdx.x & 31;
  const Share sh(p, lane);
  double m = 0.0, r = 1.0;
  if (p.softmax) {
    float top = -INFINITY;
    for (int j = 0; j < sh.n; ++j) top = fmaxf(top, to_f32(row[sh.base + j]));
    m = static_cast<double>(warp_max(top));
    double sum = 0.0;
    for (int j = 0; j < sh.n; ++j) sum += exp(static_cast<double>(to_f32(row[sh.base + j])) - m);
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(kAllLanes, sum, off);
    r = 1.0 / sum;
  }
  auto score = [&](float l) {
    const double d = static_cast<double>(l);
    return p.softmax ? exp(d - m) * r : 1.0 / (1.0 + exp(-d));
  };
  double c[kMost];
  for (int j = 0; j < kMost; ++j) {
    c[j] = -INFINITY;
    if (j >= sh.n) continue;
    const float l = to_f32(row[sh.base + j]);
    if (l == -INFINITY) continue;
    c[j] = p.bias ? score(l) + static_cast<double>(p.bias[sh.base + j]) : static_cast<double>(l);
  }
  bool kept = sh.in;
  if (p.group_top < p.groups) {
    double a = -INFINITY, b = -INFINITY;  // the group's two largest
    auto put = [&](double v) {
      if (order_key(v) > order_key(a)) {
        b = a;
        a = v;
      } else if (order_key(v) > order_key(b)) {
        b = v;
      }
    };
    for (int j = 0; j < sh.n; ++j) put(c[j]);
    for (int off = 1; off < p.lanes; off <<= 1) {
      const double oa = __shfl_xor_sync(kAllLanes, a, off), ob = __shfl_xor_sync(kAllLanes, b, off);
      put(oa);
      put(ob);
    }
    double v = a;
    if (p.top2 && p.size > 1) {
      if (p.bias)
        v = a + b;
      else
        v = (a == -INFINITY ? a : score(static_cast<float>(a))) +
            (b == -INFINITY ? b : score(static_cast<float>(b)));
    }
    const uint64_t mine = order_key(v);
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const uint64_t o = __shfl_sync(kAllLanes, mine, g * p.lanes);
      rank += o > mine || (o == mine && g < sh.group);
    }
    kept = kept && rank < p.group_top;
  }
  uint32_t open = 0u;  // the lane's experts that are still to be chosen
  if (kept) open = sh.n >= 32 ? 0xFFFFFFFFu : (1u << sh.n) - 1u;
  int id = 0;
  for (int k = 0; k < p.K; ++k) {
    uint64_t best = 0;
    int at = -1;
    for (int j = 0; j < sh.n; ++j)
      if ((open >> j & 1u) && order_key(c[j]) > best) {
        best = order_key(c[j]);
        at = j;
      }
    uint64_t top = best;
    for (int off = 16; off; off >>= 1) {
      const uint64_t o = __shfl_xor_sync(kAllLanes, top, off);
      top = o > top ? o : top;
    }
    const int winner = __ffs(__ballot_sync(kAllLanes, best == top)) - 1;
    const int e = __shfl_sync(kAllLanes, sh.base + at, winner);
    if (lane == winner) open &= ~(1u << at);
    if (lane == k) id = e;
  }
  return id;
}

// ---------------------------------------------------------------- forward
// Unnormalised weight of a chosen logit; top: the largest chosen logit.  Stable
// for any logits: sigmoid(l) = e^min(l, 0) / (1 + e^-|l|), and the ratios of
// several stay as they are when e^min(top, 0) is divided out.
__device__ __forceinline__ float ratio_term(bool softmax, float l, float top) {
  if (l == -INFINITY) return 0.0f;
  if (softmax) return expf(l - top);
  return expf(fminf(l, 0.0f) - fminf(top, 0.0f)) / (1.0f + expf(-fabsf(l)));
}
__device__ __forceinline__ float sigmoid_exactly(float l) {
  return expf(fminf(l, 0.0f)) / (1.0f + expf(-fabsf(l)));
}

// One token by a warp.  bias: this lane's share (0 where there is none).
// Returns whether the token is live; lane k < K receives the k-th expert and its
// weight.
template <int NL, typename T>
__device__ __forceinline__ bool gate_token(const T* __restrict__ row, const GateArgs& p,
                                           const Share& sh, const float (&bias)[NL], int lane,
                                           int* id_out, float* w_out) {
  const bool softmax = p.softmax != 0;
  float x[NL];
  load_share<NL>(row, sh, p.vec != 0, x);
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < NL; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(x[j]));
  top = warp_max(top);
  if (top == -INFINITY) return false;
  // the softmax's sum, where scores are wanted: with a bias, for sums of two, or
  // for weights that are not normalised
  float inv = 1.0f;
  if (softmax && (p.bias || p.top2 || !p.normalize)) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NL; ++j) sum += exp_fast(x[j] - top);
    inv = 1.0f / warp_sum(sum);
  }
  auto score = [&](float l) {
    return softmax ? exp_fast(l - top) * inv : __fdividef(1.0f, 1.0f + exp_fast(-l));
  };
  // the choices; without a bias the logits, which order the same
  float c[NL];
#pragma unroll
  for (int j = 0; j < NL; ++j)
    c[j] = p.bias && x[j] != -INFINITY ? score(x[j]) + bias[j] : x[j];
  bool unsure = false, kept = sh.in;
  if (p.group_top < p.groups) {
    float a = -INFINITY, b = -INFINITY;  // the group's two largest
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      float low = a;
      asm("min.NaN.f32 %0, %0, %1;" : "+f"(low) : "f"(c[j]));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(c[j]));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(low));
    }
    for (int off = 1; off < p.lanes; off <<= 1) {
      const float oa = __shfl_xor_sync(kAllLanes, a, off), ob = __shfl_xor_sync(kAllLanes, b, off);
      float low = a;
      asm("min.NaN.f32 %0, %0, %1;" : "+f"(low) : "f"(oa));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(oa));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(low));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(ob));
    }
    float v = a;
    const bool pair = p.top2 && p.size > 1;
    if (pair) {
      if (p.bias)
        v = a + b;
      else
        v = (a == -INFINITY ? a : score(a)) + (b == -INFINITY ? b : score(b));
    }
    // (a NaN anywhere in the sums above: the exact choice orders it)
    const uint32_t mine = order_key(v);
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const uint32_t o = __shfl_sync(kAllLanes, mine, g * p.lanes);
      rank += o > mine || (o == mine && g < sh.group);
    }
    kept = kept && rank < p.group_top;
    unsure = v != v;
    if (p.bias || pair) {
      const uint32_t last = __reduce_min_sync(kAllLanes, kept ? mine : 0xFFFFFFFFu);
      const uint32_t next = __reduce_max_sync(kAllLanes, sh.in && !kept ? mine : 0u);
      const float vl = key_logit(last), vn = key_logit(next);
      // (two choices, so twice the doubt; their scores are at most 1 each)
      unsure |= vl - vn <= 2.0f * doubt(softmax, 1.0f, fmaxf(fabsf(vl), fabsf(a) + fabsf(b)));
    }
  }
  // K rounds: the largest key, the lowest lane that has it, the lane's lowest
  // expert.  A lane keeps its two largest; one that wins a second time looks
  // through its share for the next.
  uint32_t first = 0u, second = 0u;
  int at1 = 0, at2 = 0;
  uint32_t key[NL];
#pragma unroll
  for (int j = 0; j < NL; ++j) {
    key[j] = kept && j < sh.n ? order_key(c[j]) : 0u;
    if (key[j] > first) {
      second = first;
      at2 = at1;
      first = key[j];
      at1 = j;
    } else if (key[j] > second) {
      second = key[j];
      at2 = j;
    }
  }
  int id = 0;
  uint32_t chosen = 0u;
  for (int k = 0; k < p.K; ++k) {
    const uint32_t w = __reduce_max_sync(kAllLanes, first);
    const int winner = __ffs(__ballot_sync(kAllLanes, first == w)) - 1;
    const int e = __shfl_sync(kAllLanes, sh.base + at1, winner);
    if (lane == k) {
      id = e;
      chosen = w;
    }
    bool search = false;
    uint32_t won = 0u;
    int won_at = 0;
    if (lane == winner) {
      search = second == 0u;
      won = first;
      won_at = at1;
      first = second;
      at1 = at2;
      second = 0u;
    }
    if (__any_sync(kAllLanes, search)) {
      uint32_t f = 0u;
      int fa = 0;
#pragma unroll
      for (int j = 0; j < NL; ++j)
        if ((key[j] < won || (key[j] == won && j > won_at)) && key[j] > f) {
          f = key[j];
          fa = j;
        }
      if (search) {
        first = f;
        at1 = fa;
      }
    }
  }
  // (fp32 keys of choices with a bias: the order of neighbours, and that nothing
  // that was left out belongs before the last)
  const float l = lane < p.K ? to_f32(row[id]) : -INFINITY;
  if (p.bias) {
    const float mine = lane < p.K ? key_logit(chosen) : 0.0f;
    const float b = lane < p.K ? p.bias[id] : 0.0f;
    const float next = __shfl_down_sync(kAllLanes, mine, 1);
    const float nl = __shfl_down_sync(kAllLanes, l, 1), nb = __shfl_down_sync(kAllLanes, b, 1);
    if (lane + 1 < p.K)
      unsure |= mine - next <= doubt(softmax, fmaxf(fabsf(mine - b), fabsf(next - nb)),
                                     fmaxf(fabsf(mine), fabsf(next))) &&
                !(l == nl && b == nb);
    const float last = __shfl_sync(kAllLanes, mine, p.K - 1);
    const float ll = __shfl_sync(kAllLanes, l, p.K - 1), lb = __shfl_sync(kAllLanes, b, p.K - 1);
    const int last_id = __shfl_sync(kAllLanes, id, p.K - 1);
    const uint32_t last_key = order_key(last);
    const float least = last - doubt(softmax, last - lb, last), own = softmax ? 0x1p-17f : 0.0f;
    bool near = false;
#pragma unroll
    for (int j = 0; j < NL; ++j)
      near |= key[j] != 0u && fmaf(own, fabsf(c[j] - bias[j]), c[j]) >= least;
    if (__any_sync(kAllLanes, near)) {
      // (the chosen ones are near too: those come before the last by key and index)
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const bool after = key[j] < last_key || (key[j] == last_key && sh.base + j > last_id);
        unsure |= key[j] != 0u && fmaf(own, fabsf(c[j] - bias[j]), c[j]) >= least && after &&
                  !(x[j] == ll && bias[j] == lb);
      }
    }
  }
  float mine_l = l;
  if (__any_sync(kAllLanes, unsure)) {
    id = choose_exact(row, p);
    mine_l = lane < p.K ? to_f32(row[id]) : -INFINITY;
  }
  const bool used = lane < p.K;
  float w;
  if (p.normalize) {
    const float m = warp_max(used ? mine_l : -INFINITY);
    const float t = used ? ratio_term(softmax, mine_l, m) : 0.0f;
    const float sum = warp_sum(t);
    w = sum == 0.0f ? 0.0f : t / sum;
  } else if (softmax) {
    // (the sum of powers above, once more with the exact ones)
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NL; ++j) sum += j < sh.n ? expf(x[j] - top) : 0.0f;
    sum = warp_sum(sum);
    w = used ? expf(mine_l - top) / sum : 0.0f;
  } else {
    w = used ? sigmoid_exactly(mine_l) : 0.0f;
  }
  *id_out = id;
  *w_out = p.scale * w;
  return true;
}

constexpr int kGateWarps = 16;
// A token per warp up to this many: one block, which then writes the counts by
// itself (16 tokens of 64 experts: one launch instead of two).
constexpr int kGateSmall = 32;

// SMALL: one block.  Else the counts are zero already (once the kernel before
// this one is over) and the blocks add theirs: whole numbers, so the order does
// not matter.
template <int NL, bool SMALL, typename T>
__global__ void __launch_bounds__(SMALL ? 1024 : 32 * kGateWarps, SMALL ? 1 : NL > 16 ? 1 : 2)
    gate_forward_kernel(const T* __restrict__ logits, const __grid_constant__ GateArgs p) {
  __shared__ int s_count[kMaxExperts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) s_count[e] = 0;
  __syncthreads();
  const Share sh(p, lane);
  float bias[NL];
#pragma unroll
  for (int j = 0; j < NL; ++j) bias[j] = p.bias && j < sh.n ? p.bias[sh.base + j] : 0.0f;
  for (int t = blockIdx.x + gridDim.x * warp; t < p.T; t += gridDim.x * warps) {
    int id = -1;
    float w = 0.0f;
    const bool live =
        (!p.mask || p.mask[t]) &&
        gate_token<NL>(logits + static_cast<int64_t>(t) * p.ld, p, sh, bias, lane, &id, &w);
    if (lane < p.K) {
      p.ids[static_cast<int64_t>(t) * p.K + lane] = live ? id : -1;
      p.weights[static_cast<int64_t>(t) * p.K + lane] = live ? w : 0.0f;
      if (live) atomicAdd(&s_count[id], 1);
    }
  }
  __syncthreads();
  if constexpr (!SMALL) pdl_wait();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    const int n = s_count[e];
    if (SMALL)
      p.counts[e] = n;
    else if (n)
      atomicAdd(&p.counts[e], n);
  }
}

__global__ void gate_zero_kernel(int32_t* counts, int E) {
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < E; e += blockDim.x) counts[e] = 0;
}

// ---------------------------------------------------------------- backward
constexpr int kGateBackWarps = 8;

struct GateBackArgs {
  int64_t ld, ld_d;
  int T, E, K, softmax, normalize, vec;
  float scale;
  const int32_t* ids;
  const float* d_weights;
};

// A warp per token: the row without the chosen experts (zeros, or the softmax's
// dense part), then the K chosen ones' values over it.
template <typename T>
__global__ void __launch_bounds__(32 * kGateBackWarps)
    gate_backward_kernel(const T* logits, T* d_logits,
                         const __grid_constant__ GateBackArgs p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool softmax = p.softmax != 0, dense = softmax && !p.normalize;
  for (int t = blockIdx.x * kGateBackWarps + warp; t < p.T; t += gridDim.x * kGateBackWarps) {
    const T* row = logits + static_cast<int64_t>(t) * p.ld;
    T* d = d_logits + static_cast<int64_t>(t) * p.ld_d;
    const bool used = lane < p.K;
    const int64_t at = static_cast<int64_t>(t) * p.K + lane;
    const int id = used ? p.ids[at] : -1;
    const bool real = used && id >= 0 && id < p.E;
    const bool live = __any_sync(kAllLanes, real);
    const float dw = real ? p.d_weights[at] : 0.0f;
    const float l = real ? to_f32(row[id]) : -INFINITY;
    float value = 0.0f, rest = 0.0f, top = 0.0f, inv = 0.0f;
    if (live && p.normalize) {
      const float m = warp_max(l);
      const float term = real ? ratio_term(softmax, l, m) : 0.0f;
      const float sum = warp_sum(term);
      const float u = sum == 0.0f ? 0.0f : term / sum;
      const float mean = warp_sum(u * dw);
      value = p.scale * u * (dw - mean);
      // d s / d l: s (1 - s) with 1 - s = sigmoid(-l), or the softmax's, whose
      // sum over the chosen is 0
      if (!softmax && real) value *= sigmoid_exactly(-l);
    } else if (live && !softmax) {
      if (real) value = p.scale * dw * sigmoid_exactly(l) * sigmoid_exactly(-l);
    } else if (live) {
      top = -INFINITY;
      for (int e = lane; e < p.E; e += 32) {
        const float v = to_f32(row[e]);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(v));
      }
      top = warp_max(top);
      float sum = 0.0f;
      for (int e = lane; e < p.E; e += 32) sum += expf(to_f32(row[e]) - top);
      inv = 1.0f / warp_sum(sum);
      const float pk = real ? expf(l - top) * inv : 0.0f;
      rest = p.scale * warp_sum(pk * dw);
      value = pk * (p.scale * dw - rest);
    }
    if (dense && live) {
      for (int e = lane; e < p.E; e += 32) {
        const float pe = expf(to_f32(row[e]) - top) * inv;
        set(d[e], -pe * rest);
      }
    } else if (p.vec) {
      constexpr int kPer = 16 / sizeof(T);
      const int whole = p.E / kPer;
      for (int i = lane; i < whole; i += 32)
        reinterpret_cast<uint4*>(d)[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int e = whole * kPer + lane; e < p.E; e += 32) set(d[e], 0.0f);
    } else {
      for (int e = lane; e < p.E; e += 32) set(d[e], 0.0f);
    }
    __syncwarp();
    if (real) set(d[id], value);
  }
}

// ---------------------------------------------------------------- expert order
// A stable counting sort of n expert ids: bin E takes the ids outside [0, E).
// A block takes a run of slots and each of its warps a run of those, 32 at a
// time; equal ids of a 32 are ranked by the lanes that hold them.
constexpr int kOrderWarps = 32;
constexpr int kOrderBlocks = 128;
constexpr int kOrderRun = 64;  // slots per warp at least

struct OrderArgs {
  const int32_t* ids;
  int n, E, run;      // run: slots per warp, a multiple of 32
  int32_t* hist;      // [blocks][E + 1]
  int32_t *slots, *offsets, *rows;
};

__device__ __forceinline__ int bin_of(const OrderArgs& p, int64_t i) {
  const int id = p.ids[i];
  return id >= 0 && id < p.E ? id : p.E;
}

// Each warp's counts of its run: s[warp][bin].
__device__ __forceinline__ void count_runs(const OrderArgs& p, int* s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bins = p.E + 1;
  for (int i = threadIdx.x; i < kOrderWarps * bins; i += blockDim.x) s[i] = 0;
  __syncthreads();
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kOrderWarps + warp) * p.run;
  for (int j = lane; j < p.run; j += 32)
    if (first + j < p.n) atomicAdd(&s[warp * bins + bin_of(p, first + j)], 1);
  __syncthreads();
}

__global__ void __launch_bounds__(32 * kOrderWarps)
    order_count_kernel(const __grid_constant__ OrderArgs p) {
  extern __shared__ int s_bins[];
  const int bins = p.E + 1;
  pdl_launch_dependents();
  count_runs(p, s_bins);
  for (int e = threadIdx.x; e < bins; e += blockDim.x) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < kOrderWarps; ++w) sum += s_bins[w * bins + e];
    p.hist[static_cast<int64_t>(blockIdx.x) * bins + e] = sum;
  }
}

// ALONE: the only block (no counts of others).
template <bool ALONE>
__global__ void __launch_bounds__(32 * kOrderWarps)
    order_place_kernel(const __grid_constant__ OrderArgs p) {
  extern __shared__ int s_bins[];  // [kOrderWarps][bins], then [2][1024]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bins = p.E + 1;
  int* s_before = s_bins + kOrderWarps * bins;
  int* s_total = s_before + 1024;
  count_runs(p, s_bins);
  // bin e: slots of earlier blocks, and of all blocks
  int before = 0, total = 0;
  if (!ALONE) {
    pdl_wait();
    const int width = (bins + 31) / 32 * 32, parts = 1024 / width;
    const int e = threadIdx.x % width, part = threadIdx.x / width;
    if (e < bins && part < parts) {
#pragma unroll 8
      for (int b = part; b < static_cast<int>(gridDim.x); b += parts) {
        const int h = p.hist[static_cast<int64_t>(b) * bins + e];
        total += h;
        before += b < static_cast<int>(blockIdx.x) ? h : 0;
      }
    }
    s_before[threadIdx.x] = before;
    s_total[threadIdx.x] = total;
    __syncthreads();
    if (part == 0)
      for (int q = 1; q < parts; ++q) {
        before += s_before[q * width + e];
        total += s_total[q * width + e];
      }
    __syncthreads();
  }
  // this block's own counts become each warp's first rank in the bin
  const int e = threadIdx.x;
  if (e < bins) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < kOrderWarps; ++w) {
      const int c = s_bins[w * bins + e];
      s_bins[w * bins + e] = run;
      run += c;
    }
    if (ALONE) total = run;
  }
  // exclusive scan of the totals over the bins
  int inc = e < bins ? total : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(kAllLanes, inc, off);
    if (lane >= off) inc += o;
  }
  if (lane == 31) s_total[warp] = inc;
  __syncthreads();
  int base = inc - (e < bins ? total : 0);
  for (int w = 0; w < warp; ++w) base += s_total[w];
  if (e < bins) {
    s_before[e] = base + before;
    if (blockIdx.x == 0) p.offsets[e] = base;
  }
  __syncthreads();
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kOrderWarps + warp) * p.run;
  for (int j = 0; j < p.run; j += 32) {
    const int64_t i = first + j + lane;
    const bool in = i < p.n;
    const int b = in ? bin_of(p, i) : bins;
    const unsigned same = __match_any_sync(kAllLanes, b);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int at = 0;
    if (in) at = s_bins[warp * bins + b] + rank;
    __syncwarp();
    if (in && rank == 0) s_bins[warp * bins + b] = at + __popc(same);
    __syncwarp();
    if (in) {
      const int row = s_before[b] + at;
      p.slots[row] = static_cast<int32_t>(i);
      if (p.rows) p.rows[i] = b < p.E ? row : -1;
    }
  }
}

// ---------------------------------------------------------------- host
bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int kSms = 152;
// Most tokens: a warp's next token (the stride is that of all warps) stays in 32 bits.
constexpr int kGateMaxTokens = INT32_MAX - 65535;
static_assert(2 * kSms * kGateWarps <= 65535 && 8 * kSms * kGateBackWarps <= 65535);

moe_status check_gate(const void* logits, int dtype, int64_t ld, int T, int E, int K,
                      const moe_gate_config* c) {
  if (!c || T < 0 || E < 1 || K < 1 || K > E || ld < E) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (c->group_score != MOE_GROUP_MAX && c->group_score != MOE_GROUP_TOP2)
    return MOE_ERR_INVALID_ARG;
  if (c->groups < 1 || E % c->groups || c->group_top < 1 || c->group_top > c->groups ||
      static_cast<int64_t>(c->group_top) * (E / c->groups) < K || !std::isfinite(c->scale))
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || K > kMaxTopK || c->groups > kMaxGroups || T > kGateMaxTokens ||
      static_cast<int64_t>(T) * K > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!logits || !aligned_to(logits, dtype == MOE_DTYPE_F32 ? 4 : 2)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Experts per lane that are kept in registers: 4 / 8 / 12 / 16 / 32.
template <typename F>
cudaError_t by_share(int per, F&& f) {
  if (per <= 4) return f(std::integral_constant<int, 4>{});
  if (per <= 8) return f(std::integral_constant<int, 8>{});
  if (per <= 12) return f(std::integral_constant<int, 12>{});
  if (per <= 16) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

template <typename T>
cudaError_t run_forward(const T* logits, GateArgs p, cudaStream_t s) {
  // Lanes per group: as many as there are, a power of two.  Shares in whole
  // fours where the rows are read in fours.
  p.lanes = 32;
  while (p.lanes * p.groups > 32) p.lanes /= 2;
  p.per = (p.size + p.lanes - 1) / p.lanes;
  p.vec = aligned_to(logits, 4 * sizeof(T)) && p.ld % 4 == 0 && p.size % 4 == 0;
  if (p.vec) p.per = (p.per + 3) / 4 * 4;
  return by_share(p.per, [&](auto nl) {
    constexpr int kN = decltype(nl)::value;
    if (p.T <= kGateSmall)
      return launch_pdl(false, gate_forward_kernel<kN, true, T>, dim3(1),
                        dim3(32 * std::max(p.T, 1)), 0, s, logits, p);
    cudaError_t e =
        launch_pdl(false, gate_zero_kernel, dim3(1), dim3(kMaxExperts), 0, s, p.counts, p.E);
    if (e == cudaSuccess)
      e = launch_pdl(true, gate_forward_kernel<kN, false, T>,
                     dim3(std::min((kN > 16 ? 1 : 2) * kSms, (p.T + kGateWarps - 1) / kGateWarps)),
                     dim3(32 * kGateWarps), 0, s, logits, p);
    return e;
  });
}

template <typename T>
cudaError_t run_backward(const T* logits, T* d_logits, GateBackArgs p, cudaStream_t s) {
  p.vec = aligned_to(d_logits, 16) && p.ld_d % (16 / sizeof(T)) == 0;
  return launch_pdl(false, gate_backward_kernel<T>,
                    dim3(std::min(8 * kSms, (p.T + kGateBackWarps - 1) / kGateBackWarps)),
                    dim3(32 * kGateBackWarps), 0, s, logits, d_logits, p);
}

// Slots per warp of a sort of n, and its blocks.
int order_run(int n) {
  const int64_t warps = static_cast<int64_t>(kOrderBlocks) * kOrderWarps;
  const int64_t run = ((n + warps - 1) / warps + 31) / 32 * 32;
  return static_cast<int>(std::max<int64_t>(run, kOrderRun));
}
int order_blocks(int n) {
  const int64_t per = static_cast<int64_t>(order_run(n)) * kOrderWarps;
  return static_cast<int>(std::max<int64_t>(1, (n + per - 1) / per));
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_gate_forward(const void* logits, int dtype, int64_t ld, const float* bias,
                            const uint8_t* mask, int T, int E, int K, const moe_gate_config* cfg,
                            int32_t* ids, float* weights, int32_t* counts, void* stream) {
  const moe_status st = check_gate(logits, dtype, ld, T, E, K, cfg);
  if (st != MOE_OK) return st;
  if (!counts || (T > 0 && (!ids || !weights))) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(counts, 4) ||
      !aligned_to(bias, 4))
    return MOE_ERR_INVALID_ARG;
  GateArgs p{};
  p.ld = ld;
  p.bias = bias;
  p.mask = mask;
  p.T = T, p.E = E, p.K = K;
  p.groups = cfg->groups;
  p.size = E / cfg->groups;
  p.group_top = cfg->group_top;
  p.softmax = cfg->score == MOE_SCORE_SOFTMAX;
  p.top2 = cfg->group_score == MOE_GROUP_TOP2;
  p.normalize = cfg->normalize != 0;
  p.scale = cfg->scale;
  p.ids = ids, p.weights = weights, p.counts = counts;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MOE_DTYPE_F32
                            ? run_forward(static_cast<const float*>(logits), p, s)
                            : run_forward(static_cast<const __nv_bfloat16*>(logits), p, s);
  return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_gate_backward(const void* logits, int dtype, int64_t ld, int T, int E, int K,
                             const moe_gate_config* cfg, const int32_t* ids,
                             const float* d_weights, void* d_logits, int64_t ld_d, void* stream) {
  const moe_status st = check_gate(logits, dtype, ld, T, E, K, cfg);
  if (st != MOE_OK) return st;
  if (ld_d < E) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!ids || !d_weights || !d_logits || !aligned_to(ids, 4) || !aligned_to(d_weights, 4) ||
      !aligned_to(d_logits, dtype == MOE_DTYPE_F32 ? 4 : 2))
    return MOE_ERR_INVALID_ARG;
  GateBackArgs p{};
  p.ld = ld, p.ld_d = ld_d;
  p.T = T, p.E = E, p.K = K;
  p.softmax = cfg->score == MOE_SCORE_SOFTMAX;
  p.normalize = cfg->normalize != 0;
  p.scale = cfg->scale;
  p.ids = ids, p.d_weights = d_weights;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == MOE_DTYPE_F32
          ? run_backward(static_cast<const float*>(logits), static_cast<float*>(d_logits), p, s)
          : run_backward(static_cast<const __nv_bfloat16*>(logits),
                         static_cast<__nv_bfloat16*>(d_logits), p, s);
  return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_order_workspace(int n, int E) {
  if (n < 0 || E < 1 || E > kMaxExperts) return 0;
  const int blocks = order_blocks(n);
  return blocks == 1 ? 0 : static_cast<size_t>(blocks) * (E + 1) * 4;
}

moe_status moe_order(const int32_t* ids, int n, int E, int32_t* slots, int32_t* offsets,
                     int32_t* rows, void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || E < 1) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  if (!offsets || (n > 0 && (!ids || !slots))) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(ids, 4) || !aligned_to(slots, 4) || !aligned_to(offsets, 4) ||
      !aligned_to(rows, 4))
    return MOE_ERR_INVALID_ARG;
  const size_t need = moe_order_workspace(n, E);
  if (need && (!workspace || !aligned_to(workspace, 4) || workspace_bytes < need))
    return MOE_ERR_INVALID_ARG;
  OrderArgs p{ids, n, E, order_run(n), static_cast<int32_t*>(workspace), slots, offsets, rows};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = order_blocks(n), counters = kOrderWarps * (E + 1) * 4;
  auto limit = [&](auto k, OncePerDevice& prepared) {
    return prepared([&] {
      return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  kOrderWarps * (kMaxExperts + 1) * 4 + 8192);
    });
  };
  cudaError_t e;
  if (blocks == 1) {
    static OncePerDevice prepared;
    e = limit(order_place_kernel<true>, prepared);
    if (e == cudaSuccess)
      e = launch_pdl(false, order_place_kernel<true>, dim3(1), dim3(32 * kOrderWarps),
                     counters + 8192, s, p);
  } else {
    static OncePerDevice counted, placed;
    e = limit(order_count_kernel, counted);
    if (e == cudaSuccess) e = limit(order_place_kernel<false>, placed);
    if (e == cudaSuccess)
      e = launch_pdl(false, order_count_kernel, dim3(blocks), dim3(32 * kOrderWarps), counters, s,
                     p);
    if (e == cudaSuccess)
      e = launch_pdl(true, order_place_kernel<false>, dim3(blocks), dim3(32 * kOrderWarps),
                     counters + 8192, s, p);
  }
  return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
