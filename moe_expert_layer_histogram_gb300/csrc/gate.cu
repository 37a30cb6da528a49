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
// the logits themselves.
//
// A warp takes a token; a lane holds a run of neighbouring experts of one group.
// Each choice becomes a 32-bit word that orders as it does: the float's bits (made
// positive) but the last four, which hold 15 - j for the lane's j-th expert.  So
// one redux.sync finds a round's winner and, with a vote for the lane, its index,
// and a lane's two largest words, which are all that a group's score needs too,
// take three operations an expert.  (32768 x 384 in 8 groups: keys and indices apart
// took 124 us, this 39, of which the logits' bytes are 8: instructions bound it.)
// The words are coarser than fp32, and fp32 scores are off by a few 2^-24: where the
// order of neighbours, or the border, could be another, the token is decided again
// in 64 bits, its near choices only (at E = 384 and K = 8 nine gaps of about 0.008
// against 5e-6: one token in two hundred).
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
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

__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// How far apart two scores that were worked out in fp32, s the larger at most, have
// to be for their order to be certain.  Sigmoid: the power is off by (2 + 1.5 |l|)
// 2^-24 of itself, which moves s by s (1 - s) of that (|l| s (1 - s) <= 0.23), sum
// and reciprocal by 2^-23 s: below 3 2^-23 in all, twice for two.  Softmax: sum and
// powers are off by at most 50 2^-24 of themselves beside |d| e^d <= 0.37.
__device__ __forceinline__ float doubt(bool softmax, float s) {
  return softmax ? 0x1p-17f * s + 0x1p-22f : 0x1p-20f;
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

// FULL: every lane's share is NL real experts, in fours.
template <int NL, bool FULL, typename T>
__device__ __forceinline__ void load_share(const T* __restrict__ row, const Share& sh, bool vec,
                                           float (&x)[NL]) {
#pragma unroll
  for (int j = 0; j < NL; j += 4) {
    if (FULL || (vec && j + 4 <= sh.n)) {
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
// Scores of one token in 64 bits.
template <typename T>
struct ExactScore {
  bool softmax, by_choice;
  double top = 0.0, inv = 1.0;
  // The whole warp; sum: whether a softmax's sum is wanted.
  __device__ ExactScore(const T* row, const GateArgs& p, const Share& sh, bool sum_wanted)
      : softmax(p.softmax != 0), by_choice(p.bias != nullptr) {
    if (!softmax || !sum_wanted) return;
    float m = -INFINITY;
    for (int j = 0; j < sh.n; ++j) {
      const float l = to_f32(row[sh.base + j]);
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(l));
    }
    top = static_cast<double>(warp_max(m));
    double sum = 0.0;
    for (int j = 0; j < sh.n; ++j) sum += exp(static_cast<double>(to_f32(row[sh.base + j])) - top);
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(kAllLanes, sum, off);
    inv = 1.0 / sum;
  }
  __device__ double score(float l) const {
    const double d = static_cast<double>(l);
    return softmax ? exp(d - top) * inv : 1.0 / (1.0 + exp(-d));
  }
  // What an expert is chosen by: -inf if it is disabled.
  __device__ double choice(float l, const float* bias) const {
    if (l == -INFINITY) return -INFINITY;
    return by_choice ? score(l) + static_cast<double>(*bias) : static_cast<double>(l);
  }
};

// The experts marked in the lanes' masks (bit j: the lane's j-th), one to a lane in
// order of their indices; returns how many there are, at most 33.
__device__ __forceinline__ int collect(uint32_t mask, const Share& sh, int lane, int& e, int& from) {
  int m = 0;
  for (;;) {
    const unsigned left = __ballot_sync(kAllLanes, mask != 0u);
    if (!left || m == 33) return m;
    const int owner = __ffs(left) - 1;
    const int found = __shfl_sync(kAllLanes, sh.base + __ffs(mask) - 1, owner);
    if (lane == m) {
      e = found;
      from = owner;
    }
    if (lane == owner) mask &= mask - 1;
    ++m;
  }
}

// The choice of one token in 64 bits, by the whole warp: lane k < K receives the
// k-th expert.  all: groups and every expert; else only the experts `among` (a bit
// each).  For tokens with a NaN or masses of ties, so it keeps its values in local
// memory and takes its time.
template <typename T>
__device__ __noinline__ int choose_slowly(const T* __restrict__ row, const GateArgs& p, bool all,
                                          uint32_t among) {
  constexpr int kMost = 32;
  const int lane = threadIdx.x & 31;
  const Share sh(p, lane);
  const uint32_t wanted = !all ? among : sh.n >= 32 ? 0xFFFFFFFFu : (1u << sh.n) - 1u;
  const ExactScore<T> x(row, p, sh, true);
  double c[kMost];
  for (int j = 0; j < kMost; ++j) {
    c[j] = -INFINITY;
    if (wanted >> j & 1u) c[j] = x.choice(to_f32(row[sh.base + j]), p.bias + sh.base + j);
  }
  bool kept = sh.in;
  if (all && p.group_top < p.groups) {
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
        v = (a == -INFINITY ? a : x.score(static_cast<float>(a))) +
            (b == -INFINITY ? b : x.score(static_cast<float>(b)));
    }
    const uint64_t mine = order_key(v);
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const uint64_t o = __shfl_sync(kAllLanes, mine, g * p.lanes);
      rank += o > mine || (o == mine && g < sh.group);
    }
    kept = kept && rank < p.group_top;
  }
  uint32_t open = kept ? wanted : 0u;  // the lane's experts that are still to be chosen
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

// The same among a few experts, which are scored at once, one to a lane.
template <typename T>
__device__ __noinline__ int choose_exact(const T* __restrict__ row, const GateArgs& p,
                                         uint32_t among) {
  const int lane = threadIdx.x & 31;
  const Share sh(p, lane);
  int e = 0, from = 0;
  const int m = collect(among, sh, lane, e, from);
  if (m > 32) return choose_slowly(row, p, false, among);
  const ExactScore<T> x(row, p, sh, p.bias != nullptr);
  const double c = lane < m ? x.choice(to_f32(row[e]), p.bias + e) : -INFINITY;
  int rank = 0;
  for (int i = 0; i < m; ++i) {
    const double o = __shfl_sync(kAllLanes, c, i);
    rank += o > c || (o == c && i < lane);  // (the lanes' experts rise)
  }
  int id = 0;
  for (int i = 0; i < m; ++i) {
    const int r = __shfl_sync(kAllLanes, rank, i), found = __shfl_sync(kAllLanes, e, i);
    if (lane == r) id = found;
  }
  return id;
}

// Whether this lane's group is among the group_top best, in 64 bits.  sure: it
// certainly is; open: it may be, and `among` are the lane's experts that may be its
// two largest.  2: too many to tell this way.
template <typename T>
__device__ __noinline__ int groups_exact(const T* __restrict__ row, const GateArgs& p, bool sure,
                                         bool open, uint32_t among) {
  const int lane = threadIdx.x & 31;
  const Share sh(p, lane);
  int e = 0, from = 0;
  const int m = collect(open ? among : 0u, sh, lane, e, from);
  if (m > 32) return 2;
  const bool pair = p.top2 && p.size > 1;
  const ExactScore<T> x(row, p, sh, p.bias != nullptr || pair);
  const float l = lane < m ? to_f32(row[e]) : -INFINITY;
  double c = lane < m ? x.choice(l, p.bias + e) : -INFINITY;
  // (the logits order as their scores, and the sum is of scores)
  if (pair && !p.bias && lane < m && l != -INFINITY) c = x.score(l);
  const int of = from / p.lanes;
  double a = -INFINITY, b = -INFINITY;
  for (int i = 0; i < m; ++i) {
    const double o = __shfl_sync(kAllLanes, c, i);
    const int group = __shfl_sync(kAllLanes, of, i);
    if (group == sh.group) {
      b = o > a ? a : o > b ? o : b;
      a = o > a ? o : a;
    }
  }
  const double v = pair ? a + b : a;
  int left = p.group_top, rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const double o = __shfl_sync(kAllLanes, v, g * p.lanes);
    left -= __shfl_sync(kAllLanes, static_cast<int>(sure), g * p.lanes);
    const int other = __shfl_sync(kAllLanes, static_cast<int>(open), g * p.lanes);
    rank += other && (o > v || (o == v && g < sh.group));
  }
  return sure || (open && rank < left);
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

// How the words are made: from choices with a bias (less the least bias, plus 1/16,
// so positive), from fp32 logits, or from bf16 logits, whose 16-bit keys leave room
// for the expert's own index: those words are exact.
enum { kByChoice, kByLogit, kByShortLogit };

// One token by a warp.  bias: this lane's share, less the least bias, plus 1/16.
// exact: decide in 64 bits from the start.  Returns whether the token is live; lane
// k < K receives the k-th expert and its weight.
template <int NL, bool FULL, int MODE, typename T>
__device__ __forceinline__ bool gate_token(const T* __restrict__ row, const GateArgs& p,
                                           const Share& sh, const float (&bias)[NL], bool exact,
                                           int lane, int* id_out, float* w_out) {
  // last bits of a word: kLow - j for the lane's j-th expert
  constexpr uint32_t kLow = NL > 16 ? 31u : 15u;
  constexpr float kCut = (kLow + 1) * 0x1p-23f;  // what they are of the value, at most
  const bool softmax = p.softmax != 0;
  auto real = [&](int j) { return FULL || j < sh.n; };
  uint32_t word[NL], first = 0u, second = 0u;
  float top = 0.0f, inv = 1.0f;
  bool all = exact;  // decide everything slowly, in 64 bits
  {
    float x[NL];
    load_share<NL, FULL>(row, sh, p.vec != 0, x);
    float odd = 0.0f;
#pragma unroll
    for (int j = 0; j < NL; ++j) odd = fmaf(real(j) ? x[j] : 0.0f, 0.0f, odd);
    bool off = false;  // whether some expert's logit is -inf
    if (__any_sync(kAllLanes, odd != 0.0f)) {  // (an infinity or NaN times 0)
      bool live = false, nan = false;
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        live |= real(j) && x[j] != -INFINITY;
        nan |= x[j] != x[j];
        off |= real(j) && x[j] == -INFINITY;
      }
      if (!__any_sync(kAllLanes, live)) return false;
      all |= __any_sync(kAllLanes, nan);
      off = __any_sync(kAllLanes, off);
    }
    if (softmax && (MODE == kByChoice || p.top2)) {
      top = -INFINITY;
#pragma unroll
      for (int j = 0; j < NL; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(x[j]));
      top = warp_max(top);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < NL; ++j) sum += exp_fast(x[j] - top);
      inv = 1.0f / warp_sum(sum);
      all |= inv != inv;
    }
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      if constexpr (MODE == kByChoice) {
        const float s = softmax ? exp_fast(x[j] - top) * inv : rcp_fast(1.0f + exp_fast(-x[j]));
        word[j] = (__float_as_uint(s + bias[j]) & ~kLow) | (kLow - j);
      } else {
        const uint32_t key = logit_key(x[j]);
        word[j] = MODE == kByLogit ? (key & ~kLow) | (kLow - j)
                                   : (key & 0xFFFF0000u) | static_cast<uint32_t>(0xFFFF - sh.base - j);
      }
      if (!real(j)) word[j] = 0u;
    }
    if (MODE == kByChoice && off) {
      // (the last of all, their order left to 64 bits)
#pragma unroll
      for (int j = 0; j < NL; ++j)
        if (real(j) && x[j] == -INFINITY) word[j] = (kLow + 1) | (kLow - j);
    }
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      second = max(second, min(first, word[j]));
      first = max(first, word[j]);
    }
  }
  auto score = [&](float l) {
    return softmax ? exp_fast(l - top) * inv : rcp_fast(1.0f + exp_fast(-l));
  };
  // how near two choices, the larger of them c, may be for their order to be in doubt
  auto margin = [&](float c) {
    return doubt(softmax, fmaxf(c - 0.0625f, 0.0f)) + c * (0x1p-21f + kCut);
  };
  // whether the expert of `lo` could belong before that of `hi`
  auto near = [&](uint32_t hi, uint32_t lo) {
    if constexpr (MODE == kByShortLogit) return false;
    if constexpr (MODE == kByLogit) return ((hi ^ lo) & ~kLow) == 0u;
    const float c = __uint_as_float(hi & ~kLow);
    return !(c - __uint_as_float(lo & ~kLow) > margin(c));  // (two infinities: near)
  };
  bool kept = sh.in;
  if (p.group_top < p.groups) {
    uint32_t a = first, b = second;  // the group's two largest
    for (int o = 1; o < p.lanes; o <<= 1) {
      const uint32_t oa = __shfl_xor_sync(kAllLanes, a, o), ob = __shfl_xor_sync(kAllLanes, b, o);
      b = max(max(b, ob), min(a, oa));
      a = max(a, oa);
    }
    const bool pair = p.top2 && p.size > 1;
    int rank = 0;
    if (MODE == kByShortLogit && !pair) {
      // (the words of different groups differ, and order by index where logits tie)
      for (int g = 0; g < p.groups; ++g) rank += __shfl_sync(kAllLanes, a, g * p.lanes) > a;
      kept = kept && rank < p.group_top;
    } else {
      float v, d;
      if constexpr (MODE == kByChoice) {
        // (a disabled expert's word stands for a choice of -inf)
        const float va = a <= 2 * kLow + 1 ? -INFINITY : __uint_as_float(a & ~kLow);
        const float vb = b <= 2 * kLow + 1 ? -INFINITY : __uint_as_float(b & ~kLow);
        v = pair ? va + vb : va;
        d = pair ? 2.0f * margin(fmaxf(va, 0.0f)) + 0x1p-22f * fmaxf(v, 0.0f) : margin(fmaxf(va, 0.0f));
      } else {
        auto logit = [&](uint32_t w) {
          if (MODE == kByLogit) return key_logit(w & ~kLow);
          return key_logit(w >> 31 ? w & 0xFFFF0000u : w | 0xFFFFu);
        };
        const float la = logit(a), lb = logit(b);
        v = pair ? score(la) + score(lb) : la;
        d = pair ? 2.0f * doubt(softmax, 1.0f) + 0x1p-21f + 2.0f * kCut * (fabsf(la) + fabsf(lb)) : 0.0f;
        // (a group with fewer than two enabled experts)
        if (pair && !(lb > -FLT_MAX)) v = NAN;
      }
      // (Lanes past the last group hold no words: no part in the votes below.  Their empty
      // words are a NaN's as logits, and sent every token of 3, 5, 6, .. groups to the
      // choice in 64 bits: 32768 x 384 f32, softmax without a bias, 3 of 6 groups by "top2"
      // 2680 us where it takes 75 to 88, and 4 of 8 groups 58 to 73.)
      if (!FULL && !sh.in) {
        v = -INFINITY;
        d = 0.0f;
      }
      for (int g = 0; g < p.groups; ++g) rank += __shfl_sync(kAllLanes, v, g * p.lanes) > v;
      kept = kept && rank < p.group_top;
      // the border: the least of the kept, and the largest of the others
      const uint32_t mine = order_key(v);
      const float vl = key_logit(__reduce_min_sync(kAllLanes, kept ? mine : 0xFF800000u));
      const float vn = key_logit(__reduce_max_sync(kAllLanes, sh.in && !kept ? mine : 0x007FFFFFu));
      const int groups = __popc(__ballot_sync(kAllLanes, kept && lane % p.lanes == 0));
      // (equal ones, and NaN: more than group_top may have been kept)
      if (__any_sync(kAllLanes, v != v || !(vl - vn > d) || groups != p.group_top)) {
        // the largest doubt of any group decides which are open
        const float most = warp_max(sh.in ? d : 0.0f);
        const bool sure = kept && v > vn + most && v > vl + most, open = sh.in && !sure && v >= vl - most;
        uint32_t among = 0u;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          // (what may be its group's second largest, or largest)
          const uint32_t least = pair ? b : a;
          among |= static_cast<uint32_t>(real(j) && (word[j] >= least || near(least, word[j]))) << j;
        }
        const bool odd = __any_sync(kAllLanes, v != v || !(most < INFINITY));
        const int in = odd ? 2 : groups_exact(row, p, sure, open, among);
        all |= in == 2;
        kept = in == 1;
      }
    }
    if (!kept) first = second = 0u;
  }
  // K rounds: the largest word and the lowest lane that has it.  A lane that has won
  // twice looks through its share for the next.
  uint32_t mine = 0u;
  int from = 0;
  for (int k = 0; k < p.K; ++k) {
    const uint32_t w = __reduce_max_sync(kAllLanes, first);
    const int winner = __ffs(__ballot_sync(kAllLanes, first == w)) - 1;
    if (lane == k) {
      mine = w;
      from = winner;
    }
    const bool won = lane == winner;
    first = won ? second : first;
    second = won ? 0u : second;
    if (__any_sync(kAllLanes, won && first == 0u)) {
      uint32_t next = 0u;
#pragma unroll
      for (int j = 0; j < NL; ++j) next = max(next, word[j] < w ? word[j] : 0u);
      if (won) first = next;
    }
  }
  int id = 0;
  bool unsure = all;
  const uint32_t last = __shfl_sync(kAllLanes, mine, p.K - 1);
  if constexpr (MODE == kByShortLogit) {
    id = 0xFFFF - static_cast<int>(mine & 0xFFFFu);
  } else {
    id = from / p.lanes * p.size + from % p.lanes * p.per + static_cast<int>(kLow - (mine & kLow));
    const uint32_t after = __shfl_down_sync(kAllLanes, mine, 1);
    unsure |= (lane + 1 < p.K && near(mine, after)) || (first != 0u && near(last, first));
  }
  if (__any_sync(kAllLanes, unsure)) {
    uint32_t among = 0u;
#pragma unroll
    for (int j = 0; j < NL; ++j)
      among |= static_cast<uint32_t>(real(j) && kept && (word[j] >= last || near(last, word[j]))) << j;
    id = all ? choose_slowly(row, p, true, 0u) : choose_exact(row, p, among);
  }
  const bool used = lane < p.K;
  const float l = used ? to_f32(row[id]) : -INFINITY;
  float w;
  if (p.normalize) {
    const float m = warp_max(l);
    const float t = used ? ratio_term(softmax, l, m) : 0.0f;
    const float sum = warp_sum(t);
    w = sum == 0.0f ? 0.0f : t / sum;
  } else if (softmax) {
    // (the whole row once more, with expf)
    float m = -INFINITY, sum = 0.0f;
    for (int e = lane; e < p.E; e += 32) {
      const float v = to_f32(row[e]);
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(v));
    }
    m = warp_max(m);
    for (int e = lane; e < p.E; e += 32) sum += expf(to_f32(row[e]) - m);
    sum = warp_sum(sum);
    w = used ? expf(l - m) / sum : 0.0f;
  } else {
    w = used ? sigmoid_exactly(l) : 0.0f;
  }
  *id_out = id;
  *w_out = p.scale * w;
  return true;
}

constexpr int kGateWarps = 16;
// A token per warp up to this many: one block, which then writes the counts by
// itself, in one launch instead of two.  (64 experts: 16 tokens 7.2 us with the order
// behind it and 7.9 in two, 32 tokens 8.5 and 7.7; 384 experts 9.1 and 9.1, 11.5 and
// 9.3.)
constexpr int kGateSmall = 16;

// SMALL: one block.  Else the counts are zero already (once the kernel before this
// one is over) and the blocks add theirs: whole numbers, so the order does not
// matter.
template <int NL, bool FULL, int MODE, bool SMALL, typename T>
__global__ void __launch_bounds__(32 * (SMALL ? kGateSmall : kGateWarps), SMALL || NL > 16 ? 1 : 2)
    gate_forward_kernel(const T* __restrict__ logits, const __grid_constant__ GateArgs p) {
  __shared__ int s_count[kMaxExperts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) s_count[e] = 0;
  __syncthreads();
  const Share sh(p, lane);
  float bias[NL];
  bool exact = false;  // a bias that is no number
  if constexpr (MODE == kByChoice) {
    float least = INFINITY, odd = 0.0f;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      bias[j] = j < sh.n ? p.bias[sh.base + j] : INFINITY;
      least = fminf(least, bias[j]);
      if (j < sh.n) odd = fmaf(bias[j], 0.0f, odd);
    }
    least = -warp_max(-least);
    exact = __any_sync(kAllLanes, odd != 0.0f);
#pragma unroll
    for (int j = 0; j < NL; ++j) bias[j] = j < sh.n ? bias[j] - least + 0.0625f : 0.0625f;
  }
  for (int t = blockIdx.x + gridDim.x * warp; t < p.T; t += gridDim.x * warps) {
    int id = -1;
    float w = 0.0f;
    const bool live = (!p.mask || p.mask[t]) &&
                      gate_token<NL, FULL, MODE>(logits + static_cast<int64_t>(t) * p.ld, p, sh, bias,
                                           exact, lane, &id, &w);
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
    __syncwarp();  // (d may be the row itself)
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
constexpr int kOrderBlocks = 64;  // (262144 slots of 384 experts: 12.5 us; 128 blocks 18.3, 32 16.7)
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
  auto with = [&](auto nl, auto mode) {
    constexpr int kN = decltype(nl)::value, kMode = decltype(mode)::value;
    if (p.T <= kGateSmall)
      return launch_pdl(false, gate_forward_kernel<kN, false, kMode, true, T>, dim3(1),
                        dim3(32 * std::max(p.T, 1)), 0, s, logits, p);
    cudaError_t e =
        launch_pdl(false, gate_zero_kernel, dim3(1), dim3(kMaxExperts), 0, s, p.counts, p.E);
    if (e != cudaSuccess) return e;
    const dim3 grid(std::min((kN > 16 ? 1 : 2) * kSms, (p.T + kGateWarps - 1) / kGateWarps));
    // (full shares need no look at their ends: 32768 x 384 in 8 groups 43 -> 39 us)
    if constexpr (kN <= 16)
      if (p.vec && p.per == kN && p.lanes * p.per == p.size && p.lanes * p.groups == 32)
        return launch_pdl(true, gate_forward_kernel<kN, true, kMode, false, T>, grid,
                          dim3(32 * kGateWarps), 0, s, logits, p);
    return launch_pdl(true, gate_forward_kernel<kN, false, kMode, false, T>, grid,
                      dim3(32 * kGateWarps), 0, s, logits, p);
  };
  return by_share(p.per, [&](auto nl) {
    if (p.bias) return with(nl, std::integral_constant<int, kByChoice>{});
    return with(nl, std::integral_constant<int, sizeof(T) == 4 ? kByLogit : kByShortLogit>{});
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
