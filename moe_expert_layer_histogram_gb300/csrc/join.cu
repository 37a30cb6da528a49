// join.cu -- the end of a block: its parts added up, a norm after the block, the
// scaled sum with the residual stream, and the norm before the next block.
//
//   y  = sum_k w_k z[row_k] + sigmoid(a) u      (routed rows, shared expert)
//   x' = x + scale N(y; post)                   (N left out without `post`)
//   h  = N(x'; norm),   N(v; w) = w v r,  r = 1 / sqrt(mean(v^2) + eps)
//
// with h in bf16 or, for the next 8-bit product, as codes with one scale per
// token.  x' is stored in x's type and h is the norm of what was stored, so the
// backward pass, which reads x' again, differentiates the same function:
//
//   g  = d x' + r2 (v - xh mean(v xh)),   v = norm d h,  xh = x' r2
//   d x = g;  d n = scale g
//   d y = r1 (v - yh mean(v yh)),         v = post d n,  yh = y r1
//   d z[row_k] = w_k d y;  d w_k = <d y, z[row_k]>
//   d u = sigmoid(a) d y;  d a = <d y, u> s (1 - s)
//   d norm = sum_t d h xh;  d post = sum_t d n yh
//
// Both passes are bound by the rows' bytes.  A block of threads takes a token and
// keeps the whole row of every sum in registers, so each input is read once (the
// backward pass with `post` reads z twice, the second time from L2: y has to be
// complete before d y is known).  The weights' gradients are sums over tokens:
// each block keeps its columns' sums in registers over its tokens and writes one
// row of partials, which a second kernel adds in block order; the same inputs
// give the same bits.
//
// Rows come by bulk copies: a warp of the block's own walks through its tokens' rows
// ahead of the others and fills a ring of stages in shared memory, one row each, so
// that a token's dozen rows, which depend on its indices and on one another's sums,
// are all on their way at once and the next token's behind them (4096 x 7168, top-8:
// 128 us forward and 208 backward, 6.0 TB/s; with rows loaded by the threads that use
// them 143 and 318).  With few tokens to a block there is little to run ahead of, and
// narrow rows have more blocks to an SM; those, rows that do not start on 16 bytes, and
// rows of more than 7936 columns, whose vectors and filling warp are more than a block's
// threads, are loaded by their threads (use_ring).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "int8_quant.cuh"
#include "internal.h"
#include "moe.h"
#include "ptx_pipeline.cuh"

namespace moe {

namespace {

constexpr unsigned kAllLanes = 0xFFFFFFFFu;
constexpr int kSms = 152;
constexpr int kMaxWidth = 16384;  // H: 512 threads of 4 vectors
constexpr int kVec = 8;           // columns of a vector

__device__ int g_join_status;

struct JoinArgs {
  moe_join j;
  // forward
  void* x_out;
  int64_t ld_out;
  __nv_bfloat16* h;
  int64_t ld_h;
  int8_t* codes;
  int64_t ld_codes;
  float *code_scales, *post_rstd, *norm_rstd;
  int stages;  // of the ring
};

struct JoinBackArgs {
  moe_join j;
  const void *x_out, *d_x_out, *d_h;
  int64_t ld_out, ld_dxo, ld_dh;
  const float *post_rstd, *norm_rstd;
  void* d_x;
  int64_t ld_dx;
  __nv_bfloat16* d_rows;
  int64_t ld_drows;
  const int32_t* live_rows;
  float* d_weights;
  __nv_bfloat16* d_shared;
  int64_t ld_dshared;
  void* d_gate;
  float *part_post, *part_norm;  // [blocks, H] each, or null
  int stages;                    // of the ring
};

// The columns of a thread's vector i, element c: vectors of eight neighbours, or
// (rows that do not start on 16 bytes) single columns a block apart, so that
// either way a warp's accesses are neighbours.
template <bool VEC>
__device__ __forceinline__ int column(int i, int c) {
  const int n = blockDim.x, t = threadIdx.x;
  return VEC ? (i * n + t) * kVec + c : (i * kVec + c) * n + t;
}

template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int i, int H, float (&v)[kVec]) {
  if constexpr (VEC) {
    const int c0 = column<VEC>(i, 0);
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (c0 < H) q = *reinterpret_cast<const uint4*>(row + c0);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[2 * c] = __uint_as_float(w[c] << 16);
      v[2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int c = 0; c < kVec; ++c) {
      const int col = column<VEC>(i, c);
      v[c] = col < H ? __bfloat162float(row[col]) : 0.0f;
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float* row, int i, int H, float (&v)[kVec]) {
  if constexpr (VEC) {
    const int c0 = column<VEC>(i, 0);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (c0 < H) {
      a = *reinterpret_cast<const float4*>(row + c0);
      b = *reinterpret_cast<const float4*>(row + c0 + 4);
    }
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int c = 0; c < kVec; ++c) {
      const int col = column<VEC>(i, c);
      v[c] = col < H ? row[col] : 0.0f;
    }
  }
}
// A norm's weights, of either type.
template <bool VEC>
__device__ __forceinline__ void load_weights(const void* w, int type, int i, int H,
                                             float (&v)[kVec]) {
  if (type == MOE_DTYPE_F32)
    load8<VEC>(static_cast<const float*>(w), i, H, v);
  else
    load8<VEC>(static_cast<const __nv_bfloat16*>(w), i, H, v);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return reinterpret_cast<const uint32_t&>(p);
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int i, int H, const float (&v)[kVec]) {
  if constexpr (VEC) {
    const int c0 = column<VEC>(i, 0);
    if (c0 < H)
      *reinterpret_cast<uint4*>(row + c0) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]),
                                                       pack2(v[4], v[5]), pack2(v[6], v[7]));
  } else {
#pragma unroll
    for (int c = 0; c < kVec; ++c) {
      const int col = column<VEC>(i, c);
      if (col < H) row[col] = __float2bfloat16_rn(v[c]);
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float* row, int i, int H, const float (&v)[kVec]) {
  if constexpr (VEC) {
    const int c0 = column<VEC>(i, 0);
    if (c0 < H) {
      *reinterpret_cast<float4*>(row + c0) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(row + c0 + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < kVec; ++c) {
      const int col = column<VEC>(i, c);
      if (col < H) row[col] = v[c];
    }
  }
}

// What v becomes when it is stored.
__device__ __forceinline__ float stored(float v, const float*) { return v; }
__device__ __forceinline__ float stored(float v, const __nv_bfloat16*) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kAllLanes, v, off);
  return v;
}

// Sum over the block, the same in every thread; `s`: 32 words that no other sum
// uses between two syncs.
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? s[lane] : 0.0f);
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* s) {
  v = __reduce_max_sync(kAllLanes, v);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return __reduce_max_sync(kAllLanes, lane < warps ? s[lane] : 0u);
}

__device__ __forceinline__ float sigmoid(float a) {
  return expf(fminf(a, 0.0f)) / (1.0f + expf(-fabsf(a)));
}
// A token's gate, 1 without one; rest: what it leaves, 1 - gate, as sigmoid(-a) (the
// difference would have lost its digits from a = 10 on).
__device__ __forceinline__ float gate_value(const moe_join& j, float a, bool rest) {
  if (!j.gate) return rest ? 0.0f : 1.0f;
  return sigmoid(rest ? -a : a);
}
__device__ __forceinline__ float gate_of(const moe_join& j, int64_t t, bool rest = false) {
  if (!j.gate) return rest ? 0.0f : 1.0f;
  return gate_value(j,
                    j.gate_type == MOE_DTYPE_F32
                        ? static_cast<const float*>(j.gate)[t]
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(j.gate)[t]),
                    rest);
}

// The block's sum y of token t: routed rows (kAtOnce of them on their way
// together) and the shared expert.
constexpr int kAtOnce = 4;

template <int NV, bool VEC>
__device__ __forceinline__ void gather(const moe_join& j, int64_t t, float sg,
                                       float (&y)[NV][kVec]) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < kVec; ++c) y[i][c] = 0.0f;
  const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(j.expert_rows);
  for (int k0 = 0; k0 < j.K; k0 += kAtOnce) {
    int row[kAtOnce];
    float w[kAtOnce];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      row[q] = k0 + q < j.K ? j.row_of_slot[t * j.K + k0 + q] : -1;
      w[q] = k0 + q < j.K ? j.weights[t * j.K + k0 + q] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[kAtOnce][kVec];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const bool in = row[q] >= 0 && row[q] < j.rows;
        load8<VEC>(z + (in ? row[q] : 0) * j.ld_rows, i, in ? j.H : 0, v[q]);
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        // (a row of no expert is no term: not 0 times whatever its weight is)
        const float wq = row[q] >= 0 && row[q] < j.rows ? w[q] : 0.0f;
#pragma unroll
        for (int c = 0; c < kVec; ++c) y[i][c] = fmaf(wq, v[q][c], y[i][c]);
      }
    }
  }
  if (j.shared) {
    const __nv_bfloat16* u = static_cast<const __nv_bfloat16*>(j.shared) + t * j.ld_shared;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[kVec];
      load8<VEC>(u, i, j.H, v);
#pragma unroll
      for (int c = 0; c < kVec; ++c) y[i][c] = fmaf(sg, v[c], y[i][c]);
    }
  }
}

// ---------------------------------------------------------------- forward
template <typename X, int NV, bool VEC>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512)
    join_forward_kernel(const __grid_constant__ JoinArgs p) {
  __shared__ float s_post[32], s_norm[32];
  __shared__ uint32_t s_max[32];
  const moe_join& j = p.j;
  const int64_t t = blockIdx.x;
  const int H = j.H;
  const X* x = static_cast<const X*>(j.x) + t * j.ld_x;
  float v[NV][kVec];  // y, then x'
  if (j.K || j.shared) {
    gather<NV, VEC>(j, t, j.shared ? gate_of(j, t) : 1.0f, v);
    float r = 1.0f;
    if (j.post_weight) {
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < kVec; ++c) sq = fmaf(v[i][c], v[i][c], sq);
      r = 1.0f / sqrtf(block_sum(sq, s_post) / H + j.eps);
      if (p.post_rstd && threadIdx.x == 0) p.post_rstd[t] = r;
    }
    X* out = static_cast<X*>(p.x_out) + t * p.ld_out;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[kVec];
      if (j.post_weight) {
        load_weights<VEC>(j.post_weight, j.weight_type, i, H, a);
#pragma unroll
        for (int c = 0; c < kVec; ++c) v[i][c] *= r * a[c];
      }
      load8<VEC>(x, i, H, a);
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        v[i][c] = stored(fmaf(j.scale, v[i][c], a[c]), static_cast<X*>(nullptr));
      store8<VEC>(out, i, H, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) load8<VEC>(x, i, H, v[i]);
    if (p.x_out) {
      X* out = static_cast<X*>(p.x_out) + t * p.ld_out;
#pragma unroll
      for (int i = 0; i < NV; ++i) store8<VEC>(out, i, H, v[i]);
    }
  }
  if (!j.norm_weight) return;
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < kVec; ++c) sq = fmaf(v[i][c], v[i][c], sq);
  const float r = 1.0f / sqrtf(block_sum(sq, s_norm) / H + j.eps);
  if (p.norm_rstd && threadIdx.x == 0) p.norm_rstd[t] = r;
  uint32_t amax = 0u;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[kVec];
    load_weights<VEC>(j.norm_weight, j.weight_type, i, H, w);
#pragma unroll
    for (int c = 0; c < kVec; ++c) {
      v[i][c] *= r * w[c];
      amax = max(amax, __float_as_uint(v[i][c]) & 0x7FFFFFFFu);
    }
    if (p.h) store8<VEC>(p.h + t * p.ld_h, i, H, v[i]);
  }
  if (!p.codes) return;
  amax = block_max(amax, s_max);
  const float s = i8_scale(amax);
  if (threadIdx.x == 0) p.code_scales[t] = s;
  const I8Coder coder(s);
  int8_t* codes = p.codes + t * p.ld_codes;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint2 w = coder.bytes(v[i]);
    if constexpr (VEC) {
      const int c0 = column<VEC>(i, 0);
      if (c0 < H) *reinterpret_cast<uint2*>(codes + c0) = w;
    } else {
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        if (column<VEC>(i, c) < H)
          codes[column<VEC>(i, c)] = static_cast<int8_t>((c < 4 ? w.x : w.y) >> (8 * (c & 3)));
    }
  }
}

// ---------------------------------------------------------------- backward
template <typename X, int NV, bool VEC>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512)
    join_backward_kernel(const __grid_constant__ JoinBackArgs p) {
  // by token parity: a warp may write the next token's while another still reads
  __shared__ float s_norm[2][32], s_post[2][32], s_dot[2][kMaxTopK + 1][32];
  const moe_join& j = p.j;
  const int H = j.H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  const bool block = j.K || j.shared;
  float acc_norm[NV][kVec], acc_post[NV][kVec];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < kVec; ++c) acc_norm[i][c] = acc_post[i][c] = 0.0f;
  int parity = 0;
  pdl_launch_dependents();
  for (int64_t t = blockIdx.x; t < j.T; t += gridDim.x, parity ^= 1) {
    // g = d x'
    float g[NV][kVec];
    if (p.d_h) {
      const X* xo = static_cast<const X*>(p.x_out) + t * p.ld_out;
      const __nv_bfloat16* dh = static_cast<const __nv_bfloat16*>(p.d_h) + t * p.ld_dh;
      const float r = p.norm_rstd[t];
      float xh[NV][kVec], dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float w[kVec];
        load8<VEC>(xo, i, H, xh[i]);
        load8<VEC>(dh, i, H, g[i]);
        load_weights<VEC>(j.norm_weight, j.weight_type, i, H, w);
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          xh[i][c] *= r;
          acc_norm[i][c] = fmaf(g[i][c], xh[i][c], acc_norm[i][c]);
          g[i][c] *= w[c];
          dot = fmaf(g[i][c], xh[i][c], dot);
        }
      }
      const float mean = block_sum(dot, s_norm[parity]) / H;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < kVec; ++c) g[i][c] = r * fmaf(-mean, xh[i][c], g[i][c]);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < kVec; ++c) g[i][c] = 0.0f;
    }
    if (p.d_x_out) {
      const X* dxo = static_cast<const X*>(p.d_x_out) + t * p.ld_dxo;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float a[kVec];
        load8<VEC>(dxo, i, H, a);
#pragma unroll
        for (int c = 0; c < kVec; ++c) g[i][c] += a[c];
      }
    }
    if (p.d_x) {
      X* dx = static_cast<X*>(p.d_x) + t * p.ld_dx;
#pragma unroll
      for (int i = 0; i < NV; ++i) store8<VEC>(dx, i, H, g[i]);
    }
    if (!block) continue;
    const float sg = j.shared ? gate_of(j, t) : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < kVec; ++c) g[i][c] *= j.scale;
    if (j.post_weight) {
      float y[NV][kVec], dot = 0.0f;
      gather<NV, VEC>(j, t, sg, y);
      const float r = p.post_rstd[t];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float w[kVec];
        load_weights<VEC>(j.post_weight, j.weight_type, i, H, w);
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          y[i][c] *= r;
          acc_post[i][c] = fmaf(g[i][c], y[i][c], acc_post[i][c]);
          g[i][c] *= w[c];
          dot = fmaf(g[i][c], y[i][c], dot);
        }
      }
      const float mean = block_sum(dot, s_post[parity]) / H;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < kVec; ++c) g[i][c] = r * fmaf(-mean, y[i][c], g[i][c]);
    }
    // d z, d u and their dot products with d y
    float(*dots)[32] = s_dot[parity];
    const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(j.expert_rows);
    for (int k0 = 0; k0 < j.K; k0 += kAtOnce) {
      int row[kAtOnce];
      float dot[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int r = k0 + q < j.K ? j.row_of_slot[t * j.K + k0 + q] : -1;
        row[q] = r < j.rows ? r : -1;
        dot[q] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (p.d_weights) {
          float a[kAtOnce][kVec];
#pragma unroll
          for (int q = 0; q < kAtOnce; ++q)
            load8<VEC>(z + max(row[q], 0) * j.ld_rows, i, row[q] < 0 ? 0 : H, a[q]);
#pragma unroll
          for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
            for (int c = 0; c < kVec; ++c) dot[q] = fmaf(g[i][c], a[q][c], dot[q]);
        }
        if (p.d_rows) {
#pragma unroll
          for (int q = 0; q < kAtOnce; ++q) {
            if (row[q] < 0) continue;
            const float w = j.weights[t * j.K + k0 + q];
            float a[kVec];
#pragma unroll
            for (int c = 0; c < kVec; ++c) a[c] = w * g[i][c];
            store8<VEC>(p.d_rows + row[q] * p.ld_drows, i, H, a);
          }
        }
      }
      if (p.d_weights) {
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
          const float sum = warp_sum(dot[q]);
          if (lane == 0 && k0 + q < j.K) dots[k0 + q][warp] = row[q] < 0 ? 0.0f : sum;
        }
      }
    }
    if (j.shared && (p.d_shared || p.d_gate)) {
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float a[kVec];
        if (p.d_gate) {
          load8<VEC>(static_cast<const __nv_bfloat16*>(j.shared) + t * j.ld_shared, i, H, a);
#pragma unroll
          for (int c = 0; c < kVec; ++c) dot = fmaf(g[i][c], a[c], dot);
        }
        if (p.d_shared) {
#pragma unroll
          for (int c = 0; c < kVec; ++c) a[c] = sg * g[i][c];
          store8<VEC>(p.d_shared + t * p.ld_dshared, i, H, a);
        }
      }
      if (p.d_gate) {
        dot = warp_sum(dot);
        if (lane == 0) dots[kMaxTopK][warp] = dot;
      }
    }
    if (p.d_weights || p.d_gate) {
      __syncthreads();
      if (p.d_weights)
        for (int k = warp; k < j.K; k += warps) {
          const float dot = warp_sum(lane < warps ? dots[k][lane] : 0.0f);
          if (lane == 0) p.d_weights[t * j.K + k] = dot;
        }
      if (p.d_gate && warp == warps - 1) {
        const float d =
            warp_sum(lane < warps ? dots[kMaxTopK][lane] : 0.0f) * sg * gate_of(j, t, true);
        if (lane == 0) {
          if (j.gate_type == MOE_DTYPE_F32)
            static_cast<float*>(p.d_gate)[t] = d;
          else
            static_cast<__nv_bfloat16*>(p.d_gate)[t] = __float2bfloat16_rn(d);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (p.part_norm)
      store8<VEC>(p.part_norm + static_cast<int64_t>(blockIdx.x) * H, i, H, acc_norm[i]);
    if (p.part_post)
      store8<VEC>(p.part_post + static_cast<int64_t>(blockIdx.x) * H, i, H, acc_post[i]);
  }
  // rows of no expert
  if (p.d_rows && p.live_rows) {
    float zero[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) zero[c] = 0.0f;
    for (int64_t r = max(*p.live_rows, 0) + static_cast<int64_t>(blockIdx.x); r < j.rows;
         r += gridDim.x)
#pragma unroll
      for (int i = 0; i < NV; ++i) store8<VEC>(p.d_rows + r * p.ld_drows, i, H, zero);
  }
}

// ---------------------------------------------------------------- by bulk copies
// The ring's bookkeeping: the consumers (all warps but the last) and the warp that
// fills it walk through the same rows in the same order.  A token's slots' rows and
// weights travel beside it; a token has a row at least, so no more tokens than
// stages are on their way.
constexpr int kMaxStages = 30;
constexpr int kInfos = 32;
static_assert(kInfos > kMaxStages);

struct TokenInfo {
  int row[kMaxTopK];  // -1: none
  float w[kMaxTopK];
  float gate, norm_rstd, post_rstd, gate_rest;
};

struct Ring {
  uint8_t* data;
  TokenInfo* info;
  uint64_t *full, *empty;
  volatile int* abort;
  int stages, bytes;
  int stage = 0, loads = 0;
  uint32_t phase = 0;
  bool ok = true;

  __device__ Ring(uint8_t* smem, int stages, int bytes) : stages(stages), bytes(bytes) {
    data = smem;
    info = reinterpret_cast<TokenInfo*>(smem + stages * bytes);
    full = reinterpret_cast<uint64_t*>(info + kInfos);
    empty = full + kMaxStages;
    abort = reinterpret_cast<volatile int*>(empty + kMaxStages);
  }
  __device__ void init(int consumers) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], consumers);
    }
    *abort = 0;
    fence_mbar_init();
  }
  __device__ void next() {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  // The filling warp: a row of n bytes.
  __device__ void put(const void* row, int n, int lane) {
    if (!ok) return;
    ok = wait_warp(&empty[stage], phase ^ 1, abort);
    if (!ok) return;
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[stage], n);
      bulk_load(data + stage * bytes, row, n, &full[stage]);
    }
    ++loads;
    next();
  }
  // ... which leaves when no copy is in flight, also after a wait that gave up.
  __device__ void drain(int lane) {
    for (int back = 1; lane == 0 && back <= stages && back <= loads; ++back) {
      const int load = loads - back;
      mbar_wait(&full[load % stages], static_cast<uint32_t>((load / stages) & 1), nullptr);
    }
    __syncwarp();
  }
  // A consumer's vector of the next row.
  template <typename T>
  __device__ void get(int H, float (&v)[kVec]) {
#pragma unroll
    for (int c = 0; c < kVec; ++c) v[c] = 0.0f;
    if (!ok) return;
    ok = wait_warp(&full[stage], phase, abort);
    if (!ok) return;
    const int c0 = threadIdx.x * kVec;
    const uint8_t* row = data + stage * bytes;
    if (c0 < H) {
      if constexpr (sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4*>(row)[2 * threadIdx.x],
                     b = reinterpret_cast<const float4*>(row)[2 * threadIdx.x + 1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      } else {
        const uint4 q = reinterpret_cast<const uint4*>(row)[threadIdx.x];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[2 * c] = __uint_as_float(w[c] << 16);
          v[2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
        }
      }
    }
    fence_proxy_async_shared();  // (the next copy into the stage comes after these reads)
    __syncwarp();
    mbar_arrive_if((threadIdx.x & 31) == 0, smem_u32(&empty[stage]));
    next();
  }
};

// Sums over the consumers (a named barrier: the filling warp takes no part).
__device__ __forceinline__ void sync_consumers(int threads) {
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}
__device__ __forceinline__ float consumer_sum(float v, float* s, int threads) {
  v = warp_sum(v);
  const int lane = threadIdx.x & 31;
  if (lane == 0) s[threadIdx.x >> 5] = v;
  sync_consumers(threads);
  return warp_sum(lane < threads >> 5 ? s[lane] : 0.0f);
}

// y of a token from the ring: its rows, then the shared expert's.
__device__ __forceinline__ void gather_ring(const moe_join& j, Ring& ring, const TokenInfo& info,
                                            float (&y)[kVec]) {
  float v[kVec];
#pragma unroll
  for (int c = 0; c < kVec; ++c) y[c] = 0.0f;
  for (int k = 0; k < j.K; ++k) {
    if (info.row[k] < 0) continue;
    ring.get<__nv_bfloat16>(j.H, v);
    const float w = info.w[k];
#pragma unroll
    for (int c = 0; c < kVec; ++c) y[c] = fmaf(w, v[c], y[c]);
  }
  if (j.shared) {
    const float sg = info.gate;
    ring.get<__nv_bfloat16>(j.H, v);
#pragma unroll
    for (int c = 0; c < kVec; ++c) y[c] = fmaf(sg, v[c], y[c]);
  }
}

// The filling warp's part of the same: the rows `row` (a lane each, -1: none).
__device__ __forceinline__ void put_rows(const moe_join& j, Ring& ring, int64_t t, int row, int lane,
                                         bool rows, bool shared) {
  const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(j.expert_rows);
  for (int k = 0; rows && k < j.K; ++k) {
    const int r = __shfl_sync(kAllLanes, row, k);
    if (r >= 0) ring.put(z + r * j.ld_rows, j.H * 2, lane);
  }
  if (shared && j.shared)
    ring.put(static_cast<const __nv_bfloat16*>(j.shared) + t * j.ld_shared, j.H * 2, lane);
}

// What a token's threads want to know of it, a lane a word: loaded a token ahead, and
// left in the ring.  The gate's sigmoids wait until then, so that the filling warp does
// not wait for their logit (at once: 4096 x 7168, top-8, six microseconds more forward
// and seven backward).
struct TokenWords {
  int row = -1;
  float w = 0.0f;
  uint32_t gate = 0u;  // the logit's bits as they are stored
  __device__ void load(const moe_join& j, const float* norm_rstd, const float* post_rstd, int64_t t,
                       int lane) {
    row = -1;
    w = 0.0f;
    if (t >= j.T) return;
    if (lane < j.K) {
      row = j.row_of_slot[t * j.K + lane];
      w = j.weights[t * j.K + lane];
      if (row >= j.rows || row < 0) row = -1;
    } else if (lane == kMaxTopK || lane == kMaxTopK + 3) {
      if (j.gate)
        gate = j.gate_type == MOE_DTYPE_F32 ? static_cast<const uint32_t*>(j.gate)[t]
                                            : static_cast<const uint16_t*>(j.gate)[t];
    } else if (lane == kMaxTopK + 1 && norm_rstd) {
      w = norm_rstd[t];
    } else if (lane == kMaxTopK + 2 && post_rstd) {
      w = post_rstd[t];
    }
  }
  __device__ void leave(const moe_join& j, TokenInfo& info, int lane) const {
    if (lane < kMaxTopK) {
      info.row[lane] = row;
      info.w[lane] = w;
    }
    const bool rest = lane == kMaxTopK + 3;
    if (lane == kMaxTopK || rest) {
      const float a = __uint_as_float(j.gate_type == MOE_DTYPE_F32 ? gate : gate << 16);
      const float s = gate_value(j, a, rest);
      if (rest)
        info.gate_rest = s;
      else
        info.gate = s;
    }
    if (lane == kMaxTopK + 1) info.norm_rstd = w;
    if (lane == kMaxTopK + 2) info.post_rstd = w;
    __syncwarp();
  }
};

template <typename X>
__global__ void __launch_bounds__(1024, 1)
    join_forward_ring_kernel(const __grid_constant__ JoinArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_post[2][32], s_norm[2][32];
  __shared__ uint32_t s_max[2][32];
  const moe_join& j = p.j;
  const int H = j.H, consumers = blockDim.x - 32, lane = threadIdx.x & 31;
  Ring ring(smem, p.stages, H * static_cast<int>(sizeof(X)));
  if (threadIdx.x == 0) ring.init(consumers >> 5);
  __syncthreads();
  if (static_cast<int>(threadIdx.x) >= consumers) {
    TokenWords words, next;
    words.load(j, nullptr, nullptr, blockIdx.x, lane);
    int n = 0;
    for (int64_t t = blockIdx.x; ring.ok && t < j.T; t += gridDim.x, ++n) {
      next.load(j, nullptr, nullptr, t + gridDim.x, lane);
      words.leave(j, ring.info[n % kInfos], lane);
      ring.put(static_cast<const X*>(j.x) + t * j.ld_x, H * sizeof(X), lane);
      put_rows(j, ring, t, words.row, lane, true, true);
      words = next;
    }
    ring.drain(lane);
    if (!ring.ok && lane == 0) report_status(&g_join_status, kStatusTimeout);
    return;
  }
  const bool block = j.K || j.shared;
  int parity = 0, n = 0;
  // (a wait that gave up ends no loop here: the others count on this warp's arrivals)
  for (int64_t t = blockIdx.x; t < j.T; t += gridDim.x, parity ^= 1, ++n) {
    const TokenInfo& info = ring.info[n % kInfos];
    float x[kVec], v[kVec], a[kVec];
    ring.get<X>(H, x);
    if (block) {
      gather_ring(j, ring, info, v);
      if (j.post_weight) {
        load_weights<true>(j.post_weight, j.weight_type, 0, H, a);
        float sq = 0.0f;
#pragma unroll
        for (int c = 0; c < kVec; ++c) sq = fmaf(v[c], v[c], sq);
        const float r = 1.0f / sqrtf(consumer_sum(sq, s_post[parity], consumers) / H + j.eps);
        if (p.post_rstd && threadIdx.x == 0) p.post_rstd[t] = r;
#pragma unroll
        for (int c = 0; c < kVec; ++c) v[c] *= r * a[c];
      }
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        v[c] = stored(fmaf(j.scale, v[c], x[c]), static_cast<X*>(nullptr));
    } else {
#pragma unroll
      for (int c = 0; c < kVec; ++c) v[c] = x[c];
    }
    if (p.x_out) store8<true>(static_cast<X*>(p.x_out) + t * p.ld_out, 0, H, v);
    if (!j.norm_weight) continue;
    load_weights<true>(j.norm_weight, j.weight_type, 0, H, a);
    float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < kVec; ++c) sq = fmaf(v[c], v[c], sq);
    const float r = 1.0f / sqrtf(consumer_sum(sq, s_norm[parity], consumers) / H + j.eps);
    if (p.norm_rstd && threadIdx.x == 0) p.norm_rstd[t] = r;
    uint32_t amax = 0u;
#pragma unroll
    for (int c = 0; c < kVec; ++c) {
      v[c] *= r * a[c];
      amax = max(amax, __float_as_uint(v[c]) & 0x7FFFFFFFu);
    }
    if (p.h) store8<true>(p.h + t * p.ld_h, 0, H, v);
    if (!p.codes) continue;
    amax = __reduce_max_sync(kAllLanes, amax);
    if (lane == 0) s_max[parity][threadIdx.x >> 5] = amax;
    sync_consumers(consumers);
    amax = __reduce_max_sync(kAllLanes, lane < consumers >> 5 ? s_max[parity][lane] : 0u);
    const float s = i8_scale(amax);
    if (threadIdx.x == 0) p.code_scales[t] = s;
    const uint2 w = I8Coder(s).bytes(v);
    const int c0 = threadIdx.x * kVec;
    if (c0 < H) *reinterpret_cast<uint2*>(p.codes + t * p.ld_codes + c0) = w;
  }
}

template <typename X, bool POST>
__global__ void __launch_bounds__(1024, 1)
    join_backward_ring_kernel(const __grid_constant__ JoinBackArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_norm[2][32], s_post[2][32], s_dot[2][kMaxTopK + 1][32];
  const moe_join& j = p.j;
  const int H = j.H, consumers = blockDim.x - 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = consumers >> 5;
  Ring ring(smem, p.stages, H * static_cast<int>(sizeof(X)));
  if (threadIdx.x == 0) ring.init(warps);
  pdl_launch_dependents();
  __syncthreads();
  const bool block = j.K || j.shared;
  if (warp == warps) {
    TokenWords words, next;
    words.load(j, p.norm_rstd, p.post_rstd, blockIdx.x, lane);
    int n = 0;
    for (int64_t t = blockIdx.x; ring.ok && t < j.T; t += gridDim.x, ++n) {
      next.load(j, p.norm_rstd, p.post_rstd, t + gridDim.x, lane);
      words.leave(j, ring.info[n % kInfos], lane);
      // (of x', d h and d x' one is there: a token has a row at least)
      if (p.d_h) {
        ring.put(static_cast<const X*>(p.x_out) + t * p.ld_out, H * sizeof(X), lane);
        ring.put(static_cast<const __nv_bfloat16*>(p.d_h) + t * p.ld_dh, H * 2, lane);
      }
      if (p.d_x_out)
        ring.put(static_cast<const X*>(p.d_x_out) + t * p.ld_dxo, H * sizeof(X), lane);
      if (POST) put_rows(j, ring, t, words.row, lane, true, true);
      if (block) put_rows(j, ring, t, words.row, lane, p.d_weights != nullptr, p.d_gate != nullptr);
      words = next;
    }
    ring.drain(lane);
    if (!ring.ok && lane == 0) report_status(&g_join_status, kStatusTimeout);
  } else {
    float acc_norm[kVec], acc_post[POST ? kVec : 1];
#pragma unroll
    for (int c = 0; c < kVec; ++c) acc_norm[c] = 0.0f;
#pragma unroll
    for (int c = 0; c < (POST ? kVec : 1); ++c) acc_post[c] = 0.0f;
    int parity = 0, n = 0;
    for (int64_t t = blockIdx.x; t < j.T; t += gridDim.x, parity ^= 1, ++n) {
      const TokenInfo& info = ring.info[n % kInfos];
      float g[kVec], a[kVec];
      if (p.d_h) {
        float xh[kVec];
        ring.get<X>(H, xh);
        const float r = info.norm_rstd;
        float dot = 0.0f;
        load_weights<true>(j.norm_weight, j.weight_type, 0, H, a);
        ring.get<__nv_bfloat16>(H, g);
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          xh[c] *= r;
          acc_norm[c] = fmaf(g[c], xh[c], acc_norm[c]);
          g[c] *= a[c];
          dot = fmaf(g[c], xh[c], dot);
        }
        const float mean = consumer_sum(dot, s_norm[parity], consumers) / H;
#pragma unroll
        for (int c = 0; c < kVec; ++c) g[c] = r * fmaf(-mean, xh[c], g[c]);
      } else {
#pragma unroll
        for (int c = 0; c < kVec; ++c) g[c] = 0.0f;
      }
      if (p.d_x_out) {
        ring.get<X>(H, a);
#pragma unroll
        for (int c = 0; c < kVec; ++c) g[c] += a[c];
      }
      if (p.d_x) store8<true>(static_cast<X*>(p.d_x) + t * p.ld_dx, 0, H, g);
      if (!block) continue;
      const float sg = info.gate;
#pragma unroll
      for (int c = 0; c < kVec; ++c) g[c] *= j.scale;
      if constexpr (POST) {
        float y[kVec], dot = 0.0f;
        gather_ring(j, ring, info, y);
        const float r = info.post_rstd;
        load_weights<true>(j.post_weight, j.weight_type, 0, H, a);
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          y[c] *= r;
          acc_post[c] = fmaf(g[c], y[c], acc_post[c]);
          g[c] *= a[c];
          dot = fmaf(g[c], y[c], dot);
        }
        const float mean = consumer_sum(dot, s_post[parity], consumers) / H;
#pragma unroll
        for (int c = 0; c < kVec; ++c) g[c] = r * fmaf(-mean, y[c], g[c]);
      }
      // d z, d u and their dot products with d y
      float(*dots)[32] = s_dot[parity];
      for (int k = 0; k < j.K; ++k) {
        const int row = info.row[k];
        float dot = 0.0f;
        if (row >= 0) {
          if (p.d_weights) {
            ring.get<__nv_bfloat16>(H, a);
#pragma unroll
            for (int c = 0; c < kVec; ++c) dot = fmaf(g[c], a[c], dot);
          }
          if (p.d_rows && ring.ok) {
            const float w = info.w[k];
#pragma unroll
            for (int c = 0; c < kVec; ++c) a[c] = w * g[c];
            store8<true>(p.d_rows + row * p.ld_drows, 0, H, a);
          }
        }
        if (p.d_weights) {
          dot = warp_sum(dot);
          if (lane == 0) dots[k][warp] = dot;
        }
      }
      if (j.shared) {
        if (p.d_gate) {
          float dot = 0.0f;
          ring.get<__nv_bfloat16>(H, a);
#pragma unroll
          for (int c = 0; c < kVec; ++c) dot = fmaf(g[c], a[c], dot);
          dot = warp_sum(dot);
          if (lane == 0) dots[kMaxTopK][warp] = dot;
        }
        if (p.d_shared) {
#pragma unroll
          for (int c = 0; c < kVec; ++c) a[c] = sg * g[c];
          store8<true>(p.d_shared + t * p.ld_dshared, 0, H, a);
        }
      }
      if (p.d_weights || p.d_gate) {
        sync_consumers(consumers);
        if (p.d_weights)
          for (int k = warp; k < j.K; k += warps) {
            const float dot = warp_sum(lane < warps ? dots[k][lane] : 0.0f);
            if (lane == 0) p.d_weights[t * j.K + k] = dot;
          }
        if (p.d_gate && warp == warps - 1) {
          const float d =
              warp_sum(lane < warps ? dots[kMaxTopK][lane] : 0.0f) * sg * info.gate_rest;
          if (lane == 0) {
            if (j.gate_type == MOE_DTYPE_F32)
              static_cast<float*>(p.d_gate)[t] = d;
            else
              static_cast<__nv_bfloat16*>(p.d_gate)[t] = __float2bfloat16_rn(d);
          }
        }
      }
    }
    if (p.part_norm)
      store8<true>(p.part_norm + static_cast<int64_t>(blockIdx.x) * H, 0, H, acc_norm);
    if constexpr (POST)
      if (p.part_post)
        store8<true>(p.part_post + static_cast<int64_t>(blockIdx.x) * H, 0, H, acc_post);
    // rows of no expert
    if (p.d_rows && p.live_rows) {
      float zero[kVec];
#pragma unroll
      for (int c = 0; c < kVec; ++c) zero[c] = 0.0f;
      for (int64_t r = max(*p.live_rows, 0) + static_cast<int64_t>(blockIdx.x); r < j.rows;
           r += gridDim.x)
        store8<true>(p.d_rows + r * p.ld_drows, 0, H, zero);
    }
  }
}

// Column sums of the partials, in block order within each of kFinishRows runs of
// rows, then run by run.  blockIdx.y: 0 norm, 1 post.
constexpr int kFinishRows = 16;

struct JoinFinishArgs {
  const float* part[2];
  void* out[2];
  int blocks, H, type;
};

__global__ void __launch_bounds__(32 * kFinishRows)
    join_finish_kernel(const __grid_constant__ JoinFinishArgs p) {
  __shared__ float s[kFinishRows][33];
  pdl_wait();
  const float* part = p.part[blockIdx.y];
  if (!part) return;
  const int col = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  float sum = 0.0f;
  if (col < p.H)
#pragma unroll 8
    for (int b = y; b < p.blocks; b += kFinishRows) sum += part[static_cast<int64_t>(b) * p.H + col];
  s[y][threadIdx.x] = sum;
  __syncthreads();
  if (y != 0 || col >= p.H) return;
#pragma unroll
  for (int q = 1; q < kFinishRows; ++q) sum += s[q][threadIdx.x];
  if (p.type == MOE_DTYPE_F32)
    static_cast<float*>(p.out[blockIdx.y])[col] = sum;
  else
    static_cast<__nv_bfloat16*>(p.out[blockIdx.y])[col] = __float2bfloat16_rn(sum);
}

// Zeros in the rows of no expert where there is no token (the passes over tokens see
// to them themselves).
__global__ void __launch_bounds__(256)
    join_zero_rows_kernel(__nv_bfloat16* d_rows, int64_t ld, int rows, int H,
                          const int32_t* live_rows) {
  for (int64_t r = max(*live_rows, 0) + static_cast<int64_t>(blockIdx.x); r < rows; r += gridDim.x)
    for (int c = threadIdx.x; c < H; c += blockDim.x) d_rows[r * ld + c] = __float2bfloat16_rn(0.0f);
}

// ---------------------------------------------------------------- host
bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t size_of(int type) { return type == MOE_DTYPE_F32 ? 4 : 2; }
bool is_type(int t) { return t == MOE_DTYPE_F32 || t == MOE_DTYPE_BF16; }

// Whether rows can be read in vectors.
bool in_vectors(const void* p, int64_t ld, size_t size) {
  return !p || (aligned_to(p, 16) && (ld * static_cast<int64_t>(size)) % 16 == 0);
}

moe_status check_join(const moe_join* j, bool with_x) {
  if (!j || j->T < 0 || j->H < 1 || j->K < 0 || j->rows < 0) return MOE_ERR_INVALID_ARG;
  if (!is_type(j->x_type) || !is_type(j->weight_type) || !is_type(j->gate_type))
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(j->scale) || !(j->eps >= 0.0f) || !std::isfinite(j->eps))
    return MOE_ERR_INVALID_ARG;
  if (j->K > kMaxTopK || j->H > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if ((j->gate && !j->shared) || (j->post_weight && !j->K && !j->shared))
    return MOE_ERR_INVALID_ARG;
  if (j->T == 0) return MOE_OK;
  const size_t xs = size_of(j->x_type);
  if (with_x && (!j->x || !aligned_to(j->x, xs) || j->ld_x < j->H)) return MOE_ERR_INVALID_ARG;
  if (j->K && (!j->row_of_slot || !j->weights || !aligned_to(j->row_of_slot, 4) ||
               !aligned_to(j->weights, 4) || (j->rows > 0 && !j->expert_rows) ||
               !aligned_to(j->expert_rows, 2) || j->ld_rows < j->H))
    return MOE_ERR_INVALID_ARG;
  if (j->shared && (!aligned_to(j->shared, 2) || j->ld_shared < j->H)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(j->gate, size_of(j->gate_type)) ||
      !aligned_to(j->post_weight, size_of(j->weight_type)) ||
      !aligned_to(j->norm_weight, size_of(j->weight_type)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool join_vectors(const moe_join& j) {
  const size_t xs = size_of(j.x_type);
  return j.H % kVec == 0 && in_vectors(j.x, j.ld_x, xs) && in_vectors(j.expert_rows, j.ld_rows, 2) &&
         in_vectors(j.shared, j.ld_shared, 2) && in_vectors(j.post_weight, 0, 1) &&
         in_vectors(j.norm_weight, 0, 1);
}

// Vectors per thread: one up to 1024 threads, else four of 512 threads at most.
// (More threads with little to keep beat fewer with more: 4096 x 7168 in two vectors
// of 448 threads took 150 us forward and 470 backward.)
struct Shape {
  int nv, threads;
};
Shape shape_of(int H) {
  const int vectors = (H + kVec - 1) / kVec, nv = vectors <= 1024 ? 1 : 4;
  return {nv, ((vectors + nv - 1) / nv + 31) / 32 * 32};
}

// The ring's shape: blocks of an SM, and stages of each.
struct RingShape {
  int threads, blocks, stages, smem;
};
constexpr int kRingMost = 1024 - 32;  // consumers, of a vector each
constexpr int kSmSmem = 233472;       // of which each block has 1 KB more than it asks for
constexpr int kRingStatic = 5120;     // static shared memory, at most
constexpr int kRingDynamic = 232448 - kRingStatic;
bool ring_fits(int H) { return (H + kVec - 1) / kVec <= kRingMost; }
RingShape ring_shape(int H, int size) {
  constexpr int kFixed = kInfos * sizeof(TokenInfo) + 2 * kMaxStages * 8 + 16;
  const int bytes = H * size;
  RingShape r;
  r.threads = ((H + kVec - 1) / kVec + 31) / 32 * 32 + 32;
  // (64 registers a thread; several blocks, whose sums hide behind each other's
  // copies, with a dozen rows' stages each)
  r.blocks = std::max(1, std::min({16, 1024 / r.threads,
                                   kSmSmem / (12 * bytes + kFixed + kRingStatic + 1024)}));
  r.stages = std::min(kMaxStages, (kSmSmem / r.blocks - 1024 - kRingStatic - kFixed) / bytes);
  r.smem = r.stages * bytes + kFixed;
  return r;
}

// Where the ring is the faster way.  Forward pass, 7168 columns: 512 tokens 20 us
// against 15 of loads, 1024 38 and 42, 2048 70 and 75; 2048 columns: 4096 tokens 41
// and 38.  Backward pass, 7168: 304 tokens 23 and 27, 512 42 and 58, 2048 112 and
// 176; 2048 with a norm after the block: 1024 tokens 33 and 29, 4096 97 and 97; 512:
// 8192 tokens 40 and 53.  (4096 tokens, top-8, forward and backward: 7936 columns by
// the ring 136 and 228, 8192 by loads 157 and 352, 16384 467 and 957.)
bool use_ring(int T, int H, int size, bool backward) {
  if (!ring_fits(H)) return false;
  const bool wide = H > 4096;
  if (!backward && !wide) return false;
  return T >= (backward && wide ? 2 : 5) * ring_shape(H, size).blocks * kSms;
}

template <typename K, typename Args>
cudaError_t launch_ring(K kernel, OncePerDevice& prepared, const RingShape& r, int T, Args p,
                        cudaStream_t s) {
  const cudaError_t ready = prepared([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingDynamic);
  });
  if (ready != cudaSuccess) return ready;
  p.stages = r.stages;
  return launch_pdl(false, kernel, dim3(std::min(T, r.blocks * kSms)), dim3(r.threads), r.smem, s, p);
}

template <typename X, bool VEC>
cudaError_t run_forward(const JoinArgs& p, cudaStream_t s) {
  const int T = p.j.T;
  if constexpr (VEC)
    if (use_ring(T, p.j.H, sizeof(X), false)) {
      static OncePerDevice prepared;
      return launch_ring(join_forward_ring_kernel<X>, prepared, ring_shape(p.j.H, sizeof(X)), T, p, s);
    }
  const Shape q = shape_of(p.j.H);
  auto go = [&](auto k) { return launch_pdl(false, k, dim3(T), dim3(q.threads), 0, s, p); };
  return q.nv == 1 ? go(join_forward_kernel<X, 1, VEC>) : go(join_forward_kernel<X, 4, VEC>);
}

// Blocks of the backward pass: as many as run at a time (ring: 0, or the size of x's
// elements).
int back_blocks(int T, int H, int ring) {
  const Shape q = shape_of(H);
  const int resident = ring ? ring_shape(H, ring).blocks
                            : std::max(1, std::min(8, 65536 / ((q.nv == 1 ? 64 : 128) * q.threads)));
  return std::max(1, std::min(T, resident * kSms));
}

bool back_by_ring(const JoinBackArgs& p, int size) {
  return (p.d_h || p.d_x_out) && use_ring(p.j.T, p.j.H, size, true);
}

template <typename X, bool VEC>
cudaError_t run_backward(const JoinBackArgs& p, cudaStream_t s) {
  if constexpr (VEC)
    if (back_by_ring(p, sizeof(X))) {
      static OncePerDevice plain, post;
      const RingShape r = ring_shape(p.j.H, sizeof(X));
      return p.j.post_weight
                 ? launch_ring(join_backward_ring_kernel<X, true>, post, r, p.j.T, p, s)
                 : launch_ring(join_backward_ring_kernel<X, false>, plain, r, p.j.T, p, s);
    }
  const Shape q = shape_of(p.j.H);
  auto go = [&](auto k) {
    return launch_pdl(false, k, dim3(back_blocks(p.j.T, p.j.H, 0)), dim3(q.threads), 0, s, p);
  };
  return q.nv == 1 ? go(join_backward_kernel<X, 1, VEC>) : go(join_backward_kernel<X, 4, VEC>);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_join_forward(const moe_join* j, void* x_out, int64_t ld_out, void* h, int64_t ld_h,
                            void* codes, int64_t ld_codes, float* code_scales, float* post_rstd,
                            float* norm_rstd, void* stream) {
  const moe_status st = check_join(j, true);
  if (st != MOE_OK) return st;
  if (j->T == 0) return MOE_OK;
  const bool normed = h || codes;
  if (normed != (j->norm_weight != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((x_out && ld_out < j->H) || (h && ld_h < j->H) || (codes && ld_codes < j->H))
    return MOE_ERR_INVALID_ARG;
  if ((j->K || j->shared) && !x_out) return MOE_ERR_INVALID_ARG;
  if (!x_out && !normed) return MOE_ERR_INVALID_ARG;
  const size_t xs = size_of(j->x_type);
  if (!aligned_to(x_out, xs) || !aligned_to(h, 2) || (codes && !code_scales) ||
      !aligned_to(code_scales, 4) || !aligned_to(post_rstd, 4) || !aligned_to(norm_rstd, 4))
    return MOE_ERR_INVALID_ARG;
  JoinArgs p{};
  p.j = *j;
  p.x_out = x_out, p.ld_out = ld_out;
  p.h = static_cast<__nv_bfloat16*>(h), p.ld_h = ld_h;
  p.codes = static_cast<int8_t*>(codes), p.ld_codes = ld_codes;
  p.code_scales = code_scales, p.post_rstd = post_rstd, p.norm_rstd = norm_rstd;
  const bool vec = join_vectors(*j) && in_vectors(x_out, ld_out, xs) && in_vectors(h, ld_h, 2) &&
                   in_vectors(codes, ld_codes, 1);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (j->x_type == MOE_DTYPE_F32)
    e = vec ? run_forward<float, true>(p, s) : run_forward<float, false>(p, s);
  else
    e = vec ? run_forward<__nv_bfloat16, true>(p, s) : run_forward<__nv_bfloat16, false>(p, s);
  return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_join_workspace(int T, int H) {
  if (T < 1 || H < 1 || H > kMaxWidth) return 0;
  const int blocks =
      std::max({back_blocks(T, H, 0), ring_fits(H) ? back_blocks(T, H, 2) : 0,
                ring_fits(H) ? back_blocks(T, H, 4) : 0});
  return static_cast<size_t>(2) * blocks * ((H + 3) / 4 * 4) * 4;
}

moe_status moe_join_backward(const moe_join* j, const void* x_out, int64_t ld_out,
                             const float* post_rstd, const float* norm_rstd, const void* d_x_out,
                             int64_t ld_dxo, const void* d_h, int64_t ld_dh, void* d_x,
                             int64_t ld_dx, void* d_rows, int64_t ld_drows,
                             const int32_t* live_rows, float* d_weights, void* d_shared,
                             int64_t ld_dshared, void* d_gate, void* d_post, void* d_norm,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status st = check_join(j, false);
  if (st != MOE_OK) return st;
  if ((d_h || d_norm) && !j->norm_weight) return MOE_ERR_INVALID_ARG;
  if ((d_norm && !d_h && j->T > 0) || (d_post && !j->post_weight) || (d_gate && !j->gate) ||
      (d_shared && !j->shared) || ((d_rows || d_weights) && !j->K))
    return MOE_ERR_INVALID_ARG;
  if ((d_x_out && ld_dxo < j->H) || (d_h && (ld_dh < j->H || ld_out < j->H)) ||
      (d_x && ld_dx < j->H) || (d_rows && ld_drows < j->H) || (d_shared && ld_dshared < j->H))
    return MOE_ERR_INVALID_ARG;
  const size_t xs = size_of(j->x_type);
  if (!aligned_to(d_post, size_of(j->weight_type)) || !aligned_to(d_norm, size_of(j->weight_type)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  JoinFinishArgs f{{nullptr, nullptr}, {d_norm, d_post}, 0, j->H, j->weight_type};
  if (j->T > 0) {
    if ((d_h && (!x_out || !norm_rstd)) || (j->post_weight && !post_rstd) ||
        !aligned_to(x_out, xs) || !aligned_to(d_x_out, xs) || !aligned_to(d_x, xs) ||
        !aligned_to(d_h, 2) || !aligned_to(d_rows, 2) || !aligned_to(d_shared, 2) ||
        !aligned_to(d_gate, size_of(j->gate_type)) || !aligned_to(post_rstd, 4) ||
        !aligned_to(norm_rstd, 4) || !aligned_to(live_rows, 4) || !aligned_to(d_weights, 4))
      return MOE_ERR_INVALID_ARG;
    if ((d_post || d_norm) && (!workspace || !aligned_to(workspace, 16) ||
                               workspace_bytes < moe_join_workspace(j->T, j->H)))
      return MOE_ERR_INVALID_ARG;
    JoinBackArgs p{};
    p.j = *j;
    p.x_out = d_h ? x_out : nullptr;  // (read with d_h alone)
    p.ld_out = ld_out, p.d_x_out = d_x_out, p.ld_dxo = ld_dxo;
    p.d_h = d_h, p.ld_dh = ld_dh, p.post_rstd = post_rstd, p.norm_rstd = norm_rstd;
    p.d_x = d_x, p.ld_dx = ld_dx;
    p.d_rows = static_cast<__nv_bfloat16*>(d_rows), p.ld_drows = ld_drows;
    p.live_rows = live_rows;
    p.d_weights = d_weights;
    p.d_shared = static_cast<__nv_bfloat16*>(d_shared), p.ld_dshared = ld_dshared;
    p.d_gate = d_gate;
    moe_join in = *j;
    in.x = nullptr;  // (not read)
    const bool vec = join_vectors(in) && in_vectors(p.x_out, ld_out, xs) &&
                     in_vectors(d_x_out, ld_dxo, xs) && in_vectors(d_h, ld_dh, 2) &&
                     in_vectors(d_x, ld_dx, xs) && in_vectors(d_rows, ld_drows, 2) &&
                     in_vectors(d_shared, ld_dshared, 2);
    const int size = static_cast<int>(xs);
    f.blocks = back_blocks(j->T, j->H, vec && back_by_ring(p, size) ? size : 0);
    float* ws = static_cast<float*>(workspace);
    if (d_norm) f.part[0] = p.part_norm = ws;
    if (d_post)
      f.part[1] = p.part_post = ws + static_cast<int64_t>(f.blocks) * ((j->H + 3) / 4 * 4);
    cudaError_t e;
    if (j->x_type == MOE_DTYPE_F32)
      e = vec ? run_backward<float, true>(p, s) : run_backward<float, false>(p, s);
    else
      e = vec ? run_backward<__nv_bfloat16, true>(p, s) : run_backward<__nv_bfloat16, false>(p, s);
    if (take_error(e) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (j->T == 0 && d_rows && live_rows && j->rows > 0) {
    if (!aligned_to(d_rows, 2) || !aligned_to(live_rows, 4)) return MOE_ERR_INVALID_ARG;
    const cudaError_t e =
        launch_pdl(false, join_zero_rows_kernel, dim3(std::min(j->rows, 8 * kSms)), dim3(256), 0, s,
                   static_cast<__nv_bfloat16*>(d_rows), ld_drows, j->rows, j->H, live_rows);
    if (take_error(e) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (!d_post && !d_norm) return MOE_OK;
  if (j->T == 0) {
    // (sums over no tokens)
    const size_t bytes = j->H * size_of(j->weight_type);
    cudaError_t e = cudaSuccess;
    if (d_norm) e = cudaMemsetAsync(d_norm, 0, bytes, s);
    if (d_post && e == cudaSuccess) e = cudaMemsetAsync(d_post, 0, bytes, s);
    return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  const cudaError_t e =
      launch_pdl(true, join_finish_kernel, dim3((j->H + 31) / 32, d_post ? 2 : 1),
                 dim3(32, kFinishRows), 0, s, f);
  return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_join_status(void) {
  int v = 0;
  const int zero = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_join_status, sizeof(int));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_join_status, &zero, sizeof(int));
  if (take_error(e) != cudaSuccess) return MOE_ERR_CUDA;
  return v ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

}  // extern "C"
