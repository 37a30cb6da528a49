// int8.cu -- products of 8-bit integer matrices with a scale per token and a scale
// per output channel: the quantiser of the activations, and the entry points with
// their checks.  The products run in int8_gemm.cu.
//
// Quantisation of a row: s = amax / 127, codes round(x / s) to even within +-127,
// both quotients rounded to nearest in fp32.  The products take the codes as f16
// (exact), so the calls that quantise for themselves write them so at once.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "int8_quant.cuh"
#include "internal.h"
#include "moe.h"
#include "ptx.cuh"

namespace moe {

namespace {

// Largest M, N and K of a product: rounding one up to a tile, or to a block's
// stride over a row, stays in 32 bits.
constexpr int kMaxExtent = INT32_MAX - 65791;

// Eight codes to memory: bytes, or f16.
template <bool F16>
__device__ __forceinline__ void store_codes(void* row, int c0, int cols, bool vec,
                                            const I8Coder& coder, const float (&v)[8]) {
  if constexpr (F16) {
    uint16_t* d = static_cast<uint16_t*>(row) + c0;
    const uint4 w = coder.f16(v);
    if (vec && c0 + 8 <= cols) {
      *reinterpret_cast<uint4*>(d) = w;
    } else {
      const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + i < cols) d[i] = static_cast<uint16_t>(h[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    int8_t* d = static_cast<int8_t*>(row) + c0;
    const uint2 w = coder.bytes(v);
    if (vec && c0 + 8 <= cols) {
      *reinterpret_cast<uint2*>(d) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + i < cols) d[i] = static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
  }
}

// `warps` warps of a block (a power of two) take a row, the block 8 / warps of
// them.  A thread's first kKept vectors of eight stay in registers between the
// maximum and the codes; what a longer row has beyond is read again.  With many rows
// 8192 x 7168 take 43 us (5.4 TB/s), 24576 gathered ones x 2048 34 us (81 with a
// block to a row).
constexpr int kKept = 4;

template <typename X, bool F16>
__global__ void __launch_bounds__(256)
    int8_quantize_kernel(const X* x, int64_t ldx, int x_rows, const int32_t* slots, int top_k,
                         int rows, int cols, void* codes, int64_t ld_codes, float* scales, int vec,
                         int warps) {
  // A product that follows may set itself up and load weights meanwhile.  (fp32 rows
  // are those of the product before, which may not be over.)
  if (sizeof(X) == 4) pdl_wait();
  pdl_launch_dependents();
  __shared__ uint32_t s_max[8];
  const int warp = threadIdx.x >> 5, sub = warp & (warps - 1);
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (8 / warps) + warp / warps;
  const bool real = r < rows;
  const int slot = real && slots ? slots[r] : 0;
  const int64_t src = slots ? slot / top_k : r;
  const bool in = real && slot >= 0 && src < x_rows;
  const X* row = x + (in ? src : 0) * ldx;
  const int stride = warps * 256;  // columns of one vector of every thread of the row
  const int first = (sub * 32 + (threadIdx.x & 31)) * 8, end = in ? cols : 0;
  // eight values: bf16 in pairs, or fp32
  constexpr int kWords = sizeof(X) == 2 ? 4 : 8;
  auto load = [&](int c0, uint32_t (&v)[kWords]) {
    if (c0 >= end) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) v[i] = 0u;
    } else if (vec && c0 + 8 <= cols) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 q = reinterpret_cast<const uint4*>(row + c0)[i / 4];
        v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(X) == 2) {
          const uint16_t* s = reinterpret_cast<const uint16_t*>(row) + c0;
          const uint32_t lo = c0 + 2 * i < cols ? s[2 * i] : 0u;
          const uint32_t hi = c0 + 2 * i + 1 < cols ? s[2 * i + 1] : 0u;
          v[i] = lo | hi << 16;
        } else {
          v[i] = c0 + i < cols ? __float_as_uint(row[c0 + i]) : 0u;
        }
      }
    }
  };
  auto largest = [](const uint32_t (&v)[kWords], uint32_t m) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(X) == 2) m = max(m, (v[i] << 16) & 0x7FFFFFFFu);
      m = max(m, v[i] & (sizeof(X) == 2 ? 0x7FFF0000u : 0x7FFFFFFFu));
    }
    return m;
  };
  uint32_t kept[kKept][kWords], m = 0u;
#pragma unroll
  for (int i = 0; i < kKept; ++i) load(first + i * stride, kept[i]);
#pragma unroll
  for (int i = 0; i < kKept; ++i) m = largest(kept[i], m);
  for (int c0 = first + kKept * stride; c0 < end; c0 += stride) {
    uint32_t v[kWords];
    load(c0, v);
    m = largest(v, m);
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (warps > 1) {
    if ((threadIdx.x & 31) == 0) s_max[warp] = m;
    __syncthreads();
    for (int w = 0; w < warps; ++w) m = max(m, s_max[warp - sub + w]);
  }
  if (!real) return;
  const float s = i8_scale(m);
  const I8Coder coder(s);
  if (first == 0) scales[r] = s;
  void* out = F16 ? static_cast<void*>(static_cast<uint16_t*>(codes) + r * ld_codes)
                  : static_cast<void*>(static_cast<int8_t*>(codes) + r * ld_codes);
  auto put = [&](int c0, const uint32_t (&v)[kWords]) {
    if (c0 >= cols) return;
    float f[8];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(X) == 2) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
      } else {
        f[i] = __uint_as_float(v[i]);
      }
    }
    store_codes<F16>(out, c0, cols, vec, coder, f);
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i) put(first + i * stride, kept[i]);
  for (int c0 = first + kKept * stride; c0 < cols; c0 += stride) {
    uint32_t v[kWords];
    load(c0, v);
    put(c0, v);
  }
}

// int8 codes to f16 ones, eight at a time; out: rows of a multiple of eight.
__global__ void __launch_bounds__(256)
    int8_widen_kernel(const int8_t* codes, int64_t ld, int rows, int cols, uint16_t* out,
                      int64_t ld_out, int vec) {
  pdl_launch_dependents();
  const int per = (cols + 7) / 8;
  const int64_t n = static_cast<int64_t>(rows) * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / per;
    const int c0 = static_cast<int>(i - r * per) * 8;
    const int8_t* src = codes + r * ld + c0;
    uint32_t q[2] = {0u, 0u};  // four codes each
    if (vec && c0 + 8 <= cols) {
      const uint2 w = *reinterpret_cast<const uint2*>(src);
      q[0] = w.x, q[1] = w.y;
    } else {
#pragma unroll
      for (int b = 0; b < 8; ++b)
        if (c0 + b < cols)
          q[b >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(src[b])) << (8 * (b & 3));
    }
    uint4 f;
    i8_widen4(q[0], f.x, f.y);
    i8_widen4(q[1], f.z, f.w);
    // (rows of a multiple of eight codes: the last ones' padding is theirs)
    *reinterpret_cast<uint4*>(out + r * ld_out + c0) = f;
  }
}

// The experts' rows, two and more of a token, are quantised once a token and copied from
// this many codes on: 64 x (2048, 1024), top-6, 512 tokens (6.3 M codes) 104.3 us and
// 103.9 with every row quantised for itself, 1024 128.6 and 129.5, 4096 269 and 278; 64
// x (7168, 2048), top-8, 64 tokens (3.7 M) 446 and 440, 512 545 and 549.
constexpr int64_t kOnceLeast = int64_t{1} << 23;

// Rows of a token's codes for each of its slots, as f16, with their scales: a warp to a
// row.  cols: a multiple of sixteen, like all strides.
__global__ void __launch_bounds__(256)
    int8_gather_kernel(const int8_t* codes, const float* scales, int T, const int32_t* slots,
                       int top_k, int rows, int cols, uint16_t* out, float* out_scales) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int slot = slots[r], t = slot / top_k;
  const bool in = slot >= 0 && t < T;
  if (lane == 0) out_scales[r] = in ? scales[t] : 0.0f;
  const int8_t* src = codes + static_cast<int64_t>(in ? t : 0) * cols;
  uint16_t* dst = out + r * cols;
#pragma unroll 4
  for (int c0 = lane * 8; c0 < cols; c0 += 256) {
    const uint2 q = in ? *reinterpret_cast<const uint2*>(src + c0) : make_uint2(0u, 0u);
    uint4 f;
    i8_widen4(q.x, f.x, f.y);
    i8_widen4(q.y, f.z, f.w);
    *reinterpret_cast<uint4*>(dst + c0) = f;
  }
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---------------------------------------------------------------- arguments
struct Product {
  const void* w;
  int64_t ldw;
  const float* w_scales;
  const int32_t* offsets;
  int E, M, N, K;
};

// TMA wants 16-byte aligned bases and row strides; scales and offsets are read as
// 32-bit words.
moe_status check_weights(const Product& p) {
  if (p.M < 0 || p.N < 1 || p.K < 1 || p.E < 1 || (!p.offsets && p.E != 1))
    return MOE_ERR_INVALID_ARG;
  if (p.E > kMaxExperts || p.M > kMaxExtent || p.N > kMaxExtent || p.K > kMaxExtent)
    return MOE_ERR_UNSUPPORTED;
  if (p.ldw < p.K) return MOE_ERR_INVALID_ARG;
  if (p.M == 0) return MOE_OK;
  if (!p.w || !p.w_scales || !aligned_to(p.w, 16) || p.ldw % 16 || !aligned_to(p.w_scales, 4) ||
      !aligned_to(p.offsets, 4))
    return MOE_ERR_INVALID_ARG;
  // strides of the tensor maps and the item count stay in range
  if (p.ldw >= (int64_t{1} << 39) / p.N ||
      (static_cast<int64_t>(p.E) + p.M / 16 + 1) * ((p.N + 127) / 128) > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspaces: f16 codes in rows of a multiple of eight, then the scales.
int64_t padded(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
struct Coded {
  uint16_t* codes;
  int64_t ld;
  float* scales;
  static int64_t code_bytes(int64_t rows, int64_t cols) {
    return padded(rows * padded(cols, 8) * 2, 256);
  }
  static int64_t bytes(int64_t rows, int64_t cols) {
    return code_bytes(rows, cols) + padded(rows * 4, 256);
  }
  Coded(void* ws, int64_t rows, int64_t cols)
      : codes(static_cast<uint16_t*>(ws)), ld(padded(cols, 8)),
        scales(reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + code_bytes(rows, cols))) {}
};

// SwiGLU's limit: +inf for none.
float limit_of(float clamp) { return clamp > 0.0f && std::isfinite(clamp) ? clamp : INFINITY; }

// The product of f16 codes x [M, K] with their scales.
moe_status run_product(const Product& p, const uint16_t* x, int64_t ld, const float* scales,
                       bool swiglu, void* out, int64_t ldo, float clamp, cudaStream_t s) {
  const BlockscaleDevice* d = current_device();
  if (!d) return MOE_ERR_NO_DEVICE;
  auto encode = [&](CUtensorMap* m, CUtensorMapDataType type, const void* base, int rank,
                    const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    const cuuint32_t one[3] = {1, 1, 1};
    return tensor_map_encoder()(m, type, rank, const_cast<void*>(base), dims, strides, box, one,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  Int8Maps maps;
  // (one expert: all chunks take the largest box)
  const bool pairs = int8_in_pairs(p.M, p.N, p.E);
  const int most = pairs ? 128 : int8_chunk_rows(p.M, p.N, p.E);
  const int boxes = most <= 16 ? 1 : most <= 32 ? 2 : most <= 64 ? 3 : 4;
  const cuuint64_t xdims[2] = {static_cast<cuuint64_t>(p.K), static_cast<cuuint64_t>(p.M)};
  const cuuint64_t xstr[1] = {static_cast<cuuint64_t>(ld) * 2};
  for (int i = p.E == 1 && !pairs ? boxes - 1 : 0; i < boxes; ++i) {
    const cuuint32_t box[2] = {64, 16u << i};
    if (!encode(&maps.x[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, 2, xdims, xstr, box))
      return MOE_ERR_CUDA;
  }
  const cuuint64_t wdims[3] = {static_cast<cuuint64_t>(p.K), static_cast<cuuint64_t>(p.N),
                               static_cast<cuuint64_t>(p.E)};
  const cuuint64_t wstr[2] = {static_cast<cuuint64_t>(p.ldw), static_cast<cuuint64_t>(p.ldw) * p.N};
  const cuuint32_t wbox[3] = {128, pairs && swiglu ? 64u : 128u, 1};
  if (!encode(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w, 3, wdims, wstr, wbox)) return MOE_ERR_CUDA;
  Int8Args a{};
  a.a_scales = scales;
  a.w_scales = p.w_scales;
  a.offsets = p.offsets;
  a.E = p.E, a.M = p.M, a.N = p.N, a.K = p.K;
  a.out = out;
  a.ldo = ldo;
  a.out_pairs = aligned_to(out, 4) && ldo % 2 == 0;
  a.out_fours = aligned_to(out, 8) && ldo % 4 == 0;
  a.clamp = limit_of(clamp);
  return take_error(launch_int8(maps, a, swiglu, *d, s)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <bool F16, typename X>
moe_status run_quantize(const X* x, int64_t ldx, int x_rows, const int32_t* slots, int top_k,
                        int rows, int cols, void* codes, int64_t ld_codes, float* scales,
                        cudaStream_t s) {
  const bool vec = aligned_to(x, 16) && ldx % 8 == 0 && aligned_to(codes, F16 ? 16 : 8) &&
                   ld_codes % 8 == 0;
  // Warps of a row: as many as keep it in registers, and more where the rows alone
  // would leave SMs without a block.
  int warps = 1;
  while (warps < 8 && (cols > warps * 256 * kKept ||
                       (static_cast<int64_t>(rows) * warps < 152 * 8 && cols > warps * 256)))
    warps *= 2;
  const int64_t blocks = (static_cast<int64_t>(rows) * warps + 7) / 8;
  const cudaError_t e =
      launch_pdl(sizeof(X) == 4, int8_quantize_kernel<X, F16>, dim3(static_cast<unsigned>(blocks)),
                 dim3(256), 0, s, x, ldx, x_rows, slots, top_k, rows, cols, codes, ld_codes, scales,
                 static_cast<int>(vec), warps);
  return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// The product of a few rows: x in bf16, or codes a with their scales.
moe_status run_rows(const Product& p, const void* x, int64_t ldx, const int8_t* a, int64_t lda,
                    const float* scales, bool early, void* out, int64_t ldo, cudaStream_t s) {
  Int8RowsArgs r{};
  r.w = static_cast<const int8_t*>(p.w), r.ldw = p.ldw, r.w_scales = p.w_scales;
  r.x = static_cast<const __nv_bfloat16*>(x), r.ldx = ldx;
  r.x_vec = aligned_to(x, 16) && ldx % 8 == 0;
  r.a = a, r.lda = lda, r.a_vec = aligned_to(a, 16) && lda % 16 == 0, r.a_scales = scales;
  r.M = p.M, r.N = p.N, r.K = p.K;
  r.out = static_cast<__nv_bfloat16*>(out), r.ldo = ldo;
  return take_error(launch_int8_rows(r, early, s)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// The products of a few rows of several experts: codes a with their scales; swiglu:
// out is h in f32.
moe_status run_group_rows(const Product& p, const int8_t* a, int64_t lda, const float* scales,
                          bool swiglu, bool early, void* out, int64_t ldo, float clamp,
                          cudaStream_t s) {
  Int8RowsArgs r{};
  r.w = static_cast<const int8_t*>(p.w), r.ldw = p.ldw, r.w_scales = p.w_scales;
  r.a = a, r.lda = lda, r.a_vec = aligned_to(a, 16) && lda % 16 == 0, r.a_scales = scales;
  r.M = p.M, r.N = p.N, r.K = p.K;
  r.out = static_cast<__nv_bfloat16*>(out), r.h = static_cast<float*>(out), r.ldo = ldo;
  r.offsets = p.offsets, r.E = p.E;
  r.clamp = limit_of(clamp);
  return take_error(launch_int8_group_rows(r, swiglu, early, s)) == cudaSuccess ? MOE_OK
                                                                               : MOE_ERR_CUDA;
}

// Blocks of an elementwise kernel of 256 threads over n vectors.
int vector_blocks(int64_t n) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, 152 * 8 * 4)));
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_int8_quantize(const void* x, int64_t ldx, int x_rows, const int32_t* slots,
                             int top_k, int rows, int cols, void* codes, int64_t ld_codes,
                             float* scales, void* stream) {
  if (rows < 0 || cols < 1 || x_rows < 0 || ldx < cols || ld_codes < cols)
    return MOE_ERR_INVALID_ARG;
  if (slots ? top_k < 1 : x_rows < rows) return MOE_ERR_INVALID_ARG;
  if (cols > kMaxExtent) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if ((!x && x_rows > 0) || !codes || !scales || !aligned_to(x, 2) || !aligned_to(slots, 4) ||
      !aligned_to(scales, 4))
    return MOE_ERR_INVALID_ARG;
  return run_quantize<false>(static_cast<const __nv_bfloat16*>(x), ldx, x_rows, slots, top_k, rows,
                             cols, codes, ld_codes, scales, static_cast<cudaStream_t>(stream));
}

size_t moe_int8_matmul_workspace(int M, int K, int grouped) {
  if (M < 1 || K < 1 || M > kMaxExtent || K > kMaxExtent) return 0;
  return !grouped && int8_by_rows(M, K, 1) ? 0 : static_cast<size_t>(Coded::bytes(M, K));
}

moe_status moe_int8_matmul(const void* a, int64_t lda, const float* a_scales, const void* w,
                           int64_t ldw, const float* w_scales, const int32_t* offsets, int E,
                           int M, int N, int K, void* out, int64_t ldo, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const Product p{w, ldw, w_scales, offsets, E, M, N, K};
  const moe_status st = check_weights(p);
  if (st != MOE_OK) return st;
  if (lda < K || ldo < N) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const size_t need = moe_int8_matmul_workspace(M, K, offsets != nullptr);
  if (!a || !a_scales || !out || !aligned_to(a_scales, 4) || !aligned_to(out, 2) ||
      workspace_bytes < need || (need && (!workspace || !aligned_to(workspace, 16))))
    return MOE_ERR_INVALID_ARG;
  if (!current_device()) return MOE_ERR_NO_DEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!need)
    return run_rows(p, nullptr, 0, static_cast<const int8_t*>(a), lda, a_scales, false, out, ldo, s);
  if (int8_by_group_rows(M, N, K, E))
    return run_group_rows(p, static_cast<const int8_t*>(a), lda, a_scales, false, false, out, ldo, 0.0f, s);
  const Coded c(workspace, M, K);
  const int64_t vectors = static_cast<int64_t>(M) * ((K + 7) / 8);
  const cudaError_t e = launch_pdl(false, int8_widen_kernel, dim3(vector_blocks(vectors)),
                                   dim3(256), 0, s, static_cast<const int8_t*>(a), lda, M, K,
                                   c.codes, c.ld, static_cast<int>(aligned_to(a, 8) && lda % 8 == 0));
  if (take_error(e) != cudaSuccess) return MOE_ERR_CUDA;
  return run_product(p, c.codes, c.ld, a_scales, false, out, ldo, 0.0f, s);
}

size_t moe_int8_linear_workspace(int M, int N, int K) {
  return N < 1 || N > kMaxExtent || int8_rows_quantize(M, K, 1) ? 0
                                                                : moe_int8_matmul_workspace(M, K, 1);
}

moe_status moe_int8_linear(const void* x, int64_t ldx, const void* w, int64_t ldw,
                           const float* w_scales, int M, int N, int K, void* out, int64_t ldo,
                           void* workspace, size_t workspace_bytes, void* stream) {
  const Product p{w, ldw, w_scales, nullptr, 1, M, N, K};
  const moe_status st = check_weights(p);
  if (st != MOE_OK) return st;
  if (ldx < K || ldo < N) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const size_t need = moe_int8_linear_workspace(M, N, K);
  if (!x || !out || !aligned_to(x, 2) || !aligned_to(out, 2) || workspace_bytes < need ||
      (need && (!workspace || !aligned_to(workspace, 16))))
    return MOE_ERR_INVALID_ARG;
  if (!current_device()) return MOE_ERR_NO_DEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!need) return run_rows(p, x, ldx, nullptr, 0, nullptr, false, out, ldo, s);
  const Coded c(workspace, M, K);
  if (int8_by_rows(M, K, 1)) {
    // (codes of 8 bits where those of 16 would be)
    int8_t* codes = reinterpret_cast<int8_t*>(c.codes);
    const int64_t ld = padded(K, 16);
    const moe_status sq = run_quantize<false>(static_cast<const __nv_bfloat16*>(x), ldx, M, nullptr,
                                              1, M, K, codes, ld, c.scales, s);
    if (sq != MOE_OK) return sq;
    return run_rows(p, nullptr, 0, codes, ld, c.scales, true, out, ldo, s);
  }
  const moe_status sq = run_quantize<true>(static_cast<const __nv_bfloat16*>(x), ldx, M, nullptr, 1,
                                           M, K, c.codes, c.ld, c.scales, s);
  if (sq != MOE_OK) return sq;
  return run_product(p, c.codes, c.ld, c.scales, false, out, ldo, 0.0f, s);
}

size_t moe_int8_experts_workspace(int rows, int H, int I) {
  if (rows < 1 || H < 1 || I < 1 || rows > kMaxExtent || H > kMaxExtent || I > kMaxExtent / 2)
    return 0;
  // the rows' codes, h in fp32, its codes
  return static_cast<size_t>(Coded::bytes(rows, H) +
                             padded(static_cast<int64_t>(rows) * I * 4, 256) +
                             Coded::bytes(rows, I));
}

moe_status moe_int8_experts(const void* x, int64_t ldx, int T, const int32_t* slots, int top_k,
                            int rows, const int32_t* offsets, int E, const void* w13,
                            const float* w13_scales, const void* w2, const float* w2_scales, int H,
                            int I, float clamp_limit, void* out, int64_t ldo, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (I < 1 || H < 1 || T < 0 || top_k < 1 || !offsets) return MOE_ERR_INVALID_ARG;
  if (I % 16 || H % 16 || I > kMaxExtent / 2) return MOE_ERR_UNSUPPORTED;
  const Product p1{w13, H, w13_scales, offsets, E, rows, 2 * I, H};
  const Product p2{w2, I, w2_scales, offsets, E, rows, H, I};
  moe_status st = check_weights(p1);
  if (st == MOE_OK) st = check_weights(p2);
  if (st != MOE_OK) return st;
  if (ldx < H || ldo < H) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if ((!x && T > 0) || !slots || !out || !workspace || !aligned_to(x, 2) || !aligned_to(slots, 4) ||
      !aligned_to(out, 2) || !aligned_to(workspace, 16) ||
      workspace_bytes < moe_int8_experts_workspace(rows, H, I))
    return MOE_ERR_INVALID_ARG;
  if (!current_device()) return MOE_ERR_NO_DEVICE;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  const Coded c(at, rows, H);
  at += Coded::bytes(rows, H);
  float* h = reinterpret_cast<float*>(at);
  at += padded(static_cast<int64_t>(rows) * I * 4, 256);
  const Coded hc(at, rows, I);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (int8_by_group_rows(rows, std::max(2 * I, H), std::max(H, I), E)) {
    // (codes of 8 bits where those of 16 would be)
    int8_t *codes = reinterpret_cast<int8_t*>(c.codes), *h_codes = reinterpret_cast<int8_t*>(hc.codes);
    st = run_quantize<false>(static_cast<const __nv_bfloat16*>(x), ldx, T, slots, top_k, rows, H,
                             codes, H, c.scales, s);
    if (st == MOE_OK)
      st = run_group_rows(p1, codes, H, c.scales, true, true, h, I, clamp_limit, s);
    if (st == MOE_OK)
      st = run_quantize<false>(h, I, rows, nullptr, 1, rows, I, h_codes, I, hc.scales, s);
    if (st == MOE_OK)
      st = run_group_rows(p2, h_codes, I, hc.scales, false, true, out, ldo, 0.0f, s);
    return st;
  }
  const __nv_bfloat16* tokens = static_cast<const __nv_bfloat16*>(x);
  const int64_t token_codes = padded(static_cast<int64_t>(T) * H, 256);
  if (T > 0 && rows / 2 >= T && static_cast<int64_t>(rows) * H >= kOnceLeast &&
      token_codes + 4 * static_cast<int64_t>(T) <= static_cast<int64_t>(rows) * I * 4) {
    // Each token once, and its codes (where h will be) to all of its rows.
    int8_t* once = reinterpret_cast<int8_t*>(h);
    float* once_scales = reinterpret_cast<float*>(once + token_codes);
    st = run_quantize<false>(tokens, ldx, T, nullptr, 1, T, H, once, H, once_scales, s);
    if (st == MOE_OK &&
        take_error(launch_pdl(true, int8_gather_kernel, dim3((rows - 1) / 8 + 1), dim3(256), 0, s,
                              once, once_scales, T, slots, top_k, rows, H, c.codes, c.scales)) !=
            cudaSuccess)
      st = MOE_ERR_CUDA;
  } else {
    st = run_quantize<true>(tokens, ldx, T, slots, top_k, rows, H, c.codes, c.ld, c.scales, s);
  }
  if (st == MOE_OK) st = run_product(p1, c.codes, c.ld, c.scales, true, h, I, clamp_limit, s);
  if (st == MOE_OK)
    st = run_quantize<true>(h, I, rows, nullptr, 1, rows, I, hc.codes, hc.ld, hc.scales, s);
  if (st == MOE_OK) st = run_product(p2, hc.codes, hc.ld, hc.scales, false, out, ldo, 0.0f, s);
  return st;
}

moe_status moe_int8_status(void) {
  int v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess || int8_status(&v) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return v ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

}  // extern "C"
