// blockscale.cu -- products of e4m3 matrices with one fp32 scale per block of
// 128 (activations: per row and 128 columns, weights: per 128 x 128): the
// quantiser of the activations, and the entry points with their checks.  The
// products run in blockscale_gemm.cu.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "blockscale_quant.cuh"
#include "internal.h"
#include "moe.h"

namespace moe {

namespace {

constexpr int kBlk = 128;
// Largest M, N and K of a product: rounding one up to a tile stays in 32 bits.
constexpr int kMaxExtent = INT32_MAX - 255;

__host__ __device__ __forceinline__ int blocks_of(int n) { return (n + kBlk - 1) / kBlk; }

// ---------------------------------------------------------------- quantise
// A warp takes four blocks of a row, eight lanes per block and 16 columns per
// lane: with aligned rows (VEC) two 16-byte loads and one 16-byte store.
constexpr int kQuantCols = 4 * kBlk;

template <bool VEC>
__global__ void __launch_bounds__(256, VEC ? 8 : 5)
    blockscale_quantize_kernel(const __nv_bfloat16* x, int64_t ldx, int x_rows,
                               const int32_t* slots, int top_k, int rows, int cols,
                               uint8_t* __restrict__ codes, int64_t ld_codes,
                               float* __restrict__ scales, int64_t ld_scales) {
  // What came before is over when a product that follows may set itself up and
  // load weights meanwhile.
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int r = static_cast<int>(row), lane = threadIdx.x & 31;
  const int c0 = blockIdx.y * kQuantCols + lane * 16, b = c0 / kBlk;
  const bool real = c0 < cols;
  const int slot = slots ? slots[r] : r, src = slots ? slot / top_k : r;
  const bool in = real && slot >= 0 && src < x_rows;
  const __nv_bfloat16* p = x + src * ldx + c0;
  uint32_t values[1][8];  // pairs of bf16
  uint32_t(&v)[8] = values[0];
  if (VEC && in && c0 + 16 <= cols) {
    const uint4 lo = *reinterpret_cast<const uint4*>(p), hi = *reinterpret_cast<const uint4*>(p + 8);
    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
    v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t lo = 0u, hi = 0u;
      if (in && c0 + 2 * i < cols) lo = reinterpret_cast<const uint16_t*>(p)[2 * i];
      if (in && c0 + 2 * i + 1 < cols) hi = reinterpret_cast<const uint16_t*>(p)[2 * i + 1];
      v[i] = lo | (hi << 16);
    }
  }
  float scale[1];
  uint4 w4[1];
  quantize_16(values, w4, scale);
  const bool first = (lane & 7) == 0 && b * kBlk < cols;
  if (first) scales[b * ld_scales + r] = scale[0];
  if (!real) return;
  const uint32_t w[4] = {w4[0].x, w4[0].y, w4[0].z, w4[0].w};
  uint8_t* d = codes + r * ld_codes + c0;
  if (VEC && c0 + 16 <= cols) {
    *reinterpret_cast<uint4*>(d) = w4[0];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c0 + i < cols) d[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
}

// Rows of quantised activations by slot: codes in 16-byte words (row strides
// of `words`), scales block by block.  A warp copies up to kCopyWords words of
// one row, its lanes next to each other; a slot outside the activations gives
// zeros.  Bound by the writes.
constexpr int kCopyWords = 128;

__global__ void __launch_bounds__(256)
    blockscale_copy_rows_kernel(const uint4* codes, const float* scales, int x_rows, int blocks,
                                int words, const int32_t* slots, int top_k, int rows, uint4* out,
                                float* out_scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int lane = threadIdx.x & 31, slot = slots[row], src = slot / top_k;
  const bool in = slot >= 0 && src < x_rows;
  const uint4* s = codes + static_cast<int64_t>(in ? src : 0) * words;
  uint4* d = out + row * words;
  const int w0 = blockIdx.y * kCopyWords + lane;
  uint4 v[kCopyWords / 32];
#pragma unroll
  for (int i = 0; i < kCopyWords / 32; ++i)
    v[i] = in && w0 + 32 * i < words ? s[w0 + 32 * i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < kCopyWords / 32; ++i)
    if (w0 + 32 * i < words) d[w0 + 32 * i] = v[i];
  // the words' blocks' scales (8 words to a block)
  const int b = blockIdx.y * (kCopyWords / 8) + lane;
  if (lane < kCopyWords / 8 && b < blocks)
    out_scales[static_cast<int64_t>(b) * rows + row] =
        in ? scales[static_cast<int64_t>(b) * x_rows + src] : 0.0f;
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---------------------------------------------------------------- arguments
struct Product {
  const void* a;
  int64_t lda;
  const float* a_scales;
  int64_t ld_as;
  const void* w;
  int64_t ldw;
  const float* w_scales;
  const int32_t* offsets;
  int E, M, N, K;
  bool transpose;
  const void* x = nullptr;  // bf16 activations that the product quantises (no codes in `a`)
  int64_t ldx = 0;
};

// TMA wants 16-byte aligned bases and row strides; scales and offsets are
// read as 32-bit words.
moe_status check_weights(const Product& p) {
  if (p.M < 0 || p.N < 1 || p.K < 1 || p.E < 1 || (!p.offsets && p.E != 1))
    return MOE_ERR_INVALID_ARG;
  if (p.E > kMaxExperts || p.M > kMaxExtent || p.N > kMaxExtent || p.K > kMaxExtent)
    return MOE_ERR_UNSUPPORTED;
  if (p.ldw < (p.transpose ? p.N : p.K)) return MOE_ERR_INVALID_ARG;
  if (p.M == 0) return MOE_OK;
  if (!p.w || !p.w_scales || !aligned_to(p.w, 16) || p.ldw % 16 || !aligned_to(p.w_scales, 4) ||
      !aligned_to(p.offsets, 4))
    return MOE_ERR_INVALID_ARG;
  // strides of the tensor maps and the item count stay in range
  const int64_t rows = p.transpose ? p.K : p.N;
  if (p.ldw >= (int64_t{1} << 39) / rows ||
      (static_cast<int64_t>(p.E) + p.M / kBlk + 1) * blocks_of(p.N) > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_product(const Product& p) {
  if (p.lda < p.K || p.ld_as < p.M) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_weights(p);
  if (st != MOE_OK || p.M == 0) return st;
  if (!p.a || !p.a_scales || !aligned_to(p.a, 16) || p.lda % 16 || !aligned_to(p.a_scales, 4))
    return MOE_ERR_INVALID_ARG;
  return p.lda >= (int64_t{1} << 39) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t one[3] = {1, 1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base),
                              dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The current device, null unless it is an sm_103 one.  What was found out about
// a device is kept; a look-up that failed is tried again.
const BlockscaleDevice* current_device() {
  constexpr int kMaxDevices = 64;
  struct Entry {
    std::atomic<bool> known{false};
    BlockscaleDevice d{};
  };
  static Entry entries[kMaxDevices];
  static std::mutex looking_up;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return nullptr;
  }
  Entry& e = entries[dev];
  if (e.known.load(std::memory_order_acquire)) return &e.d;
  std::lock_guard<std::mutex> lock(looking_up);
  if (!e.known.load(std::memory_order_relaxed)) {
    int major = 0, minor = 0;
    const bool usable =
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&e.d.sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
        major == 10 && minor == 3 && tensor_map_encoder() && blockscale_clusters(&e.d) == cudaSuccess;
    if (!usable) {
      cudaGetLastError();
      return nullptr;
    }
    e.known.store(true, std::memory_order_release);
  }
  return &e.d;
}

// early: the product follows the library's own kernel on the stream and may
// start while it runs (programmatic dependent launch).
moe_status run_product(const Product& p, bool swiglu, void* out, int64_t ldo, float clamp,
                       float* h_scales, int64_t ld_hs, bool early, cudaStream_t s) {
  const BlockscaleDevice* d = current_device();
  if (!d) return MOE_ERR_NO_DEVICE;
  BlockscaleMaps maps;
  // (one expert: all chunks take the largest box)
  const int boxes = p.M <= 16 ? 1 : p.M <= 32 ? 2 : p.M <= 64 ? 3 : 4;
  const cuuint64_t adims[2] = {static_cast<cuuint64_t>(p.K), static_cast<cuuint64_t>(p.M)};
  const cuuint64_t astr[1] = {static_cast<cuuint64_t>(p.lda)};
  for (int i = p.E == 1 ? boxes - 1 : 0; i < boxes && !p.x; ++i) {
    const cuuint32_t box[2] = {128, 16u << i};
    if (!encode(&maps.a[i], p.a, 2, adims, astr, box)) return MOE_ERR_CUDA;
  }
  const int wrows = p.transpose ? p.K : p.N, wcols = p.transpose ? p.N : p.K;
  const cuuint64_t wdims[3] = {static_cast<cuuint64_t>(wcols), static_cast<cuuint64_t>(wrows),
                               static_cast<cuuint64_t>(p.E)};
  const cuuint64_t wstr[2] = {static_cast<cuuint64_t>(p.ldw),
                              static_cast<cuuint64_t>(p.ldw) * wrows};
  const cuuint32_t wbox[3] = {128, swiglu ? 64u : 128u, 1};
  if (!encode(&maps.w, p.w, 3, wdims, wstr, wbox)) return MOE_ERR_CUDA;
  BlockscaleArgs a{};
  a.a_scales = p.a_scales;
  a.ld_as = p.ld_as;
  a.w_scales = p.w_scales;
  a.w_blocks = static_cast<int64_t>(blocks_of(p.N)) * blocks_of(p.K);
  a.w_stride_n = p.transpose ? 1 : blocks_of(p.K);
  a.w_stride_k = p.transpose ? blocks_of(p.N) : 1;
  a.offsets = p.offsets;
  a.E = p.E;
  a.M = p.M;
  a.N = p.N;
  a.K = p.K;
  a.out = out;
  a.ldo = ldo;
  a.out_vec = aligned_to(out, 32) && ldo % 16 == 0;
  a.clamp = clamp > 0.0f && std::isfinite(clamp) ? clamp : INFINITY;
  a.h_scales = h_scales;
  a.ld_hs = ld_hs;
  a.x = static_cast<const __nv_bfloat16*>(p.x);
  a.ldx = p.ldx;
  a.x_vec = aligned_to(p.x, 16) && p.ldx % 8 == 0;
  a.early = early;
  return take_error(launch_blockscale(maps, a, swiglu, p.transpose, *d, s)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status run_quantize(const void* x, int64_t ldx, int x_rows, const int32_t* slots, int top_k,
                        int rows, int cols, void* codes, int64_t ld_codes, float* scales,
                        int64_t ld_scales, cudaStream_t s) {
  if (rows < 0 || cols < 1 || x_rows < 0 || ldx < cols || ld_codes < cols || ld_scales < rows)
    return MOE_ERR_INVALID_ARG;
  if (slots ? top_k < 1 : x_rows < rows) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if ((!x && x_rows > 0) || !codes || !scales || !aligned_to(x, 2) || !aligned_to(slots, 4) ||
      !aligned_to(scales, 4))
    return MOE_ERR_INVALID_ARG;
  const dim3 grid((static_cast<unsigned>(rows) + 7) / 8, (cols - 1) / kQuantCols + 1);
  if (grid.y > 65535) return MOE_ERR_UNSUPPORTED;
  const bool vec = aligned_to(x, 16) && ldx % 8 == 0 && aligned_to(codes, 16) && ld_codes % 16 == 0;
  const cudaError_t e = launch_pdl(
      true, vec ? blockscale_quantize_kernel<true> : blockscale_quantize_kernel<false>,
      grid, dim3(256), 0, s, static_cast<const __nv_bfloat16*>(x),
      ldx, x_rows, slots, top_k, rows, cols, static_cast<uint8_t*>(codes), ld_codes, scales,
      ld_scales);
  return take_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Quantised activations in a workspace: codes in rows of a multiple of 16
// bytes, then the scales.
int64_t padded(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
int64_t quantized_bytes(int64_t rows, int64_t cols) {
  return padded(rows * padded(cols, 16), 256) + padded(rows * ((cols + 127) / 128) * 4, 256);
}
struct Quantized {
  uint8_t* codes;
  int64_t ld;
  float* scales;
  int64_t ld_scales;
  Quantized(void* ws, int64_t rows, int64_t cols)
      : codes(static_cast<uint8_t*>(ws)), ld(padded(cols, 16)),
        scales(reinterpret_cast<float*>(codes + padded(rows * ld, 256))), ld_scales(rows) {}
};

// Whether moe_blockscale_experts quantises the tokens and copies their codes
// to the rows, instead of quantising the rows: for several rows per token and
// enough of them.  A whole call, copied against quantised: 8192 tokens of 8
// rows x 7168 2.59 ms against 2.65, 4096 of 8 x 2048 289 us against 299, 1024
// of 8 x 2048 128 against 130, fewer the same, and it is a launch more on the
// host.  The tokens' codes are kept where h will be, so they have to fit there.
constexpr int64_t kCopyMinBytes = int64_t{1} << 24;
bool copies_rows(int T, int rows, int H, int I) {
  return T > 0 && rows >= 2 * static_cast<int64_t>(T) &&
         static_cast<int64_t>(rows) * H >= kCopyMinBytes &&
         quantized_bytes(T, H) <= quantized_bytes(rows, I);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_blockscale_quantize(const void* x, int64_t ldx, int x_rows, const int32_t* slots,
                                   int top_k, int rows, int cols, void* codes, int64_t ld_codes,
                                   float* scales, int64_t ld_scales, void* stream) {
  return run_quantize(x, ldx, x_rows, slots, top_k, rows, cols, codes, ld_codes, scales, ld_scales,
                      static_cast<cudaStream_t>(stream));
}

moe_status moe_blockscale_matmul(const void* a, int64_t lda, const float* a_scales, int64_t ld_as,
                                 const void* w, int64_t ldw, const float* w_scales,
                                 const int32_t* offsets, int E, int M, int N, int K,
                                 int transpose_w, void* out, int64_t ldo, void* stream) {
  const Product p{a, lda, a_scales, ld_as, w, ldw, w_scales, offsets, E, M, N, K, transpose_w != 0};
  const moe_status st = check_product(p);
  if (st != MOE_OK) return st;
  if (ldo < N) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!out || !aligned_to(out, 2)) return MOE_ERR_INVALID_ARG;
  return run_product(p, false, out, ldo, 0.0f, nullptr, 0, false,
                     static_cast<cudaStream_t>(stream));
}

moe_status moe_blockscale_swiglu(const void* a, int64_t lda, const float* a_scales, int64_t ld_as,
                                 const void* w13, int64_t ldw, const float* w13_scales,
                                 const int32_t* offsets, int E, int M, int I, int K,
                                 float clamp_limit, void* h, int64_t ldh, float* h_scales,
                                 int64_t ld_hs, void* stream) {
  if (I < 1 || I > (1 << 29)) return MOE_ERR_INVALID_ARG;
  if (I % kBlk) return MOE_ERR_UNSUPPORTED;
  const Product p{a, lda, a_scales, ld_as, w13, ldw, w13_scales, offsets, E, M, 2 * I, K, false};
  const moe_status st = check_product(p);
  if (st != MOE_OK) return st;
  if (ldh < I || ld_hs < M) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!h || !h_scales || !aligned_to(h_scales, 4) || !aligned_to(h, 16) || ldh % 16)
    return MOE_ERR_INVALID_ARG;
  return run_product(p, true, h, ldh, clamp_limit, h_scales, ld_hs, false,
                     static_cast<cudaStream_t>(stream));
}

size_t moe_blockscale_linear_workspace(int M, int N, int K) {
  if (M < 1 || N < 1 || K < 1 || M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return 0;
  const BlockscaleDevice* d = current_device();
  return d && blockscale_quantizes(M, N, K, *d) ? 0 : static_cast<size_t>(quantized_bytes(M, K));
}

size_t moe_blockscale_experts_workspace(int rows, int H, int I) {
  if (rows < 1 || H < 1 || I < 1 || rows > kMaxExtent || H > kMaxExtent || I > kMaxExtent) return 0;
  return static_cast<size_t>(quantized_bytes(rows, H) + quantized_bytes(rows, I));
}

moe_status moe_blockscale_linear(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                 const float* w_scales, int M, int N, int K, int transpose_w,
                                 void* out, int64_t ldo, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  Product p{nullptr, 0, nullptr, 0, w, ldw, w_scales, nullptr, 1, M, N, K, transpose_w != 0};
  const moe_status st = check_weights(p);
  if (st != MOE_OK) return st;
  if (ldx < K || ldo < N) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const size_t need = moe_blockscale_linear_workspace(M, N, K);
  if (!x || !out || !aligned_to(x, 2) || !aligned_to(out, 2) || workspace_bytes < need ||
      (need && (!workspace || !aligned_to(workspace, 16))))
    return MOE_ERR_INVALID_ARG;
  if (!current_device()) return MOE_ERR_NO_DEVICE;
  if (!need) {
    p.x = x;
    p.ldx = ldx;
    return run_product(p, false, out, ldo, 0.0f, nullptr, 0, false,
                       static_cast<cudaStream_t>(stream));
  }
  const Quantized q(workspace, M, K);
  p.a = q.codes;
  p.lda = q.ld;
  p.a_scales = q.scales;
  p.ld_as = q.ld_scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const moe_status sq =
      run_quantize(x, ldx, M, nullptr, 1, M, K, q.codes, q.ld, q.scales, q.ld_scales, s);
  if (sq != MOE_OK) return sq;
  return run_product(p, false, out, ldo, 0.0f, nullptr, 0, true, s);
}

moe_status moe_blockscale_experts(const void* x, int64_t ldx, int T, const int32_t* slots,
                                  int top_k, int rows, const int32_t* offsets, int E,
                                  const void* w13, const float* w13_scales, const void* w2,
                                  const float* w2_scales, int H, int I, float clamp_limit,
                                  void* out, int64_t ldo, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (I < 1 || I > (1 << 29) || T < 0 || top_k < 1 || !offsets) return MOE_ERR_INVALID_ARG;
  if (I % kBlk || H % 16) return MOE_ERR_UNSUPPORTED;
  Product p1{nullptr, 0, nullptr, 0, w13, H, w13_scales, offsets, E, rows, 2 * I, H, false};
  Product p2{nullptr, 0, nullptr, 0, w2, I, w2_scales, offsets, E, rows, H, I, false};
  moe_status st = check_weights(p1);
  if (st == MOE_OK) st = check_weights(p2);
  if (st != MOE_OK) return st;
  if (ldx < H || ldo < H) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if ((!x && T > 0) || !slots || !out || !workspace || !aligned_to(x, 2) || !aligned_to(slots, 4) ||
      !aligned_to(out, 2) || !aligned_to(workspace, 16) ||
      workspace_bytes < moe_blockscale_experts_workspace(rows, H, I))
    return MOE_ERR_INVALID_ARG;
  if (!current_device()) return MOE_ERR_NO_DEVICE;
  const Quantized q(workspace, rows, H);
  uint8_t* rest = static_cast<uint8_t*>(workspace) + quantized_bytes(rows, H);
  const Quantized h(rest, rows, I);
  p1.a = q.codes, p1.lda = q.ld, p1.a_scales = q.scales, p1.ld_as = q.ld_scales;
  p2.a = h.codes, p2.lda = h.ld, p2.a_scales = h.scales, p2.ld_as = h.ld_scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (copies_rows(T, rows, H, I)) {
    // (the tokens' codes lie where h will be)
    const Quantized t(rest, T, H);
    st = run_quantize(x, ldx, T, nullptr, 1, T, H, t.codes, t.ld, t.scales, t.ld_scales, s);
    const int words = static_cast<int>(t.ld / 16);
    const dim3 grid((static_cast<unsigned>(rows) + 7) / 8, (words + kCopyWords - 1) / kCopyWords);
    if (st == MOE_OK &&
        take_error(launch_pdl(true, blockscale_copy_rows_kernel, grid, dim3(256), 0, s,
                              reinterpret_cast<const uint4*>(t.codes), t.scales, T, blocks_of(H),
                              words, slots, top_k, rows, reinterpret_cast<uint4*>(q.codes),
                              q.scales)) != cudaSuccess)
      st = MOE_ERR_CUDA;
  } else {
    st = run_quantize(x, ldx, T, slots, top_k, rows, H, q.codes, q.ld, q.scales, q.ld_scales, s);
  }
  if (st == MOE_OK)
    st = run_product(p1, true, h.codes, h.ld, clamp_limit, h.scales, h.ld_scales, true, s);
  if (st == MOE_OK) st = run_product(p2, false, out, ldo, 0.0f, nullptr, 0, true, s);
  return st;
}

moe_status moe_blockscale_status(void) {
  int v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess || blockscale_status(&v) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return v ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

}  // extern "C"
