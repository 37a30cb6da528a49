// int8_rows.cu -- 8-bit integer products of a few rows: y[m][n] = sx[m] sw[n]
// sum_k cx[m][k] cw[n][k] for up to four m, or up to 24 rows of as many experts or
// more.
//
// Such a product is as fast as its weights come out of HBM, and a row's dot products
// of four codes (dp4a, int32 sums: exact) keep up with that without the tensor
// cores' staging.  A warp takes four channels and a slice of the reduction, 16 codes
// a lane and channel at a time; it has its first loads under way before anything
// else: one or two rows are quantised by every block for itself meanwhile (QUANT),
// more by a kernel that this one overlaps.  On the GPU, 7168 -> 4096: one row 7.0
// us, two 9.7, three 9.4, four 10.0; five, through the tensor cores, 11.1.  4096 ->
// 14592 (60 MB, 8.8 us of HBM): one row 8.7, two 10.9, three 12.6, four 13.5 (the dot
// products take the time by then); five 14.3.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "expert_table.cuh"
#include "int8_quant.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsChannels = 4;  // of a warp
constexpr int kRowsAhead = 2;     // blocks of 512 codes that are loaded together
constexpr int kRowsSms = 152, kRowsResident = 3;  // blocks of an SM at a time
constexpr int kRowsOwn = 32768;   // codes that a block quantises for itself, at most
constexpr unsigned kAllLanes = 0xFFFFFFFFu;

// Sixteen codes from column k on; past K: zeros.
__device__ __forceinline__ uint4 load16(const int8_t* row, int k, int K, bool aligned) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (aligned && k + 16 <= K) {
    v = *reinterpret_cast<const uint4*>(row + k);
  } else if (k < K) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k + i < K) w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + i])) << (8 * (i & 3));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int acc) {
  acc = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), acc);
  acc = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), acc);
  acc = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), acc);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), acc);
}

// M: rows (some may be past p.M).  QUANT: p.x in bf16, else codes p.a and scales.
// p.slices warps of a block share four channels' reduction.
template <int M, bool QUANT>
__global__ void __launch_bounds__(kRowsThreads, kRowsResident)
    int8_rows_kernel(const __grid_constant__ Int8RowsArgs p) {
  extern __shared__ uint8_t s_codes[];  // QUANT: [M][K rounded up to 16]
  __shared__ uint32_t s_max[8][M];
  __shared__ int s_sum[2][8][kRowsChannels * M];  // by turns
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = warp % p.slices, group = warp / p.slices, groups = 8 / p.slices;
  // this block's units (groups * kRowsChannels channels), and the warp's channels
  const int units = (p.N + groups * kRowsChannels - 1) / (groups * kRowsChannels);
  int unit = blockIdx.x, n0 = (unit * groups + group) * kRowsChannels;
  const int step = p.slices * 512;
  uint4 w[kRowsAhead][kRowsChannels];
  auto load_w = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i)
#pragma unroll
      for (int c = 0; c < kRowsChannels; ++c) {
        const int k = k0 + i * step;
        w[i][c] = n0 + c < p.N ? load16(p.w + static_cast<int64_t>(n0 + c) * p.ldw, k, p.K, true)
                               : make_uint4(0u, 0u, 0u, 0u);
      }
  };
  int k0 = (slice * 32 + lane) * 16;
  if (!QUANT) pdl_launch_dependents();
  load_w(k0);
  const int ld = (p.K + 15) / 16 * 16;
  float scale[QUANT ? M : 1];
  if constexpr (QUANT) {
    const int vectors = (p.K + 7) / 8;
    auto load_x = [&](int m, int v, float (&f)[8]) {
      const uint16_t* src =
          reinterpret_cast<const uint16_t*>(p.x) + static_cast<int64_t>(m) * p.ldx + v * 8;
      if (p.x_vec && v * 8 + 8 <= p.K) {
        const uint4 q = *reinterpret_cast<const uint4*>(src);
        const uint32_t b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = __uint_as_float(b[i] << 16);
          f[2 * i + 1] = __uint_as_float(b[i] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          f[i] = v * 8 + i < p.K ? __uint_as_float(static_cast<uint32_t>(src[i]) << 16) : 0.0f;
      }
    };
    uint32_t most[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      most[m] = 0u;
      if (m < p.M)
        for (int v = threadIdx.x; v < vectors; v += kRowsThreads) {
          float f[8];
          load_x(m, v, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) most[m] = max(most[m], __float_as_uint(f[i]) & 0x7FFFFFFFu);
        }
      most[m] = __reduce_max_sync(kAllLanes, most[m]);
      if (lane == 0) s_max[warp][m] = most[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int i = 0; i < 8; ++i) most[m] = max(most[m], s_max[i][m]);
      scale[m] = i8_scale(most[m]);
      const I8Coder coder(scale[m]);
      for (int v = threadIdx.x; v * 8 < ld; v += kRowsThreads) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (m < p.M && v < vectors) load_x(m, v, f);
        *reinterpret_cast<uint2*>(s_codes + m * ld + v * 8) = coder.bytes(f);
      }
    }
    __syncthreads();
  } else {
    pdl_wait();
  }
  for (int turn = 0;; turn ^= 1) {
    int acc[kRowsChannels][M];
#pragma unroll
    for (int c = 0; c < kRowsChannels; ++c)
#pragma unroll
      for (int m = 0; m < M; ++m) acc[c][m] = 0;
    for (;;) {
#pragma unroll
      for (int i = 0; i < kRowsAhead; ++i) {
        const int k = k0 + i * step;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if constexpr (QUANT) {
            if (k < p.K) x = *reinterpret_cast<const uint4*>(s_codes + m * ld + k);
          } else if (m < p.M) {
            x = load16(p.a + static_cast<int64_t>(m) * p.lda, k, p.K, p.a_vec != 0);
          }
#pragma unroll
          for (int c = 0; c < kRowsChannels; ++c) acc[c][m] = dot16(w[i][c], x, acc[c][m]);
        }
      }
      k0 += kRowsAhead * step;
      if (k0 - (slice * 32 + lane) * 16 >= p.K) break;  // (the same for all lanes)
      load_w(k0);
    }
    // the next unit's weights are on their way while this one's sums are joined
    const int done = unit;
    unit += gridDim.x;
    k0 = (slice * 32 + lane) * 16;
    if (unit < units) {
      n0 = (unit * groups + group) * kRowsChannels;
      load_w(k0);
    }
#pragma unroll
    for (int c = 0; c < kRowsChannels; ++c)
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int sum = __reduce_add_sync(kAllLanes, acc[c][m]);
        if (lane == 0) s_sum[turn][warp][c * M + m] = sum;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < groups * kRowsChannels * M; i += kRowsThreads) {
      const int g = i / (kRowsChannels * M), c = i / M % kRowsChannels, m = i % M;
      const int n = (done * groups + g) * kRowsChannels + c;
      if (n >= p.N || m >= p.M) continue;
      int sum = 0;
      for (int s = 0; s < p.slices; ++s) sum += s_sum[turn][g * p.slices + s][c * M + m];
      float sx;
      if constexpr (QUANT) {
        sx = scale[0];
#pragma unroll
        for (int q = 1; q < M; ++q) sx = m == q ? scale[q] : sx;
      } else {
        sx = p.a_scales[m];
      }
      p.out[m * p.ldo + n] = __float2bfloat16_rn(static_cast<float>(sum) * (sx * p.w_scales[n]));
    }
    if (unit >= units) break;
  }
}

// The rows of several experts, no more than there are experts: items of up to four
// rows of an expert, its weights read once for each.  A unit is an item's rows and a
// block's channels; with SWIGLU a warp's four are two gates and the ups that go with
// them.  Small units keep all SMs at work to the end, where tiles of 256 channels are
// one round and a part of them.
constexpr int kGroupRows = 24;  // rows in all, at most
constexpr int kItemRows = 4;

template <bool SWIGLU>
__global__ void __launch_bounds__(kRowsThreads, kRowsResident)
    int8_group_rows_kernel(const __grid_constant__ Int8RowsArgs p) {
  constexpr int kOut = SWIGLU ? kRowsChannels / 2 : kRowsChannels;  // results of a warp and row
  __shared__ int s_tab[3 * kMaxExperts + 1];
  __shared__ int s_expert[kGroupRows], s_row[kGroupRows], s_rows[kGroupRows];
  __shared__ int s_sum[2][8][kRowsChannels * kItemRows];  // by turns
  const ExpertTable tab{s_tab, s_tab + p.E + 1, s_tab + 2 * p.E + 1};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = warp % p.slices, group = warp / p.slices, groups = 8 / p.slices;
  const int width = SWIGLU ? p.N / 2 : p.N;  // results of a row
  const int tiles = (width - 1) / (groups * kOut) + 1;
  pdl_launch_dependents();
  // (offsets and weights are not the kernel's before this one)
  if (warp == 0) {
    fill_expert_table(p, tab, kItemRows, lane);
    __syncwarp();
    for (int e = lane; e < p.E; e += 32)
      for (int i = tab.chunk_off[e]; i < tab.chunk_off[e + 1]; ++i) {
        const int row = tab.start[e] + (i - tab.chunk_off[e]) * kItemRows;
        s_expert[i] = e;
        s_row[i] = row;
        s_rows[i] = min(kItemRows, tab.end[e] - row);
      }
  }
  __syncthreads();
  const int units = tab.chunk_off[p.E] * tiles;
  int unit = blockIdx.x;
  if (unit >= units) {
    // (no row may have an expert, and no block a unit: this kernel is not over before the
    // one that it overlaps, whose end the kernels after it rely on)
    pdl_wait();
    return;
  }
  const int step = p.slices * 512, k_first = (slice * 32 + lane) * 16;
  uint4 w[kRowsAhead][kRowsChannels];
  int k0 = k_first;
  auto load_w = [&]() {
    const int item = unit / tiles, n0 = ((unit - item * tiles) * groups + group) * kOut;
    const int8_t* base = p.w + static_cast<int64_t>(s_expert[item]) * p.N * p.ldw;
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i)
#pragma unroll
      for (int c = 0; c < kRowsChannels; ++c) {
        const int n = n0 + c % kOut;
        const int8_t* row = base + static_cast<int64_t>(n + c / kOut * width) * p.ldw;
        w[i][c] = n < width ? load16(row, k0 + i * step, p.K, true) : make_uint4(0u, 0u, 0u, 0u);
      }
  };
  load_w();
  pdl_wait();
  int turn = 0;
  // a unit of up to M rows; the next one's first weights are on their way before its
  // sums are joined
  auto run = [&](auto rows_of_item) {
    constexpr int M = decltype(rows_of_item)::value;
    const int item = unit / tiles, tile = unit - item * tiles;
    const int row0 = s_row[item], rows = s_rows[item], e = s_expert[item];
    const int8_t* a = p.a + row0 * p.lda;
    int acc[kRowsChannels][M];
#pragma unroll
    for (int c = 0; c < kRowsChannels; ++c)
#pragma unroll
      for (int m = 0; m < M; ++m) acc[c][m] = 0;
    for (;;) {
#pragma unroll
      for (int i = 0; i < kRowsAhead; ++i)
#pragma unroll
        for (int m = 0; m < M; ++m) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (m < rows) x = load16(a + m * p.lda, k0 + i * step, p.K, p.a_vec != 0);
#pragma unroll
          for (int c = 0; c < kRowsChannels; ++c) acc[c][m] = dot16(w[i][c], x, acc[c][m]);
        }
      k0 += kRowsAhead * step;
      if (k0 - k_first >= p.K) break;  // (the same for all lanes)
      load_w();
    }
    unit += gridDim.x;
    k0 = k_first;
    if (unit < units) load_w();
#pragma unroll
    for (int c = 0; c < kRowsChannels; ++c)
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int sum = __reduce_add_sync(kAllLanes, acc[c][m]);
        if (lane == 0) s_sum[turn][warp][c * M + m] = sum;
      }
    __syncthreads();
    const float* sw = p.w_scales + static_cast<int64_t>(e) * p.N;
    for (int i = threadIdx.x; i < groups * kOut * M; i += kRowsThreads) {
      const int g = i / (kOut * M), c = i / M % kOut, m = i % M;
      const int n = (tile * groups + g) * kOut + c;
      if (n >= width || m >= rows) continue;
      auto value = [&](int channel, int row_of_w) {
        int sum = 0;
        for (int s = 0; s < p.slices; ++s) sum += s_sum[turn][g * p.slices + s][channel * M + m];
        return static_cast<float>(sum) * (p.a_scales[row0 + m] * sw[row_of_w]);
      };
      const int64_t at = (row0 + m) * p.ldo + n;
      if constexpr (SWIGLU)
        p.h[at] = swiglu(value(c, n), value(c + kOut, n + width), p.clamp);
      else
        p.out[at] = __float2bfloat16_rn(value(c, n));
    }
    turn ^= 1;
  };
  while (unit < units) {
    const int rows = s_rows[unit / tiles];  // (the same for all threads)
    if (rows == 1)
      run(std::integral_constant<int, 1>{});
    else if (rows == 2)
      run(std::integral_constant<int, 2>{});
    else
      run(std::integral_constant<int, kItemRows>{});
  }
}

// Warps to a reduction: as many as leave each the blocks that it loads at once.
int slices_of(int K) {
  const int blocks = (K + 511) / 512;
  int slices = 1;
  while (slices < 8 && slices * kRowsAhead < blocks) slices *= 2;
  return slices;
}

template <int M, bool QUANT>
cudaError_t launch(const Int8RowsArgs& p, bool early, cudaStream_t s) {
  const int groups = 8 / p.slices;
  const int units = (p.N - 1) / (groups * kRowsChannels) + 1;
  const int blocks = std::min(units, kRowsResident * kRowsSms);
  const int smem = QUANT ? M * ((p.K + 15) / 16 * 16) : 0;
  static OncePerDevice prepared;
  if (QUANT) {
    const cudaError_t e = prepared([&] {
      return cudaFuncSetAttribute(int8_rows_kernel<M, QUANT>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsOwn + 64);
    });
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(early, int8_rows_kernel<M, QUANT>, dim3(blocks),
                    dim3(kRowsThreads), smem, s, p);
}

}  // namespace

// See internal.h.  Int32 sums hold K products of 128 x 128 below 2^17 of them.
bool int8_by_rows(int M, int K, int E) { return E == 1 && M <= 4 && K < 131072; }
// The experts' products on the GPU, here and on the tensor cores.  64 x (2048, 1024),
// top-6: one token 13.0 and 27.1 us, four 43.7 and 53.3, five 55.6 and 53.8.  64 x
// (7168, 2048), top-8: one token 65.4 and 79.8, two 116.7 and 127.2, three 166 and
// 179, four 225 and 192.  More rows than experts: 8 x (4096, 14336), top-2: 16 rows
// 280 and 219, where 8 rows take 176 and 176.  (Units stay in 32 bits.)
bool int8_by_group_rows(int M, int N, int K, int E) {
  return E > 1 && M <= std::min(E, kGroupRows) && K < 131072 && M * static_cast<int64_t>(N) <= INT32_MAX;
}
bool int8_rows_quantize(int M, int K, int E) {
  return int8_by_rows(M, K, E) && M <= 2 && M * static_cast<int64_t>(K) <= kRowsOwn;
}

cudaError_t launch_int8_rows(Int8RowsArgs p, bool early, cudaStream_t s) {
  p.slices = slices_of(p.K);
  if (p.x) return p.M == 1 ? launch<1, true>(p, false, s) : launch<2, true>(p, false, s);
  if (p.M == 1) return launch<1, false>(p, early, s);
  if (p.M == 2) return launch<2, false>(p, early, s);
  return launch<4, false>(p, early, s);
}

cudaError_t launch_int8_group_rows(Int8RowsArgs p, bool swiglu, bool early, cudaStream_t s) {
  // (two warps to a reduction at most: with more the blocks wait for their slowest warp
  // more often.  64 x (7168, 2048), top-8, two tokens: eight 127.5 us, four 123.0, two
  // 116.7, one 115.9; 8 x (4096, 14336), top-2, four: 179, 181, 176 and 208)
  p.slices = std::min(slices_of(p.K), 2);
  const int groups = 8 / p.slices, width = swiglu ? p.N / 2 : p.N;
  const int64_t tiles = (width - 1) / (groups * (swiglu ? 2 : kRowsChannels)) + 1;
  // (an expert has an item for each of its rows at most)
  const int blocks = static_cast<int>(std::min<int64_t>(p.M * tiles, kRowsResident * kRowsSms));
  return swiglu ? launch_pdl(early, int8_group_rows_kernel<true>, dim3(blocks), dim3(kRowsThreads), 0, s, p)
                : launch_pdl(early, int8_group_rows_kernel<false>, dim3(blocks), dim3(kRowsThreads), 0, s, p);
}

}  // namespace moe
