// int8_gemm.cu -- products of 8-bit integer matrices with a scale per token and a
// scale per output channel, on the sm_103a tensor cores.
//
//   y[m][n] = sx[m] sw[n] sum_k cx[m][k] cw[n][k]
//
// sm_103a's tensor cores have no fast integer kind, but an 8-bit code is exact in
// f16 and so is the product of two in the fp32 accumulator (|sum| <= 2^24, that
// is 1024 products of largest codes, is exact; a longer sum rounds as fp32 sums
// do).  So the codes run as kind::f16, and the weights stay 8 bits wide in HBM,
// in L2 and in shared memory: they are the A operand, which the tensor cores can
// read from TMEM, and are widened on the way from shared memory into it.  A code
// c becomes the f16 with the bits 0x6400 + (c + 128), which is 1152 + c, and a
// subtraction takes the 1152 away: five instructions for four codes.  The tokens
// are the B operand, as f16 codes in shared memory.
//
// So D[channel][token]: a tile is 256 channels (two halves of 128 TMEM lanes) by
// up to 128 tokens.  Structure: one persistent CTA per SM walks the items (expert,
// tile, chunk of at most 128 rows).  Warps 0 and 3 (a thread each) fill two rings of
// stages by TMA, of 128 columns of the reduction: 8-bit weights (32 KB), and f16
// codes of the chunk's rows (box height 16 / 32 / 64 / 128).  Warps 4-11 widen: warp
// w takes the TMEM lanes 32 (w % 4).. of half (w - 4) / 4 and writes its rows' f16
// into one of two TMEM buffers; a stage of weights is free then, before its MMAs (in
// one ring with the tokens: 64 experts of 2048 x 1024, 6144 rows, 144 us for 130).  Warp
// 1 issues the MMAs.  The widening warps also read
// the results out: after the first two blocks of the next item have been widened,
// so the tensor cores go on as soon as the results are in registers, and the
// scaling and the stores run beside them.
//
// Few rows leave most SMs without an item; there a cluster of two to eight CTAs
// splits the reduction of each item and joins its fp32 partial sums through
// distributed shared memory, in rank order, so the result does not depend on
// timing.
//
// With SWIGLU the halves are 128 gate channels and the 128 up channels that go
// with them; h = silu(gate) up is stored in fp32, for a row's scale is known only
// when all of its tiles are.
#include <cuda_bf16.h>

#include <algorithm>

#include "expert_table.cuh"
#include "int8_quant.cuh"
#include "internal.h"
#include "ptx_pipeline.cuh"

namespace moe {

namespace {

constexpr int kI8Threads = 384;
constexpr int kI8WideWarp0 = 4;     // warps 4-11 widen the weights and read the results
constexpr int kI8WideWarps = 8;
constexpr int kI8Tile = 256;        // channels of an item
constexpr int kI8MaxStages = 6;   // of weights, and of tokens
constexpr int kI8WBytes = kI8Tile * 128;
constexpr int kI8SmemLimit = 232448;
constexpr int kI8Buffers = 2;       // TMEM buffers of widened weights, 128 columns each
constexpr uint32_t kI8Results = 0;  // TMEM columns: results (2 x 128), then the buffers
constexpr uint32_t kI8Weights = 256;
constexpr int kI8PartLd = kI8Tile + 4;

__device__ int g_int8_status;

// kind::f16 with f16 inputs, f32 accumulator, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// A from TMEM (lane = row, a column holds two neighbouring k), B from shared
// memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                           uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

// No copy of this thread is in flight when it leaves, also after a wait that gave up:
// `loads` so far, the latest in the stages before the next one's.
__device__ __forceinline__ void drain_loads(uint64_t* full, int stages, int loads) {
  for (int back = 1; back <= stages && back <= loads; ++back) {
    const int load = loads - back;
    mbar_wait(&full[load % stages], static_cast<uint32_t>((load / stages) & 1), nullptr);
  }
}

struct I8Item {
  int e, tile, row0, rows;
};

// Items of an expert: groups of up to `group` chunks of `rows` rows, tile by tile within a group,
// chunk by chunk within a tile, so that CTAs that run together share both weights
// and tokens in L2.  e: the expert of this or an earlier item, moved up.
__device__ __forceinline__ I8Item map_i8_item(const ExpertTable& t, int tiles, int group, int rows,
                                              int item, int& e) {
  while (t.chunk_off[e + 1] * tiles <= item) ++e;
  const int chunks = t.chunk_off[e + 1] - t.chunk_off[e];
  const int local = item - t.chunk_off[e] * tiles;
  const int g = local / (group * tiles), in = local - g * group * tiles;
  const int size = min(group, chunks - g * group);
  I8Item it;
  it.e = e;
  it.tile = in / size;
  it.row0 = t.start[e] + (g * group + in - it.tile * size) * rows;
  it.rows = min(rows, t.end[e] - it.row0);
  return it;
}

__device__ __forceinline__ void st_if_b32(bool on, void* p, uint32_t v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.b32 [%0], %1;\n\t}" ::"l"(p),
               "r"(v), "r"(static_cast<uint32_t>(on))
               : "memory");
}
__device__ __forceinline__ void st_if_b16(bool on, void* p, uint32_t v) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b16 h;\n\tsetp.ne.u32 p, %2, 0;\n\tcvt.u16.u32 h, %1;\n\t"
      "@p st.global.b16 [%0], h;\n\t}" ::"l"(p),
      "r"(v), "r"(static_cast<uint32_t>(on))
      : "memory");
}

// bf16 results of 128 tokens (columns) and the warp's 32 channels (lane = channel):
// v times the tokens' scales and the channel's, n the lane's channel of N, out the
// first token's row, rows how many are real.  Two tokens at a time: a lane packs its
// channel's values of both, an even lane takes the first token's pair of channels
// from it and its neighbour, the odd one the second's.  No branches within 32
// tokens: with them the steps of one pair waited for those of the one before, 9000
// cycles for the 128 tokens.
__device__ __forceinline__ void store_tokens(const uint32_t (&v)[4][32], const float* scales,
                                             float s, uint16_t* out, int64_t ldo, int n, int N,
                                             int rows, bool pairs, int lane) {
  const bool odd = lane & 1;
  // (the last channel of an odd N has no partner; its pair's even lane stores it)
  const bool both = (n | 1) < N, one = (n & ~1) < N && !both;
  uint16_t* d = pairs ? out + (n & ~1) + (odd ? ldo : 0) : out + n;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (32 * i >= rows) break;
    uint32_t w[16];
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
      const float4 f = *reinterpret_cast<const float4*>(scales + 32 * i + c);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(__uint_as_float(v[i][c]) * (f.x * s),
                                                      __uint_as_float(v[i][c + 1]) * (f.y * s));
      const __nv_bfloat162 hi = __floats2bfloat162_rn(__uint_as_float(v[i][c + 2]) * (f.z * s),
                                                      __uint_as_float(v[i][c + 3]) * (f.w * s));
      w[c / 2] = reinterpret_cast<const uint32_t&>(lo);
      w[c / 2 + 1] = reinterpret_cast<const uint32_t&>(hi);
    }
    const int left = rows - 32 * i;
    if (pairs) {
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w[c], 1);
        w[c] = odd ? __byte_perm(o, w[c], 0x7632) : __byte_perm(w[c], o, 0x5410);
      }
      const int first = left - (odd ? 1 : 0);
#pragma unroll
      for (int c = 0; c < 16; ++c) st_if_b32(both && 2 * c < first, d + 2 * c * ldo, w[c]);
      if (__any_sync(0xFFFFFFFFu, one))
#pragma unroll
        for (int c = 0; c < 16; ++c) st_if_b16(one && 2 * c < first, d + 2 * c * ldo, w[c]);
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        st_if_b16(n < N && 2 * c < left, d + 2 * c * ldo, w[c]);
        st_if_b16(n < N && 2 * c + 1 < left, d + (2 * c + 1) * ldo, w[c] >> 16);
      }
    }
    d += 32 * ldo;
  }
}

template <bool SWIGLU, bool SPLIT>
__global__ void __launch_bounds__(kI8Threads, 1)
    int8_gemm_kernel(const __grid_constant__ Int8Maps maps, const __grid_constant__ Int8Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int x_bytes = p.a_rows * 256, w_stages = p.w_stages, x_stages = p.x_stages;
  uint8_t* s_x = smem + w_stages * kI8WBytes;
  // per widening warp: the scales of a chunk's rows
  float* s_scale = reinterpret_cast<float*>(s_x + x_stages * x_bytes);
  uint64_t* wfull = reinterpret_cast<uint64_t*>(s_scale + kI8WideWarps * 128);
  uint64_t* wempty = wfull + kI8MaxStages;
  uint64_t* xfull = wempty + kI8MaxStages;
  uint64_t* xempty = xfull + kI8MaxStages;
  uint64_t* afull = xempty + kI8MaxStages;
  uint64_t* aempty = afull + kI8Buffers;
  uint64_t* dfull = aempty + kI8Buffers;
  uint64_t* dempty = dfull + 1;
  uint64_t* drained = dempty + 1;  // all MMAs are over
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_tab = reinterpret_cast<int*>(tmem_holder + 2);
  const ExpertTable tab{s_tab, s_tab + p.E + 1, s_tab + 2 * p.E + 1};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < w_stages; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], kI8WideWarps);
    }
    for (int s = 0; s < x_stages; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int b = 0; b < kI8Buffers; ++b) {
      mbar_init(&afull[b], kI8WideWarps);
      mbar_init(&aempty[b], 1);
    }
    mbar_init(dfull, 1);
    mbar_init(dempty, kI8WideWarps);
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // The kernel before this one is the library's own: it writes the codes and their
  // scales, neither offsets nor weights, and has let this one start only when all
  // before it was over.
  pdl_launch_dependents();
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == 2) fill_expert_table(p, tab, p.a_rows, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int kb_all = (p.K + 127) / 128;
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int kb0 = SPLIT ? kb_all * rank / p.split : 0;
  const int kb1 = SPLIT ? kb_all * (rank + 1) / p.split : kb_all;
  const int first = SPLIT ? blockIdx.x / p.split : blockIdx.x;
  const int step = SPLIT ? gridDim.x / p.split : gridDim.x;
  const int total = tab.chunk_off[p.E] * p.tiles;
  int expert = 0;  // of the role's latest item
  auto map_item = [&](int item) {
    return map_i8_item(tab, p.tiles, p.chunk_group, p.a_rows, item, expert);
  };
  // (one expert: the box that all its chunks take, the last one short)
  auto box_of = [&](int rows) {
    rows = p.E == 1 ? p.a_rows : rows;
    return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3;
  };

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------- weights by TMA
      // (they are not the kernel's before this one: no wait for it)
      const uint64_t once = l2_policy_evict_first(), reused = l2_policy_evict_normal();
      int stage = 0, loads = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int item = first; ok && item < total; item += step) {
        const I8Item it = map_item(item);
        // weights of an expert with one chunk are read once
        const uint64_t policy = tab.chunk_off[it.e + 1] - tab.chunk_off[it.e] > 1 ? reused : once;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&wempty[stage], phase ^ 1, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(&wfull[stage], kI8WBytes);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int n0 = SWIGLU ? it.tile * 128 + h * (p.N / 2) : it.tile * kI8Tile + h * 128;
            tma_load_3d_hint(smem + stage * kI8WBytes + h * (kI8WBytes / 2), &maps.w, &wfull[stage],
                             kb * 128, n0, it.e, policy);
          }
          ++loads;
          if (++stage == w_stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      drain_loads(wfull, w_stages, loads);
      if (!ok) report_status(&g_int8_status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp == 3) {
    if (lane == 0) {
      // -------------------------------------------------- tokens by TMA
      const uint64_t reused = l2_policy_evict_normal();
      int stage = 0, loads = 0;
      uint32_t phase = 0;
      bool ok = true;
      pdl_wait();
      fence_proxy_async_global();
      for (int item = first; ok && item < total; item += step) {
        const I8Item it = map_item(item);
        const int box = box_of(it.rows);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&xempty[stage], phase ^ 1, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(&xfull[stage], (16u << box) * 256u);
          uint8_t* sx = s_x + stage * x_bytes;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_2d_hint(sx + h * (16 << box) * 128, &maps.x[box], &xfull[stage],
                             kb * 128 + h * 64, it.row0, reused);
          ++loads;
          if (++stage == x_stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      drain_loads(xfull, x_stages, loads);
      if (!ok) report_status(&g_int8_status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------- MMA issuer
    int stage = 0, buf = 0;
    uint32_t phase = 0, aphase = 0, dphase = 0;
    bool ok = true;
    for (int item = first; ok && item < total; item += step) {
      const I8Item it = map_item(item);
      const int box = box_of(it.rows), n = 16 << box;
      const uint32_t idesc = idesc_f16(128, n);
      ok = wait_warp(dempty, dphase ^ 1, abort_flag);
      dphase ^= 1;
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        ok = wait_warp(&xfull[stage], phase, abort_flag) &&
             wait_warp(&afull[buf], aphase, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t sx = smem_u32(s_x + stage * x_bytes);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // 16 of the 128 columns: 32 bytes further in a row of 64 f16
            const uint64_t b = desc_sw128(sx + (k >> 2) * n * 128 + (k & 3) * 32);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_f16_ts(tmem + kI8Results + h * 128, tmem + kI8Weights + buf * 128 + h * 64 + k * 8,
                         b, idesc, kb > kb0 || k > 0);
          }
          tc_commit(&xempty[stage]);
          tc_commit(&aempty[buf]);
          if (kb + 1 == kb1) tc_commit(dfull);
        }
        __syncwarp();
        if (++stage == x_stages) {
          stage = 0;
          phase ^= 1;
        }
        if (++buf == kI8Buffers) {
          buf = 0;
          aphase ^= 1;
        }
      }
    }
    // (the same lane is elected every time: its commit covers all that it issued)
    if (elect_one()) tc_commit(drained);
    __syncwarp();
    if (lane == 0) mbar_wait(drained, 0, nullptr);
    __syncwarp();
    if (!ok && lane == 0) report_status(&g_int8_status, kStatusTimeout);
  } else if (warp >= kI8WideWarp0) {
    // ---------------------------------------------------- widen, and results
    const int quarter = warp & 3, half = (warp - kI8WideWarp0) >> 2;
    const int row = quarter * 32 + lane;  // of the half: the thread's TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* scales = s_scale + (warp - kI8WideWarp0) * 128;
    int stage = 0, buf = 0;
    uint32_t phase = 0, aphase = 0, dphase = 0;
    bool ok = true, waited = false;

    auto widen = [&]() {
      if (!wait_warp(&wfull[stage], phase, abort_flag)) return false;
      const uint8_t* src = smem + stage * kI8WBytes + half * (kI8WBytes / 2) + row * 128;
      uint4 v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        v[c] = *reinterpret_cast<const uint4*>(src + ((c ^ (row & 7)) << 4));
      // (without the fence the next copy into the stage could overtake these reads: up to
      // four of five calls that split the reduction of 65 and more rows, and went round the
      // ring, took channels of a later block.  16 rows of 7168 -> 4096 10.9 us without,
      // 11.4 with)
      fence_proxy_async_shared();
      __syncwarp();
      mbar_arrive_if(lane == 0, smem_u32(&wempty[stage]));
      if (!wait_warp(&aempty[buf], aphase ^ 1, abort_flag)) return false;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          i8_widen4(v[4 * q + c].x, w[8 * c], w[8 * c + 1]);
          i8_widen4(v[4 * q + c].y, w[8 * c + 2], w[8 * c + 3]);
          i8_widen4(v[4 * q + c].z, w[8 * c + 4], w[8 * c + 5]);
          i8_widen4(v[4 * q + c].w, w[8 * c + 6], w[8 * c + 7]);
        }
        tmem_st32(lanes + kI8Weights + buf * 128 + half * 64 + q * 32, w);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive_if(lane == 0, smem_u32(&afull[buf]));
      if (++stage == w_stages) {
        stage = 0;
        phase ^= 1;
      }
      if (++buf == kI8Buffers) {
        buf = 0;
        aphase ^= 1;
      }
      return true;
    };

    // Results of 32 columns (tokens) from `col` on.
    auto read32 = [&](uint32_t col, uint32_t (&v)[32]) { tmem_ld32(lanes + kI8Results + col, v); };

    auto results = [&](const I8Item& it) {
      if (!waited) {
        // (the scales are the kernel's before this one)
        pdl_wait();
        waited = true;
      }
      const float* sx = p.a_scales + it.row0;
      const float* sw = p.w_scales + static_cast<int64_t>(it.e) * p.N;
      float sr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sr[i] = 32 * i + lane < it.rows ? sx[32 * i + lane] : 0.0f;
      if (!wait_warp(dfull, dphase, abort_flag)) return false;
      dphase ^= 1;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 4; ++i) scales[32 * i + lane] = sr[i];
      __syncwarp();
      if constexpr (SPLIT) {
        // fp32 sums to [token][channel] in what were the rings of stages
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          if (c >= it.rows) break;
          uint32_t v[32];
          read32(half * 128 + c, v);
          tmem_ld_wait();
          reg_fence32(v);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < it.rows)
              part[(c + i) * kI8PartLd + half * 128 + row] = __uint_as_float(v[i]);
        }
        tc_fence_before();
      } else if constexpr (SWIGLU) {
        // all channels of one half of the tokens: gate and up of each
        uint32_t g[2][32], u[2][32];
        const int c0 = half * 64;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          read32(c0 + 32 * i, g[i]);
          read32(128 + c0 + 32 * i, u[i]);
        }
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          reg_fence32(g[i]);
          reg_fence32(u[i]);
        }
        tc_fence_before();
        mbar_arrive_if(lane == 0, smem_u32(dempty));
        const int I = p.N / 2, n = it.tile * 128 + row;
        const float sg = n < I ? sw[n] : 0.0f, su = n < I ? sw[I + n] : 0.0f;
        float* out = static_cast<float*>(p.out) + static_cast<int64_t>(it.row0) * p.ldo + n;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (c0 + 32 * i >= it.rows) break;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(scales + c0 + 32 * i + c);
            const float sc[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              g[i][c + k] = __float_as_uint(swiglu(__uint_as_float(g[i][c + k]) * (sc[k] * sg),
                                                   __uint_as_float(u[i][c + k]) * (sc[k] * su),
                                                   p.clamp));
          }
          const int rest = it.rows - c0 - 32 * i;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            st_if_b32(c < rest && n < I, out + (c0 + 32 * i + c) * p.ldo, g[i][c]);
        }
        return true;
      } else {
        uint32_t v[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) read32(half * 128 + 32 * i, v[i]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) reg_fence32(v[i]);
        tc_fence_before();
        mbar_arrive_if(lane == 0, smem_u32(dempty));
        const int n = it.tile * kI8Tile + half * 128 + row;
        const float s = n < p.N ? sw[n] : 0.0f;
        uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(it.row0) * p.ldo;
        store_tokens(v, scales, s, out, p.ldo, n, p.N, it.rows, p.out_pairs, lane);
      }
      return true;
    };

    // (one place in the code for each: copies of `results` cost registers)
    I8Item before{};
    bool pending = false;
    for (int item = first; ok; item += step) {
      const bool more = item < total;
      const int blocks = more ? kb1 - kb0 : 0, ahead = min(kI8Buffers, blocks);
      for (int kb = 0;; ++kb) {
        if (pending && kb == ahead) {
          ok = results(before);
          pending = false;
        }
        if (!ok || kb == blocks) break;
        ok = widen();
      }
      if (!more) break;
      before = map_item(item);
      pending = true;
    }
    if (!ok && lane == 0) report_status(&g_int8_status, kStatusTimeout);
  }

  if constexpr (SPLIT) {
    // Join: the ranks' partial sums in rank order, four channels to a thread, all
    // ranks' loads under way before the first is added (one after the other they took
    // most of a small product's time: 333 x 2000 -> 1001 in 19 us).
    __syncwarp();
    cluster_sync();
    if (first < total && warp >= kI8WideWarp0) {
      const I8Item it = map_item(first);
      const float* sw = p.w_scales + static_cast<int64_t>(it.e) * p.N;
      constexpr int kChannels = SWIGLU ? 128 : 256;   // of a token
      constexpr int kAtOnce = 1024 / kChannels;       // tokens of 256 threads
      const int id = threadIdx.x - 32 * kI8WideWarp0;
      const int c = id % (kChannels / 4) * 4, sub = id / (kChannels / 4);
      const int n = it.tile * kChannels + c, width = SWIGLU ? p.N / 2 : p.N;
      const float* part = reinterpret_cast<const float*>(smem) + c;
      pdl_wait();
      auto sum_of = [&](const float* at) {
        float4 v[kBsMaxSplit], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kBsMaxSplit; ++k)
          if (k < p.split) v[k] = ld_cluster_f4(smem_u32(at), k);
#pragma unroll
        for (int k = 0; k < kBsMaxSplit; ++k)
          if (k < p.split) sum.x += v[k].x, sum.y += v[k].y, sum.z += v[k].z, sum.w += v[k].w;
        return sum;
      };
      float sn[4], su[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sn[i] = n + i < width ? sw[n + i] : 0.0f;
        su[i] = SWIGLU && n + i < width ? sw[width + n + i] : 0.0f;
      }
      for (int t = rank * kAtOnce + sub; t < it.rows; t += kAtOnce * p.split) {
        const float4 f = sum_of(part + t * kI8PartLd);
        const float s = p.a_scales[it.row0 + t];
        const float v[4] = {f.x * (s * sn[0]), f.y * (s * sn[1]), f.z * (s * sn[2]), f.w * (s * sn[3])};
        if constexpr (SWIGLU) {
          const float4 g = sum_of(part + t * kI8PartLd + 128);
          const float u[4] = {g.x * (s * su[0]), g.y * (s * su[1]), g.z * (s * su[2]), g.w * (s * su[3])};
          float* out = static_cast<float*>(p.out) + (it.row0 + t) * p.ldo + n;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            st_if_b32(n + i < width, out + i, __float_as_uint(swiglu(v[i], u[i], p.clamp)));
        } else {
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (it.row0 + t) * p.ldo + n;
          if (p.out_fours && n + 4 <= width) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]),
                                 hi = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2*>(out) = make_uint2(reinterpret_cast<const uint32_t&>(lo),
                                                        reinterpret_cast<const uint32_t&>(hi));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n + i < width) out[i] = __float2bfloat16_rn(v[i]);
          }
        }
      }
    }
    __syncwarp();
    cluster_sync();  // the other ranks' shared memory stays until it has been read
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- CTA pairs
// Many rows.  A single CTA's 256 x 128 block of 128 columns moves 64 KB into shared
// memory, 32 KB out of it for the widening and 64 KB for the MMAs (the tokens once
// for each half), and 64 KB into TMEM, which takes the same path: 1800 cycles of it
// against 1024 of MMA.  In a pair (cta_group::2) two CTAs share 256 channels x up
// to 256 tokens: each widens its own 128 channels and loads half of the tokens: 48
// KB in, 16 and 32 KB out, 32 KB into TMEM, 1024 cycles.
//
// Rank 0 issues; each CTA's results are its own 128 channels (TMEM lanes) of all
// tokens.  An item's tokens are cut in two halves of a multiple of 16, and an
// expert's rows evenly into items, so that short and odd ones share the work.  The
// widening warps take every other block of 128 columns: four on one, four on the
// next.  With SWIGLU the CTA's channels are 64 gate and the 64 up channels that go
// with them, 16 of each to a warp's 32 lanes, so that a gate and its up meet by a
// shuffle.
//
// Weights and tokens have rings of their own: a stage of weights is free as soon as
// it has been widened, long before its MMAs, and their loads have that much longer
// (in one ring of four stages the widening waited 900 cycles a block for its
// weights; 64 experts, 24576 rows, 2048 x 1024, with the quantisation: 309 us for
// 282).  The stores take 4000 cycles an item, most of them beside the MMAs of the
// next item's first blocks, which have been widened by then (in four parts with the
// widening of further blocks between them: 293 us).
constexpr int kP8WStages = 5, kP8XStages = 4;
// Barriers of filled weights, two to a stage by turns: the stages' number is odd, so a
// stage's uses go to the two halves of the widening warps by turns, and a barrier's
// phase tells only neighbouring uses apart.  (One to a stage: where a load came after
// those of the two blocks behind it, the half that had skipped a use took the stage for
// its own next one, with what was there.)
constexpr int kP8WFull = 2 * kP8WStages;
constexpr int kP8WBytes = 128 * 128;
constexpr int kP8Buffers = 4;      // TMEM buffers of widened weights, 64 columns each
constexpr uint32_t kP8Weights = 256;
constexpr int kP8Tokens = 256;     // most tokens of an item
constexpr int kP8XBytes = kP8Tokens / 2 * 256;
constexpr int kP8Ahead = 3;        // blocks of the next item that come before an item's results

__device__ __forceinline__ void mma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                                uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kI8Threads, 1)
    int8_pair_kernel(const __grid_constant__ Int8Maps maps, const __grid_constant__ Int8Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_x = smem + kP8WStages * kP8WBytes;
  // per widening warp: the scales of its 128 tokens
  float* s_scale = reinterpret_cast<float*>(s_x + kP8XStages * kP8XBytes);
  uint64_t* wfull = reinterpret_cast<uint64_t*>(s_scale + kI8WideWarps * 128);
  uint64_t* wempty = wfull + kP8WFull;
  uint64_t* xfull = wempty + kP8WStages;  // (rank 0's: both CTAs' tokens)
  uint64_t* xempty = xfull + kP8XStages;
  uint64_t* afull = xempty + kP8XStages;  // (rank 0's: both CTAs' weights)
  uint64_t* aempty = afull + kP8Buffers;
  uint64_t* dfull = aempty + kP8Buffers;
  uint64_t* dempty = dfull + 1;            // (rank 0's)
  uint64_t* drained = dempty + 1;          // all MMAs are over
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_tab = reinterpret_cast<int*>(tmem_holder + 2);
  const ExpertTable tab{s_tab, s_tab + p.E + 1, s_tab + 2 * p.E + 1};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kP8WFull; ++s) mbar_init(&wfull[s], 1);
    for (int s = 0; s < kP8WStages; ++s) mbar_init(&wempty[s], 4);  // the warps that widen it
    for (int s = 0; s < kP8XStages; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int b = 0; b < kP8Buffers; ++b) {
      mbar_init(&afull[b], 8);  // four warps of each CTA
      mbar_init(&aempty[b], 1);
    }
    mbar_init(dfull, 1);
    mbar_init(dempty, 2 * kI8WideWarps);
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_launch_dependents();
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  if (warp == 2) fill_expert_table(p, tab, p.a_rows, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers, before either arrives on the other's
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int blocks = (p.K + 127) / 128;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  const int total = tab.chunk_off[p.E] * p.tiles;
  int expert = 0;  // of the role's latest item
  // row0, rows: of the item, cut evenly among its expert's chunks
  auto map_item = [&](int item) {
    while (tab.chunk_off[expert + 1] * p.tiles <= item) ++expert;
    const int chunks = tab.chunk_off[expert + 1] - tab.chunk_off[expert];
    const int local = item - tab.chunk_off[expert] * p.tiles;
    const int g = local / (p.chunk_group * p.tiles), in = local - g * p.chunk_group * p.tiles;
    const int size = min(p.chunk_group, chunks - g * p.chunk_group);
    const int r0 = tab.start[expert], rows = tab.end[expert] - r0;
    I8Item it;
    it.e = expert;
    it.tile = in / size;
    const int c = g * p.chunk_group + in - it.tile * size;
    const int each = ((rows + chunks - 1) / chunks + 31) & ~31;  // at most a_rows
    it.row0 = r0 + c * each;
    it.rows = max(min(each, r0 + rows - it.row0), 0);
    return it;
  };
  // rows of either CTA's part of an item (the MMA's N, both parts, is a multiple of
  // 32), and their box
  auto part_of = [](const I8Item& it) { return max((it.rows + 31) / 32 * 16, 16); };
  auto box_of = [](int part) {
    // (one box that holds them all: parts of 96 rows in boxes of 64 and 32 took 315 us
    // where a box of 128 takes 294, with a quarter more bytes)
    return part <= 16 ? 0 : part <= 32 ? 1 : part <= 64 ? 2 : 3;
  };

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------- weights by TMA
      // (they are not the kernel's before this one: no wait for it)
      const uint64_t reused = l2_policy_evict_normal();
      int stage = 0, loads = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int item = first; ok && item < total; item += step) {
        const I8Item it = map_item(item);
        for (int kb = 0; kb < blocks; ++kb) {
          ok = mbar_wait(&wempty[stage], phase ^ 1, abort_flag);
          if (!ok) break;
          uint64_t* full = &wfull[loads % kP8WFull];
          mbar_arrive_expect_tx(full, kP8WBytes);
          uint8_t* sw = smem + stage * kP8WBytes;
          if constexpr (SWIGLU) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_3d_hint(sw + h * (kP8WBytes / 2), &maps.w, full, kb * 128,
                               it.tile * 128 + rank * 64 + h * (p.N / 2), it.e, reused);
          } else {
            tma_load_3d_hint(sw, &maps.w, full, kb * 128, it.tile * kI8Tile + rank * 128, it.e,
                             reused);
          }
          ++loads;
          if (++stage == kP8WStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      drain_loads(wfull, kP8WFull, loads);
      if (!ok) report_status(&g_int8_status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp == 3) {
    if (lane == 0) {
      // -------------------------------------------------- tokens by TMA
      const uint64_t reused = l2_policy_evict_normal();
      const uint32_t xfull0 = mapa_shared(smem_u32(xfull), 0);
      int stage = 0, loads = 0;
      uint32_t phase = 0;
      bool ok = true;
      pdl_wait();
      fence_proxy_async_global();
      for (int item = first; ok && item < total; item += step) {
        const I8Item it = map_item(item);
        const int part = part_of(it), box = box_of(part);
        for (int kb = 0; kb < blocks; ++kb) {
          ok = mbar_wait(&xempty[stage], phase ^ 1, abort_flag);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&xfull[stage], 2u * (16u << box) * 256u);
          uint8_t* sx = s_x + stage * kP8XBytes;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_2d_pair(sx + h * (16 << box) * 128, &maps.x[box], xfull0 + stage * 8,
                             kb * 128 + h * 64, it.row0 + rank * part, reused);
          ++loads;
          if (++stage == kP8XStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // (rank 0's barriers count both CTAs' copies, and neither leaves before the other)
      if (rank == 0) drain_loads(xfull, kP8XStages, loads);
      // every stage's last release has arrived here before this CTA may leave
      for (int s = 0; ok && s < kP8XStages; ++s) {
        ok = mbar_wait(&xempty[stage], phase ^ 1, abort_flag);
        if (++stage == kP8XStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) report_status(&g_int8_status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------- MMA issuer
    int stage = 0, buf = 0;
    uint32_t phase = 0, aphase = 0, dphase = 0;
    bool ok = true;
    for (int item = first; ok && item < total; item += step) {
      const I8Item it = map_item(item);
      const int part = part_of(it), n = 16 << box_of(part);
      const uint32_t idesc = idesc_f16(256, 2 * part);
      ok = wait_warp(dempty, dphase ^ 1, abort_flag);
      dphase ^= 1;
      for (int kb = 0; ok && kb < blocks; ++kb) {
        ok = wait_warp(&xfull[stage], phase, abort_flag) &&
             wait_warp(&afull[buf], aphase, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t sx = smem_u32(s_x + stage * kP8XBytes);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_f16_ts_pair(tmem, tmem + kP8Weights + buf * 64 + k * 8,
                            desc_sw128(sx + (k >> 2) * n * 128 + (k & 3) * 32), idesc,
                            kb > 0 || k > 0);
          tc_commit_pair(&xempty[stage], 3);
          tc_commit_pair(&aempty[buf], 3);
          if (kb + 1 == blocks) tc_commit_pair(dfull, 3);
        }
        __syncwarp();
        if (++stage == kP8XStages) {
          stage = 0;
          phase ^= 1;
        }
        if (++buf == kP8Buffers) {
          buf = 0;
          aphase ^= 1;
        }
      }
    }
    // (the same lane is elected every time: its commit covers all that it issued)
    if (elect_one()) tc_commit_pair(drained, 3);
    __syncwarp();
    if (!ok && lane == 0) report_status(&g_int8_status, kStatusTimeout);
  } else if (warp >= kI8WideWarp0) {
    // ---------------------------------------------------- widen, and results
    const int quarter = warp & 3, group = (warp - kI8WideWarp0) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    // the row of the tile that becomes this thread's TMEM lane
    const int row = SWIGLU ? (lane >> 4) * 64 + quarter * 16 + (lane & 15) : quarter * 32 + lane;
    float* scales = s_scale + (warp - kI8WideWarp0) * 128;
    const uint32_t afull0 = mapa_shared(smem_u32(afull), 0);
    const uint32_t dempty0 = mapa_shared(smem_u32(dempty), 0);
    int next = group, limit = 0;  // this group's next block; all items' so far
    uint32_t dphase = 0;
    bool ok = true, waited = false;

    // Every other block: this group's turn.
    auto widen = [&](int block) {
      const int stage = block % kP8WStages, buf = block % kP8Buffers;
      if (!wait_warp(&wfull[block % kP8WFull], (block / kP8WFull) & 1, abort_flag)) return false;
      const uint8_t* src = smem + stage * kP8WBytes + row * 128;
      uint4 v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        v[c] = *reinterpret_cast<const uint4*>(src + ((c ^ (row & 7)) << 4));
      fence_proxy_async_shared();
      __syncwarp();
      mbar_arrive_if(lane == 0, smem_u32(&wempty[stage]));
      if (!wait_warp(&aempty[buf], ((block / kP8Buffers) & 1) ^ 1, abort_flag)) return false;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          i8_widen4(v[4 * q + c].x, w[8 * c], w[8 * c + 1]);
          i8_widen4(v[4 * q + c].y, w[8 * c + 2], w[8 * c + 3]);
          i8_widen4(v[4 * q + c].z, w[8 * c + 4], w[8 * c + 5]);
          i8_widen4(v[4 * q + c].w, w[8 * c + 6], w[8 * c + 7]);
        }
        tmem_st32(lanes + kP8Weights + buf * 64 + q * 32, w);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive_if(lane == 0, afull0 + buf * 8);
      return true;
    };

    auto results = [&](const I8Item& it) {
      if (!waited) {
        // (the scales are the kernel's before this one)
        pdl_wait();
        waited = true;
      }
      const int c0 = group * 128, left = it.rows - c0;  // this group's tokens
      const float* sx = p.a_scales + it.row0 + c0;
      const float* sw = p.w_scales + static_cast<int64_t>(it.e) * p.N;
      float sr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sr[i] = 32 * i + lane < left ? sx[32 * i + lane] : 0.0f;
      if (!wait_warp(dfull, dphase, abort_flag)) return false;
      dphase ^= 1;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 4; ++i) scales[32 * i + lane] = sr[i];
      __syncwarp();
      uint32_t v[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(lanes + c0 + 32 * i, v[i]);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 4; ++i) reg_fence32(v[i]);
      tc_fence_before();
      mbar_arrive_if(lane == 0, dempty0);
      if constexpr (SWIGLU) {
        // lanes below 16 take the first of two tokens, the others the second
        const int I = p.N / 2, n = it.tile * 128 + rank * 64 + quarter * 16 + (lane & 15);
        const bool high = lane & 16;
        const float sg = n < I ? sw[n] : 0.0f, su = n < I ? sw[I + n] : 0.0f;
        float* out = static_cast<float*>(p.out) +
                     static_cast<int64_t>(it.row0 + c0 + (high ? 1 : 0)) * p.ldo + n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (32 * i >= left) break;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(scales + 32 * i + c);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const uint32_t x = v[i][c + k], y = v[i][c + k + 1];
              const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, high ? x : y, 16);
              const float sc = k ? (high ? f.w : f.z) : (high ? f.y : f.x);
              v[i][c + k] = __float_as_uint(swiglu(__uint_as_float(high ? o : x) * (sc * sg),
                                                   __uint_as_float(high ? y : o) * (sc * su),
                                                   p.clamp));
            }
          }
          // (the stores after all 32 tokens' sums: no load or step waits for one)
          const int rest = left - 32 * i - (high ? 1 : 0);
#pragma unroll
          for (int c = 0; c < 32; c += 2) st_if_b32(c < rest && n < I, out + c * p.ldo, v[i][c]);
          out += 32 * p.ldo;
        }
      } else {
        const int n = it.tile * kI8Tile + rank * 128 + quarter * 32 + lane;
        const float s = n < p.N ? sw[n] : 0.0f;
        uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(it.row0 + c0) * p.ldo;
        store_tokens(v, scales, s, out, p.ldo, n, p.N, left, p.out_pairs, lane);
      }
      return true;
    };

    I8Item before{};
    bool pending = false;
    for (int item = first; ok; item += step) {
      const bool more = item < total;
      const int ahead = limit + kP8Ahead;
      limit += more ? blocks : 0;
      for (;;) {
        if (pending && next >= min(ahead, limit)) {
          ok = results(before);
          pending = false;
        }
        if (!ok || next >= limit) break;
        ok = widen(next);
        next += 2;
      }
      if (!more) break;
      before = map_item(item);
      pending = true;
    }
    // the last releases of the buffers, before this CTA may leave
    for (int b = 0; ok && b < kP8Buffers; ++b)
      if (limit - 1 - b >= 0)
        ok = wait_warp(&aempty[(limit - 1 - b) % kP8Buffers],
                       ((limit - 1 - b) / kP8Buffers) & 1, abort_flag);
    if (!ok && lane == 0) report_status(&g_int8_status, kStatusTimeout);
  }

  tc_fence_before();
  __syncthreads();
  // every MMA of the pair is over
  if (warp == 1 && lane == 0) mbar_wait(drained, 0, nullptr);
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------- host
int extra_smem(int E) {
  return kI8WideWarps * 128 * 4 + (4 * kI8MaxStages + 2 * kI8Buffers + 3) * 8 + 8 +
         (3 * E + 1) * 4;
}

template <bool SWIGLU, bool SPLIT>
cudaError_t launch_i8(const Int8Maps& maps, Int8Args p, int grid, cudaStream_t s) {
  auto k = int8_gemm_kernel<SWIGLU, SPLIT>;
  static OncePerDevice prepared;
  const cudaError_t ready = prepared([&] {
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kI8SmemLimit);
  });
  if (ready != cudaSuccess) return ready;
  const int fixed = 1024 + extra_smem(p.E), x_bytes = p.a_rows * 256;
  // (three to six stages of weights.  128 rows: two stages of tokens and four of weights
  // 136 us where these take 130, for 64 experts of 2048 x 1024 and 6144 rows)
  p.x_stages = p.a_rows <= 64 ? 4 : 3;
  p.w_stages = std::min(kI8MaxStages, (kI8SmemLimit - fixed - p.x_stages * x_bytes) / kI8WBytes);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kI8Threads);
  cfg.dynamicSmemBytes = fixed + p.w_stages * kI8WBytes + p.x_stages * x_bytes;
  cfg.stream = s;
  cfg.attrs = attr;
  attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  if (SPLIT) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = p.split;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, k, maps, p);
}

template <bool SWIGLU>
cudaError_t launch_i8_pair(const Int8Maps& maps, Int8Args p, int pairs, cudaStream_t s) {
  auto k = int8_pair_kernel<SWIGLU>;
  static OncePerDevice prepared;
  const cudaError_t ready = prepared([&] {
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kI8SmemLimit);
  });
  if (ready != cudaSuccess) return ready;
  constexpr int fixed = 1024 + kP8WStages * kP8WBytes + kP8XStages * kP8XBytes +
                        kI8WideWarps * 128 * 4 +
                        (kP8WFull + kP8WStages + 2 * kP8XStages + 2 * kP8Buffers + 3) * 8 + 8;
  static_assert(fixed + (3 * kMaxExperts + 1) * 4 <= kI8SmemLimit);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kI8Threads);
  cfg.dynamicSmemBytes = fixed + (3 * p.E + 1) * 4;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  return cudaLaunchKernelEx(&cfg, k, maps, p);
}

}  // namespace

// Pairs where every pair of SMs has an item and the experts' rows fill most of one.
bool int8_in_pairs(int M, int N, int E) {
  return M / 192 >= E && static_cast<int64_t>(M / kP8Tokens) * ((N + kI8Tile - 1) / kI8Tile) >= 76;
}

int int8_chunk_rows(int M, int N, int E) {
  if (int8_in_pairs(M, N, E)) return kP8Tokens;
  const int64_t most = E == 1 ? M : std::min<int64_t>(M, std::max<int64_t>(32, 2 * (static_cast<int64_t>(M) / E)));
  return most <= 16 ? 16 : most <= 32 ? 32 : most <= 64 ? 64 : 128;
}

// See internal.h.  Chunks: of all rows where there are few, else 128; with several
// experts of few rows each on average, twice that average at least, since a lower
// chunk leaves room for more stages of weights (64 experts, 512 rows, 7168 x 2048:
// chunks of 128 rows and three stages 319 + 171 us, of 32 rows and five 301 + 160, in
// one ring),
// and an expert with more rows reads its weights again from L2.  Fewer items than
// half the SMs: the reduction is split over clusters of as many CTAs (up to eight)
// as still run all at once.  Several experts only with a token's rows or two in
// all, so that with more a row's sums keep their order whatever the other experts'
// number.
cudaError_t launch_int8(const Int8Maps& maps, Int8Args p, bool swiglu, const BlockscaleDevice& d,
                        cudaStream_t s) {
  p.a_rows = int8_chunk_rows(p.M, p.N, p.E);
  const int kb = (p.K + 127) / 128;
  const int64_t chunks = p.E == 1 ? (p.M + p.a_rows - 1) / p.a_rows
                                  : std::min<int64_t>(p.E, p.M) + p.M / p.a_rows;
  p.tiles = swiglu ? (p.N / 2 + 127) / 128 : (p.N + kI8Tile - 1) / kI8Tile;
  p.chunk_group = 8;
  const int64_t items = chunks * p.tiles;
  if (items > INT32_MAX) return cudaErrorInvalidValue;
  if (int8_in_pairs(p.M, p.N, p.E)) {
    const int pairs = static_cast<int>(std::min<int64_t>(d.clusters[2], items));
    return swiglu ? launch_i8_pair<true>(maps, p, pairs, s) : launch_i8_pair<false>(maps, p, pairs, s);
  }
  p.split = 1;
  if (p.E == 1 || p.M <= 16)
    for (int n = 2; n <= std::min(kBsMaxSplit, kb); ++n)
      if (items <= d.clusters[n] && (kb + n - 1) / n < (kb + p.split - 1) / p.split) p.split = n;
  if (p.split > 1) {
    const int grid = static_cast<int>(items) * p.split;
    return swiglu ? launch_i8<true, true>(maps, p, grid, s) : launch_i8<false, true>(maps, p, grid, s);
  }
  const int grid = static_cast<int>(std::min<int64_t>(d.sms, items));
  return swiglu ? launch_i8<true, false>(maps, p, grid, s) : launch_i8<false, false>(maps, p, grid, s);
}

cudaError_t int8_status(int* code) {
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_int8_status, sizeof(int));
  if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_int8_status, &zero, sizeof(int));
  return e;
}

}  // namespace moe
