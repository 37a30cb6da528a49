// blockscale_gemm.cu -- the block-scaled FP8 products on the sm_103a tensor
// cores.
//
//   y[m][n] = sum_b sa[b][m] sw[n/128][b] sum_{k in block b} a[m][k] w[n][k]
//
// The scales are general fp32 numbers, so the tensor cores cannot apply them;
// they change with every 128 columns of the reduction.  Each block's plain
// e4m3 product therefore goes into a TMEM buffer of its own (four MMAs of
// K = 32, the first one overwriting), and the epilogue warps add it, times
// sa sw, to fp32 accumulators that stay in registers for the whole item: one
// scaled fused multiply-add per output and block, two at a time
// (fma.f32x2).  The buffers are double (256 columns) or fourfold (128), so
// the tensor pipe works on the next block meanwhile.
//
// Structure: one persistent CTA per SM walks the items (expert, tile of NT
// weight rows, chunk of at most 128 rows), expert-major, then tile, then
// chunk, so that CTAs running together share a weight tile in L2.  Warp 0
// (one thread) fills a ring of stages by TMA: 128 columns of the chunk's
// rows (box height 16 / 32 / 64 / 128, so short chunks pull no padding) and
// of the NT weight rows.  Warp 1 (one thread) issues the MMAs.  Warp 2 runs
// ahead through the same blocks and leaves every row's scale product in a
// ring in shared memory.  Warps 4-11 are the epilogue: warp w reads TMEM
// lanes 32 (w % 4).. and half of the tile's columns, so a thread owns one row
// and NT / 2 columns.
//
// With the weights transposed (input gradient) the reduction runs along the
// stored rows: the tile is 128 rows of 128 bytes of output columns, an
// MN-major operand for the tensor cores; nothing is copied or re-laid out.
//
// Few rows of one expert leave most SMs without an item; there a cluster of
// 2, 4 or 8 CTAs splits the reduction of each item and joins its fp32
// partial sums through distributed shared memory, in rank order, so the
// result does not depend on timing.
#include <cuda_bf16.h>

#include <algorithm>

#include "blockscale_quant.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kBsThreads = 384;
constexpr int kBsEpiWarp0 = 4;
constexpr int kBsLeanRegs = 72;
constexpr int kBsEpiRegs = 216;
// registers per thread at launch: the lean warpgroup gives up 96 of 168, the
// two epilogue warpgroups claim 48 each
constexpr int kBsLaunchRegs = 168;
static_assert(kBsLeanRegs + 2 * kBsEpiRegs <= 3 * kBsLaunchRegs, "register split");
constexpr int kBsMaxStages = 8;
constexpr int kBsScaleSlots = 8;  // blocks the scale warp may run ahead
constexpr int kBsSmemLimit = 232448;
constexpr int kBsSplitRows = 32;  // largest chunk whose reduction is split

__device__ int g_blockscale_status;

// kind::f8f6f4, e4m3 x e4m3, f32 accumulator; transpose_b: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool transpose_b) {
  return (1u << 4) | (static_cast<uint32_t>(transpose_b) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

// MN-major operand staged by TMA with the 128-byte swizzle: rows of 128
// bytes along M/N, one per reduction index, 8-row atoms of 1024 bytes
// stacked along the reduction (stride 1024); the next 128 columns of M/N
// follow `chunk` bytes later.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t chunk) {
  return desc_sw128(saddr) | (static_cast<uint64_t>((chunk >> 4) & 0x3FFFu) << 16);
}

__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, uint64_t* bar,
                                                 int32_t x, int32_t y, int32_t z,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z),
      "l"(policy)
      : "memory");
}

// 32 consecutive 32-bit columns of the thread's TMEM lane; not valid before
// tmem_ld_wait() and reg_fence32().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19,"
      " %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void reg_fence32(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                   "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// acc += {lo, hi} * {s, s}, two fp32 fused multiply-adds.
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s2) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(lo), "r"(hi));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(p), "l"(s2));
}

__device__ __forceinline__ uint64_t pack2(float s) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %1};" : "=l"(p) : "f"(s));
  return p;
}

__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t saddr, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(mapa_shared(saddr, rank))
               : "memory");
  return v;
}

struct BsItem {
  int e, tile, row0, rows;
};

// Chunk table in shared memory: off[0..E] exclusive chunk counts, start[e]
// and the row end of every expert, clamped into [0, M].
struct BsTable {
  int* chunk_off;  // [E + 1]
  int* start;      // [E]
  int* end;        // [E]
};

__device__ __forceinline__ BsItem map_bs_item(const BsTable& t, int E, int tiles, int item) {
  int lo = 0, hi = E;  // chunk_off[lo] * tiles <= item < chunk_off[hi] * tiles
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.chunk_off[mid] * tiles <= item) lo = mid;
    else hi = mid;
  }
  const int chunks = t.chunk_off[lo + 1] - t.chunk_off[lo];
  const int local = item - t.chunk_off[lo] * tiles;
  BsItem it;
  it.e = lo;
  it.tile = local / chunks;
  it.row0 = t.start[lo] + (local % chunks) * 128;
  it.rows = min(128, t.end[lo] - it.row0);
  return it;
}

// One warp fills the table: lane l takes kMaxExperts / 32 consecutive experts.
__device__ __forceinline__ void fill_bs_table(const BlockscaleArgs& p, const BsTable& t, int lane) {
  constexpr int kPer = kMaxExperts / 32;
  int chunks = 0;
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    if (e >= p.E) break;
    const int r0 = p.offsets ? min(max(p.offsets[e], 0), p.M) : 0;
    const int r1 = p.offsets ? min(max(p.offsets[e + 1], r0), p.M) : p.M;
    t.start[e] = r0;
    t.end[e] = r1;
    chunks += (r1 - r0 + 127) / 128;
  }
  int inc = chunks;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
    if (lane >= off) inc += o;
  }
  int run = inc - chunks;
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    if (e >= p.E) break;
    t.chunk_off[e] = run;
    run += (t.end[e] - t.start[e] + 127) / 128;
    if (e == p.E - 1) t.chunk_off[p.E] = run;
  }
}

// bf16 of 32 consecutive fp32 columns n0 .. n0 + 31 of one row (n0 + 32 may
// pass N).
__device__ __forceinline__ void store_bf16_32(__nv_bfloat16* row, int n0, int N, bool vec,
                                              const uint64_t* acc) {
  uint32_t v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 f = unpack2(acc[i]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    v[i] = reinterpret_cast<const uint32_t&>(b);
  }
  if (vec && n0 + 32 <= N) {
    uint4* d = reinterpret_cast<uint4*>(row + n0);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (n0 + i < N)
      reinterpret_cast<uint16_t*>(row)[n0 + i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
}

__device__ __forceinline__ float swiglu(float g, float u, float clamp) {
  g = fminf(fmaxf(g, -clamp), clamp);
  u = fminf(fmaxf(u, -clamp), clamp);
  return g / (1.0f + expf(-g)) * u;
}

// NT: weight rows per item.  SWIGLU: the tile is 128 gate rows and the 128
// up rows of the same columns (NT = 256).  SPLIT: the grid is clusters of
// args.split CTAs, one item each (one expert, at most kBsSplitRows rows).
template <int NT, bool SWIGLU, bool TRANS, bool SPLIT>
__global__ void __launch_bounds__(kBsThreads, 1)
    blockscale_gemm_kernel(const __grid_constant__ BlockscaleMaps maps,
                           const __grid_constant__ BlockscaleArgs p) {
  constexpr int kBufs = 512 / NT;  // TMEM accumulators of one block each
  constexpr int kCols = NT / 2;    // columns per epilogue thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int a_bytes = p.a_rows * 128;
  const int stage_bytes = a_bytes + NT * 128;
  const int stages = p.stages;
  float* s_part = reinterpret_cast<float*>(smem + stages * stage_bytes);  // SPLIT: [32][NT + 4]
  uint32_t* s_amax = reinterpret_cast<uint32_t*>(s_part);                 // SWIGLU: [2][128]
  constexpr int kSets = NT / 128;  // weight blocks of the tile: scale sets of a slot
  float* s_scale = s_part + (SPLIT ? kBsSplitRows * (NT + 4) : SWIGLU ? 256 : 0);
  uint64_t* full = reinterpret_cast<uint64_t*>(s_scale + kBsScaleSlots * kSets * 128);
  uint64_t* empty = full + kBsMaxStages;
  uint64_t* tfull = empty + kBsMaxStages;
  uint64_t* tempty = tfull + 4;
  uint64_t* sfull = tempty + 4;
  uint64_t* sempty = sfull + kBsScaleSlots;
  uint64_t* drained = sempty + kBsScaleSlots;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_tab = reinterpret_cast<int*>(tmem_holder + 2);
  const BsTable tab{s_tab, s_tab + p.E + 1, s_tab + 2 * p.E + 1};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 8);
    }
    for (int i = 0; i < kBsScaleSlots; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], 8);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  // (early: the only kernel this one may overlap is the library's own before
  // it, which writes the activations and their scales but no offsets or
  // weights)
  if (!p.early) pdl_wait();
  if (warp == 2) fill_bs_table(p, tab, lane);
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

  if (warp < kBsEpiWarp0) {
    regs_release<kBsLeanRegs>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------ TMA producer
      const uint64_t once = l2_policy_evict_first(), reused = l2_policy_evict_normal();
      int stage = 0, slots = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto box_of = [](int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; };
      // announce a stage's bytes and load its weight tile
      auto load_w = [&](const BsItem& it, int st, int kb) {
        // weights of an expert with one chunk are read once
        const uint64_t policy =
            tab.chunk_off[it.e + 1] - tab.chunk_off[it.e] > 1 ? reused : once;
        uint8_t* sb = smem + st * stage_bytes + a_bytes;
        mbar_arrive_expect_tx(&full[st], (16u << box_of(it.rows)) * 128u + NT * 128u);
#pragma unroll
        for (int h = 0; h < NT / 128; ++h) {
          const int n0 = SWIGLU ? it.tile * 128 + h * (p.N / 2) : it.tile * NT + h * 128;
          if constexpr (TRANS)
            tma_load_3d_hint(sb + h * 16384, &maps.w, &full[st], n0, kb * 128, it.e, policy);
          else
            tma_load_3d_hint(sb + h * 16384, &maps.w, &full[st], kb * 128, n0, it.e, policy);
        }
      };
      int ahead = 0;  // stages of the first item whose weights are on their way
      if (p.early) {
        if (first < total) {
          const BsItem it = map_bs_item(tab, p.E, p.tiles, first);
          for (; ahead < min(stages, kb1 - kb0); ++ahead) load_w(it, ahead, kb0 + ahead);
        }
        pdl_wait();
      }
      for (int item = first; item < total && ok; item += step) {
        const BsItem it = map_bs_item(tab, p.E, p.tiles, item);
        const int box = box_of(it.rows);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (slots >= ahead) load_w(it, stage, kb);
          tma_load_2d(smem + stage * stage_bytes, &maps.a[box], &full[stage], kb * 128, it.row0);
          ++slots;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // no copy of this thread is in flight when it leaves
      for (int back = 1; back <= stages && back <= slots; ++back) {
        const int idx = slots - back;
        mbar_wait(&full[idx % stages], static_cast<uint32_t>((idx / stages) & 1), nullptr);
      }
      if (!ok) report_status(&g_blockscale_status, kStatusTimeout);
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------ MMA issuer
      constexpr uint32_t idesc = idesc_e4m3(128, NT, TRANS);
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      for (int item = first; item < total && ok; item += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&tempty[buf], bphase ^ 1u, abort_flag) ||
              !mbar_wait(&full[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * stage_bytes);
          const uint64_t da = desc_sw128(sa);
          const uint64_t db = TRANS ? desc_mn_sw128(sa + a_bytes, 16384) : desc_sw128(sa + a_bytes);
          const uint32_t d = tmem + buf * NT;
          // 32 reduction columns are 32 bytes along a K-major row, 32 rows
          // (4096 bytes) of an MN-major tile
          constexpr uint64_t kStepB = TRANS ? 256 : 2;
          mma_e4m3(d, da, db, idesc, 0u);
          mma_e4m3(d, da + 2, db + kStepB, idesc, 1u);
          mma_e4m3(d, da + 4, db + 2 * kStepB, idesc, 1u);
          mma_e4m3(d, da + 6, db + 3 * kStepB, idesc, 1u);
          tc_commit(&empty[stage]);
          tc_commit(&tfull[buf]);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == kBufs) {
            buf = 0;
            bphase ^= 1u;
          }
        }
      }
      tc_commit(drained);
      mbar_wait(drained, 0, nullptr);
      if (!ok) report_status(&g_blockscale_status, kStatusTimeout);
    } else if (warp == 2) {
      // ------------------------------------------------ scales
      // Lane l takes rows l, l + 32, ..; four blocks' loads are in flight at
      // a time, and the ring lets them run ahead of the tensor pipe.
      constexpr int kAhead = 4;
      if (p.early) pdl_wait();
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int item = first; item < total && ok; item += step) {
        const BsItem it = map_bs_item(tab, p.E, p.tiles, item);
        const float* sa = p.a_scales + it.row0 + lane;
        // SWIGLU: the gate's block and the up half's; else the tile's blocks
        // (one past N has no scale of its own and is not stored)
        const float* sw[kSets];
#pragma unroll
        for (int h = 0; h < kSets; ++h) {
          const int nb = SWIGLU ? it.tile + h * (p.N / 256)
                                : min(it.tile * kSets + h, (p.N + 127) / 128 - 1);
          sw[h] = p.w_scales + it.e * p.w_blocks + nb * p.w_stride_n;
        }
        for (int kb = kb0; kb < kb1 && ok; kb += kAhead) {
          float a[kAhead][4], w[kAhead][kSets];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              a[i][j] = kb + i < kb1 && lane + 32 * j < it.rows
                            ? __ldg(sa + (kb + i) * p.ld_as + 32 * j)
                            : 0.0f;
#pragma unroll
            for (int h = 0; h < kSets; ++h)
              w[i][h] = kb + i < kb1 ? __ldg(sw[h] + (kb + i) * p.w_stride_k) : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            if (kb + i >= kb1) break;
            const bool free = mbar_wait(&sempty[slot], phase ^ 1u, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, free)) {
              ok = false;
              break;
            }
            float* d = s_scale + slot * kSets * 128 + lane;
#pragma unroll
            for (int h = 0; h < kSets; ++h)
#pragma unroll
              for (int j = 0; j < 4; ++j) d[h * 128 + 32 * j] = a[i][j] * w[i][h];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfull[slot]);
            if (++slot == kBsScaleSlots) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
      }
      if (!ok && lane == 0) report_status(&g_blockscale_status, kStatusTimeout);
    }
    if constexpr (SPLIT) {
      // the epilogue warps' two barriers take every thread of the cluster;
      // the second keeps this CTA's shared memory alive for its peers
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    regs_claim<kBsEpiRegs>();
    // ------------------------------------------------ epilogue warps
    const int q = warp & 3, g = (warp - kBsEpiWarp0) >> 2;
    int buf = 0, slot = 0;
    uint32_t bphase = 0, sphase = 0;
    bool ok = true;
    for (int item = first; item < total && ok; item += step) {
      const BsItem it = map_bs_item(tab, p.E, p.tiles, item);
      const int r = q * 32 + lane;
      const bool active = q * 32 < it.rows, live = r < it.rows;
      const int64_t row = it.row0 + (live ? r : 0);
      uint64_t acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = 0ull;
      for (int kb = kb0; kb < kb1; ++kb) {
        const bool landed = mbar_wait(&sfull[slot], sphase, abort_flag) &&
                            mbar_wait(&tfull[buf], bphase, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, landed)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (active) {
          const float* ss = s_scale + slot * kSets * 128 + r;
          const uint64_t p0 = pack2(ss[SWIGLU || kSets == 1 ? 0 : g * 128]),
                         p1 = SWIGLU ? pack2(ss[128]) : p0;
          const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * NT;
          // SWIGLU: columns 64 g.. of the gate, then of the up half
          auto col = [&](int c) {
            return SWIGLU ? (c < 2 ? 0 : 128) + g * 64 + (c & 1) * 32 : g * kCols + c * 32;
          };
          // the next 32 columns are read while these are added
          uint32_t v[2][32];
          tmem_ld32(t0 + col(0), v[0]);
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            tmem_ld_wait();
            reg_fence32(v[c & 1]);
            if (c + 1 < kCols / 32) tmem_ld32(t0 + col(c + 1), v[(c + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              fma2(acc[c * 16 + i], v[c & 1][2 * i], v[c & 1][2 * i + 1],
                   SWIGLU && c >= 2 ? p1 : p0);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&tempty[buf]);
          mbar_arrive(&sempty[slot]);
        }
        if (++buf == kBufs) {
          buf = 0;
          bphase ^= 1u;
        }
        if (++slot == kBsScaleSlots) {
          slot = 0;
          sphase ^= 1u;
        }
      }
      if (!ok) break;
      if constexpr (SPLIT) {
        // this rank's partial sums; joined below
        if (live) {
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            const int col = SWIGLU ? (c < 2 ? 0 : 128) + g * 64 + (c & 1) * 32 : g * kCols + c * 32;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 lo = unpack2(acc[c * 16 + 2 * i]), hi = unpack2(acc[c * 16 + 2 * i + 1]);
              *reinterpret_cast<float4*>(s_part + r * (NT + 4) + col + 4 * i) =
                  make_float4(lo.x, lo.y, hi.x, hi.y);
            }
          }
        }
      } else if constexpr (SWIGLU) {
        // h of 64 columns; the block's maximum is over both warpgroups
        float h[64];
        uint32_t amax = 0u;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 gg = unpack2(acc[i]), uu = unpack2(acc[32 + i]);
          h[2 * i] = swiglu(gg.x, uu.x, p.clamp);
          h[2 * i + 1] = swiglu(gg.y, uu.y, p.clamp);
          amax = max(amax, max(abs_bits(h[2 * i]), abs_bits(h[2 * i + 1])));
        }
        s_amax[g * 128 + r] = amax;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        amax = max(s_amax[r], s_amax[128 + r]);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (live) {
          const BlockQuant bq(amax);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = bq.code4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
          uint4* d = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + row * p.ldo +
                                              it.tile * 128 + g * 64);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            d[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          if (g == 0) p.h_scales[it.tile * p.ld_hs + row] = bq.scale;
        }
      } else if (live) {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.out) + row * p.ldo;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c)
          store_bf16_32(d, it.tile * NT + g * kCols + c * 32, p.N, p.out_vec, acc + c * 16);
      }
    }
    if (!ok && lane == 0) report_status(&g_blockscale_status, kStatusTimeout);
    if constexpr (SPLIT) {
      // Join: epilogue warp w of rank k takes row groups 8 k + w, ... and adds
      // the ranks' partial sums in rank order.
      __syncwarp();
      cluster_sync();
      if (first < total) {
        const BsItem it = map_bs_item(tab, p.E, p.tiles, first);
        constexpr int kGroups = SWIGLU ? 1 : NT / 128;  // 128-column groups of a row
        for (int u = rank * 8 + warp - kBsEpiWarp0; u < it.rows * kGroups; u += 8 * p.split) {
          const int r = u / kGroups, c = (u % kGroups) * 128 + lane * 4;
          const int64_t row = it.row0 + r;
          float s[SWIGLU ? 8 : 4];
#pragma unroll
          for (int i = 0; i < (SWIGLU ? 8 : 4); ++i) s[i] = 0.0f;
          for (int k = 0; k < p.split; ++k)
#pragma unroll
            for (int i = 0; i < (SWIGLU ? 8 : 4); i += 4) {
              const float4 v = ld_cluster_f4(smem_u32(s_part + r * (NT + 4) + c + 32 * i), k);
              s[i] += v.x, s[i + 1] += v.y, s[i + 2] += v.z, s[i + 3] += v.w;
            }
          if constexpr (SWIGLU) {
            float h[4];
            uint32_t amax = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              h[i] = swiglu(s[i], s[4 + i], p.clamp);
              amax = max(amax, abs_bits(h[i]));
            }
            const BlockQuant bq(__reduce_max_sync(0xFFFFFFFFu, amax));
            reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row * p.ldo +
                                        it.tile * 128)[lane] = bq.code4(h[0], h[1], h[2], h[3]);
            if (lane == 0) p.h_scales[it.tile * p.ld_hs + row] = bq.scale;
          } else {
            __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.out) + row * p.ldo;
            const int n0 = it.tile * NT + c;
            if (p.out_vec && n0 + 4 <= p.N) {
              const __nv_bfloat162 lo = __floats2bfloat162_rn(s[0], s[1]),
                                   hi = __floats2bfloat162_rn(s[2], s[3]);
              *reinterpret_cast<uint2*>(d + n0) =
                  make_uint2(reinterpret_cast<const uint32_t&>(lo),
                             reinterpret_cast<const uint32_t&>(hi));
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n0 + i < p.N) d[n0 + i] = __float2bfloat16_rn(s[i]);
            }
          }
        }
      }
      cluster_sync();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- host
using Kernel = void (*)(BlockscaleMaps, BlockscaleArgs);

template <int NT, bool SWIGLU, bool TRANS, bool SPLIT>
constexpr int extra_smem() {
  return (SPLIT ? kBsSplitRows * (NT + 4) * 4 : SWIGLU ? 1024 : 0) + kBsScaleSlots * NT * 4 +
         (2 * kBsMaxStages + 2 * kBsScaleSlots + 9) * 8 + 8;
}

template <int NT, bool SWIGLU, bool TRANS, bool SPLIT>
cudaError_t launch_bs(const BlockscaleMaps& maps, BlockscaleArgs p, int grid, bool pdl,
                      cudaStream_t s) {
  auto k = blockscale_gemm_kernel<NT, SWIGLU, TRANS, SPLIT>;
  // Once per instance: the shared-memory limit, and that the launch
  // allocation covers the register split (setmaxnreg would wait forever).
  static const cudaError_t ready = [&] {
    cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBsSmemLimit);
    cudaFuncAttributes fa{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, k);
    if (e == cudaSuccess && fa.numRegs != kBsLaunchRegs) e = cudaErrorInvalidConfiguration;
    return e;
  }();
  if (ready != cudaSuccess) return ready;
  const int stage = p.a_rows * 128 + NT * 128;
  const int fixed = 1024 + extra_smem<NT, SWIGLU, TRANS, SPLIT>() + (3 * p.E + 1) * 4;
  p.stages = std::min(kBsMaxStages, (kBsSmemLimit - fixed) / stage);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kBsThreads);
  cfg.dynamicSmemBytes = fixed + p.stages * stage;
  cfg.stream = s;
  cfg.attrs = attr;
  if (pdl) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (SPLIT) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = p.split;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, k, maps, p);
}

}  // namespace

// See internal.h.
cudaError_t launch_blockscale(const BlockscaleMaps& maps, BlockscaleArgs p, bool swiglu,
                              bool transpose, bool pdl, int sms, cudaStream_t s) {
  const int64_t chunks =
      p.E == 1 ? (p.M + 127) / 128 : std::min<int64_t>(p.E, p.M) + p.M / 128;
  p.a_rows = p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
  const bool wide = swiglu || chunks * ((p.N + 255) / 256) >= sms;
  const int nt = wide ? 256 : 128;
  p.tiles = swiglu ? p.N / 256 : (p.N + nt - 1) / nt;
  const int64_t items = chunks * p.tiles;
  if (items > INT32_MAX) return cudaErrorInvalidValue;
  p.split = 1;
  if (p.E == 1 && p.M <= kBsSplitRows)
    while (p.split < 8 && items * p.split * 2 <= sms && p.split * 2 <= (p.K + 127) / 128)
      p.split *= 2;
  if (p.split > 1) {
    const int grid = static_cast<int>(items) * p.split;
    if (swiglu) return launch_bs<256, true, false, true>(maps, p, grid, pdl, s);
    return transpose ? launch_bs<128, false, true, true>(maps, p, grid, pdl, s)
                     : launch_bs<128, false, false, true>(maps, p, grid, pdl, s);
  }
  const int grid = static_cast<int>(std::min<int64_t>(sms, items));
  if (swiglu) return launch_bs<256, true, false, false>(maps, p, grid, pdl, s);
  if (wide)
    return transpose ? launch_bs<256, false, true, false>(maps, p, grid, pdl, s)
                     : launch_bs<256, false, false, false>(maps, p, grid, pdl, s);
  return transpose ? launch_bs<128, false, true, false>(maps, p, grid, pdl, s)
                   : launch_bs<128, false, false, false>(maps, p, grid, pdl, s);
}

cudaError_t blockscale_status(int* code) {
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_blockscale_status, sizeof(int));
  if (e == cudaSuccess && *code)
    e = cudaMemcpyToSymbol(g_blockscale_status, &zero, sizeof(int));
  return e;
}

}  // namespace moe
