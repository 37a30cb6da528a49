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
// fused multiply-add per output and block, two outputs to an instruction.
//
// A buffer's turn is an MMA, the hand-off to the epilogue, its reads and the
// hand-off back, about 600 cycles besides the work.  So TMEM holds four buffers
// of 128 columns, and the epilogue hands a buffer back as soon as it has read
// it.  An issuing warp stays whole and elects a thread for each group of MMAs:
// the same code under `lane == 0` spent 631 cycles on a block, longer than the
// tensor pipe's 512.  For the same reason the epilogue's waits branch on votes
// and its arrivals are predicated.
//
// Structure: one persistent CTA per SM walks the items (expert, tile of NT
// weight rows, chunk of at most 128 rows), expert-major, then tile, then
// chunk, so that CTAs running together share a weight tile in L2.  Warp 0
// (one thread) fills a ring of stages by TMA: 128 columns of the chunk's
// rows (box height 16 / 32 / 64 / 128, so short chunks pull no padding) and
// of the NT weight rows.  Of a tile of 256 rows each half is a product of its
// own: warp 1 issues the first half's MMAs and warp 3 the second's, into two
// buffers each, read by one epilogue warpgroup each (warps 4-7 and 8-11; warp
// w reads TMEM lanes 32 (w % 4)..).  A tile of 128 has one issuer and all four
// buffers, and each warpgroup reads half of the columns.  Warp 2 runs ahead
// through the same blocks and leaves the product of the scales of every row,
// four blocks at a time, in a ring in shared memory.
//
// Full chunks come in pairs (PAIR): a cluster of two CTAs shares MMAs of 256
// rows x 128 columns (cta_group::2), each CTA loading its own 128 rows and
// half of the weight tile.  A single CTA's 128 x 256 block moves 48 KB into
// shared memory and reads 64 KB of operands back out (the rows once for each
// half), 875 cycles at 128 bytes a cycle against 512 of MMA; in a pair it is
// 32 and 48 KB, 640 cycles.
//
// Small products of one matrix (QUANT): the CTA's warps but the producer first
// quantise the bf16 activations of its rows and its part of the reduction
// into shared memory, in the swizzled order the MMAs expect, while the first
// weight tiles are on their way.  Every CTA does so for itself, but there is
// no kernel before this one and no workspace, which is most of such a call's
// time.
//
// With the weights transposed (input gradient) the reduction runs along the
// stored rows: the tile is 128 rows of 128 bytes of output columns, an
// MN-major operand for the tensor cores; nothing is copied or re-laid out.
//
// Few rows leave most SMs without an item; there a cluster of two to eight
// CTAs splits the reduction of each item and joins its fp32 partial sums
// through distributed shared memory, in rank order, so the result does not
// depend on timing.
//
// What bounds it: with many rows, the hand-offs between the issuers and the
// warps that read TMEM (8192 x 4096 x 7168: 183 us, 2620 TFLOP/s; a build
// without the epilogue's sums took 163).  Nothing is saturated: per active
// cycle the tensor pipe is busy 57 %, shared memory 72 %, the TMEM ports 62 %
// (4096 x 4096 x 7168).  With few rows per expert, the weights' bytes (64
// tokens over 64 experts of 44 MB: 420 us, 6.7 TB/s).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

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
constexpr int kBsAhead = 4;       // blocks whose scales are passed on together, a float4 per row
constexpr int kBsGroups = 2;      // such groups in the scale ring
constexpr int kBsSmemLimit = 232448;
// Most rows of a SwiGLU product that is split: the partial sums lie beside the
// ring of stages.  A whole call of one expert, split against not, 7168 -> 2048:
// 32 rows 30.4 us against 40.4, 64 rows 32.9 against 41, 100 rows 46.1 against
// 41.7 (two stages are left).
constexpr int kBsSplitSwigluRows = 64;
// Most rows in all of several experts whose products are split: a token's or
// two (a whole call of one token, 64 x (2048, 1024), top-6: 20.9 us against
// 24.6 in one piece; 64 x (7168, 2048), top-2: 28.2 against 42.8).  With more
// rows a row's sums keep their order whatever the other experts' number.
constexpr int kBsSplitGroupRows = 16;

__device__ int g_blockscale_status;

// kind::f8f6f4, e4m3 x e4m3, f32 accumulator; transpose_b: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool transpose_b) {
  return (1u << 4) | (static_cast<uint32_t>(transpose_b) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// PAIR: issued by rank 0 for both CTAs of the cluster (A rows and B rows half
// from each), else for this CTA alone.
template <bool PAIR>
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accum) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}

// (An MN-major operand tile, staged by TMA with the 128-byte swizzle, has one
// row of 128 bytes per reduction index and 8-row atoms of 1024 bytes stacked
// along the reduction: desc_sw128 describes it too, with the transpose bit of
// the instruction descriptor set.)

// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait by a whole warp, with its branches on votes: the lanes stay
// together without the compiler's reconvergence points, which made a wait on
// a phase that had completed cost 62 cycles instead of 36 in eight warps (and
// 176 when one lane waited for the others).
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity,
                                               volatile int* abort) {
  uint32_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    if ((i & 127u) == 0) {
      // (the low half of the timer: its differences are good for 4 s)
      uint32_t now;
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
      if (i == 0) t0 = now;
      if (__any_sync(0xFFFFFFFFu, *abort != 0 || now - t0 > static_cast<uint32_t>(kWaitTimeoutNs))) {
        *abort = 1;
        return false;
      }
    }
  }
}

// One thread of a whole warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t x, int32_t y,
                                                 int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
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

// Arrive, where `on`, on a barrier at a shared::cluster address (an address
// of this CTA's own shared memory is one; see also mbar_arrive_cluster): a
// predicated instruction, no branch.
__device__ __forceinline__ void mbar_arrive_if(bool on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(static_cast<uint32_t>(on))
      : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t saddr, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(mapa_shared(saddr, rank))
               : "memory");
  return v;
}

// Rows of scales (one per activation row) for QUANT's resident blocks: the
// epilogue reads them kBsAhead at a time.
__host__ __device__ constexpr int scale_rows(int resident) {
  return (resident + kBsAhead - 1) / kBsAhead * kBsAhead;
}

struct BsItem {
  int e, tile, row0, rows;
};

// Chunk table in shared memory: exclusive counts of the items' chunk groups
// (`group` chunks of 128 rows each), and the first and last row of every
// expert.  The offsets are clamped into [0, M] and each is raised to the
// largest before it, so no row has two experts and the host's bound on the
// number of items holds whatever the offsets are: the split products have one
// item per cluster and no more.
struct BsTable {
  int* chunk_off;  // [E + 1]
  int* start;      // [E]
  int* end;        // [E]
};

// group: chunks per item (a pair's two; the second may have no rows), rank:
// the chunk of the item that is wanted.  e: the expert of this or an earlier
// item, moved up to the item's: a CTA's items come in expert order, so the
// search is a step or two of the way.
__device__ __forceinline__ BsItem map_bs_item(const BsTable& t, int tiles, int item, int group,
                                              int rank, int& e) {
  while (t.chunk_off[e + 1] * tiles <= item) ++e;
  const int chunks = t.chunk_off[e + 1] - t.chunk_off[e];
  const int local = item - t.chunk_off[e] * tiles;
  BsItem it;
  it.e = e;
  it.tile = local / chunks;
  it.row0 = t.start[e] + (local - it.tile * chunks) * (128 * group) + rank * 128;
  it.rows = min(128, t.end[e] - it.row0);
  return it;
}

// One warp fills the table, 32 experts at a time; all offsets are on their way
// before the first is used.
__device__ __forceinline__ void fill_bs_table(const BlockscaleArgs& p, const BsTable& t, int group,
                                              int lane) {
  if (!p.offsets) {
    if (lane == 0) {
      t.start[0] = 0;
      t.end[0] = p.M;
      t.chunk_off[0] = 0;
      t.chunk_off[1] = (p.M + 128 * group - 1) / (128 * group);
    }
    return;
  }
  constexpr int kPer = kMaxExperts / 32;
  const int per_item = 128 * group;
  int first[kPer], last[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = 32 * i + lane;
    first[i] = e < p.E ? p.offsets[e] : 0;
    last[i] = e < p.E ? p.offsets[e + 1] : 0;
  }
  bool falls = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) falls |= last[i] < first[i];
  if (__any_sync(0xFFFFFFFFu, falls)) {
    int top = 0;
    for (int i = 0; i < kPer && 32 * i < p.E; ++i) {
      const int e = 32 * i + lane;
      int m = max(e < p.E ? p.offsets[e] : 0, top);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, m, off);
        if (lane >= off) m = max(m, o);
      }
      if (e < p.E) t.start[e] = m;
      top = __shfl_sync(0xFFFFFFFFu, m, 31);
    }
    // (every lane reads back what it wrote itself)
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (32 * i + lane < p.E) first[i] = t.start[32 * i + lane];
  }
  int run = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (32 * i >= p.E) break;
    const int e = 32 * i + lane;
    const int r0 = min(max(first[i], 0), p.M), r1 = min(max(last[i], r0), p.M);
    const int chunks = e < p.E ? (r1 - r0 + per_item - 1) / per_item : 0;
    int inc = chunks;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
      if (lane >= off) inc += o;
    }
    if (e < p.E) {
      t.start[e] = r0;
      t.end[e] = r1;
      t.chunk_off[e] = run + inc - chunks;
    }
    run += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
  if (lane == 0) t.chunk_off[p.E] = run;
}

// acc += s v for 32 columns.
__device__ __forceinline__ void add_scaled(float* acc, const uint32_t (&v)[32], float s) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 t = __ffma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])),
                                make_float2(s, s), make_float2(acc[i], acc[i + 1]));
    acc[i] = t.x;
    acc[i + 1] = t.y;
  }
}

// bf16 of 32 consecutive fp32 columns n0 .. n0 + 31 of the warp's 32 rows
// (lane = row; row0 the first one's, rows how many are real; n0 + 32 may pass
// N).  Whole sectors where the rows start on one (vec).  Else the block is
// turned in `turn` (32 x kTurnWords words of shared memory, the warp's own),
// so that a store covers consecutive columns of one row instead of one column
// of 32 rows.
constexpr int kTurnWords = 17;  // per row of 32 bf16: odd, so columns differ in bank
__device__ __forceinline__ void store_bf16_32(__nv_bfloat16* row0, int64_t ldo, int rows, int lane,
                                              int n0, int N, bool vec, uint32_t* turn,
                                              const float* acc) {
  uint32_t v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
    v[i] = reinterpret_cast<const uint32_t&>(b);
  }
  if (vec && n0 + 32 <= N) {
    if (lane < rows) {
      // (32 bytes each: whole sectors)
      __nv_bfloat16* d = row0 + lane * ldo + n0;
      st_global_v8(d, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
      st_global_v8(d + 16, v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i) turn[lane * kTurnWords + i] = v[i];
  __syncwarp();
  if (n0 + lane < N) {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(turn) + lane;
    uint16_t* d = reinterpret_cast<uint16_t*>(row0) + n0 + lane;
    for (int r = 0; r < min(rows, 32); ++r) d[r * ldo] = src[r * 2 * kTurnWords];
  }
}

// v in [-limit, limit]; a NaN stays one (fminf and fmaxf would drop it).
__device__ __forceinline__ float clamp_to(float v, float limit) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(-limit));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(limit));
  return v;
}

__device__ __forceinline__ float swiglu(float g, float u, float clamp) {
  g = clamp_to(g, clamp);
  u = clamp_to(u, clamp);
  // e^-g by the hardware's power of two, off by two ulp and |g| 2^-24 of itself,
  // and an approximate quotient of two ulp: as near as the sums of the product
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  return __fdividef(g, 1.0f + e) * u;
}

// NT: weight rows per item.  SWIGLU: the tile is 128 gate rows and the 128
// up rows of the same columns (NT = 256).  SPLIT: the grid is clusters of
// args.split CTAs, one item each at most.
// PAIR: the grid is clusters of two CTAs that share each item (NT = 256).
// QUANT: the activations are args.x, and every CTA (or split cluster) has one
// item (NT = 128, one expert).
template <int NT, bool SWIGLU, bool TRANS, bool SPLIT, bool PAIR, bool QUANT>
__global__ void __launch_bounds__(kBsThreads, 1)
    blockscale_gemm_kernel(const __grid_constant__ BlockscaleMaps maps,
                           const __grid_constant__ BlockscaleArgs p) {
  constexpr int kHalves = NT / 128;  // 128-column halves of the tile
  constexpr int kBufs = 4;           // TMEM buffers of 128 columns, used in turn
  constexpr int kSets = kHalves;     // weight blocks of the tile: its scale sets
  constexpr int kCols = NT / 2;      // columns per epilogue thread
  constexpr int kGroup = PAIR ? 2 : 1;
  constexpr int kBBytes = NT / kGroup * 128;  // this CTA's part of the weight tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // QUANT: the resident activations, then the ring of weight tiles
  const int a_bytes = p.a_rows * 128;
  const int stage_bytes = (QUANT ? 0 : a_bytes) + kBBytes;
  const int b_off = QUANT ? 0 : a_bytes;
  const int stages = p.stages;
  uint8_t* const s_a = smem;
  if constexpr (QUANT) smem += p.resident * a_bytes;
  float* s_part = reinterpret_cast<float*>(smem + stages * stage_bytes);  // SPLIT: [a_rows][NT + 4]
  uint32_t* s_amax = reinterpret_cast<uint32_t*>(s_part);                 // SWIGLU: [2][128]
  // [group][weight block of the tile][row][block] (QUANT: [block][row])
  float* s_scale = s_part + (SPLIT    ? p.a_rows * (NT + 4)
                             : SWIGLU ? 256
                                      : 8 * 32 * kTurnWords);
  const int scale_words =
      QUANT ? scale_rows(p.resident) * p.a_rows : kBsGroups * kBsAhead * kSets * 128;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_scale + scale_words);
  uint64_t* empty = full + kBsMaxStages;
  uint64_t* tfull = empty + kBsMaxStages;
  uint64_t* tempty = tfull + 4;
  uint64_t* sfull = tempty + 4;
  uint64_t* sempty = sfull + kBsGroups;
  uint64_t* drained = sempty + kBsGroups;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_tab = reinterpret_cast<int*>(tmem_holder + 2);
  const BsTable tab{s_tab, s_tab + p.E + 1, s_tab + 2 * p.E + 1};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // (not early: below)
  if (p.early) pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kHalves);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      // the epilogue warps that read it (of both CTAs)
      mbar_init(&tempty[b], 8 / kHalves * kGroup);
    }
    for (int i = 0; i < kBsGroups; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], 8);
    }
    mbar_init(drained, kHalves);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // The launch may overlap the kernel before it.  Early: that is the library's
  // own, which writes the activations and their scales but no offsets or
  // weights, and which has let this one start only when all before it was
  // over.  Else nothing is read, no TMEM held that the other could be waiting
  // for, and no kernel after this one started, before it is over.  (What it
  // may have written is not read with __ldg, which is for memory that stays as
  // it is.)
  if (!p.early) {
    pdl_wait();
    pdl_launch_dependents();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_holder, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, 512);
      tmem_relinquish();
    }
  }
  if (warp == 2) fill_bs_table(p, tab, kGroup, lane);
  tc_fence_before();
  __syncthreads();
  // both CTAs' barriers are initialised before either arrives on the other's
  if constexpr (PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int kb_all = (p.K + 127) / 128;
  const int rank = SPLIT || PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int kb0 = SPLIT ? kb_all * rank / p.split : 0;
  const int kb1 = SPLIT ? kb_all * (rank + 1) / p.split : kb_all;
  const int first = blockIdx.x / (SPLIT ? p.split : kGroup);
  const int step = gridDim.x / (SPLIT ? p.split : kGroup);
  const int total = tab.chunk_off[p.E] * p.tiles;
  int expert = 0;  // of the role's latest item
  auto map_item = [&](int item) {
    return map_bs_item(tab, p.tiles, item, kGroup, PAIR ? rank : 0, expert);
  };

  if (QUANT && warp > 0 && first < total) {
    // Eight lanes per (row, block), 16 columns each: kUnits of those at a time,
    // three times over (all loads before the first is used) while more than
    // one time is left.
    constexpr int kUnits = (kBsThreads - 32) / 8;
    const BsItem it = map_item(first);
    const int units = it.rows * (kb1 - kb0), chunk = lane & 7;
    const float* sw = p.w_scales + it.tile * p.w_stride_n;
    // u / rows by a multiplication (exact: u and rows stay far below 2^16)
    const uint32_t inv = 0xFFFFFFFFu / static_cast<uint32_t>(it.rows) + 1u;
    auto block_of = [&](int u) {
      return it.rows == 1 ? u : static_cast<int>(__umulhi(static_cast<uint32_t>(u), inv));
    };
    auto quantise = [&](auto batch, int u0) {
      constexpr int N = decltype(batch)::value;
      uint32_t v[N][8];
      float w[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int u = u0 + k * kUnits;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = 0u;
        w[k] = 0.0f;
        if (u >= units) continue;
        const int block = block_of(u), r = u - block * it.rows, kb = kb0 + block;
        const int c0 = kb * 128 + chunk * 16;
        const __nv_bfloat16* src = p.x + (it.row0 + r) * p.ldx + c0;
        w[k] = sw[kb * p.w_stride_k];
        if (p.x_vec && c0 + 16 <= p.K) {
          const uint4 lo = *reinterpret_cast<const uint4*>(src),
                      hi = *reinterpret_cast<const uint4*>(src + 8);
          v[k][0] = lo.x, v[k][1] = lo.y, v[k][2] = lo.z, v[k][3] = lo.w;
          v[k][4] = hi.x, v[k][5] = hi.y, v[k][6] = hi.z, v[k][7] = hi.w;
        } else if (c0 < p.K) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t lo = 0u, hi = 0u;
            if (c0 + 2 * i < p.K) lo = reinterpret_cast<const uint16_t*>(src)[2 * i];
            if (c0 + 2 * i + 1 < p.K) hi = reinterpret_cast<const uint16_t*>(src)[2 * i + 1];
            v[k][i] = lo | (hi << 16);
          }
        }
      }
      uint4 codes[N];
      float scale[N];
      quantize_16(v, codes, scale);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int u = u0 + k * kUnits;
        if (u < units) {
          const int block = block_of(u), r = u - block * it.rows;
          // row r's 16-byte chunk c lies at chunk c ^ (r % 8)
          *reinterpret_cast<uint4*>(s_a + block * a_bytes + r * 128 + ((chunk ^ (r & 7)) << 4)) =
              codes[k];
          if (chunk == 0) s_scale[block * p.a_rows + r] = scale[k] * w[k];
        }
      }
    };
    const int unit = (static_cast<int>(threadIdx.x) - 32) / 8;
    int done = 0;
    for (; done + kUnits < units; done += 3 * kUnits)
      quantise(std::integral_constant<int, 3>(), done + unit);
    if (done < units) quantise(std::integral_constant<int, 1>(), done + unit);
    // the codes are read by the tensor core, the scales by the epilogue
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("bar.sync 5, %0;" ::"n"(kBsThreads - 32) : "memory");
  }

  if (warp < kBsEpiWarp0) {
    if constexpr (!QUANT) regs_release<kBsLeanRegs>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------ TMA producer
      const uint64_t once = l2_policy_evict_first(), reused = l2_policy_evict_normal();
      int stage = 0, slots = 0;
      uint32_t phase = 0;
      bool ok = true;
      // (one expert: the box that all its chunks take, the last one short)
      auto box_of = [&](int rows) {
        rows = p.E == 1 ? p.a_rows : rows;
        return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3;
      };
      auto a_size = [&](int rows) { return rows > 0 ? (16u << box_of(rows)) * 128u : 0u; };
      const uint32_t full_lead = PAIR ? mapa_shared(smem_u32(full), 0) : 0u;
      // announce a stage's bytes (a pair's on rank 0) and load its weight tile
      auto load_w = [&](const BsItem& it, int st, int kb) {
        // weights of an expert with one chunk are read once
        const uint64_t policy =
            tab.chunk_off[it.e + 1] - tab.chunk_off[it.e] > 1 ? reused : once;
        uint8_t* sb = smem + st * stage_bytes + b_off;
        if constexpr (PAIR) {
          if (rank == 0)
            mbar_arrive_expect_tx(&full[st],
                                  a_size(it.rows) + a_size(min(128, tab.end[it.e] - it.row0 - 128)) +
                                      NT * 128u);
        } else {
          mbar_arrive_expect_tx(&full[st], (QUANT ? 0u : a_size(it.rows)) + NT * 128u);
        }
        // A single CTA's half h is tile columns 128 h..; a pair's CTA `rank`
        // supplies tile columns 128 rank.., 64 of them to each half.  SWIGLU:
        // a half is 64 gate columns, then the up columns that go with them
        // (of a pair, rank 0 has the gate rows and rank 1 the up rows).
        constexpr int kBoxRows = SWIGLU ? 64 : 128;
#pragma unroll
        for (int i = 0; i < kBBytes / 128 / kBoxRows; ++i) {
          int n0;
          if constexpr (SWIGLU)
            n0 = it.tile * 128 + (PAIR ? i * 64 + rank * (p.N / 2)
                                       : (i >> 1) * 64 + (i & 1) * (p.N / 2));
          else
            n0 = it.tile * NT + (PAIR ? rank : i) * 128;
          const int x = TRANS ? n0 : kb * 128, y = TRANS ? kb * 128 : n0;
          uint8_t* d = sb + i * kBoxRows * 128;
          if constexpr (PAIR)
            tma_load_3d_pair(d, &maps.w, full_lead + st * 8, x, y, it.e, policy);
          else
            tma_load_3d_hint(d, &maps.w, &full[st], x, y, it.e, policy);
        }
      };
      int ahead = 0;  // stages of the first item whose weights are on their way
      if (p.early) {
        if (first < total) {
          const BsItem it = map_item(first);
          for (; ahead < min(stages, kb1 - kb0); ++ahead) load_w(it, ahead, kb0 + ahead);
        }
        pdl_wait();
      }
      for (int item = first; item < total && ok; item += step) {
        const BsItem it = map_item(item);
        const int box = box_of(it.rows);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (slots >= ahead) load_w(it, stage, kb);
          uint8_t* sa = smem + stage * stage_bytes;
          if constexpr (PAIR) {
            if (it.rows > 0)
              tma_load_2d_pair(sa, &maps.a[box], full_lead + stage * 8, kb * 128, it.row0, reused);
          } else if constexpr (!QUANT) {
            tma_load_2d(sa, &maps.a[box], &full[stage], kb * 128, it.row0);
          }
          ++slots;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // no copy of this thread is in flight when it leaves (a pair's complete
      // on rank 0's barriers, and neither CTA leaves before the other)
      for (int back = 1; back <= stages && back <= slots && (!PAIR || rank == 0); ++back) {
        const int idx = slots - back;
        mbar_wait(&full[idx % stages], static_cast<uint32_t>((idx / stages) & 1), nullptr);
      }
      if (!ok) report_status(&g_blockscale_status, kStatusTimeout);
    } else if ((warp == 1 || (kHalves == 2 && warp == 3)) && (!PAIR || rank == 0)) {
      // ------------------------------------------------ MMA issuers
      constexpr uint32_t idesc = idesc_e4m3(128 * kGroup, 128, TRANS);
      // 32 reduction columns are 32 bytes along a K-major row, 32 rows (4096
      // bytes) of an MN-major tile.  The second half is 128 / kGroup weight
      // rows on; of an MN-major tile as many bytes along its rows, or the
      // next 16 KB box.
      constexpr uint64_t kStepB = TRANS ? 256 : 2;
      constexpr int kHalfB = TRANS && PAIR ? 64 : 16384 / kGroup;
      const int half = warp >> 1;
      const uint64_t da0 = desc_sw128(smem_u32(QUANT ? s_a : smem));
      const uint64_t db0 = desc_sw128(smem_u32(smem) + b_off + half * kHalfB);
      int stage = 0, buf = half;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      for (int item = first; item < total && ok; item += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_warp(&full[stage], phase, abort_flag) ||
              !mbar_wait_warp(&tempty[buf], bphase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = static_cast<uint64_t>(stage * (stage_bytes >> 4));
          const uint64_t da =
              da0 + (QUANT ? static_cast<uint64_t>((kb - kb0) * (a_bytes >> 4)) : off);
          const uint64_t db = db0 + off;
          const uint32_t d = tmem + buf * 128;
          if (elect_one()) {
            mma_e4m3<PAIR>(d, da, db, idesc, 0u);
            mma_e4m3<PAIR>(d, da + 2, db + kStepB, idesc, 1u);
            mma_e4m3<PAIR>(d, da + 4, db + 2 * kStepB, idesc, 1u);
            mma_e4m3<PAIR>(d, da + 6, db + 3 * kStepB, idesc, 1u);
            if constexpr (PAIR) {
              tc_commit_pair(&tfull[buf], 3);
              tc_commit_pair(&empty[stage], 3);
            } else {
              tc_commit(&tfull[buf]);
              tc_commit(&empty[stage]);
            }
          }
          __syncwarp();
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
          if ((buf += kHalves) >= kBufs) {
            buf = half;
            bphase ^= 1u;
          }
        }
      }
      // (the same lane is elected every time: its commit covers what it issued)
      if (elect_one()) {
        if constexpr (PAIR) tc_commit_pair(drained, 3);
        else tc_commit(drained);
      }
      __syncwarp();
      if constexpr (!PAIR) mbar_wait_warp(drained, 0, abort_flag);
      if (!ok && lane == 0) report_status(&g_blockscale_status, kStatusTimeout);
    } else if (!QUANT && warp == 2) {
      // ------------------------------------------------ scales
      // Lane l takes rows l, l + 32, ..; four blocks' loads are in flight at a
      // time, and the ring lets the warp run ahead of the tensor pipe.
      if (p.early) pdl_wait();
      int item = first, kb = kb0;  // the block the loads have come to
      BsItem it{};
      float a[kBsAhead][4], w[kBsAhead][kSets];
      auto load = [&]() {
        // up to four blocks of one item
        if (kb == kb0) it = map_item(item);
        const int n = min(kBsAhead, kb1 - kb);
        const float* sa = p.a_scales + it.row0 + lane + kb * p.ld_as;
#pragma unroll
        for (int i = 0; i < kBsAhead; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            a[i][j] = i < n && lane + 32 * j < it.rows ? sa[i * p.ld_as + 32 * j] : 0.0f;
        // SWIGLU: the gate's block and the up half's; else the tile's blocks
        // (one past N has no scale of its own and is not stored)
#pragma unroll
        for (int h = 0; h < kSets; ++h) {
          const int nb = SWIGLU ? it.tile + h * (p.N / 256)
                                : min(it.tile * kSets + h, (p.N + 127) / 128 - 1);
          const float* sw = p.w_scales + it.e * p.w_blocks + nb * p.w_stride_n + kb * p.w_stride_k;
#pragma unroll
          for (int i = 0; i < kBsAhead; ++i) w[i][h] = i < n ? sw[i * p.w_stride_k] : 0.0f;
        }
        kb += n;
        if (kb == kb1) {
          kb = kb0;
          item += step;
        }
      };
      int group = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto write = [&]() {
        if (!mbar_wait_warp(&sempty[group], phase ^ 1u, abort_flag)) {
          ok = false;
          return;
        }
        float4* d = reinterpret_cast<float4*>(s_scale) + group * kSets * 128 + lane;
#pragma unroll
        for (int h = 0; h < kSets; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            d[h * 128 + 32 * j] = make_float4(a[0][j] * w[0][h], a[1][j] * w[1][h],
                                              a[2][j] * w[2][h], a[3][j] * w[3][h]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[group]);
        if (++group == kBsGroups) {
          group = 0;
          phase ^= 1u;
        }
      };
      while (item < total && kb0 < kb1 && ok) {
        load();
        write();
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
    if constexpr (!QUANT) regs_claim<kBsEpiRegs>();
    // Where warpgroup g's c-th 32 columns lie in the tile (SWIGLU: in its 128
    // gate columns, then its 128 up columns).  NT = 256: the half of its own,
    // two times 64 columns of the halves that a pair's CTAs supplied or that
    // are gate and up; NT = 128: 64 columns of the one half.
    auto tile_col = [](int c, int g) {
      return SWIGLU || PAIR ? (c >> 1) * 128 + g * 64 + (c & 1) * 32 : g * kCols + c * 32;
    };
    // ------------------------------------------------ epilogue warps
    const int q = warp & 3, g = (warp - kBsEpiWarp0) >> 2, r = q * 32 + lane;
    const uint32_t tempty_lead = PAIR ? mapa_shared(smem_u32(tempty), 0) : smem_u32(tempty);
    int buf = kHalves == 2 ? g : 0, group = 0;
    uint32_t bphase = 0, gphase = 0;
    bool ok = true;
    for (int item = first; item < total && ok; item += step) {
      // (a vote: the compiler then knows that the warp goes one way)
      const bool active = __any_sync(0xFFFFFFFFu, q * 32 < map_item(item).rows);
      // a warp whose rows are all past the chunk's only hands the buffers back
      auto hand_back = [&](int b, bool group_done) {
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(lane == 0, tempty_lead + b * 8);
        if constexpr (!QUANT)
          mbar_arrive_if(lane == 0 && group_done, smem_u32(&sempty[group]));
        if (group_done && ++group == kBsGroups) {
          group = 0;
          gphase ^= 1u;
        }
      };
      auto last_of_group = [&](int kb) {
        return ((kb + 1 - kb0) & (kBsAhead - 1)) == 0 || kb + 1 == kb1;
      };
      float acc[kCols];
      if (active && kb0 < kb1) {
        // The warp's reads and sums run on across the blocks: while 32 columns
        // are added the next 32 are read, the first of the next block before
        // the last of this one are added.
        constexpr int kParts = kCols / 32;
        constexpr bool kTwoSets = SWIGLU || PAIR;  // the second 64 columns have other scales
        const uint32_t t_lane =
            tmem + (static_cast<uint32_t>(q * 32) << 16) + (kHalves == 1 ? g * kCols : 0);
        uint32_t v[2][32];
        float4 s0, s1;  // the scales of kBsAhead blocks
        s0 = s1 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // wait for a block's buffer and scales, and read its first columns
        auto open = [&](int block, int b, uint32_t ph, bool known) {
          if ((block & (kBsAhead - 1)) == 0) {
            if constexpr (QUANT) {
              const float* ss = s_scale + block * p.a_rows + r;
              s0 = make_float4(ss[0], ss[p.a_rows], ss[2 * p.a_rows], ss[3 * p.a_rows]);
            } else {
              ok &= mbar_wait_warp(&sfull[group], gphase, abort_flag);
              const float4* ss = reinterpret_cast<const float4*>(s_scale) + group * kSets * 128 + r;
              s0 = ss[kTwoSets || kSets == 1 ? 0 : g * 128];
              if (kTwoSets) s1 = ss[128];
            }
          } else {
            // the next block's scales move to the front
            s0 = make_float4(s0.y, s0.z, s0.w, 0.0f);
            if (kTwoSets) s1 = make_float4(s1.y, s1.z, s1.w, 0.0f);
          }
          if (!known) ok &= mbar_wait_warp(&tfull[b], ph, abort_flag);
          tc_fence_after();
          tmem_ld32(t_lane + b * 128, v[0]);
        };
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
        open(0, buf, bphase, false);
        // (a wait that gave up is followed by nothing but quick ones, so the
        // loop just runs to its end)
        for (int kb = kb0; kb < kb1; ++kb) {
          const int nbuf = (buf + kHalves) & (kBufs - 1);
          const uint32_t nphase = bphase ^ (nbuf < kHalves ? 1u : 0u);
          bool next = false;
          const float c0 = s0.x, c1 = s1.x;
#pragma unroll
          for (int c = 0; c < kParts; ++c) {
            const float sc = kTwoSets && c >= 2 ? c1 : c0;
            tmem_ld_wait();
            reg_fence32(v[c & 1]);
            if (c + 1 < kParts) {
              tmem_ld32(t_lane + buf * 128 + (c + 1) * 32, v[(c + 1) & 1]);
              if (c + 2 == kParts) next = mbar_test(&tfull[nbuf], nphase);
            } else {
              hand_back(buf, last_of_group(kb));
              if (kb + 1 < kb1)
                open(kb + 1 - kb0, nbuf, nphase, __all_sync(0xFFFFFFFFu, next));
            }
            add_scaled(acc + c * 32, v[c & 1], sc);
          }
          buf = nbuf;
          bphase = nphase;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
        for (int kb = kb0; kb < kb1 && ok; ++kb) {
          if (!QUANT && ((kb - kb0) & (kBsAhead - 1)) == 0)
            ok = mbar_wait_warp(&sfull[group], gphase, abort_flag);
          ok = ok && mbar_wait_warp(&tfull[buf], bphase, abort_flag);
          if (!ok) break;
          hand_back(buf, last_of_group(kb));
          buf = (buf + kHalves) & (kBufs - 1);
          if (buf < kHalves) bphase ^= 1u;
        }
      }
      if (!ok) break;
      // (mapped again: nothing of it stays in registers during the sums)
      const BsItem it = map_item(item);
      const bool live = r < it.rows;
      const int64_t row = it.row0 + (live ? r : 0);
      if constexpr (SPLIT) {
        // this rank's partial sums; joined below
        if (live) {
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            const int col = tile_col(c, g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(s_part + r * (NT + 4) + col + 4 * i) =
                  make_float4(acc[c * 32 + 4 * i], acc[c * 32 + 4 * i + 1], acc[c * 32 + 4 * i + 2],
                              acc[c * 32 + 4 * i + 3]);
          }
        }
      } else if constexpr (SWIGLU) {
        // h of 64 columns, in place of the gate; the block's maximum is that of
        // both warps with these rows
        uint32_t amax = 0u;
        if (active) {
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            acc[i] = swiglu(acc[i], acc[64 + i], p.clamp);
            amax = max(amax, abs_bits(acc[i]));
          }
          s_amax[g * 128 + r] = amax;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
          amax = max(amax, s_amax[(1 - g) * 128 + r]);
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
        }
        if (live) {
          const BlockQuant bq(amax);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = bq.code4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
          uint4* d = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + row * p.ldo +
                                              it.tile * 128 + g * 64);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            d[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          if (g == 0) p.h_scales[it.tile * p.ld_hs + row] = bq.scale;
        }
      } else if (active) {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.out) + (it.row0 + q * 32) * p.ldo;
        uint32_t* turn = reinterpret_cast<uint32_t*>(s_part) + (warp - kBsEpiWarp0) * 32 * kTurnWords;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c)
          store_bf16_32(d, p.ldo, it.rows - q * 32, lane, it.tile * NT + tile_col(c, g), p.N,
                        p.out_vec, turn, acc + c * 32);
      }
    }
    if (!ok && lane == 0) report_status(&g_blockscale_status, kStatusTimeout);
    if constexpr (SPLIT) {
      // Join: epilogue warp w of rank k takes row groups 8 k + w, ... and adds
      // the ranks' partial sums in rank order.
      __syncwarp();
      cluster_sync();
      if (first < total) {
        const BsItem it = map_item(first);
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
  if constexpr (PAIR) {
    // every MMA of the pair has completed, and neither CTA leaves while the
    // other may still arrive on its barriers
    if (warp == 1 && lane == 0) mbar_wait(drained, 0, nullptr);
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
  } else {
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- host
using Kernel = void (*)(BlockscaleMaps, BlockscaleArgs);

// Shared memory beside the stages (and, QUANT, the resident activations).
template <int NT, bool SWIGLU, bool SPLIT, bool QUANT>
int extra_smem(int a_rows, int resident) {
  return (SPLIT    ? a_rows * (NT + 4) * 4
          : SWIGLU ? 1024
                   : 8 * 32 * kTurnWords * 4) +
         (QUANT ? scale_rows(resident) * a_rows * 4 : kBsGroups * kBsAhead * NT * 4) +
         (2 * kBsMaxStages + 2 * kBsGroups + 9) * 8 + 8;
}

template <int NT, bool SWIGLU, bool TRANS, bool SPLIT, bool PAIR = false, bool QUANT = false>
cudaError_t launch_bs(const BlockscaleMaps& maps, BlockscaleArgs p, int grid, cudaStream_t s) {
  auto k = blockscale_gemm_kernel<NT, SWIGLU, TRANS, SPLIT, PAIR, QUANT>;
  // Once per instance and device: the shared-memory limit, and that the launch
  // allocation covers the register split (setmaxnreg would wait forever).
  static OncePerDevice prepared;
  const cudaError_t ready = prepared([&] {
    cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBsSmemLimit);
    cudaFuncAttributes fa{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, k);
    if (e == cudaSuccess && !QUANT && fa.numRegs != kBsLaunchRegs) e = cudaErrorInvalidConfiguration;
    return e;
  });
  if (ready != cudaSuccess) return ready;
  const int a_bytes = p.a_rows * 128;
  const int stage = (QUANT ? 0 : a_bytes) + NT / (PAIR ? 2 : 1) * 128;
  const int fixed = 1024 + extra_smem<NT, SWIGLU, SPLIT, QUANT>(p.a_rows, p.resident) +
                    p.resident * a_bytes + (3 * p.E + 1) * 4;
  // (either eight stages of 16 KB and more or all that there is: one CTA to an
  // SM, so no CTA waits for TMEM that another of its cluster holds)
  p.stages = std::min(kBsMaxStages, (kBsSmemLimit - fixed) / stage);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kBsThreads);
  cfg.dynamicSmemBytes = fixed + p.stages * stage;
  cfg.stream = s;
  cfg.attrs = attr;
  attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  if (SPLIT || PAIR) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = PAIR ? 2 : p.split;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, k, maps, p);
}

}  // namespace

namespace {

// How a product is cut up.  An item of 256 columns takes about 1.5 times as
// long as one of 128 (4096 x 4096 x 7168: 105 us in 256s, 133 in 128s), so NT
// = 256 where its rounds of items over the SMs are at most two thirds of
// those of NT = 128 (1024 x 4096 x 7168, one round against two: 30 us, 41 in
// 128s; 512 rows, one round of either: 128).  With few rows per expert the
// weights' bytes are what takes the time, and finer items share them out more
// evenly (64 experts of 64 rows, 2048 -> 2048: a whole call 144 us in 128s,
// 147 in 256s; of 128 rows 128.5 and 128; of 512 rows 299 and 285).  Fewer
// items than half the SMs: the reduction is split over clusters of as many
// CTAs (up to eight) as still run all at once, which is fewer than SMs /
// items: 16 items in eight pieces each, 15 of 16 clusters at a time, took
// 15.1 us where four pieces take 8.5 and six 9.1 (128 x 2048 x 2048 with a
// kernel that quantises; 16 x 2048 x 7168 in one kernel: four pieces 10.9,
// six 9.5).  333 x 1001 x 2000: 8.2 us in four pieces, 10.7 in one; 512 x
// 1024 x 7168: 11.5 and 21.6.
struct Plan {
  bool wide;
  int a_rows, tiles, split, resident;
  int64_t items;  // an upper bound where the experts' rows are not known
};

Plan plan_product(int M, int N, int K, int E, bool swiglu, const BlockscaleDevice& d) {
  Plan p{};
  const int64_t chunks = E == 1 ? (M + 127) / 128 : std::min<int64_t>(E, M) + M / 128;
  const int kb = (K + 127) / 128;
  p.a_rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  auto rounds = [&](int nt) { return (chunks * ((N + nt - 1) / nt) + d.sms - 1) / d.sms; };
  p.wide = swiglu || (3 * rounds(256) <= 2 * rounds(128) && (E == 1 || M > 64 * E));
  const int nt = p.wide ? 256 : 128;
  p.tiles = swiglu ? N / 256 : (N + nt - 1) / nt;
  p.items = chunks * p.tiles;
  p.split = 1;
  if (E > 1 ? M <= kBsSplitGroupRows : !p.wide || M <= kBsSplitSwigluRows)
    for (int s = 2; s <= std::min(kBsMaxSplit, kb); ++s)
      if (p.items <= d.clusters[s] && (kb + s - 1) / s < (kb + p.split - 1) / p.split) p.split = s;
  p.resident = (kb + p.split - 1) / p.split;
  return p;
}

// Row blocks that a CTA quantises for itself at most (QUANT).  On the GPU one
// row x 7168 into 4096 takes 8.5 us where a quantising kernel and the product
// take 10.1; 16 rows 10.4 and 10.6; 48 rows x 2048 into 7168 (384 a CTA) 10.4
// and 9.1; 333 x 2000 into 1001 (512) 11.6 and 8.8; 64 x 7168 into 2048 (640)
// 13.7 and 10.5; 16 x 4096 into 14592 (512, not split) 17.1 and 15.3, one row of
// it (32) 13.9 and 15.1.  But the second launch and the workspace make a call
// 21 us for the host, against 12, so up to 512 the one kernel is the faster
// call from eager code; replayed from a graph it is up to a third slower.
constexpr int kBsQuantUnits = 512;

}  // namespace

// See internal.h.
cudaError_t blockscale_clusters(BlockscaleDevice* d) {
  auto k = blockscale_gemm_kernel<128, false, false, true, false, false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBsSmemLimit);
  for (int n = 1; n <= kBsMaxSplit && e == cudaSuccess; ++n) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(n * d->sms);
    cfg.blockDim = dim3(kBsThreads);
    cfg.dynamicSmemBytes = kBsSmemLimit;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&d->clusters[n], k, &cfg);
  }
  return e;
}

bool blockscale_quantizes(int M, int N, int K, const BlockscaleDevice& d) {
  const Plan p = plan_product(M, N, K, 1, false, d);
  // (two stages of weights beside the rows)
  const int extra = p.split > 1 ? extra_smem<128, false, true, true>(p.a_rows, p.resident)
                                : extra_smem<128, false, false, true>(p.a_rows, p.resident);
  const int64_t smem = int64_t{p.resident} * p.a_rows * 128 + 2 * 128 * 128 + 1024 + extra + 16;
  return !p.wide && std::min(M, 128) * p.resident <= kBsQuantUnits && smem <= kBsSmemLimit &&
         p.items * p.split <= d.sms;
}

cudaError_t launch_blockscale(const BlockscaleMaps& maps, BlockscaleArgs p, bool swiglu,
                              bool transpose, const BlockscaleDevice& d, cudaStream_t s) {
  const Plan plan = plan_product(p.M, p.N, p.K, p.E, swiglu, d);
  if (plan.items * plan.split > INT32_MAX) return cudaErrorInvalidValue;
  p.a_rows = plan.a_rows;
  p.tiles = plan.tiles;
  p.split = plan.split;
  p.resident = p.x ? plan.resident : 0;
  const bool wide = plan.wide;
  const int items = static_cast<int>(plan.items);
  if (p.split > 1) {
    const int grid = items * p.split;
    if (p.x)
      return transpose ? launch_bs<128, false, true, true, false, true>(maps, p, grid, s)
                       : launch_bs<128, false, false, true, false, true>(maps, p, grid, s);
    if (swiglu) return launch_bs<256, true, false, true>(maps, p, grid, s);
    return transpose ? launch_bs<128, false, true, true>(maps, p, grid, s)
                     : launch_bs<128, false, false, true>(maps, p, grid, s);
  }
  if (p.x)
    return transpose ? launch_bs<128, false, true, false, false, true>(maps, p, items, s)
                     : launch_bs<128, false, false, false, false, true>(maps, p, items, s);
  const int grid = std::min(d.sms, items);
  // (pairs for full chunks: one expert of 8192 rows, 4096 x 7168, 183 us
  // against 192; 8 experts of 1024 rows, a whole call, 93 against 100; 64 of
  // 256 rows, where the second chunk is often short, 195 against 174; averages
  // between 256 and 1024 and uneven experts were not measured)
  if (wide && p.M / 1024 >= p.E) {
    const int pairs = std::min(d.clusters[2], (items + 1) / 2);
    if (swiglu) return launch_bs<256, true, false, false, true>(maps, p, 2 * pairs, s);
    return transpose ? launch_bs<256, false, true, false, true>(maps, p, 2 * pairs, s)
                     : launch_bs<256, false, false, false, true>(maps, p, 2 * pairs, s);
  }
  if (swiglu) return launch_bs<256, true, false, false>(maps, p, grid, s);
  if (wide)
    return transpose ? launch_bs<256, false, true, false>(maps, p, grid, s)
                     : launch_bs<256, false, false, false>(maps, p, grid, s);
  return transpose ? launch_bs<128, false, true, false>(maps, p, grid, s)
                   : launch_bs<128, false, false, false>(maps, p, grid, s);
}

cudaError_t blockscale_status(int* code) {
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_blockscale_status, sizeof(int));
  if (e == cudaSuccess && *code)
    e = cudaMemcpyToSymbol(g_blockscale_status, &zero, sizeof(int));
  return e;
}

}  // namespace moe
