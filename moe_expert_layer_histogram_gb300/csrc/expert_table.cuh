// expert_table.cuh -- the rows of each expert and the items they are cut into, in
// shared memory: what the grouped products' roles walk through.
#pragma once

#include "internal.h"

namespace moe {

// Exclusive counts of the experts' items (`per_item` rows each), and the first and
// last row of every expert.  The offsets are clamped into [0, M] and each is
// raised to the largest before it, so no row has two experts and the host's bound
// on the number of items holds whatever the offsets are: the split products have
// one item per cluster and no more.
struct ExpertTable {
  int* chunk_off;  // [E + 1]
  int* start;      // [E]
  int* end;        // [E]
};

// One warp fills the table, 32 experts at a time; all offsets are on their way
// before the first is used.
template <typename Args>
__device__ __forceinline__ void fill_expert_table(const Args& p, const ExpertTable& t,
                                                  int per_item, int lane) {
  if (!p.offsets) {
    if (lane == 0) {
      t.start[0] = 0;
      t.end[0] = p.M;
      t.chunk_off[0] = 0;
      t.chunk_off[1] = (p.M + per_item - 1) / per_item;
    }
    return;
  }
  constexpr int kPer = kMaxExperts / 32;
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

}  // namespace moe
