// Ragged segments of tokens grouped by agent: what the grouped-delta kernels share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "lora_attn.h"

namespace la {

constexpr int kDevSegment = 16;   // bit of the device error word

struct GroupedParams {
  const void* x;
  int64_t ldx;
  const void* y;
  int64_t ldy;
  void* out;
  int64_t ldo;
  const void* A;
  int64_t a_agent;          // elements between agents' A; 0: one A
  const void* B;
  const int32_t* seg_start;   // [n_segs + 1]
  const int32_t* seg_agent;   // [n_segs]
  int n_segs, n_agents, n_tokens, hidden, n_out, r;
  float s;
  int* err;
};

// Rows per tile: bf16 (tensor cores); fp32 where segments have 64 rows on average (their
// sizes are known only on the device), and fp32 otherwise
constexpr int kRowsTC = 128, kRowsWide = 64, kRowsNarrow = 16;
inline int grouped_tile_rows(bool bf16, int n_tokens, int n_segs) {
  if (bf16) return kRowsTC;
  return n_tokens >= (int64_t)kRowsWide * n_segs ? kRowsWide : kRowsNarrow;
}
// Tiles a launch has to offer: every segment ends in at most one short tile
inline int64_t grouped_tiles(int n_tokens, int n_segs, int rows) {
  return ((int64_t)n_tokens + rows - 1) / rows + n_segs;
}

// One row tile of a segment.  rows == 0: no such tile.
struct SegTile {
  int row0, rows, agent, bad;
};

// One warp: the tile-th tile of tm rows over all segments (each segment's rows
// cut into its own tiles), and whether any segment is out of range (the same
// verdict in every CTA, since each looks at all of them).
__device__ __forceinline__ SegTile find_seg_tile(const GroupedParams& p, int tile, int tm) {
  const int lane = threadIdx.x & 31;
  SegTile t = {0, 0, -1, 0};
  int base = 0;   // tiles of the segments before this group of 32
  for (int s0 = 0; s0 < p.n_segs; s0 += 32) {
    const int s = s0 + lane;
    int lo = 0, n = 0, a = -1;
    bool bad = false;
    if (s < p.n_segs) {
      lo = p.seg_start[s];
      const int hi = p.seg_start[s + 1];
      a = p.seg_agent[s];
      bad = lo < 0 || hi < lo || hi > p.n_tokens || a < -1 || a >= p.n_agents;
      n = bad ? 0 : hi - lo;
    }
    if (__any_sync(0xffffffffu, bad)) t.bad = 1;
    const int mine = (n + tm - 1) / tm;
    int incl = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, k);
      if (lane >= k) incl += v;
    }
    const int first = base + incl - mine;
    const uint32_t own = __ballot_sync(0xffffffffu, tile >= first && tile < first + mine);
    if (own) {
      const int src = __ffs(own) - 1;
      const int row = __shfl_sync(0xffffffffu, lo + (tile - first) * tm, src);
      const int left = __shfl_sync(0xffffffffu, n - (tile - first) * tm, src);
      t.row0 = row;
      t.rows = min(tm, left);
      t.agent = __shfl_sync(0xffffffffu, a, src);
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return t;
}

}  // namespace la
