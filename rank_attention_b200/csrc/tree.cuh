// Drafted trees over the shared caches: what lora_attn_tree's kernels and
// lora_qk_norm_rope share.
//
// Tree t of sequence s has `nodes` slots.  Node j (j < tree_len) sits in cache
// row C + t * nodes + j, C = kv_len[s] the committed length, at position
// C + depth(j), depth(j) its number of ancestors; it sees rows [0, C), its
// ancestors and itself.  parent[j] in [-1, j): -1 hangs below the context.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace la {

constexpr int kTreeMaxNodes = 64;   // one 64-bit word of ancestors a node

struct TreeParams {
  const int32_t* parent;     // [n_seqs][n_trees][nodes], or null: node j's parent is j - 1
  const int32_t* tree_len;   // [n_seqs][n_trees], or null: all nodes
  int n_trees;               // 1 (one tree shared by the agents) or n_agents (one each)
  int nodes;
};

constexpr int kDevKvLen = 1, kDevPipeWait = 2, kDevTree = 8;   // bits of the device error word

// One warp: every node's ancestors (itself included) as a 64-bit mask, by
// pointer doubling over shuffles: after k rounds a node holds its nearest
// 2^k - 1 ancestors, and six rounds cover 64 nodes.  Lane l keeps nodes l and
// l + 32 of the tree's n slots (read without waiting for m) and writes
// mask[node]; nodes at or past m get 0.  False (in every lane) if one of the m
// parents is out of range.
__device__ __forceinline__ bool tree_masks_warp(const int32_t* parent, int n, int m, uint64_t* mask) {
  const int lane = threadIdx.x & 31;
  int an[2];
  uint64_t mk[2];
  bool bad = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 32 * h;
    an[h] = parent && j < n ? parent[j] : j - 1;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 32 * h;
    mk[h] = 0;
    if (j >= m) {
      an[h] = -1;
    } else {
      mk[h] = 1ull << j;
      if (an[h] < -1 || an[h] >= j) {
        bad = true;
        an[h] = -1;
      }
    }
  }
  if (__any_sync(0xffffffffu, bad)) return false;
#pragma unroll
  for (int k = 0; k < 6; ++k) {
    uint64_t m2[2];
    int a2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int src = an[h] & 31;
      const uint64_t mlo = __shfl_sync(0xffffffffu, mk[0], src), mhi = __shfl_sync(0xffffffffu, mk[1], src);
      const int alo = __shfl_sync(0xffffffffu, an[0], src), ahi = __shfl_sync(0xffffffffu, an[1], src);
      const bool hi = an[h] >= 32;
      m2[h] = an[h] < 0 ? 0 : (hi ? mhi : mlo);
      a2[h] = an[h] < 0 ? -1 : (hi ? ahi : alo);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mk[h] |= m2[h];
      an[h] = a2[h];
    }
  }
  mask[lane] = mk[0];
  mask[lane + 32] = mk[1];
  return true;
}

}  // namespace la
