// ssd_tree_attention.cuh -- parameters of the attention of drafted nodes, and the
// division of its work over workers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd.h"
#include "ssd_attention_dev.cuh"

namespace ssd {

constexpr int kTreeNodes = 256;

struct TreeAttnParams {
  ssd_tree_attn a;
  Divisor by_page, by_gqa;
  float scale_log2;        // |scale| * log2(e): scores in base 2
  uint32_t q_and, q_xor;   // of pairs of the queries' elements, which have the scale's sign
  int q_plain;             // they change nothing
  int wide_rows;           // rows of the output are on 32-byte boundaries
  int gqa;                 // query heads per key/value head
  int pairs;               // (node, head) pairs of a sequence's key/value head
  int block_pairs;         // of a block: 128, or fewer that are whole nodes
  int blocks;              // items of a sequence's key/value head
  int hg, sets;            // key/value heads of a set, sets
  int bg, block_sets;      // items of a head side by side, sets of those
  int side;                // CTAs of a worker: hg * bg
  int workers;
  int box_rows;            // tokens of a box of the cache (0: tiles do not come by TMA)
  int node_rows;           // rows of a box of nodes
  int q_nodes;             // nodes of a box of queries (0: copied row by row)
  int chain;               // the tree is one
  int part_rows;           // pairs of an item, in eights: rows of a partial
  float* po;               // [2 * CTAs, D / 4, part_rows, 4] sums (part_at)
  float2* pml;             // [2 * CTAs, part_rows] largest score (base 2), weight
  int2* begun;             // [CTAs] item that it began and did not end, or -1, and its partials
  int32_t* status;
  uint8_t parent[kTreeNodes];  // of node u > 0; 0 for node 0
};

// Tokens of a tile: tensor memory has room for sums of 256 dimensions and twice 64 scores.
__host__ __device__ constexpr int tree_tile(int D) { return D == 256 ? 64 : 128; }
// Blocks of 128 pairs of an item.  Two share each tile in shared memory: 32 sequences with 256
// pairs a head 129 us instead of 164 one by one (D = 64: 103 and 121), with 132 pairs 115 instead
// of 156, with 512 230 instead of 292.  The sums of D = 256 leave room for one.
__host__ __device__ constexpr int tree_blocks(int D, int pairs) {
  return D < 256 && pairs > 128 ? 2 : 1;
}

__device__ __forceinline__ void flag_bits(const TreeAttnParams& p, int bits) {
  if (p.status) atomicOr(p.status, bits);
}

// Sequence b: its tokens, clamped into range.
struct Seq {
  int len;
  int cached, tiles;       // tiles of the cache, of cache and nodes
  bool bad;
};
__device__ __forceinline__ Seq seq_of(const TreeAttnParams& p, int b) {
  Seq q;
  const int len = p.a.lens[b];
  const int most = p.a.cols * p.a.page_size;
  q.len = min(max(len, 0), most);
  q.bad = q.len != len;
  const int tile = tree_tile(p.a.D);
  q.cached = (q.len + tile - 1) / tile;
  q.tiles = q.cached + (p.a.N + tile - 1) / tile;
  return q;
}

// The units and the workers that share them, at most one worker per unit.
struct TreeSplit {
  int total, workers;
  __device__ __forceinline__ int first(int w) const {  // unit of worker w
    return w >= workers ? total : (int)((long long)w * total / workers);
  }
  __device__ __forceinline__ int worker(int unit) const {  // whose share a unit is in
    int w = (int)((long long)unit * workers / total);
    while (first(w + 1) <= unit) ++w;            // a step or none
    while (first(w) > unit) --w;
    return w;
  }
};
struct TreeStart {
  int b, unit;             // the sequence of a worker's first unit, and the units before it
};

// Running sums over the sequences, by the whole CTA (NT threads), which finds the sequence
// of worker w's first unit.  Up to NT sequences the sums that form the total find it too.
template <int NT>
__device__ __forceinline__ TreeSplit tree_starts(const TreeAttnParams& p, int w, TreeStart* s_start,
                                             int2* s_warp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.a.B, items = p.sets * p.block_sets;
  TreeSplit all{0, 0};
  for (int pass = 0; pass < 2; ++pass) {
    int base = 0;
    for (int b0 = 0; b0 < B; b0 += NT) {
      const int b = b0 + tid;
      int mine = 0;
      if (b < B) {
        const Seq q = seq_of(p, b);
        mine = items * (q.tiles + 1);
        if (pass == 0 && blockIdx.x == 0 && q.bad) flag_bits(p, SSD_DEV_BAD_LENGTH);
      }
      int x = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (lane == 31) s_warp[warp].x = x;
      __syncthreads();
      int before = base;
      for (int i = 0; i < NT / 32; ++i) {
        if (i < warp) before += s_warp[i].x;
        base += s_warp[i].x;
      }
      if (B <= NT) {
        all = TreeSplit{base, min(p.workers, base)};
        pass = 1;
      }
      if (pass == 1 && b < B) {
        const int u = before + x - mine, f = all.first(w);
        if (f >= u && f < u + mine) *s_start = TreeStart{b, u};
      }
      __syncthreads();
    }
    if (pass == 0) all = TreeSplit{base, min(p.workers, base)};
  }
  return all;
}

// A worker's stretches, one after the other.
struct TreeStretch {
  Seq q;
  int b, h, mb;            // the item,
  int item, slot;          // its number; the partial's, or -1 when it is done whole
  int tile0, tile1;
  int end;                 // the item's first unit no more
};
struct TreeWalk {
  int u, u1;               // units still to do
  int b, unit;
  int w, x;                // worker, its CTA: head of a set, block of a set
};
__device__ __forceinline__ bool next_stretch(const TreeAttnParams& p, TreeWalk& k, TreeStretch& s) {
  const int items = p.sets * p.block_sets;
  while (k.u < k.u1) {
    Seq q = seq_of(p, k.b);
    int n = items * (q.tiles + 1);
    while (k.u >= k.unit + n) {  // ends: u < u1 <= total
      k.unit += n;
      q = seq_of(p, ++k.b);
      n = items * (q.tiles + 1);
    }
    const int cost = q.tiles + 1;
    const int local = (k.u - k.unit) / cost;     // item within the sequence
    const int at = (k.u - k.unit) - local * cost;
    const int take = min(cost - at, k.u1 - k.u);
    k.u += take;
    s.q = q;
    s.b = k.b;
    const int set = local / p.block_sets, bb = k.x / p.hg;
    s.h = set * p.hg + k.x - bb * p.hg;
    s.mb = (local - set * p.block_sets) * p.bg + bb;
    s.tile0 = max(at - 1, 0);
    s.tile1 = at + take - 1;
    s.end = k.unit + (local + 1) * cost;
    s.item = (k.b * items + local) * p.side + k.x;
    s.slot = s.tile0 == 0 && s.tile1 == q.tiles
                 ? -1 : 2 * (k.w * p.side + k.x) + (s.tile0 == 0);
    if (s.tile1 > s.tile0) return true;  // not only the unit of the item's start
  }
  return false;
}

cudaError_t launch_tree_bf16(const TreeAttnParams& p, cudaStream_t s);
cudaError_t launch_tree_f16(const TreeAttnParams& p, cudaStream_t s);

}  // namespace ssd
