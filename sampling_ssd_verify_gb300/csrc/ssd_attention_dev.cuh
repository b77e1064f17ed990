// ssd_attention_dev.cuh -- what the attention kernels share: parameters, the
// split of the prefixes' work over workers, and the layout of partial results.
//
// A prefix is attended to by all rows of its group.  The rows' query heads
// that read one key/value head, (row, head) in row-major order, are cut into
// blocks of MT; an item is (group, key/value head, block), and costs one unit
// for its start and end (queries, partial) and one for each tile of TN tokens of
// the group's prefix.  The units of all items, in order, are divided evenly
// among the workers, so every worker has the same share however the lengths
// differ; a worker that gets a stretch of an item leaves a partial
// result (unnormalised sums, their largest score and weight), and the rows'
// partials are joined afterwards.  The partial of item i by worker w has slot
// i + w: along the sequence of stretches one of the two steps up each time,
// so slots are never shared, and need no counter.
//
// Where the key/value heads of a token lie side by side, a worker is `hg` CTAs
// that go through the same stretches, each for its head of a set of hg: they
// read neighbouring pieces of memory at about the same time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd.h"
#include "ssd_device.cuh"
#include "ssd_internal.cuh"

namespace ssd {

// 16 bytes global -> shared; zeros when !ok (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x to about 2^-22 of the value, results below 2^-126 as zero: far below the half step
// (2^-8 or 2^-11) of the 16-bit weights that are made of it.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

struct AttnParams {
  ssd_attention a;
  Divisor by_page, by_gqa;
  float scale_log2;       // scale * log2(e): scores in base 2
  int gqa;                // query heads per key/value head
  // prefixes: items, partials
  int mt, tn;             // rows of a block, tokens of a tile
  int hg, sets;           // key/value heads of a set, sets
  int workers;            // of hg CTAs each
  int nslots;
  float* po;              // [nslots, D / 4, mt, 4] unnormalised sums (part_at)
  float2* pml;            // [nslots, mt] largest score (base 2), weight
  int4* row_items;        // [R] row_items_of
  int2* item_workers;     // [items] first and last worker of an item with tokens; items of a
                          // set are hg in a row
  // own tokens: nsplit stretches per row, each with its partial
  int in_step;            // workers may be left out to keep the others in step,
  int own_apart;          // or for own tokens in a kernel of their own
  int nsplit;
  float* so;              // [R, Hq, nsplit, D]
  float2* sml;            // [R, Hq, nsplit]
  int32_t* status;
};

// Place of dimension d (a multiple of 4, or within one) of row i of a prefix's
// partial: the rows of four dimensions stand together, so that a kernel with a
// row per thread writes whole lines, and the rows of a key/value head's query
// heads are read as one piece.
template <int D>
__device__ __forceinline__ int64_t part_at(int slot, int mt, int i, int d) {
  return (((int64_t)slot * (D / 4) + d / 4) * mt + i) * 4 + d % 4;
}

// The kernels of a call follow one another on the stream, each launched so that
// its CTAs may start as soon as SMs fall free at the end of the one before:
// `start_next` lets it, `wait_previous` waits until all of it is done and seen.
__device__ __forceinline__ void start_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// What the join needs of a row's group: the number of the group's first set of items,
// or -1 when there is no prefix to join; the row's first pair in the group; the
// blocks of a key/value head.
__device__ __forceinline__ int4 row_items_of(int item, int pair, int blocks) {
  return make_int4(item, pair, blocks, 0);
}

__device__ __forceinline__ void flag(const AttnParams& p, int bit) {
  if (p.status) atomicOr(p.status, bit);
}

// Group g: its rows and tokens, clamped into range.
struct Group {
  int row0, rows, len;
  int blocks, tiles;      // blocks of its (row, head) pairs, tiles of its prefix
  int cost;               // units of an item
  bool torn;              // its rows are no range within [0, R]
  bool bad;               // that, or its length was clamped
};
__device__ __forceinline__ Group group_of(const AttnParams& p, int g) {
  Group q;
  const int o0 = p.a.group_off[g], o1 = p.a.group_off[g + 1];
  const int len = p.a.prefix_len[g];
  q.row0 = min(max(o0, 0), p.a.R);
  q.rows = min(max(o1, 0), p.a.R) - q.row0;
  const long long most = (long long)p.a.prefix_cols * p.a.page_size;
  q.len = len < 0 ? 0 : len > most ? (int)most : len;
  q.torn = q.row0 != o0 || q.rows < 0 || q.row0 + q.rows != o1;
  q.bad = q.torn || q.len != len;
  q.rows = max(q.rows, 0);
  q.blocks = (q.rows * p.gqa + p.mt - 1) / p.mt;
  q.tiles = (q.len + p.tn - 1) / p.tn;
  q.cost = q.tiles > 0 ? q.tiles + 1 : 0;
  return q;
}

// The units and the workers that share them, at most one worker per unit, so
// that the partials of an item are by consecutive workers.
struct Split {
  int total, workers;
  __device__ __forceinline__ int first(int w) const {  // unit of worker w
    return w >= workers ? total : (int)((long long)w * total / workers);
  }
};

// Blocks of the same prefix read its tiles from L2 if they come to them at about
// the same time.  They do if the workers are a multiple of the items, each of which
// then begins with a worker of its own; that pays where no more than a quarter of
// them is left idle and most units are of prefixes with several blocks.  Measured
// without own tokens, 32 heads on 8, of 19 workers (8 CTAs each): 8 blocks over
// 40000 tokens take 144 us by 16, 201 by 19; over 16000, 68 and 69; over 3000, 29 and 33;
// 3 blocks over 24000 take 47 us by 18, 57 by 19; but 10 blocks 170 by 10, 116 by 19.
//
// A prefix of several blocks leaves the memory idle, which own tokens in a kernel of
// their own wait for.  With enough of those, half the workers take the prefixes and
// the other SMs go to the own tokens at once.  `own` counts 16 tokens a unit.  The rule
// goes by own tokens x heads x D / 128 to prefix tokens x heads x blocks, half or more.
// Half and all of the workers, 256 rows over a prompt of 16000: at 0.2 119 and 91 us, 0.45
// 120 and 112, 0.6 120 and 124, 0.9 128 and 150, 3.4 348 and 363.  Where the lines cross
// differs by 0.3 either way: 64 rows over 16000 at 0.25 47 and 52, 256 rows over 40000 at
// 0.6 264 and 260.  With 16 items, more than the 9 workers left, 183 and 174.
__device__ __forceinline__ Split split_of(const AttnParams& p, int total, int items, int shared,
                                          int own) {
  Split s{total, min(p.workers, total)};
  if (p.own_apart && shared >= total - shared && 2 * items <= s.workers &&
      2ll * own * 16 * p.a.Hkv * p.a.D >= 128ll * total * p.hg * p.tn)
    s.workers /= 2;
  if (p.in_step && items > 0 && shared >= total - shared) {
    const int idle = s.workers % items;
    if (items <= s.workers && 4 * idle <= s.workers) s.workers -= idle;
  }
  return s;
}

// Running sums over the groups, by the whole CTA (NT threads), which finds for
// each of its NW workers w0 .. w0 + NW - 1 the group that holds its first
// tile.  Leaves each row's items for the join.  Returns the split.
struct Start {
  int g, unit, item;      // the group, and the sums before it
};
template <int NT, int NW>
__device__ __forceinline__ Split find_starts(const AttnParams& p, int w0, Start* s_start,
                                             int4* s_warp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.a.G;
  // pass 0 forms the total, pass 1 the starts that it determines; up to NT
  // groups, the sums of pass 0 serve for pass 1
  int torn = 0, own = 0;
  Split all{0, 0};
  if (p.own_apart) {
    const int most = p.a.cols * p.a.page_size;
    for (int r = tid; r < p.a.R; r += NT) own += min(max(p.a.lens[r], 0), most) >> 4;
    own = __reduce_add_sync(0xffffffffu, own);
  }
  for (int pass = 0; pass < 2; ++pass) {
    int4 base = make_int4(0, 0, 0, 0);
    for (int g0 = 0; g0 < G; g0 += NT) {
      const int g = g0 + tid;
      int2 mine = make_int2(0, 0);
      Group q{};
      if (g < G) {
        q = group_of(p, g);
        torn |= q.torn;
        mine = torn ? mine : make_int2(p.sets * q.blocks * q.cost, p.sets * q.blocks);
        if (pass == 0 && blockIdx.x == 0 && q.bad) flag(p, SSD_DEV_BAD_LENGTH);
      }
      int2 x = mine;
      const int shared = __reduce_add_sync(0xffffffffu, q.blocks > 1 ? mine.x : 0);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x.x, d);
        const int b = __shfl_up_sync(0xffffffffu, x.y, d);
        if (lane >= d) { x.x += a; x.y += b; }
      }
      if (lane == 31) s_warp[warp] = make_int4(x.x, x.y, shared, own);
      const int any_torn = __syncthreads_or(torn);
      int4 before = base;
      base.w = 0;  // the same for all groups
      for (int w = 0; w < NT / 32; ++w) {
        const int4 y = s_warp[w];
        if (w < warp) { before.x += y.x; before.y += y.y; }
        base = make_int4(base.x + y.x, base.y + y.y, base.z + y.z, base.w + y.w);
      }
      if (G <= NT) {
        torn = any_torn;
        all = split_of(p, torn ? 0 : base.x, base.y, base.z, base.w);
        pass = 1;
      }
      if (pass == 1 && g < G) {
        const int u = before.x + x.x - mine.x, i = before.y + x.y - mine.y;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          const int f = all.first(w0 + k);
          if (!torn && f >= u && f < u + mine.x) s_start[k] = Start{g, u, i};
        }
      }
      // the groups that fall to this CTA, one at a time by their warp
      if (pass == 1 && !torn) {
        const int item = before.y + x.y - mine.y;
        unsigned todo = __ballot_sync(0xffffffffu, g < G && g % (int)gridDim.x == (int)blockIdx.x);
        for (; todo != 0; todo &= todo - 1) {
          const int src = __ffs(todo) - 1;
          const int first = __shfl_sync(0xffffffffu, q.tiles > 0 ? item : -1, src);
          const int row0 = __shfl_sync(0xffffffffu, q.row0, src);
          const int rows = __shfl_sync(0xffffffffu, q.rows, src);
          const int blocks = __shfl_sync(0xffffffffu, q.blocks, src);
          for (int r = lane; r < rows; r += 32)
            p.row_items[row0 + r] = row_items_of(first, r * p.gqa, blocks);
        }
      }
      __syncthreads();
    }
    if (pass == 0) {
      torn = __syncthreads_or(torn);
      all = split_of(p, torn ? 0 : base.x, base.y, base.z, base.w);
    }
  }
  // rows of no group
  const int r0 = torn ? 0 : p.a.group_off[0], r1 = torn ? 0 : p.a.group_off[G];
  const int step = gridDim.x * NT, at = blockIdx.x * NT + tid;
  for (int r = at; r < r0; r += step) p.row_items[r] = row_items_of(-1, 0, 0);
  for (int r = r1 + at; r < p.a.R; r += step) p.row_items[r] = row_items_of(-1, 0, 0);
  return all;
}

// A worker's stretches, one after the other.
struct Stretch {
  int g, h, mb;           // the item,
  int item, slot;         // its number, and the partial's
  Group q;
  int tile0, tile1;       // tiles of the prefix
};
struct Walk {
  int u, u1;              // tiles still to do
  int g, unit, item;
  int w, hh;              // worker, head of a set
};
__device__ __forceinline__ bool next_stretch(const AttnParams& p, Walk& k, Stretch& s) {
  while (k.u < k.u1) {
    Group q = group_of(p, k.g);
    int n = p.sets * q.blocks * q.cost;
    while (k.u >= k.unit + n) {  // ends: u < u1 <= total
      k.unit += n;
      k.item += p.sets * q.blocks;
      q = group_of(p, ++k.g);
      n = p.sets * q.blocks * q.cost;
    }
    const int local = (k.u - k.unit) / q.cost;   // item within the group
    const int at = (k.u - k.unit) - local * q.cost;
    const int take = min(q.cost - at, k.u1 - k.u);
    k.u += take;
    s.q = q;
    s.g = k.g;
    const int set = local / q.blocks;
    s.h = set * p.hg + k.hh;
    s.mb = local - set * q.blocks;
    s.tile0 = max(at - 1, 0);
    s.tile1 = at + take - 1;
    s.item = (k.item + local) * p.hg + k.hh;
    s.slot = s.item + k.w * p.hg;
    if (s.tile1 > s.tile0) return true;  // not only the unit of the item's start
  }
  return false;
}

// One thread per stretch tells the join which workers have the item.
__device__ __forceinline__ void leave_worker(const AttnParams& p, const Stretch& s, int w) {
  if (s.slot >= p.nslots) return;
  if (s.tile0 == 0) p.item_workers[s.item].x = w;
  if (s.tile1 == s.q.tiles) p.item_workers[s.item].y = w;
}

// The tensor-core kernel (ssd_attention_tc.cu): blocks of kTcBlock pairs, tiles
// of kTcTile tokens, one worker per SM.
constexpr int kTcBlock = 128, kTcTile = 128;
bool prefix_tc_fits(const ssd_attention& a);
cudaError_t launch_prefix_tc(const AttnParams& p, cudaStream_t s);

}  // namespace ssd
