// ssd_tree_attention_kernel.cuh -- attention of drafted nodes over a paged cache and
// the nodes on their paths, on the 5th-generation tensor cores.
//
// A block is up to 128 (node, head) pairs of one sequence and key/value head, a tile kTile
// tokens: of the cache, and after those of the sequence's nodes, where each pair's
// weights of nodes off its path are zero.  S = Q K^T, P = exp2(S * scale - m), O += P V,
// out = O / sum P.  An item is a sequence's key/value head and one or two blocks, and
// costs a unit for its start and end and one for each tile; the units of all items, in
// order, are divided evenly among the workers, so every worker has the same share
// however the lengths differ.  An item that one worker does alone is written
// out by it; of the others every stretch leaves a partial (unnormalised sums, their
// largest score and weight), which the join puts together.  A worker has two such
// stretches at most, one that goes on with an item and one that begins one, so
// partials have places by the CTA.
//
// A tile's 64 KB (D = 128) take an SM 1.4 us of the memory's time (7.1 TB/s below), its products
// 2 x 512 cycles of the tensor cores for each block of pairs and its exponentials 512 of
// the four units of an SM: with one block the memory is the bound, and padding a few pairs to 128
// costs nothing; with two, which share the tile, both are near.  Copies, products and
// exponentials of different tiles overlap (warps of their own, barriers between them), and
// no barrier gets two phases ahead of a waiter.
//
// Measured in a graph, 32 heads on 8, D = 128: 256 sequences of 200 to 8000 tokens, one node
// each, 593 to 603 us (7.1 TB/s; a copy has 6.8); two contexts of 131072 for 16 nodes 157
// (6.8 TB/s); 64 sequences of 500 to 8191 in pages of 16 for trees of 11 177 (6.5 TB/s); 32 of
// them for 64 nodes 126 (1.16 PFLOP/s: the tensor cores are busy for 57% of the cycles; their
// operands come from shared memory at its rate, and a block's next scores wait for its weights).
// One stream of 700 tokens and 5 nodes 11.7, from L2 11.1: 5.5 until a tile's weights are there,
// 7.6 until the last partials are, and the join from 8.6 on.  256 sequences of 10 to 200 tokens
// 65, where memory would take 17: an item of one or two tiles is a chain of 3.4 us (scores,
// weights, sums, output) in the threads of the exponentials.  Float16 takes as long.
// A figure "instead of" another, here and below, is of the step that made the choice: with it and
// without it then, when other steps were still to come.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ssd_attention_dev.cuh"
#include "ssd_tc_dev.cuh"
#include "ssd_tree_attention.cuh"

namespace ssd {
namespace {

constexpr int kRows = 128;                // pairs of a block (M)
constexpr int kSoftmax = 256;             // threads of the two warpgroups
constexpr int kHeaderBytes = 3 << 10;     // of shared memory before the rings
constexpr int kTreeThreads = kSoftmax + 128;  // a third warpgroup: copies and products
constexpr int kCopyK = 8, kCopyV = 9, kMmaWarp = 10, kQueryWarp = 11;
// Registers per thread: launched with 168 (12 warps), of which the third warpgroup
// gives up 80 and the others take 40 each: 8 * 208 + 4 * 88 = 12 * 168.
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
constexpr float kRise = 8.f;              // scores may pass the kept maximum by this (base 2)
// Half has no weights below 2^-24: beside one that is the largest the many small ones of a long
// cache would be lost from the sums.  So all of a half's weights are 2^kLift larger, up to
// 2^(kRise + kLift) of the 2^16 that there are: what is lost then is at most 2^-32 of the largest
// weight for each token (2^-15 for 131072 of them).  Large scores are rounded when they are
// scaled, by 2^4 from 2^27 on; half's maxima are rounded up, so that no weight grows by it.
template <typename T>
constexpr float kLift = __is_same(T, __half) ? 7.f : 0.f;

constexpr int kColS = 0, kColStep = 128;  // scores (and weights) of a buffer in tensor memory

// BLOCKS: of an item.  The rings and the queries take 224 KB, one CTA per SM.
template <int D, int BLOCKS> struct TreeShape {
  static constexpr int kTile = tree_tile(D);
  static constexpr int kPanels = D / 64;
  static constexpr int kPanel = kTile * 128;          // kTile rows x 64 elements, swizzled
  static constexpr int kSlot = kPanels * kPanel;      // K or V of a tile
  static constexpr int kQueryPanel = kRows * 128;
  static constexpr int kQueries = kPanels * kQueryPanel;  // of a block
  // V stays until its weights are there, K not: two contexts of 131072 tokens in pages of 64
  // take 162 us with 2 and 4, 172 with 3 and 3 (16 tokens: 169 and 168).  At D = 256 copies of
  // 16 bytes want it the other way: 548 us with 2 and 3, 492 with 3 and 2 (boxes 359, 363).
  static constexpr int kSlotsK = D == 64 ? 5 : D == 128 ? 2 : 3;
  static constexpr int kSlotsV = D == 64 ? 7 : D == 128 ? (BLOCKS == 1 ? 4 : 3) : 2;
  static constexpr int kSmem = kHeaderBytes + (kSlotsK + kSlotsV) * kSlot + BLOCKS * kQueries;
  static_assert(kSmem <= 227 << 10, "shared memory");
  // How the two warpgroups of exponentials share the work:
  //   tiles   the even and the odd tiles of a block, each with sums of its own;
  //   blocks  a block each, of every tile;
  //   one     the first does all: the sums (256 columns) have room for one stream.
  static constexpr bool kByBlocks = BLOCKS == 2;
  static constexpr bool kOne = D == 256;
  static constexpr bool kByTiles = !kByBlocks && !kOne;
  // Of a tile, the 32s of tokens whose weights and sums are computed: those with some of
  // the `left` from its first on (256 sequences of 10 to 200 tokens 75 us instead of 82, 32 of 100
  // to 1500 28.9 instead of 30.6).  With two blocks and at D = 256 the test before each product
  // costs more than that gives (32 x 64 nodes 133 us instead of 129, at D = 256 303
  // instead of 289): all.
  static __device__ __forceinline__ int parts(int left) {
    return kByTiles ? (min(kTile, left) + 31) / 32 : kTile / 32;
  }
  // Buffers of scores, and where the sums are.  Where the sums leave room for three, the scores
  // are two tiles ahead of the sums, and the exponentials need not wait for them (64 x 11 nodes
  // 107 us instead of 113).
  static constexpr int kBuffers = kByTiles && D == 64 ? 3 : 2;
  static constexpr int kLead = kBuffers - 1;
  static constexpr int kColO = kColS + kBuffers * kColStep, kStepO = kBuffers == 3 ? 64 : 128;
};

// What the product and exponential warps know of a stretch.
struct TreeJob {
  int tiles;        // 0: no more
  int cached;       // of them, of the cache (may be negative or more than tiles)
  int tokens;       // of the cache from the first tile on
  int seq, head, pair0, pairs;  // sequence, key/value head, the item's pairs
  int slot;         // of the partial; -1: the item is done here
};

struct TreeHeader {
  float2 ml[2][kRows];              // the streams' maxima and weights, handed over at the end
  uint64_t k_full[7], k_empty[7];   // ring slots
  uint64_t v_full[7], v_empty[7];
  uint64_t q_full, q_empty;         // a stretch's job and queries; its scores are all done
  uint64_t job_read;                // its job is known to the exponentials' threads
  uint64_t s_full[3];               // scores of a tile are there, by buffer
  uint64_t p_half[3];               // its weights of the first half of the tokens are
  uint64_t p_full[3];               // all of them are
  uint64_t o_done[4];               // its part of the sums is, by block or by tile
  uint64_t ml_full;                 // both streams' maxima and weights are in place
  uint64_t o_empty;                 // the sums of a stretch have been read
  uint64_t drained;
  TreeJob job[2];                   // by the parity of the stretch
  int2 warp_sums[kTreeThreads / 32];
  TreeStart start;
  uint32_t tmem;
  volatile int err;
  volatile int odd[2];              // 1 + the last stretch with values that are no numbers
  uint8_t parent[kTreeNodes];
};
static_assert(sizeof(TreeHeader) <= kHeaderBytes, "header");

// Whether a wait of the CTA ran out (to every lane of a warp alike): no new
// work is begun then.
__device__ __forceinline__ bool gave_up(const TreeHeader& sh) {
  return __any_sync(0xffffffffu, sh.err) != 0;
}

// Whether one of two 16-bit numbers is infinite or NaN: which, as masks.
template <typename T>
__device__ __forceinline__ uint32_t odd_mask(uint32_t x) {
  constexpr uint32_t e = __is_same(T, __half) ? 0x7c00u : 0x7f80u;
  return ((x & e) == e ? 0xffffu : 0u) | ((x & e << 16) == e << 16 ? 0xffff0000u : 0u);
}
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// 32 bytes, a whole sector, to an address of that alignment.
__device__ __forceinline__ void store32(void* to, const uint32_t (&z)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(z[0]),
               "r"(z[1]), "r"(z[2]), "r"(z[3]), "r"(z[4]), "r"(z[5]), "r"(z[6]), "r"(z[7])
               : "memory");
}

// Leaves in ok (a bit per node, from node `at` on) those on node u's path.
template <int TILE>
__device__ __forceinline__ void on_path(uint32_t (&ok)[TILE / 32], const uint8_t* parent,
                                        bool chain, int u, int at) {
  uint32_t path[TILE / 32];
#pragma unroll
  for (int q = 0; q < TILE / 32; ++q) {
    const int left = u + 1 - at - q * 32;
    path[q] = !chain || left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1;
  }
  for (int v = u; !chain && v >= at; v = parent[v]) {
#pragma unroll
    for (int q = 0; q < TILE / 32; ++q)
      if ((v - at) >> 5 == q) path[q] |= 1u << (v & 31);
    if (v == 0) break;
  }
#pragma unroll
  for (int q = 0; q < TILE / 32; ++q) ok[q] &= path[q];
}

template <typename T, int D, int BLOCKS>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_tc_kernel(const __grid_constant__ TreeAttnParams p,
                   const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap knodes,
                   const __grid_constant__ CUtensorMap vnodes,
                   const __grid_constant__ CUtensorMap qmap) {
  using S = TreeShape<D, BLOCKS>;
  constexpr int kTile = S::kTile;
  extern __shared__ __align__(1024) unsigned char s_raw[];
  TreeHeader& sh = *reinterpret_cast<TreeHeader*>(s_raw);
  const ssd_tree_attn& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t kring = smem_addr(s_raw) + kHeaderBytes;
  const uint32_t vring = kring + S::kSlotsK * S::kSlot;
  const uint32_t qs = vring + S::kSlotsV * S::kSlot;

  start_next();
  if (warp == kMmaWarp) tmem_alloc(&sh.tmem);
  if (p.box_rows > 0 && warp == kQueryWarp && lane < 4)
    prefetch_map(lane == 0 ? &kmap : lane == 1 ? &vmap : lane == 2 ? &knodes : &vnodes);
  if (p.q_nodes > 0 && warp == kQueryWarp && lane == 4) prefetch_map(&qmap);
  if (tid == 0) {
    sh.err = 0;
    sh.odd[0] = sh.odd[1] = 0;
    // a tile by boxes: one arrival and its bytes; by copies of the lanes: theirs
    const int copies = p.box_rows > 0 ? 1 : 32;
    for (int i = 0; i < S::kSlotsK; ++i) {
      mbar_init(&sh.k_full[i], copies);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < S::kSlotsV; ++i) {
      mbar_init(&sh.v_full[i], copies);
      mbar_init(&sh.v_empty[i], 1);
    }
    mbar_init(&sh.q_full, 32);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_half[i], kRows);
      mbar_init(&sh.p_full[i], kRows);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.o_done[i], 1);
    mbar_init(&sh.job_read, kSoftmax);
    mbar_init(&sh.ml_full, kSoftmax);
    mbar_init(&sh.o_empty, kSoftmax);
    mbar_init(&sh.drained, 1);
    fence_barrier_init();
  }
  if (tid < a.N) sh.parent[tid] = p.parent[tid];
  const int w = blockIdx.x / p.side;
  const TreeSplit all = tree_starts<kTreeThreads>(p, w, &sh.start, sh.warp_sums);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;

  // the third warpgroup's warps walk the stretches by themselves
  TreeWalk k;
  k.u = all.first(w);
  k.u1 = all.first(w + 1);
  k.w = w;
  k.x = blockIdx.x - w * p.side;
  if (k.u < k.u1) {
    k.b = sh.start.b;
    k.unit = sh.start.unit;
  }
  TreeStretch s;

  if (warp >= kSoftmax / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kCopyK || warp == kCopyV) {
      // ---- copies: a warp for K and one for V ---------------------------------------------
      const bool v = warp == kCopyV;
      uint64_t* full = v ? sh.v_full : sh.k_full;
      uint64_t* empty = v ? sh.v_empty : sh.k_empty;
      const uint32_t slots = v ? vring : kring;
      const int nslots = v ? S::kSlotsV : S::kSlotsK;
      const int P = a.page_size;
      uint32_t slot = 0, use = 0;                // of the next tile: its slot, turns of the ring
      auto next_slot = [&] {
        if (++slot == (uint32_t)nslots) {
          slot = 0;
          ++use;
        }
      };
      if (p.box_rows > 0) {
        // a lane per box: some tokens of a page, 64 dimensions
        const int rows = p.box_rows, boxes = kTile / rows;  // tokens; of a whole tile, at most 32
        // Tokens that one item reads are not read again: they leave L2 first (64 x 11 nodes
        // 185 us instead of 198; at D = 64 107 instead of 116).
        uint64_t once, again;
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
        const uint64_t policy = p.blocks == 1 ? once : again;
        while (next_stretch(p, k, s)) {
          const int32_t* table = a.tables + (int64_t)s.b * a.table_stride;
          auto page_at = [&](int tile) {  // not looked at here: the load stays in flight
            const int t = tile * kTile + lane * rows;
            return lane < boxes && tile < s.tile1 && t < s.q.len ? table[p.by_page.quotient(t)]
                                                                 : 0;
          };
          // pages are looked up two tiles ahead of their copies
          int page = page_at(s.tile0), next = page_at(s.tile0 + 1);
          for (int tile = s.tile0; tile < s.tile1; ++tile) {
            if (gave_up(sh)) {
              k.u = k.u1;
              break;
            }
            const int after = page_at(tile + 2);
            if (use > 0) mbar_wait(&empty[slot], (use - 1) & 1, &sh.err, p.status);
            const uint32_t dst = slots + slot * S::kSlot;
            if (tile < s.q.cached) {
              if ((unsigned)page >= (unsigned)a.num_pages) {
                flag_bits(p, SSD_DEV_BAD_PAGE);
                page = a.num_pages;              // past the end: the box is zeros
              }
              const int here = min(kTile, s.q.len - tile * kTile);
              const int n = (here + rows - 1) / rows;  // boxes with tokens
              const int t = tile * kTile + lane * rows;
              const int in_page = t - p.by_page.quotient(t) * P;
              if (lane == 0)
                mbar_arrive_expect_tx(&full[slot], (uint32_t)(n * rows * 128 * S::kPanels));
              __syncwarp();
              if (lane < n) {
#pragma unroll
                for (int d = 0; d < S::kPanels; ++d)
                  tma_box(dst + lane * rows * 128 + d * S::kPanel, v ? &vmap : &kmap, d * 64, s.h,
                          in_page, page, &full[slot], policy);
              }
            } else {
              if (lane == 0)
                mbar_arrive_expect_tx(&full[slot], (uint32_t)(p.node_rows * 128 * S::kPanels));
              __syncwarp();
              if (lane < S::kPanels)
                tma_box(dst + lane * S::kPanel, v ? &vnodes : &knodes, lane * 64, s.h,
                        (tile - s.q.cached) * kTile, s.b, &full[slot], again);
            }
            next_slot();
            page = next;
            next = after;
          }
        }
        if (sh.err) {  // let the copies in flight land before the memory is given up
          for (int i = 0; i < nslots; ++i) {
            const uint32_t turns = use + ((uint32_t)i < slot ? 1 : 0);
            int none = 0;
            if (turns > 0) mbar_wait(&full[i], (turns - 1) & 1, &none, nullptr);
          }
        }
      } else {
        // any pages and strides: 16 bytes a lane at a time, the tokens' places dealt to the lanes
        constexpr int kLanes = D / 8;            // lanes of a token
        constexpr int kGroups = kTile / 32;
        const ssd_paged& cache = v ? a.v_cache : a.k_cache;
        const ssd_paged& nodes = v ? a.v : a.k;
        uint32_t told = 0, told_slot = 0, issued = 0;  // tiles whose arrival is told, begun
        auto tell = [&] {
          fence_async();
          mbar_arrive(&full[told_slot]);
          if (++told_slot == (uint32_t)nslots) told_slot = 0;
          ++told;
        };
        auto flush = [&] {
          copies_wait<0>();
          while (told != issued) tell();
        };
        while (next_stretch(p, k, s)) {
          const int32_t* table = a.tables + (int64_t)s.b * a.table_stride;
          int page[kGroups];
          auto pages_of = [&](int tile) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              const int t = tile * kTile + g * 32 + lane;
              page[g] = tile < s.q.cached && t < s.q.len ? table[p.by_page.quotient(t)] : 0;
            }
          };
          pages_of(s.tile0);
          for (int tile = s.tile0; tile < s.tile1; ++tile) {
            if (gave_up(sh)) {
              k.u = k.u1;
              break;
            }
            const bool old = tile < s.q.cached;
            const int first = (old ? tile : tile - s.q.cached) * kTile;
            const int here = min(kTile, (old ? s.q.len : a.N) - first);
            int64_t at[kGroups];                 // of the tokens; negative: zeros
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              const int r = g * 32 + lane, t = first + r;
              at[g] = -1;
              if (r < here) {
                if (!old) {
                  at[g] = s.b * nodes.page_stride + t * nodes.token_stride;
                } else if ((unsigned)page[g] < (unsigned)a.num_pages) {
                  at[g] = page[g] * cache.page_stride +
                          (t - p.by_page.quotient(t) * P) * cache.token_stride;
                } else {
                  flag_bits(p, SSD_DEV_BAD_PAGE);
                }
              }
            }
            pages_of(tile + 1);
            const T* from = static_cast<const T*>(old ? cache.ptr : nodes.ptr) +
                            s.h * (old ? cache.head_stride : nodes.head_stride) + lane % kLanes * 8;
            if (use > 0 && !__all_sync(0xffffffffu, mbar_try_wait(&empty[slot], (use - 1) & 1))) {
              flush();                           // what is waited for may need it
              mbar_wait(&empty[slot], (use - 1) & 1, &sh.err, p.status);
            }
            __syncwarp();
            const int ch = lane % kLanes;
            const uint32_t dst = slots + slot * S::kSlot + (ch / 8) * S::kPanel;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              if (g * 32 >= here) break;
#pragma unroll 8
              for (int i = 0; i < kLanes; ++i) {
                const int r = i * (32 / kLanes) + lane / kLanes;  // of the group
                const int64_t x = __shfl_sync(0xffffffffu, at[g], r);
                const int row = g * 32 + r;
                if (row < here)
                  copy16(dst + row * 128 + (((ch & 7) ^ (row & 7)) << 4), from + (x < 0 ? 0 : x),
                         x >= 0);
              }
            }
            copies_commit();
            ++issued;
            next_slot();
            if (issued - told == 2) {            // the one before has had its time
              copies_wait<1>();
              tell();
            }
          }
        }
        flush();
      }
    } else if (warp == kQueryWarp) {
      // ---- queries: a stretch's, as soon as the scores of the one before are done ------
      uint32_t i = 0;
      uint64_t q_policy;
      asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(q_policy));
      if (lane == 0) p.begun[blockIdx.x] = make_int2(-1, 0);
      while (next_stretch(p, k, s)) {
        const int rows = BLOCKS * p.block_pairs;  // of an item
        const int pair0 = s.mb * rows, pairs = min(rows, p.pairs - pair0);
        auto query = [&](const TreeStretch& z, int row) {
          const int pair = z.mb * rows + row, node = p.by_gqa.quotient(pair);
          return static_cast<const T*>(a.q) + z.b * a.q_seq_stride + node * a.q_node_stride +
                 (int64_t)(z.h * p.gqa + pair - node * p.gqa) * a.q_head_stride;
        };
        if (i > 0) mbar_wait(&sh.q_empty, (i - 1) & 1, &sh.err, p.status);
        // rows past the last pair hold whatever was there: a row's scores are its own
        if (p.q_nodes == 0) {
          constexpr int kLanes = D / 8;          // lanes of a row, 16 bytes each
          const int ch = lane % kLanes;
          auto place = [&](int row) {
            const int block = BLOCKS == 2 && row >= p.block_pairs, r = row - block * p.block_pairs;
            return qs + block * S::kQueries + (ch / 8) * S::kQueryPanel + r * 128 +
                   (((ch & 7) ^ (r & 7)) << 4);
          };
          for (int r0 = 0; r0 < pairs; r0 += 32) {  // the rows' places dealt to the lanes
            const int64_t at = query(s, min(r0 + lane, pairs - 1)) - static_cast<const T*>(a.q);
#pragma unroll 8
            for (int j = 0; j < kLanes; ++j) {
              const int r = j * (32 / kLanes) + lane / kLanes, row = r0 + r;
              const int64_t x = __shfl_sync(0xffffffffu, at, r);
              if (row < pairs) copy16(place(row), static_cast<const T*>(a.q) + x + ch * 8, true);
            }
          }
          if (!p.q_plain) {                      // a scale that is not positive: -q, or 0
            copies_commit();
            copies_wait<0>();
#pragma unroll 4
            for (int row = lane / kLanes; row < pairs; row += 32 / kLanes) {
              uint32_t x[4];                     // which this lane copied
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                           : "r"(place(row))
                           : "memory");
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place(row)),
                           "r"((x[0] & p.q_and) ^ p.q_xor), "r"((x[1] & p.q_and) ^ p.q_xor),
                           "r"((x[2] & p.q_and) ^ p.q_xor), "r"((x[3] & p.q_and) ^ p.q_xor)
                           : "memory");
            }
          }
        }
        // a thread that waits for the last job must not find two newer ones: a
        // barrier tells only the parity of its phase
        if (i > 0) mbar_wait(&sh.job_read, (i - 1) & 1, &sh.err, p.status);
        if (lane == 0)
          sh.job[i & 1] = TreeJob{s.tile1 - s.tile0, s.q.cached - s.tile0,
                                  s.q.len - s.tile0 * kTile, s.b, s.h, pair0, pairs, s.slot};
        // 32 arrivals: lane 0's follows the job
        if (p.q_nodes > 0) {
          // boxes of a block's nodes, their heads side by side, and 64 dimensions
          const int boxes = (pairs > p.block_pairs ? 2 : 1) * S::kPanels;
          if (lane == 0)
            mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(boxes * p.q_nodes * p.gqa * 128));
          __syncwarp();
          if (lane < boxes) {
            const int block = lane / S::kPanels, d = lane % S::kPanels;
            tma_box(qs + block * S::kQueries + d * S::kQueryPanel, &qmap, d * 64, s.h * p.gqa,
                    (s.mb * BLOCKS + block) * p.q_nodes, s.b, &sh.q_full, q_policy);
          }
          if (lane > 0) mbar_arrive(&sh.q_full);
        } else {
          copies_commit();
          copies_wait<0>();
          fence_async();
          mbar_arrive(&sh.q_full);
        }
        ++i;
        // the join goes by the worker that began the item, up to that of its last unit
        if (lane == 0 && s.slot >= 0 && s.tile0 == 0)
          p.begun[blockIdx.x] = make_int2(s.item, all.worker(s.end - 1) - w + 1);
        // the next ones into L2 meanwhile
        TreeWalk k1 = k;
        TreeStretch s1;
        if (next_stretch(p, k1, s1)) {
          const int n = min(rows, p.pairs - s1.mb * rows);
          for (int row = lane; row < n; row += 32)
#pragma unroll
            for (int d = 0; d < D; d += 64)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(query(s1, row) + d));
        }
      }
      if (i > 0) {
        mbar_wait(&sh.q_empty, (i - 1) & 1, &sh.err, p.status);
        mbar_wait(&sh.job_read, (i - 1) & 1, &sh.err, p.status);
      }
      if (p.q_nodes > 0 && i > 0 && sh.err) {  // let the last copies land
        int none = 0;
        mbar_wait(&sh.q_full, (i - 1) & 1, &none, nullptr);
      }
      if (lane == 0) sh.job[i & 1].tiles = 0;
      __syncwarp();
      mbar_arrive(&sh.q_full);
    } else {
      // ---- products: the warp runs in step, one elected thread issues ------------------
      constexpr uint32_t score = product<T>(kTile, false), sum = product<T>(D, true);
      uint32_t ks = 0, k_use = 0, vs = 0, v_use = 0;  // ring slots and turns
      uint32_t c = 0, c1 = 0;                    // tiles so far; of the second block
      auto scores = [&](int block, uint32_t col) {
        const uint64_t q_op = operand(qs + block * S::kQueries, 16);
        const uint64_t k_op = operand(kring + ks * S::kSlot, 16);
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
          mma_ss(tmem + kColS + col * kColStep,
                 q_op + (((e / 4) * S::kQueryPanel + (e % 4) * 32) >> 4),
                 k_op + (((e / 4) * S::kPanel + (e % 4) * 32) >> 4), score, e > 0);
      };
      // half a tile's tokens at a time: the first while the weights of the others are computed
      auto sums = [&](uint32_t weights, uint32_t col, int half, bool add, int steps) {
        const uint64_t v_op = operand(vring + vs * S::kSlot, S::kPanel);
        constexpr int kSteps = kTile / 32;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int e = half * kSteps + i;
          if (e < steps)
            mma_ts(tmem + S::kColO + col * S::kStepO, tmem + kColS + weights * kColStep + e * 8,
                   v_op + ((e * 16 * 128) >> 4), sum, add || e > 0);
        }
      };
      auto turn = [](uint32_t& slot, uint32_t& use, int n) {
        if (++slot == (uint32_t)n) {
          slot = 0;
          ++use;
        }
      };
      for (uint32_t i = 0;; ++i) {
        mbar_wait(&sh.q_full, i & 1, &sh.err, p.status);
        const int n = gave_up(sh) ? 0 : sh.job[i & 1].tiles;
        if (n == 0) break;
        const bool two = S::kByBlocks && sh.job[i & 1].pairs > p.block_pairs;
        const int cached = sh.job[i & 1].cached, tokens = sh.job[i & 1].tokens;
        auto steps_of = [&](int j) {             // 16 tokens each
          return 2 * S::parts(j < cached ? tokens - j * kTile : a.N - (j - cached) * kTile);
        };
        fence_after();
        // a step more for each tile that the sums are behind; n tiles may be fewer than that
        for (int j = 0; j < n + S::kLead; ++j) {
          if constexpr (S::kByBlocks) {
            // a block's weights, then its next scores in their place
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (x == 1 && !two) break;
              const uint32_t t = (x == 0 ? c : c1) + j;
              const bool end = x == 1 || !two;
              if (j > 0) {
                if (x == 0 && j == 1 && i > 0)
                  mbar_wait(&sh.o_empty, (i - 1) & 1, &sh.err, p.status);
                mbar_wait(&sh.p_half[x], (t - 1) & 1, &sh.err, p.status);
                if (x == 0) mbar_wait(&sh.v_full[vs], v_use & 1, &sh.err, p.status);
                fence_after();
                if (elected()) sums(x, x, 0, j > 1, kTile / 16);
                __syncwarp();
                mbar_wait(&sh.p_full[x], (t - 1) & 1, &sh.err, p.status);
                fence_after();
                if (elected()) {
                  sums(x, x, 1, j > 1, kTile / 16);
                  commit(&sh.o_done[x]);
                  if (end) commit(&sh.v_empty[vs]);
                }
                __syncwarp();
                if (end) turn(vs, v_use, S::kSlotsV);
              }
              if (j < n) {
                if (x == 0) mbar_wait(&sh.k_full[ks], k_use & 1, &sh.err, p.status);
                fence_after();
                if (elected()) {
                  scores(x, x);
                  commit(&sh.s_full[x]);
                  if (end) commit(&sh.k_empty[ks]);
                  if (end && j == n - 1) commit(&sh.q_empty);
                }
                __syncwarp();
                if (end) turn(ks, k_use, S::kSlotsK);
              }
            }
          } else {
            auto next_scores = [&] {
              const uint32_t t = c + j, buf = t % S::kBuffers;
              mbar_wait(&sh.k_full[ks], k_use & 1, &sh.err, p.status);
              fence_after();
              if (elected()) {
                scores(0, buf);
                commit(&sh.s_full[buf]);
                commit(&sh.k_empty[ks]);
                if (j == n - 1) commit(&sh.q_empty);
              }
              __syncwarp();
              turn(ks, k_use, S::kSlotsK);
            };
            // the scores of a tile go before the sums of an earlier one, but where they
            // have to wait for its keys
            const bool late = j >= S::kLead && j < n &&
                              !__any_sync(0xffffffffu, mbar_try_wait(&sh.k_full[ks], k_use & 1));
            if (j < n && !late) next_scores();
            if (j >= S::kLead) {
              const int jj = j - S::kLead;
              const uint32_t t = c + jj, buf = t % S::kBuffers, o = S::kOne ? 0 : t & 1;
              const uint32_t at = t / S::kBuffers & 1;
              if (jj == 0 && i > 0) mbar_wait(&sh.o_empty, (i - 1) & 1, &sh.err, p.status);
              mbar_wait(&sh.p_half[buf], at, &sh.err, p.status);
              mbar_wait(&sh.v_full[vs], v_use & 1, &sh.err, p.status);
              fence_after();
              const bool add = jj >= (S::kOne ? 1 : 2);
              const int steps = steps_of(jj);
              if (elected()) sums(buf, o, 0, add, steps);
              __syncwarp();
              mbar_wait(&sh.p_full[buf], at, &sh.err, p.status);
              fence_after();
              if (elected()) {
                sums(buf, o, 1, add, steps);
                commit(&sh.v_empty[vs]);
                commit(&sh.o_done[t & 3]);
              }
              __syncwarp();
              turn(vs, v_use, S::kSlotsV);
            }
            if (late) next_scores();
          }
        }
        c += n;
        if (two) c1 += n;
      }
      if (elected()) commit(&sh.drained);
      __syncwarp();
      int none = 0;
      mbar_wait(&sh.drained, 0, &none, p.status);
    }
  } else {
    // ---- exponentials: warpgroup b, a pair per thread ---------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const uint32_t b = warp >> 2, m = tid & (kRows - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t acc = S::kOne ? 0 : b;        // its sums
    const uint32_t to = tmem + lanes + S::kColO + acc * S::kStepO;
    uint32_t c = 0;                              // tiles before the stretch (its block's)
    uint32_t all_tiles = 0;                      // before the stretch, of any block
    for (uint32_t i = 0;; ++i) {
      mbar_wait(&sh.q_full, i & 1, &sh.err, p.status);
      // of the job only what the tiles need is kept in registers; it stays until the next
      // one's is read
      const TreeJob& job = sh.job[i & 1];
      const int n = gave_up(sh) ? 0 : job.tiles, cached = job.cached, tokens = job.tokens;
      // of the item's pairs; in a block's rows past its pairs there is none
      const int row = (S::kByBlocks ? (int)b * p.block_pairs : 0) + (int)m;
      const bool mine = (int)m < p.block_pairs && row < job.pairs;
      const bool busy = __any_sync(0xffffffffu, mine);
      const bool second = job.pairs > p.block_pairs;  // two blocks
      // who looks after a tile's values: warps without pairs where there are any (256 sequences
      // of 10 to 200 tokens 64.9 us instead of 66.8)
      const int taken = S::kByBlocks ? 0 : (job.pairs + 31 & ~31) % kRows;
      const int fixer = (int)m - taken, fixers = kRows - taken;
      const bool fixes = (!S::kByBlocks || b == 0) && fixer >= 0;
      const int mine_node = p.by_gqa.quotient(job.pair0 + min(row, job.pairs - 1));
      mbar_arrive(&sh.job_read);
      if (n == 0) break;
      // its tiles: j0, j0 + step, ..
      const int step = S::kByTiles ? 2 : 1;
      const int j0 = S::kByTiles ? (int)((b ^ c) & 1) : S::kOne ? (b == 0 ? 0 : n)
                                 : (b == 0 || second ? 0 : n);
      float top = -INFINITY, l = 0.f;
      for (int j = j0; j < n; j += step) {
        const uint32_t t = c + j;
        // where its scores are, and the parity of their turn
        const uint32_t buf = S::kByBlocks ? b : t % S::kBuffers;
        const uint32_t turn = (S::kByBlocks ? t : t / S::kBuffers) & 1;
        const uint32_t ts = tmem + lanes + kColS + buf * kColStep;
        const bool nodes = j >= cached;
        const int at = nodes ? (j - cached) * kTile : j * kTile;
        const int here = min(kTile, (nodes ? a.N : tokens) - at);
        const bool some = nodes || here < kTile; // not all of the tile's tokens count
        const int parts = S::parts(here);
        uint32_t ok[kTile / 32];                 // those that do, for this pair
        if (some && busy) {
#pragma unroll
          for (int q = 0; q < kTile / 32; ++q) {
            const int left = here - q * 32;
            ok[q] = left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1;
          }
          if (nodes) on_path<kTile>(ok, sh.parent, p.chain, mine_node, at);
        }
        mbar_wait(&sh.s_full[buf], turn, &sh.err, p.status);
        __syncwarp();
        fence_after();
        if (some && fixes) {
          // Zero weights must not meet what is no number (0 * NaN): rows of V past the
          // last token are whatever the page or the slot held, and a node's values may be
          // off the path of others.  Those that are no numbers are put aside, and
          // added at the end to the nodes below theirs.  (Not before the tile's scores: they
          // follow the sums that had this slot's tile before, so its barrier is at this turn.)
          const uint32_t nth = all_tiles + (uint32_t)j, slot = nth % S::kSlotsV;
          mbar_wait(&sh.v_full[slot], nth / S::kSlotsV & 1, &sh.err, p.status);
          const uint32_t vs = vring + slot * S::kSlot;
          for (int e = here * 8 + fixer; e < parts * 32 * 8; e += fixers)
#pragma unroll
            for (int d = 0; d < S::kPanels; ++d)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vs + d * S::kPanel +
                                                                           e * 16),
                           "r"(0)
                           : "memory");
          if (nodes) {
            for (int e = fixer; e < here * 8; e += fixers)
#pragma unroll
              for (int d = 0; d < S::kPanels; ++d) {
                const uint32_t where = vs + d * S::kPanel + e * 16;
                uint32_t y[4], bad = 0;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                             : "r"(where)
                             : "memory");
#pragma unroll
                for (int z = 0; z < 4; ++z) bad |= odd_mask<T>(y[z]);
                if (bad) {
                  sh.odd[i & 1] = (int)i + 1;
                  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(where),
                               "r"(y[0] & ~odd_mask<T>(y[0])), "r"(y[1] & ~odd_mask<T>(y[1])),
                               "r"(y[2] & ~odd_mask<T>(y[2])), "r"(y[3] & ~odd_mask<T>(y[3]))
                               : "memory");
                }
              }
          }
          fence_async();
        }
        if (busy) {
          constexpr int kParts = kTile / 32;
          auto mask = [&](uint32_t (&x)[32], uint32_t word) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(word & 1u << e)) x[e] = 0xff800000u;  // -inf
          };
          auto scaled = [&](float x) {
            return kLift<T> > 0.f ? __fmul_ru(x, p.scale_log2) : x * p.scale_log2;
          };
          // The kept maximum moves when a score passes it by kRise; gives the weights' offset.
          auto raise = [&](float now) {
            const bool move = now > top + kRise;
            const float old = top;
            if (move) top = now;
            const float off = top == -INFINITY ? 0.f : top;
            if (j > j0 && __any_sync(0xffffffffu, move)) {
              const float f = move ? exp2_fast(old - off) : 1.f;
              l *= f;
              // the sums of the tile before are done; of the four barriers each tile's was at
              // this turn when its scores came, two or three tiles after an earlier one's sums
              const uint32_t before = t - (S::kByTiles ? 2 : 1);
              mbar_wait(&sh.o_done[S::kByBlocks ? b : before & 3],
                        (S::kByBlocks ? before : before >> 2) & 1, &sh.err, p.status);
              fence_after();
#pragma unroll 1
              for (int q = 0; q < D; q += 8) {   // few registers: the scores may have 128
                uint32_t y[8];
                tmem_ld8(y, to + q);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                tmem_st8(to + q, y);
              }
            }
            return off;
          };
          const float2 by = make_float2(p.scale_log2, p.scale_log2);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          // Weights of 32 tokens in the type of V, as the product takes them: each is off by at
          // most half a step (bf16 2^-8, half 2^-11, or 2^-32 of the largest where that is more),
          // and an output by at most that part of sum p |v|: by less where the steps are of both
          // signs, by all of it where many weights are equal.  Their sum is of the unrounded ones.
          auto weights = [&](const uint32_t (&x)[32], int q, float off, bool half) {
            const float2 less = make_float2(kLift<T> - off, kLift<T> - off);
            uint32_t z[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float2 y = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), by, less);
              y = make_float2(exp2_fast(y.x), exp2_fast(y.y));
              sum[e >> 1 & 1] = add2(sum[e >> 1 & 1], y);
              z[e / 2] = pack2<T>(y.x, y.y);
            }
            tmem_st16(ts + q * 16, z);
            if (half) {
              tmem_wait_st();
              fence_before();
              mbar_arrive(&sh.p_half[buf]);
            }
          };
          if constexpr (S::kByTiles) {
            // 32 tokens at a time, from tensor memory for their largest score and again for their
            // weights: short code, which a stretch of a few tiles has to fetch first, and
            // registers for all of it.  One stream 11.6 us instead of 12.1, 19 x 13 short ones
            // 16.7 instead of 17.7, 64 x 11 nodes 178 instead of 182, 256 x 1 594 instead of 605;
            // but with two blocks, where the scores' chain counts, 137 instead of 126.
            uint32_t x[32];
            auto load = [&](int q) {
              tmem_ld32(x, ts + q * 32);
              tmem_wait_ld();
              if (some) {
                uint32_t word = ok[0];
#pragma unroll
                for (int y = 1; y < kParts; ++y)
                  if (q == y) word = ok[y];
                if (!__all_sync(0xffffffffu, word == ~0u)) mask(x, word);
              }
            };
            float now = -INFINITY;
#pragma unroll 1
            for (int q = 0; q < parts; ++q) {
              load(q);
              float high[4] = {now, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int e = 0; e < 32; e += 8)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  high[y] = fmax3(high[y], __uint_as_float(x[e + y]), __uint_as_float(x[e + 4 + y]));
              now = fmax3(fmaxf(high[0], high[1]), high[2], high[3]);
            }
            const float off = raise(scaled(now));
#pragma unroll 1
            for (int q = 0; q < parts; ++q) {
              load(q);
              weights(x, q, off, q == min(kParts / 2, parts) - 1);
            }
          } else {
            uint32_t x[kParts][32];
#pragma unroll
            for (int q = 0; q < kParts; ++q) tmem_ld32(x[q], ts + q * 32);
            tmem_wait_ld();
            if (some) {
#pragma unroll
              for (int q = 0; q < kParts; ++q) mask(x[q], ok[q]);
            }
            float high[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) high[y] = -INFINITY;
#pragma unroll
            for (int e = 0; e < kTile; e += 16)
#pragma unroll
              for (int y = 0; y < 8; ++y)
                high[y] = fmax3(high[y], __uint_as_float(x[e / 32][e % 32 + y]),
                               __uint_as_float(x[e / 32][e % 32 + 8 + y]));
            const float off =
                raise(scaled(fmax3(fmax3(high[0], high[1], high[2]),
                                   fmax3(high[3], high[4], high[5]), fmaxf(high[6], high[7]))));
#pragma unroll
            for (int q = 0; q < kParts; ++q) weights(x[q], q, off, q == kParts / 2 - 1);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_wait_st();
        } else {
          mbar_arrive(&sh.p_half[buf]);
        }
        fence_before();
        mbar_arrive(&sh.p_full[buf]);
      }

      // ---- the stretch's sums: both streams', half of the columns each, or the block's ----
      // The maxima and weights are handed over, and what follows from them is computed, while
      // the last products are under way (256 sequences of 10 to 200 tokens 66.6 us instead of 68.2,
      // 32 x 64 nodes 126 instead of 129).
      const bool mine_has = S::kOne || j0 < n, other_has = S::kByTiles && (j0 ^ 1) < n;
      if (i > 0) mbar_wait(&sh.o_empty, (i - 1) & 1, &sh.err, p.status);  // ml has been read
      if (!S::kOne || b == 0) sh.ml[b][m] = make_float2(top - kLift<T>, l);
      mbar_arrive(&sh.ml_full);
      mbar_wait(&sh.ml_full, i & 1, &sh.err, p.status);
      __syncwarp();
      const bool odd = sh.odd[i & 1] == (int)i + 1;
      float mx, sum, f0, f1 = 0.f;
      if constexpr (S::kByTiles) {
        const float2 m0 = sh.ml[b][m], m1 = sh.ml[b ^ 1][m];
        mx = fmaxf(m0.x, m1.x);
        const float off = mx == -INFINITY ? 0.f : mx;
        f0 = exp2_fast(m0.x - off);
        f1 = exp2_fast(m1.x - off);
        sum = m0.y * f0 + m1.y * f1;
      } else {
        const float2 m0 = sh.ml[S::kOne ? 0 : b][m];
        mx = m0.x;
        sum = m0.y;
        f0 = 1.f;
      }
      const int pair = job.pair0 + row, node = mine_node;
      const int head = job.head * p.gqa + pair - node * p.gqa;
      const bool whole = job.slot < 0;
      if (mine && (S::kByBlocks || b == 0)) {
        if (!whole)
          p.pml[(int64_t)job.slot * p.part_rows + row] = make_float2(mx, sum);
        else if (a.lse)
          a.lse[((int64_t)job.seq * a.N + node) * a.Hq + head] =
              (mx + log2f(sum)) * 0.6931471805599453f;
      }
      // no token with a score: zeros and -inf
      const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
      constexpr int kCols = S::kByBlocks ? D : D / 2;  // of this warpgroup
      const uint32_t first = S::kByBlocks ? 0 : b * kCols;
      const uint32_t other = tmem + lanes + S::kColO + (b ^ 1) * S::kStepO;
      // The last tile's sums, and with them all before: its barrier is at this turn, the scores
      // of that tile having come to one of the two warpgroups.
      if (!S::kByBlocks || j0 < n) {
        const uint32_t last = c + n - 1;
        mbar_wait(&sh.o_done[S::kByBlocks ? b : last & 3], (S::kByBlocks ? last : last >> 2) & 1,
                  &sh.err, p.status);
        __syncwarp();
      }
      fence_after();
      if (busy && mine_has | other_has) {
#pragma unroll 1
        for (int q = 0; q < kCols; q += 32) {
          const int col = (int)first + q;
          uint32_t y[32], z[S::kByTiles ? 32 : 1];
          __syncwarp();                          // the loads are the whole warp's
          // the sums of a stream without tiles are whatever the columns held
          auto load = [&](uint32_t (&x)[32], bool has, uint32_t from) {
            if (has) {
              tmem_ld32(x, from);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = 0u;
            }
          };
          load(y, mine_has, to + col);
          if constexpr (S::kByTiles) load(z, other_has, other + col);
          tmem_wait_ld();
          const float2 by0 = make_float2(f0 * inv, f0 * inv), by1 = make_float2(f1 * inv, f1 * inv);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 x = mul2(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), by0);
            if constexpr (S::kByTiles)
              x = fma2(make_float2(__uint_as_float(z[e]), __uint_as_float(z[e + 1])), by1, x);
            y[e] = __float_as_uint(x.x);
            y[e + 1] = __float_as_uint(x.y);
          }
          if (odd && mine && !(whole && sum == 0.f)) {
            // values that are no numbers, of the nodes on the path whose tiles were here
            const int v0 = max(0, -cached) * kTile, v1 = (n - cached) * kTile;
            for (int v = node;; v = sh.parent[v]) {
              if (v < v0) break;
              const T* value = static_cast<const T*>(a.v.ptr) + job.seq * a.v.page_stride +
                               v * a.v.token_stride + job.head * a.v.head_stride + col;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float z = to_float(value[e]);
                if (v < v1 && !(fabsf(z) < INFINITY))
                  y[e] = __float_as_uint(__uint_as_float(y[e]) + z);
              }
              if (v == 0) break;
            }
          }
          if (mine && whole) {
            T* out = static_cast<T*>(a.out) + job.seq * a.out_seq_stride +
                     node * a.out_node_stride + head * a.out_head_stride + col;
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t z[8];
#pragma unroll
              for (int g = 0; g < 8; ++g)
                z[g] = pack2<T>(__uint_as_float(y[e + 2 * g]), __uint_as_float(y[e + 2 * g + 1]));
              if (p.wide_rows) {
                store32(out + e, z);
              } else {
                *reinterpret_cast<uint4*>(out + e) = make_uint4(z[0], z[1], z[2], z[3]);
                *reinterpret_cast<uint4*>(out + e + 8) = make_uint4(z[4], z[5], z[6], z[7]);
              }
            }
          } else if (mine) {
            float* out = p.po + part_at<D>(job.slot, p.part_rows, row, col);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(out + e * p.part_rows) =
                  make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
      }
      fence_before();
      mbar_arrive(&sh.o_empty);
      if (!S::kByBlocks || b == 0 || second) c += n;
      all_tiles += (uint32_t)n;
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    fence_after();
    tmem_free(tmem);
  }
}

// ---- the join -------------------------------------------------------------------------------
// Bound by the latency of its loads, and from many pairs on by L2: 40 MB of partials take 8 us
// at 32 x 64 nodes.  (The last CTA of an item as the one that joins it, in the same launch, was
// slower: one stream 17.0 us instead of 13.7, 32 x 64 nodes 135 instead of 128.)
// A CTA per worker's CTA that began an item that others went on with, and eight of the
// item's pairs; a warp per 32 dimensions, whose lanes read a line of four dimensions of the
// eight pairs at a time.
template <typename T, int D, int BLOCKS>
__global__ void __launch_bounds__(D) tree_join_kernel(const __grid_constant__ TreeAttnParams p) {
  const ssd_tree_attn& a = p.a;
  const int groups = p.part_rows / 8;
  const int cta = blockIdx.x / groups, group = blockIdx.x - cta * groups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_previous();
  const int2 begun = p.begun[cta];
  const int item = begun.x, np = begun.y;
  if (item < 0) return;
  const int i = group * 8 + (lane & 7);
  const int x = cta % p.side, bb = x / p.hg;
  int rest = item / p.side;
  const int mb = rest % p.block_sets * p.bg + bb;
  rest /= p.block_sets;
  const int h = rest % p.sets * p.hg + x - bb * p.hg, seq = rest / p.sets;
  const int pair = mb * (BLOCKS * p.block_pairs) + i;
  const bool mine = i < BLOCKS * p.block_pairs && pair < p.pairs;
  // the partial of the worker that began it, then those of workers that went on
  auto slot_of = [&](int j) { return 2 * (cta + j * p.side) + (j == 0); };
  // the loads of so many partials are in flight together (one stream of 4000 tokens 16.2 us
  // instead of 18.8 with four); items of many pairs have few, and want the registers
  constexpr int kBatch = BLOCKS == 2 ? 4 : 8;
  const int d = warp * 32 + (lane >> 3) * 4;
  float top = -INFINITY, l = 0.f;
  float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int j0 = 0; j0 < np; j0 += kBatch) {
    float2 ml[kBatch];
    float4 x[kBatch][2];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      ml[j] = make_float2(-INFINITY, 0.f);
      if (j0 + j < np) {
        const int slot = slot_of(j0 + j);
        ml[j] = p.pml[(int64_t)slot * p.part_rows + i];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[j][e] =
              *reinterpret_cast<const float4*>(p.po + part_at<D>(slot, p.part_rows, i, d + e * 16));
      }
    }
    float now = top;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) now = fmaxf(now, ml[j].x);
    const float off = now == -INFINITY ? 0.f : now, keep = exp2_fast(top - off);
    top = now;
    l *= keep;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      o[e] = make_float4(o[e].x * keep, o[e].y * keep, o[e].z * keep, o[e].w * keep);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (j0 + j >= np) break;
      const float f = exp2_fast(ml[j].x - off);
      l = fmaf(ml[j].y, f, l);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        o[e].x = fmaf(x[j][e].x, f, o[e].x);
        o[e].y = fmaf(x[j][e].y, f, o[e].y);
        o[e].z = fmaf(x[j][e].z, f, o[e].z);
        o[e].w = fmaf(x[j][e].w, f, o[e].w);
      }
    }
  }
  if (!mine) return;
  const int node = p.by_gqa.quotient(pair), head = h * p.gqa + pair - node * p.gqa;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (l == 0.f) o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);  // of values that are no numbers too
  T* out = static_cast<T*>(a.out) + seq * a.out_seq_stride + node * a.out_node_stride +
           head * a.out_head_stride + d;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    *reinterpret_cast<uint2*>(out + e * 16) =
        make_uint2(pack2<T>(o[e].x * inv, o[e].y * inv), pack2<T>(o[e].z * inv, o[e].w * inv));
  if (d == 0 && a.lse)
    a.lse[((int64_t)seq * a.N + node) * a.Hq + head] = (top + log2f(l)) * 0.6931471805599453f;
}

template <typename T, int D, int BLOCKS>
cudaError_t launch_tree(const TreeAttnParams& p, cudaStream_t s) {
  constexpr int smem = TreeShape<D, BLOCKS>::kSmem;
  const auto kernel = tree_tc_kernel<T, D, BLOCKS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  CUtensorMap km{}, vm{}, kn{}, vn{}, qm{};
  const ssd_tree_attn& a = p.a;
  if (p.box_rows > 0) {
    if (!box_map(&km, a.dtype, a.k_cache, D, a.Hkv, a.page_size, a.num_pages, p.box_rows) ||
        !box_map(&vm, a.dtype, a.v_cache, D, a.Hkv, a.page_size, a.num_pages, p.box_rows) ||
        !box_map(&kn, a.dtype, a.k, D, a.Hkv, a.N, a.B, p.node_rows) ||
        !box_map(&vn, a.dtype, a.v, D, a.Hkv, a.N, a.B, p.node_rows))
      return cudaErrorInvalidValue;
  }
  if (p.q_nodes > 0 &&
      !box_map(&qm, a.dtype, {a.q, a.q_seq_stride, a.q_node_stride, a.q_head_stride}, D, a.Hq, a.N,
               a.B, p.q_nodes, p.gqa))
    return cudaErrorInvalidValue;
  kernel<<<p.workers * p.side, kTreeThreads, smem, s>>>(p, km, vm, kn, vn, qm);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(p.workers * p.side * (p.part_rows / 8)));
  c.blockDim = dim3(D);
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, tree_join_kernel<T, D, BLOCKS>, p);
}

template <typename T>
cudaError_t launch_tree_type(const TreeAttnParams& p, cudaStream_t s) {
  const bool two = tree_blocks(p.a.D, p.pairs) == 2;
  switch (p.a.D) {
    case 64: return two ? launch_tree<T, 64, 2>(p, s) : launch_tree<T, 64, 1>(p, s);
    case 128: return two ? launch_tree<T, 128, 2>(p, s) : launch_tree<T, 128, 1>(p, s);
    default: return launch_tree<T, 256, 1>(p, s);
  }
}

}  // namespace
}  // namespace ssd
