// ssd_attention_tc.cu -- attention of a group's rows over its shared prefix on
// the 5th-generation tensor cores.
//
// A block is 128 (row, head) pairs of one key/value head, a tile 128 tokens:
// S = Q K^T (128 x 128 x D), P = exp2(S * scale - m), O += P V.  The bytes of a
// tile (64 KB at D = 128) take an SM 1.4 us at the copy rate of the memory, its
// two products 0.5 us of the tensor cores and its 16384 exponentials as long,
// so up to one full block of pairs the prefix is read at the rate of the
// memory whatever the number of rows: padding a few rows to 128 costs nothing
// that is short.  What has to hold is that the products, the exponentials and
// the copies of different tiles overlap:
//   - two warps issue the copies, of K and of V: a TMA box per page and 64
//     dimensions, into rings of tiles;
//   - one thread issues the products.  Two streams of tiles, the even and the
//     odd ones, each with its own scores and sums in tensor memory, so that the
//     products of one run during the exponentials of the other;
//   - two warpgroups compute the exponentials, one per stream, a row of scores
//     per thread.  Each keeps its own maximum and weight; P replaces S in
//     tensor memory and is the A operand from there, in the type of V as the
//     product takes it: each weight is off by at most half a step, which an
//     output averages over its tokens (against 64 bits 0.0022 of the outputs'
//     norm instead of the 0.0017 of their own rounding, in bf16); its sum is of
//     the unrounded weights.  Any offset gives the same quotient, so the sums
//     are rescaled only when the maximum rose by more than 2^8.
// At the end of a stretch the two streams' sums are joined, each warpgroup
// half of the columns, and written as one partial.
//
// Measured: 32 prefixes of 500 to 8191 tokens for 12 rows each take 93 us, 6.1 TB/s
// (90% of a copy); one prompt of 16000 tokens for 256 rows, 36 us of products at the
// library's rate, 59 us by all SMs, bound by the chain of a tile (scores, exponentials,
// sums) of which two run at a time.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ssd_attention_dev.cuh"

namespace ssd {
namespace {

constexpr int kBlock = kTcBlock;  // pairs of a block (M)
constexpr int kTile = kTcTile;    // tokens of a tile
constexpr int kSoftmax = 256;     // threads of the two warpgroups
constexpr int kHeader = 3 << 10;  // bytes of shared memory before the rings
constexpr int kThreads = kSoftmax + 128;  // a third warpgroup: copies and products
constexpr int kCopyK = 8, kCopyV = 9, kMmaWarp = 10, kQueryWarp = 11;
// Registers per thread: launched with 168 (12 warps), of which the third
// warpgroup gives up 80 and the others take 40 each: 8 * 208 + 4 * 88 = 12 * 168.
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
constexpr int kPanel = kTile * 128;  // bytes of 128 rows x 64 elements, 128-byte swizzle
constexpr float kRise = 8.f;      // scores may pass the kept maximum by this (base 2)

template <int D> struct Shape {
  static constexpr int kPanels = D / 64;
  static constexpr int kSlot = kPanels * kPanel;    // K or V of a tile
  static constexpr int kSlots = D == 64 ? 6 : 3;    // K and V: 192 KB, one CTA per SM
  static constexpr int kSmem = kHeader + (2 * kSlots + 1) * kSlot;  // header, rings, queries
};

// tensor memory columns: scores (and weights) of the two streams, their sums
constexpr int kColS = 0, kColO = 256, kColStep = 128, kCols = 512;

__device__ __forceinline__ void tmem_alloc(uint32_t* where) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(where)),
               "n"(kCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "n"(kCols)
               : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One thread of a converged warp: the compiler then knows that what it issues
// is uniform.
__device__ __forceinline__ bool elected() {
  uint32_t is;
  asm volatile(
      "{.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;}" : "=r"(is));
  return is != 0;
}

// Shared-memory operand: 128-byte swizzle; `lead` bytes between 64-element
// columns of atoms (operands whose rows are the K dimension), 1024 bytes
// between atoms of 8 rows.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Product of 16-bit types into float32, M = 128.
template <typename T>
__device__ __forceinline__ constexpr uint32_t product(int n, bool b_rows_are_k) {
  const uint32_t type = sizeof(T) == 2 && !__is_same(T, __half) ? 1u : 0u;
  return 1u << 4 | type << 7 | type << 10 | (b_rows_are_k ? 1u << 16 : 0u) |
         (uint32_t)(n >> 3) << 17 | (uint32_t)(kBlock >> 4) << 24;
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                        int c2, int c3, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// What the product and exponential warps know of a stretch.
struct Job {
  int tiles;        // 0: no more
  int tokens;       // from the first tile on
  int pairs;        // of the block
  int slot;         // of the partial
};

struct Header {
  float2 ml[2][kBlock];             // the streams' maxima and weights, handed over at the end
  uint64_t k_full[6], k_empty[6];   // ring slots
  uint64_t v_full[6], v_empty[6];
  uint64_t q_full, q_empty;         // a stretch's job and queries; its scores are all done
  uint64_t job_read;                // its job is known to the exponentials' threads
  uint64_t s_full[2];               // scores of a tile are there
  uint64_t p_full[2];               // its weights are
  uint64_t o_done[2];               // its part of the sums is
  uint64_t ml_full;                 // both streams' maxima and weights are in place
  uint64_t o_empty;                 // the sums of a stretch have been read
  uint64_t drained;
  Job job[2];                       // by the parity of the stretch
  int4 warp_sums[kThreads / 32];
  Start start;
  uint32_t tmem;
  volatile int err;
};
// With the rings it fills the 227 KB of an SM: it ends where they start, on a
// 1024-byte boundary.
static_assert(sizeof(Header) <= kHeader, "header");

// Whether a wait of the CTA ran out (to every lane of a warp alike): no new
// work is begun then.
__device__ __forceinline__ bool gave_up(const Header& sh) {
  return __any_sync(0xffffffffu, sh.err) != 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<D>;
  extern __shared__ __align__(1024) unsigned char s_raw[];
  Header& sh = *reinterpret_cast<Header*>(s_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t kring = smem_addr(s_raw) + kHeader;
  const uint32_t vring = kring + S::kSlots * S::kSlot;
  const uint32_t qs = vring + S::kSlots * S::kSlot;

  start_next();
  if (warp == kMmaWarp) tmem_alloc(&sh.tmem);
  if (tid == 0) {
    sh.err = 0;
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 1);
    }
    mbar_init(&sh.q_full, 32);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], kBlock);
      mbar_init(&sh.o_done[i], 1);
    }
    mbar_init(&sh.job_read, kSoftmax);
    mbar_init(&sh.ml_full, kSoftmax);
    mbar_init(&sh.o_empty, kSoftmax);
    mbar_init(&sh.drained, 1);
    fence_barrier_init();
  }
  const int w = blockIdx.x / p.hg;
  const Split all = find_starts<kThreads, 1>(p, w, &sh.start, sh.warp_sums);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;

  // the third warpgroup's warps walk the stretches by themselves
  Walk k;
  k.u = all.first(w);
  k.u1 = all.first(w + 1);
  k.w = w;
  k.hh = blockIdx.x - w * p.hg;
  if (k.u < k.u1) {
    k.g = sh.start.g;
    k.unit = sh.start.unit;
    k.item = sh.start.item;
  }
  Stretch s;

  if (warp >= kSoftmax / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kCopyK || warp == kCopyV) {
      // ---- copies: a warp for K and one for V, one lane per page of a tile -------------
      const bool v = warp == kCopyV;
      const CUtensorMap* map = v ? &vmap : &kmap;
      uint64_t* full = v ? sh.v_full : sh.k_full;
      uint64_t* empty = v ? sh.v_empty : sh.k_empty;
      const uint32_t slots = v ? vring : kring;
      const int P = p.a.page_size;
      const int rows = min(P, kTile);            // tokens of a box
      const int boxes = kTile / rows;            // boxes of a whole tile, at most 16
      // A prefix that one block reads is not read again: it leaves L2 first, so
      // that the partials stay there for the join.  With more blocks it stays.
      uint64_t once, again;
      asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
      asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
      uint32_t c = 0;                            // tiles so far
      while (next_stretch(p, k, s)) {
        const uint64_t policy = s.q.blocks == 1 ? once : again;
        const int32_t* table = p.a.prefix_tables + (int64_t)s.g * p.a.prefix_table_stride;
        auto page_at = [&](int tile) {  // not looked at here: the load stays in flight
          const int t = tile * kTile + lane * rows;
          return lane < boxes && tile < s.tile1 && t < s.q.len ? table[p.by_page.quotient(t)] : 0;
        };
        // pages are looked up two tiles ahead of their copies
        int page = page_at(s.tile0), next = page_at(s.tile0 + 1);
        for (int tile = s.tile0; tile < s.tile1; ++tile, ++c) {
          if (gave_up(sh)) {
            k.u = k.u1;
            break;
          }
          const int after = page_at(tile + 2);
          if ((unsigned)page >= (unsigned)p.a.num_pages) {
            flag(p, SSD_DEV_BAD_PAGE);
            page = p.a.num_pages;                // past the end: the box is zeros
          }
          const int here = min(kTile, s.q.len - tile * kTile);
          const int n = (here + rows - 1) / rows;  // boxes with tokens
          const int in_page = boxes == 1 ? tile * kTile % P : 0;
          const int slot = c % S::kSlots;
          const uint32_t use = c / S::kSlots;
          if (use > 0) mbar_wait(&empty[slot], (use - 1) & 1, &sh.err, p.status);
          if (lane == 0)
            mbar_arrive_expect_tx(&full[slot], (uint32_t)(n * rows * 128 * S::kPanels));
          __syncwarp();
          if (lane < n) {
            const uint32_t dst = slots + slot * S::kSlot + lane * rows * 128;
#pragma unroll
            for (int d = 0; d < S::kPanels; ++d)
              tma_box(dst + d * kPanel, map, d * 64, s.h, in_page, page, &full[slot],
                      policy);
          }
          page = next;
          next = after;
        }
      }
      if (sh.err) {  // let the copies in flight land before the memory is given up
        for (uint32_t i = c > S::kSlots ? c - S::kSlots : 0; i < c; ++i) {
          int none = 0;
          mbar_wait(&full[i % S::kSlots], (i / S::kSlots) & 1, &none, nullptr);
        }
      }
    } else if (warp == kQueryWarp) {
      // ---- queries: a stretch's, as soon as the scores of the one before are done ------
      uint32_t i = 0;
      while (next_stretch(p, k, s)) {
        const int pair0 = s.mb * kBlock, pairs = min(kBlock, s.q.rows * p.gqa - pair0);
        auto query = [&](const Stretch& z, int row) {
          const int pair = z.mb * kBlock + row;
          return static_cast<const T*>(p.a.q) +
                 (int64_t)(z.q.row0 + p.by_gqa.quotient(pair)) * p.a.q_row_stride +
                 (int64_t)(z.h * p.gqa + pair - p.by_gqa.quotient(pair) * p.gqa) *
                     p.a.q_head_stride;
        };
        if (i > 0) mbar_wait(&sh.q_empty, (i - 1) & 1, &sh.err, p.status);
        constexpr int kLanes = D / 8;            // lanes of a row, 16 bytes each
#pragma unroll 8
        for (int r0 = 0; r0 < kBlock; r0 += 32 / kLanes) {
          const int row = r0 + lane / kLanes, ch = lane % kLanes;
          const bool ok = row < pairs;           // past the last pair: zeros
          copy16(qs + (ch / 8) * kPanel + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                 query(s, ok ? row : 0) + ch * 8, ok);
        }
        // a thread that waits for the last job must not find two newer ones: a
        // barrier tells only the parity of its phase
        if (i > 0) mbar_wait(&sh.job_read, (i - 1) & 1, &sh.err, p.status);
        if (lane == 0)
          sh.job[i & 1] = Job{s.tile1 - s.tile0, s.q.len - s.tile0 * kTile, pairs, s.slot};
        copies_commit();
        copies_wait<0>();
        fence_async();
        mbar_arrive(&sh.q_full);  // 32 arrivals: lane 0's follows the job
        ++i;
        if (lane == 0) leave_worker(p, s, w);
        // the next ones into L2 meanwhile
        Walk k1 = k;
        Stretch s1;
        if (next_stretch(p, k1, s1)) {
          const int n = min(kBlock, s1.q.rows * p.gqa - s1.mb * kBlock);
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
      if (lane == 0) sh.job[i & 1].tiles = 0;
      __syncwarp();
      mbar_arrive(&sh.q_full);
    } else {
      // ---- products: the warp runs in step, one elected thread issues ------------------
      constexpr uint32_t score = product<T>(kTile, false), sum = product<T>(D, true);
      const uint64_t q_op = operand(qs, 16);
      uint32_t c = 0;                            // tiles so far
      for (uint32_t i = 0;; ++i) {
        mbar_wait(&sh.q_full, i & 1, &sh.err, p.status);
        const int n = gave_up(sh) ? 0 : sh.job[i & 1].tiles;
        if (n == 0) break;
        fence_after();
        for (int j = 0; j <= n; ++j) {
          if (j < n) {
            const uint32_t t = c + j;
            const int slot = t % S::kSlots;
            mbar_wait(&sh.k_full[slot], t / S::kSlots & 1, &sh.err, p.status);
            fence_after();
            if (elected()) {
              const uint64_t k_op = operand(kring + slot * S::kSlot, 16);
              const uint32_t d = tmem + kColS + (t & 1) * kColStep;
#pragma unroll
              for (int e = 0; e < D / 16; ++e) {
                const uint32_t off = ((e / 4) * kPanel + (e % 4) * 32) >> 4;
                mma_ss(d, q_op + off, k_op + off, score, e > 0);
              }
              commit(&sh.s_full[t & 1]);
              commit(&sh.k_empty[slot]);
              if (j == n - 1) commit(&sh.q_empty);
            }
            __syncwarp();
          }
          if (j > 0) {
            const uint32_t t = c + j - 1, b = t & 1;
            const int slot = t % S::kSlots;
            if (j == 1 && i > 0) mbar_wait(&sh.o_empty, (i - 1) & 1, &sh.err, p.status);
            mbar_wait(&sh.p_full[b], t >> 1 & 1, &sh.err, p.status);
            mbar_wait(&sh.v_full[slot], t / S::kSlots & 1, &sh.err, p.status);
            fence_after();
            if (elected()) {
              const uint64_t v_op = operand(vring + slot * S::kSlot, kPanel);
              const uint32_t d = tmem + kColO + b * kColStep, a = tmem + kColS + b * kColStep;
#pragma unroll
              for (int e = 0; e < kTile / 16; ++e)
                mma_ts(d, a + e * 8, v_op + ((e * 16 * 128) >> 4), sum, j > 2 || e > 0);
              commit(&sh.v_empty[slot]);
              commit(&sh.o_done[b]);
            }
            __syncwarp();
          }
        }
        c += n;
      }
      if (elected()) commit(&sh.drained);
      __syncwarp();
      int none = 0;
      mbar_wait(&sh.drained, 0, &none, p.status);
    }
  } else {
    // ---- exponentials: stream b (the tiles of one parity), pair m of the block ----------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const uint32_t b = warp >> 2, m = tid & (kBlock - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t ts = tmem + lanes + kColS + b * kColStep;
    const uint32_t to = tmem + lanes + kColO + b * kColStep;
    uint32_t c = 0;                              // tiles before the stretch
    for (uint32_t i = 0;; ++i) {
      mbar_wait(&sh.q_full, i & 1, &sh.err, p.status);
      const Job job = sh.job[i & 1];
      const int n = gave_up(sh) ? 0 : job.tiles;
      mbar_arrive(&sh.job_read);
      if (n == 0) break;
      const int j0 = (int)((b ^ c) & 1);         // this stream's first tile of the stretch

      float top = -INFINITY, l = 0.f;
      for (int j = j0; j < n; j += 2) {
        const uint32_t t = c + j;
        mbar_wait(&sh.s_full[b], t >> 1 & 1, &sh.err, p.status);
        __syncwarp();
        fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int e = 0; e < 4; ++e) tmem_ld32(x[e], ts + e * 32);
        tmem_wait_ld();
        const int here = job.tokens - j * kTile;
        if (here < kTile) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q * 32 + e >= here) x[q][e] = 0xff800000u;  // -inf
        }
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            t0 = fmaxf(t0, __uint_as_float(x[q][e]));
            t1 = fmaxf(t1, __uint_as_float(x[q][e + 1]));
          }
        const float now = fmaxf(t0, t1) * p.scale_log2;
        // the kept maximum moves when a score passes it by 2^kRise
        const bool move = now > top + kRise;
        const float old = top;
        if (move) top = now;
        const float off = top == -INFINITY ? 0.f : top;
        if (j > j0 && __any_sync(0xffffffffu, move)) {
          const float f = move ? exp2_fast(old - off) : 1.f;
          l *= f;
          mbar_wait(&sh.o_done[b], (t >> 1) - 1 & 1, &sh.err, p.status);
          fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t y[32];
            tmem_ld32(y, to + q * 32);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
            tmem_st32(to + q * 32, y);
          }
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float y = exp2_fast(fmaf(__uint_as_float(x[q][e]), p.scale_log2, -off));
            sum[e & 3] += y;
            x[q][e] = __float_as_uint(y);
          }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            y[e] = pack2<T>(__uint_as_float(x[2 * q + e / 16][2 * (e % 16)]),
                            __uint_as_float(x[2 * q + e / 16][2 * (e % 16) + 1]));
          tmem_st32(ts + q * 32, y);
        }
        tmem_wait_st();
        if (here < kTile) {
          // rows of V past the last token: whatever the page or the slot held
          // must not meet the zero weights (0 * NaN)
          const int slot = t % S::kSlots;
          mbar_wait(&sh.v_full[slot], t / S::kSlots & 1, &sh.err, p.status);
          const uint32_t vs = vring + slot * S::kSlot;
          for (int e = here * 8 + (int)m; e < kTile * 8; e += kBlock)
#pragma unroll
            for (int d = 0; d < S::kPanels; ++d)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vs + d * kPanel +
                                                                           e * 16),
                           "r"(0)
                           : "memory");
          fence_async();
        }
        fence_before();
        mbar_arrive(&sh.p_full[b]);
      }

      // ---- the stretch's partial: both streams' sums, half of the columns each ----------
      const bool mine_has = j0 < n, other_has = (j0 ^ 1) < n;
      if (mine_has) {
        const uint32_t last = c + j0 + ((n - 1 - j0) & ~1);
        mbar_wait(&sh.o_done[b], last >> 1 & 1, &sh.err, p.status);
      }
      if (i > 0) mbar_wait(&sh.o_empty, (i - 1) & 1, &sh.err, p.status);  // ml has been read
      sh.ml[b][m] = make_float2(top, l);
      fence_before();
      mbar_arrive(&sh.ml_full);
      mbar_wait(&sh.ml_full, i & 1, &sh.err, p.status);
      __syncwarp();
      fence_after();
      const float2 m0 = sh.ml[b][m], m1 = sh.ml[b ^ 1][m];
      const float mx = fmaxf(m0.x, m1.x), off = mx == -INFINITY ? 0.f : mx;
      const float f0 = exp2_fast(m0.x - off), f1 = exp2_fast(m1.x - off);
      const bool mine = (int)m < job.pairs && job.slot < p.nslots;
      if (mine && b == 0)
        p.pml[(int64_t)job.slot * kBlock + m] = make_float2(mx, m0.y * f0 + m1.y * f1);
      uint32_t y0[D / 64][32];
      const uint32_t half = b * (D / 2);         // this warpgroup's columns of both sums
      const uint32_t from0 = to + half, from1 = tmem + lanes + kColO + (b ^ 1) * kColStep + half;
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        uint32_t y1[32];
        tmem_ld32(y0[q], from0 + q * 32);
        tmem_ld32(y1, from1 + q * 32);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          // the sums of a stream without tiles are whatever the columns held
          const float y = mine_has ? __uint_as_float(y0[q][e]) * f0 : 0.f;
          const float z = other_has ? __uint_as_float(y1[e]) * f1 : 0.f;
          y0[q][e] = __float_as_uint(y + z);
        }
      }
      fence_before();
      mbar_arrive(&sh.o_empty);
      if (mine) {
        float* out = p.po + part_at<D>(job.slot, kBlock, m, half);
#pragma unroll
        for (int q = 0; q < D / 64; ++q)
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(out + (q * 32 + e) * kBlock) =
                make_uint4(y0[q][e], y0[q][e + 1], y0[q][e + 2], y0[q][e + 3]);
      }
      c += n;
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

using Encode = decltype(&cuTensorMapEncodeTiled);
Encode encoder() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  return fn;
}

bool make_map(CUtensorMap* map, const ssd_attention& a, const ssd_paged& c) {
  const Encode encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.Hkv, (cuuint64_t)a.page_size,
                              (cuuint64_t)a.num_pages};
  // the stride of a dimension of one is never used
  auto bytes = [](int64_t stride, int64_t n) { return (cuuint64_t)(n > 1 ? stride * 2 : 16); };
  const cuuint64_t strides[3] = {bytes(c.head_stride, a.Hkv), bytes(c.token_stride, a.page_size),
                                 bytes(c.page_stride, a.num_pages)};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)std::min(a.page_size, kTile), 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return encode(map,
                a.dtype == SSD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                4, const_cast<void*>(c.ptr), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm,
                   cudaStream_t s) {
  constexpr int smem = Shape<D>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(
      prefix_tc_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prefix_tc_kernel<T, D><<<p.workers * p.hg, kThreads, smem, s>>>(p, km, vm);
  return cudaGetLastError();
}

}  // namespace

// Boxes have to tile a page and a tile alike, and lie on the copy's grid.
bool prefix_tc_fits(const ssd_attention& a) {
  if (a.D != 64 && a.D != 128) return false;
  if (a.page_size % 8 != 0 || (kTile % a.page_size != 0 && a.page_size % kTile != 0)) return false;
  if (!(a.scale > 0.f)) return false;  // the maximum is taken before the scale
  for (const ssd_paged* c : {&a.k, &a.v}) {
    const int64_t most = (int64_t)1 << 39;  // elements of a stride
    if ((a.Hkv > 1 && (c->head_stride < 1 || c->head_stride >= most)) ||
        (a.page_size > 1 && (c->token_stride < 1 || c->token_stride >= most)) ||
        (a.num_pages > 1 && (c->page_stride < 1 || c->page_stride >= most)))
      return false;
  }
  return true;
}

cudaError_t launch_prefix_tc(const AttnParams& p, cudaStream_t s) {
  CUtensorMap km, vm;
  if (!make_map(&km, p.a, p.a.k) || !make_map(&vm, p.a, p.a.v)) return cudaErrorInvalidValue;
  if (p.a.dtype == SSD_BF16)
    return p.a.D == 64 ? launch<__nv_bfloat16, 64>(p, km, vm, s)
                       : launch<__nv_bfloat16, 128>(p, km, vm, s);
  return p.a.D == 64 ? launch<__half, 64>(p, km, vm, s) : launch<__half, 128>(p, km, vm, s);
}

}  // namespace ssd
