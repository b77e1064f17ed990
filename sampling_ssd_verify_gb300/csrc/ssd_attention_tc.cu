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
//   - one warp issues the copies: a TMA box per page and 64 dimensions, into a
//     ring of K and V slots;
//   - one thread issues the products.  Two streams of tiles, the even and the
//     odd ones, each with its own scores and sums in tensor memory, so that the
//     products of one run during the exponentials of the other;
//   - two warpgroups compute the exponentials, one per stream, a row of scores
//     per thread.  Each keeps its own maximum and weight; P replaces S in
//     tensor memory and is the A operand from there.  The sums are rescaled
//     only when the maximum rose by more than 2^8.
// At the end of a stretch the two streams' sums are joined, each warpgroup
// half of the columns, and written as one partial.

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
constexpr int kThreads = kSoftmax + 128;  // a third warpgroup: copies, products, hints
constexpr int kCopyWarp = 8, kMmaWarp = 9, kHintWarp = 10;
// Registers per thread: launched with 168 (12 warps), of which the third
// warpgroup gives up 80 and the others take 40 each: 8 * 208 + 4 * 88 = 12 * 168.
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
constexpr int kPanel = kTile * 128;  // bytes of 128 rows x 64 elements, 128-byte swizzle
constexpr float kRise = 8.f;      // scores may pass the kept maximum by this (base 2)

template <int D> struct Shape {
  static constexpr int kPanels = D / 64;
  static constexpr int kSlot = kPanels * kPanel;    // K or V of a tile
  static constexpr int kSlots = D == 64 ? 12 : 6;   // 192 KB: one CTA per SM
  static constexpr int kSmem = (kSlots + 1) * kSlot + 1024;
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
                                        int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// Ring positions of K and V of tile j of a stretch of n tiles, counted from the
// stretch's first: in the order in which the products take them (K0, K1, V0, K2,
// V1, ..), so that slots fall free in order and the copies in flight are the
// next ones needed.
__device__ __forceinline__ uint32_t at_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t at_v(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

struct Bars {
  uint64_t full[12], empty[12];   // ring slots
  uint64_t q_full;                // queries of a stretch are in place, its sums' columns free
  uint64_t s_full[2];             // scores of a tile are there
  uint64_t p_full[2];             // its weights are
  uint64_t o_done[2];             // its part of the sums is
  uint64_t drained;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<D>;
  extern __shared__ unsigned char s_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_err;
  __shared__ Start s_start[1];
  __shared__ int2 s_warp[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // operands start on 1024-byte boundaries: ring slots, then the queries
  const uint32_t ring = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t qs = ring + S::kSlots * S::kSlot;
  // the streams' maxima and weights, handed over where the queries were
  float2* s_ml = reinterpret_cast<float2*>(s_raw + (qs - smem_addr(s_raw)));  // [2][kBlock]

  if (warp == kMmaWarp) tmem_alloc(&s_tmem);
  if (tid == 0) {
    s_err = 0;
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    mbar_init(&bars.q_full, kSoftmax);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], kBlock);
      mbar_init(&bars.o_done[i], 1);
    }
    mbar_init(&bars.drained, 1);
    fence_barrier_init();
  }
  const int w = blockIdx.x;
  const int total = find_starts<kThreads, 1>(p, w, s_start, s_warp);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;

  Walk k;
  k.u = first_unit(p, w, total);
  k.u1 = first_unit(p, w + 1, total);
  k.w = w;
  if (k.u < k.u1) {
    k.g = s_start[0].g;
    k.unit = s_start[0].unit;
    k.item = s_start[0].item;
  }
  Stretch s;

  if (warp >= kCopyWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kCopyWarp) {
      // ---- copies: one lane per page of a tile -----------------------------------------
      const int P = p.a.page_size;
      const int rows = min(P, kTile);            // tokens of a box
      const int boxes = kTile / rows;            // boxes of a whole tile, at most 16
      uint32_t c = 0;                            // slots used so far
      while (next_stretch(p, k, s)) {
        const int32_t* table = p.a.prefix_tables + (int64_t)s.g * p.a.prefix_table_stride;
        auto page_at = [&](int tile) {
          const int t = tile * kTile + lane * rows;
          int page = -1;
          if (lane < boxes && tile < s.tile1 && t < s.q.len) {
            page = table[t / P];
            if ((unsigned)page >= (unsigned)p.a.num_pages) {
              flag(p, SSD_DEV_BAD_PAGE);
              page = p.a.num_pages;              // past the end: the box is zeros
            }
          }
          return page;
        };
        // one K or V tile: wait for its slot, announce its bytes, copy its boxes
        auto load = [&](const CUtensorMap* map, int tile, int page) {
          const int here = min(kTile, s.q.len - tile * kTile);
          const int n = (here + rows - 1) / rows;  // boxes with tokens
          const int in_page = boxes == 1 ? tile * kTile % P : 0;
          const int slot = c % S::kSlots;
          const uint32_t use = c / S::kSlots;
          ++c;
          if (use > 0) mbar_wait(&bars.empty[slot], (use - 1) & 1, &s_err, p.status);
          if (lane == 0)
            mbar_arrive_expect_tx(&bars.full[slot], (uint32_t)(n * rows * 128 * S::kPanels));
          __syncwarp();
          if (lane < n) {
            const uint32_t dst = ring + slot * S::kSlot + lane * rows * 128;
#pragma unroll
            for (int d = 0; d < S::kPanels; ++d)
              tma_box(dst + d * kPanel, map, d * 64, s.h, in_page, page, &bars.full[slot]);
          }
        };
        // pages are looked up one tile ahead of their copies
        int page = page_at(s.tile0), last = -1;
        for (int tile = s.tile0; tile < s.tile1; ++tile) {
          const int next = page_at(tile + 1);
          load(&kmap, tile, page);
          if (tile > s.tile0) load(&vmap, tile - 1, last);
          last = page;
          page = next;
        }
        load(&vmap, s.tile1 - 1, last);
      }
      if (s_err) {  // let the copies in flight land before the memory is given up
        for (uint32_t i = c > S::kSlots ? c - S::kSlots : 0; i < c; ++i) {
          int none = 0;
          mbar_wait(&bars.full[i % S::kSlots], (i / S::kSlots) & 1, &none, nullptr);
        }
      }
    } else if (warp == kMmaWarp) {
      // ---- products: one thread ----------------------------------------------------------
      if (lane == 0) {
        constexpr uint32_t score = product<T>(kTile, false), sum = product<T>(D, true);
        uint32_t c = 0, stretch = 0, done[2] = {0, 0};  // slots, stretches, weights used
        while (next_stretch(p, k, s)) {
          const int n = s.tile1 - s.tile0;
          mbar_wait(&bars.q_full, stretch++ & 1, &s_err, p.status);
          fence_after();
          for (int j = 0; j <= n; ++j) {
            if (j < n) {
              const uint32_t at = c + at_k(j);
              const int slot = at % S::kSlots;
              mbar_wait(&bars.full[slot], (at / S::kSlots) & 1, &s_err, p.status);
              fence_after();
              const uint32_t ks = ring + slot * S::kSlot;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint32_t off = (i / 4) * kPanel + (i % 4) * 32;
                mma_ss(tmem + kColS + (j & 1) * kColStep, operand(qs + off, 16),
                       operand(ks + off, 16), score, i > 0);
              }
              commit(&bars.s_full[j & 1]);
              commit(&bars.empty[slot]);
            }
            if (j > 0) {
              const int b = (j - 1) & 1;
              const uint32_t at = c + at_v(j - 1, n);
              const int slot = at % S::kSlots;
              mbar_wait(&bars.p_full[b], done[b]++ & 1, &s_err, p.status);
              mbar_wait(&bars.full[slot], (at / S::kSlots) & 1, &s_err, p.status);
              fence_after();
              const uint32_t vs = ring + slot * S::kSlot;
#pragma unroll
              for (int i = 0; i < kTile / 16; ++i)
                mma_ts(tmem + kColO + b * kColStep, tmem + kColS + b * kColStep + i * 8,
                       operand(vs + i * 16 * 128, kPanel), sum, j > 2 || i > 0);
              commit(&bars.empty[slot]);
              commit(&bars.o_done[b]);
            }
          }
          c += 2 * n;
        }
        commit(&bars.drained);
        int none = 0;
        mbar_wait(&bars.drained, 0, &none, p.status);
      }
    } else if (warp == kHintWarp) {
      // ---- queries of all stretches into L2, so that a stretch starts without a
      // trip to memory (stretches are few: this runs far ahead) -----------------------
      while (next_stretch(p, k, s)) {
        const int n = min(kBlock, s.q.rows * p.gqa - s.mb * kBlock);
        for (int i = lane; i < n; i += 32) {
          const int pair = s.mb * kBlock + i;
          const char* q = reinterpret_cast<const char*>(
              static_cast<const T*>(p.a.q) +
              (int64_t)(s.q.row0 + pair / p.gqa) * p.a.q_row_stride +
              (int64_t)(s.h * p.gqa + pair % p.gqa) * p.a.q_head_stride);
#pragma unroll
          for (int d = 0; d < D * 2; d += 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q + d));
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---- exponentials: stream b, pair m of the block ------------------------------------
    const int b = warp >> 2, m = tid & (kBlock - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t ts = tmem + lanes + kColS + b * kColStep;
    const uint32_t to = tmem + lanes + kColO + b * kColStep;
    uint32_t c = 0, done = 0;                 // slots before the stretch, tiles of this stream
    while (next_stretch(p, k, s)) {
      const int n = s.tile1 - s.tile0, npairs = s.q.rows * p.gqa, pair0 = s.mb * kBlock;
      // queries: 16-byte chunks in the swizzled layout, zeros past the last pair
#pragma unroll
      for (int i = 0; i < kBlock * (D / 8) / kSoftmax; ++i) {
        const int idx = i * kSoftmax + tid, row = idx / (D / 8), ch = idx % (D / 8);
        const int pair = pair0 + row;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (pair < npairs) {
          const T* q = static_cast<const T*>(p.a.q) +
                       (int64_t)(s.q.row0 + pair / p.gqa) * p.a.q_row_stride +
                       (int64_t)(s.h * p.gqa + pair % p.gqa) * p.a.q_head_stride + ch * 8;
          x = *reinterpret_cast<const uint4*>(q);
        }
        const uint32_t d =
            qs + (ch / 8) * kPanel + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(d), "r"(x.x), "r"(x.y),
                     "r"(x.z), "r"(x.w)
                     : "memory");
      }
      fence_async();
      fence_before();
      mbar_arrive(&bars.q_full);

      float top = -INFINITY, l = 0.f;
      for (int j = b; j < n; j += 2) {
        mbar_wait(&bars.s_full[b], done & 1, &s_err, p.status);
        fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(x[i], ts + i * 32);
        tmem_wait_ld();
        const int here = s.q.len - (s.tile0 + j) * kTile;
        if (here < kTile) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (i * 32 + e >= here) x[i][e] = 0xff800000u;  // -inf
        }
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            t0 = fmaxf(t0, __uint_as_float(x[i][e]));
            t1 = fmaxf(t1, __uint_as_float(x[i][e + 1]));
          }
        const float now = fmaxf(t0, t1) * p.scale_log2;
        // the kept maximum moves when a score passes it by 2^kRise
        const bool move = now > top + kRise;
        const float old = top;
        if (move) top = now;
        const float off = top == -INFINITY ? 0.f : top;
        if (j > b && __any_sync(0xffffffffu, move)) {
          const float f = move ? exp2_fast(old - off) : 1.f;
          l *= f;
          mbar_wait(&bars.o_done[b], (done - 1) & 1, &s_err, p.status);
          fence_after();
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            uint32_t y[32];
            tmem_ld32(y, to + i * 32);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
            tmem_st32(to + i * 32, y);
          }
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float y = exp2_fast(fmaf(__uint_as_float(x[i][e]), p.scale_log2, -off));
            sum[e & 3] += y;
            x[i][e] = __float_as_uint(y);
          }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            y[e] = pack2<T>(__uint_as_float(x[2 * i + e / 16][2 * (e % 16)]),
                            __uint_as_float(x[2 * i + e / 16][2 * (e % 16) + 1]));
          tmem_st32(ts + i * 32, y);
        }
        tmem_wait_st();
        if (here < kTile) {
          // rows of V past the last token: whatever the page or the slot held
          // must not meet the zero weights (0 * NaN)
          const uint32_t at = c + at_v(j, n);
          const int slot = at % S::kSlots;
          mbar_wait(&bars.full[slot], (at / S::kSlots) & 1, &s_err, p.status);
          const uint32_t vs = ring + slot * S::kSlot;
          for (int i = here * 8 + m; i < kTile * 8; i += kBlock)
#pragma unroll
            for (int d = 0; d < S::kPanels; ++d)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vs + d * kPanel +
                                                                           i * 16),
                           "r"(0)
                           : "memory");
          fence_async();
        }
        fence_before();
        mbar_arrive(&bars.p_full[b]);
        ++done;
      }

      // ---- the stretch's partial: both streams' sums, half of the columns each ----------
      if (n > b) mbar_wait(&bars.o_done[b], (done - 1) & 1, &s_err, p.status);
      fence_after();
      softmax_sync();  // the products have read the queries: both streams are done
      s_ml[b * kBlock + m] = make_float2(top, l);
      fence_before();
      softmax_sync();
      fence_after();
      const float2 m0 = s_ml[m], m1 = s_ml[kBlock + m];
      const float mx = fmaxf(m0.x, m1.x), off = mx == -INFINITY ? 0.f : mx;
      const float f0 = exp2_fast(m0.x - off), f1 = n > 1 ? exp2_fast(m1.x - off) : 0.f;
      const bool mine = pair0 + m < npairs && s.slot < p.nslots;
      const int64_t row = (int64_t)s.slot * kBlock + m;
      if (mine && b == 0) p.pml[row] = make_float2(mx, m0.y * f0 + m1.y * f1);
      float* out = p.po + part_at<D>(s.slot, kBlock, m, b * (D / 2));
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint32_t y0[32], y1[32];
        const uint32_t col = tmem + lanes + kColO + b * (D / 2) + i * 32;
        tmem_ld32(y0, col);
        if (n > 1) tmem_ld32(y1, col + kColStep);
        tmem_wait_ld();
        if (n > 1) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            y0[e] = __float_as_uint(__uint_as_float(y0[e]) * f0 + __uint_as_float(y1[e]) * f1);
        }
        if (mine) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(out + (i * 32 + e) * kBlock) =
                make_uint4(y0[e], y0[e + 1], y0[e + 2], y0[e + 3]);
        }
      }
      c += 2 * n;
      softmax_sync();  // s_ml is read before the next queries replace it
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
  prefix_tc_kernel<T, D><<<p.workers, kThreads, smem, s>>>(p, km, vm);
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
