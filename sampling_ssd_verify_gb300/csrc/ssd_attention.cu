// ssd_attention.cu -- attention over shared prefixes and own tokens of a
// paged cache (ssd_prefix_attention): the kernel of few rows, the join of
// partial results, and the entry point.
//
// out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), with m the running
// maximum, over any stretch of tokens; two stretches join by weighting each
// with exp(m_i - max m).
//
// The join is bound by the latency of its loads (partials from L2, own tokens from
// memory), not by bytes: 96 us for 6144 rows with 1 to 8 own tokens, whose queries,
// own tokens and outputs would be 31 us at the copy rate.  The kernel of long own caches with
// the join reads them at 5.7 TB/s (256 rows of 0 to 3000 tokens) to 6.7 (64 of 8000) of the
// 6.8 of a copy when it has the memory to itself.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ssd_attention_dev.cuh"

namespace ssd {
namespace {

// ---- a stretch of tokens by one warp -----------------------------------------------
// 16 (row, head) pairs are the M of the matrix instructions, 16 tokens a step.
// Each warp keeps its own ring of steps in shared memory, filled by 16-byte
// asynchronous copies, so warps never wait for one another.
constexpr int kWarpsPerCta = 4;
constexpr int kStep = 16;           // tokens of a step
constexpr int kRing = 3;            // steps of the ring
constexpr int kTileTokens = 64;     // tokens of a tile (the unit of the split)
constexpr int kBlockRows = 16;

template <int D>
__host__ __device__ constexpr int step_bytes() { return 2 * kStep * D * 2; }  // K and V

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4],
                                                 uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Where a stretch's partial goes: dimension d of pair i of the block at
// o + i * o_step + (d / 4) * d_step + d % 4.
struct Partial {
  float* o;
  int64_t o_step, d_step;
  float2* ml;
  int64_t ml_step;
};

// Pairs [pair0, min(pair0 + 16, npairs)) of the rows from row0 on, key/value
// head h, tokens [t0, t1) of `table`.
template <typename T, int D>
__device__ __forceinline__ void warp_stretch(const AttnParams& p, uint32_t ring, int row0,
                                             int pair0, int npairs, int h, const int32_t* table,
                                             int t0, int t1, const Partial& out) {
  constexpr int KK = D / 16;        // k-steps of the scores, 16-dimension groups of the output
  constexpr int CH = D / 8;         // 16-byte chunks of a token
  const int lane = threadIdx.x & 31, quad = lane & 3, gid = lane >> 2;
  const ssd_attention& a = p.a;

  // the queries as A fragments; pairs past the end are zeros
  uint32_t qf[KK][4];
  {
    const T* q0 = nullptr;
    const T* q1 = nullptr;
    const int i0 = pair0 + gid, i1 = i0 + 8;
    auto query = [&](int i) {
      const int r = p.by_gqa.quotient(i);
      return static_cast<const T*>(a.q) + (int64_t)(row0 + r) * a.q_row_stride +
             (int64_t)(h * p.gqa + i - r * p.gqa) * a.q_head_stride;
    };
    if (i0 < npairs)
      q0 = query(i0);
    if (i1 < npairs)
      q1 = query(i1);
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      const int c = k * 16 + quad * 2;
      qf[k][0] = q0 ? *reinterpret_cast<const uint32_t*>(q0 + c) : 0u;
      qf[k][1] = q1 ? *reinterpret_cast<const uint32_t*>(q1 + c) : 0u;
      qf[k][2] = q0 ? *reinterpret_cast<const uint32_t*>(q0 + c + 8) : 0u;
      qf[k][3] = q1 ? *reinterpret_cast<const uint32_t*>(q1 + c + 8) : 0u;
    }
  }

  float o[2 * KK][4];
#pragma unroll
  for (int n = 0; n < 2 * KK; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  const int steps = (t1 - t0 + kStep - 1) / kStep;
  // lane i (and i + 16) looks up the page of token i of a step, one step
  // before its copies are issued
  auto page_of = [&](int step) {
    const int t = t0 + step * kStep + (lane & 15);
    return t < t1 ? table[p.by_page.quotient(t)] : -1;
  };
  auto issue = [&](int step, int page) {
    const int t = t0 + step * kStep + (lane & 15);
    bool ok = t < t1;
    if (ok && (unsigned)page >= (unsigned)a.num_pages) {
      ok = false;
      flag(p, SSD_DEV_BAD_PAGE);
    }
    const int in_page = ok ? t - p.by_page.quotient(t) * a.page_size : 0;
    const int64_t pg = ok ? page : 0;
    // a token that is not there: a negative offset, no read
    const int64_t ko = ok ? pg * a.k.page_stride + in_page * a.k.token_stride : -1;
    const int64_t vo = ok ? pg * a.v.page_stride + in_page * a.v.token_stride : -1;
    const T* kb = static_cast<const T*>(a.k.ptr) + h * a.k.head_stride;
    const T* vb = static_cast<const T*>(a.v.ptr) + h * a.v.head_stride;
    const uint32_t ks = ring + (step % kRing) * step_bytes<D>();
    const uint32_t vs = ks + kStep * D * 2;
#pragma unroll
    for (int i = 0; i < kStep * CH / 32; ++i) {
      const int idx = i * 32 + lane, tok = idx / CH, c = idx % CH;
      const int64_t k_at = __shfl_sync(0xffffffffu, ko, tok);
      const int64_t v_at = __shfl_sync(0xffffffffu, vo, tok);
      const uint32_t d = tok * (D * 2) + ((c ^ (tok & 7)) << 4);
      copy16(ks + d, kb + (k_at < 0 ? 0 : k_at + c * 8), k_at >= 0);
      copy16(vs + d, vb + (v_at < 0 ? 0 : v_at + c * 8), v_at >= 0);
    }
  };

  __syncwarp();  // the ring's last readers are done
  int page = page_of(0);
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) {
    if (s < steps) issue(s, page);
    copies_commit();
    page = s + 1 < steps ? page_of(s + 1) : -1;
  }
  for (int s = 0; s < steps; ++s) {
    copies_wait<kRing - 2>();
    __syncwarp();
    if (s + kRing - 1 < steps) issue(s + kRing - 1, page);
    copies_commit();
    if (s + kRing < steps) page = page_of(s + kRing);

    const uint32_t ks = ring + (s % kRing) * step_bytes<D>();
    const uint32_t vs = ks + kStep * D * 2;
    float sc[2][4] = {};
    {
      const int tok = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        uint32_t b[4];
        ldsm4<false>(b, ks + tok * (D * 2) + (((2 * k + half) ^ (tok & 7)) << 4));
        mma16816<T>(sc[0], qf[k], b[0], b[1]);
        mma16816<T>(sc[1], qf[k], b[2], b[3]);
      }
    }
    const int left = t1 - (t0 + s * kStep);  // tokens of this step that are there
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = n * 8 + quad * 2 + (i & 1);
        sc[n][i] = col < left ? sc[n][i] * p.scale_log2 : -INFINITY;
        top[i >> 1] = fmaxf(top[i >> 1], sc[n][i]);
      }
    float keep[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      const float m1 = fmaxf(m[r], top[r]);
      const float off = m1 == -INFINITY ? 0.f : m1;
      keep[r] = exp2_fast(m[r] - off);
      m[r] = m1;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sc[n][2 * r + i] = exp2_fast(sc[n][2 * r + i] - off);
          sum += sc[n][2 * r + i];
        }
      l[r] = l[r] * keep[r] + sum;
    }
    // weights in the type of the values, as the product takes them: half a step of each,
    // which an output averages over its tokens; their sum l is of the unrounded ones
    const uint32_t pf[4] = {pack2<T>(sc[0][0], sc[0][1]), pack2<T>(sc[0][2], sc[0][3]),
                            pack2<T>(sc[1][0], sc[1][1]), pack2<T>(sc[1][2], sc[1][3])};
    const int tok = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      uint32_t b[4];
      ldsm4<true>(b, vs + tok * (D * 2) + (((2 * k + (lane >> 4)) ^ (tok & 7)) << 4));
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float(&c)[4] = o[2 * k + n];
        c[0] *= keep[0];
        c[1] *= keep[0];
        c[2] *= keep[1];
        c[3] *= keep[1];
        mma16816<T>(c, pf, b[2 * n], b[2 * n + 1]);
      }
    }
  }
  copies_wait<0>();

#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int i = gid + 8 * r;
    if (pair0 + i >= npairs) continue;
    if (quad == 0) out.ml[i * out.ml_step] = make_float2(m[r], l[r]);
    float* to = out.o + i * out.o_step + (quad >> 1) * out.d_step + (quad & 1) * 2;
#pragma unroll
    for (int n = 0; n < 2 * KK; ++n)
      *reinterpret_cast<float2*>(to + 2 * n * out.d_step) =
          make_float2(o[n][2 * r], o[n][2 * r + 1]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarpsPerCta * 32)
    prefix_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(128) unsigned char s_ring[];
  __shared__ Start s_start[kWarpsPerCta];
  __shared__ int4 s_warp[kWarpsPerCta];
  start_next();
  const int w0 = blockIdx.x * kWarpsPerCta, warp = threadIdx.x >> 5, w = w0 + warp;
  const Split all = find_starts<kWarpsPerCta * 32, kWarpsPerCta>(p, w0, s_start, s_warp);
  const uint32_t ring = smem_addr(s_ring) + warp * kRing * step_bytes<D>();
  Walk k;
  k.u = all.first(w);
  k.u1 = all.first(w + 1);
  if (k.u >= k.u1) return;
  k.g = s_start[warp].g;
  k.unit = s_start[warp].unit;
  k.item = s_start[warp].item;
  k.w = w;
  k.hh = 0;
  Stretch s;
  while (next_stretch(p, k, s)) {
    if (s.slot >= p.nslots) break;  // cannot happen: the host sized the slots for every split
    if ((threadIdx.x & 31) == 0) leave_worker(p, s, w);
    const Partial out{p.po + part_at<D>(s.slot, kBlockRows, 0, 0), 4, kBlockRows * 4,
                      p.pml + (int64_t)s.slot * kBlockRows, 1};
    warp_stretch<T, D>(p, ring, s.q.row0, s.mb * kBlockRows, s.q.rows * p.gqa, s.h,
                       p.a.prefix_tables + (int64_t)s.g * p.a.prefix_table_stride,
                       s.tile0 * kTileTokens, min(s.q.len, s.tile1 * kTileTokens), out);
  }
}

// Tokens of row r's own cache, clamped into range.
__device__ __forceinline__ int own_len(const AttnParams& p, int r) {
  if (!p.a.lens) return 0;
  const long long most = (long long)p.a.cols * p.a.page_size;
  const int n = p.a.lens[r];
  return n < 0 ? 0 : n > most ? (int)most : n;
}
// Tokens of one of the nsplit stretches, whole steps.
__device__ __forceinline__ int own_stretch(const AttnParams& p, int len) {
  return ((len + p.nsplit - 1) / p.nsplit + kStep - 1) / kStep * kStep;
}

template <typename T, int D>
__device__ __forceinline__ void own_task(const AttnParams& p, uint32_t ring, int64_t task,
                                         int blocks) {
  // heads side by side: a token's lie next to each other (256 rows with 0 to 900 tokens
  // on 8 heads over a prompt of 16000: 128.0 us instead of 128.7; own caches of 0 to 1800
  // over 40000 and 19 groups of a few rows on 4 heads: the same)
  const int h = (int)(task % p.a.Hkv);
  task /= p.a.Hkv;
  const int split = (int)(task % p.nsplit);
  task /= p.nsplit;
  const int mb = (int)(task % blocks), r = (int)(task / blocks);
  const int len = own_len(p, r), n = own_stretch(p, len);
  const int t0 = min(len, split * n), t1 = min(len, t0 + n);
  if (h == 0 && mb == 0 && split == 0 && (threadIdx.x & 31) == 0 && len != p.a.lens[r])
    flag(p, SSD_DEV_BAD_LENGTH);
  if (t0 >= t1) return;  // the join does not look at it
  const int64_t at = ((int64_t)r * p.a.Hq + h * p.gqa + mb * kBlockRows) * p.nsplit + split;
  const Partial out{p.so + at * D, (int64_t)p.nsplit * D, 4, p.sml + at, p.nsplit};
  warp_stretch<T, D>(p, ring, r, mb * kBlockRows, p.gqa, h, p.a.tables + (int64_t)r * p.a.table_stride, t0, t1, out);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarpsPerCta * 32)
    own_kernel(const __grid_constant__ AttnParams p, int blocks) {
  extern __shared__ __align__(128) unsigned char s_ring[];
  start_next();
  const int warp = threadIdx.x >> 5;
  int64_t task = (int64_t)blockIdx.x * kWarpsPerCta + warp;
  if (task < (int64_t)p.a.R * p.a.Hkv * blocks * p.nsplit)
    own_task<T, D>(p, smem_addr(s_ring) + warp * kRing * step_bytes<D>(), task, blocks);
  // It needs nothing of the prefixes' kernel; but the join that waits for this one
  // must find that one done too, so one CTA stays until it is.
  if (blockIdx.x == gridDim.x - 1) wait_previous();
}

// ---- the join ------------------------------------------------------------------------
// One warp per row and up to eight of its query heads: the row's own tokens, or
// their partials, then the prefix's partials, then the output.  With few query
// heads to a key/value head a warp takes several key/value heads (eight, four or
// two), so that its lanes all have a head: their scores come from one product
// each, of which a lane keeps its own head's, and the sums add up over the
// key/value heads, with the weights of the others' heads zero.
//
// Own tokens are few in the calls that this kernel is made for (a branch's
// drafts), and such a task is a chain of loads: page, tokens, partials.  It is
// bound by their latency and by what it issues around them, so the operands of
// the products come straight from global memory, in an order of the dimensions
// that needs no exchange between lanes and in which every load of a warp takes
// whole sectors.  In 16-byte chunks of 8 dimensions: lane (gid, quad) holds
// chunks quad + 4 i of query head gid and of token gid, whose elements 4 s .. 4 s
// + 3 are the k of product s of Q K^T; and chunks gid + 8 i of tokens 2 quad and
// 2 quad + 1, whose element e is column gid of product 8 i + e of the sums: so it
// receives, of head gid, dimensions 64 i + 16 quad + e and + 8.  Long own caches
// go through own_kernel, split over many warps.
constexpr int kJoinWarps = 8;
constexpr int kJoinHeads = 8;
template <int D> constexpr int kJoinCtas = D == 256 ? 1 : 2;  // per SM, by registers
// Own caches that the join reads: of so many tokens, or of one page of so many, which
// is rarely full.  The host knows the tables' width, not the lengths.  Read by the join
// and by own_kernel: 32 x 12 branches with up to 4 tokens 106 and 109 us, up to 16 111 and
// 110, up to 30 118 and 112; 256 x 24 with up to 4 of a page of 64 291 and 415, up to 8
// 299 and 417, up to 32 406 and 437, up to 64 522 and 478; up to 16 of a page of 16 337
// and 423.  So a few tokens in wider tables, which go through own_kernel, take up to 124
// us more than they would in the join.
constexpr int kShortOwn = 16, kShortPage = 64;

// How a row's query heads are dealt to tasks: `pack` key/value heads of 8 / pack
// lanes each, or, with more than eight query heads, `blocks` tasks for one.  With
// few tasks, `split` warps (a CTA) share the partials of one: two rows over a
// prefix of 10000 tokens have a hundred.
struct Deal {
  int pack, blocks, tasks, split;
};
template <int D>
constexpr int join_bytes(int split) {  // half the warps' sums, weights and maxima
  return split / 2 * 32 * (D / 4 + 2) * 4;
}

// The prefix's partials of a pair: np of them, every hg-th from `slot` on, at row `i`.
struct Parts {
  int np, slot, i;
};
__device__ __forceinline__ Parts parts_of(const AttnParams& p, const int4& row, int h, int head) {
  if (row.x < 0) return Parts{0, 0, 0};
  const int i = row.y + head, mb = p.mt == kTcBlock ? i / kTcBlock : i / kBlockRows;
  const int set = h / p.hg, hh = h - set * p.hg;
  const int item = (row.x + set * row.z + mb) * p.hg + hh;
  const int2 w = p.item_workers[item];
  return Parts{w.y - w.x + 1, item + w.x * p.hg, i - mb * p.mt};
}

// Eight rows (heads) of the 16 that an instruction has; the others are zeros.
template <typename T>
__device__ __forceinline__ void mma_k16(float& c0, float& c1, uint32_t a0, uint32_t a2,
                                        uint32_t b0, uint32_t b1) {
  float x[4] = {c0, c1, 0.f, 0.f};
  const uint32_t a[4] = {a0, 0u, a2, 0u};
  mma16816<T>(x, a, b0, b1);
  c0 = x[0];
  c1 = x[1];
}
template <typename T>
__device__ __forceinline__ void mma_k8(float& c0, float& c1, uint32_t a0, uint32_t b0) {
  float d2, d3;
  if constexpr (__is_same(T, __half))
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
        "{%0,%1,%7,%7};"
        : "+f"(c0), "+f"(c1), "=f"(d2), "=f"(d3)
        : "r"(a0), "r"(0), "r"(b0), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
        "{%0,%1,%7,%7};"
        : "+f"(c0), "+f"(c1), "=f"(d2), "=f"(d3)
        : "r"(a0), "r"(0), "r"(b0), "f"(0.f));
}

// Chunks 0, STEP, 2 STEP, .. of 16 bytes, or zeros.
template <int STEP, int N>
__device__ __forceinline__ void load_chunks(uint4 (&x)[N], const void* from, bool ok) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    x[i] = ok ? static_cast<const uint4*>(from)[i * STEP] : make_uint4(0u, 0u, 0u, 0u);
}
// acc, a pair of zeros, or NaN where x is NaN or infinite
template <typename T>
__device__ __forceinline__ uint32_t zero_or_nan(uint32_t x, uint32_t acc) {
  uint32_t y;
  if constexpr (__is_same(T, __half))
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(0u), "r"(acc));
  else
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(0u), "r"(acc));
  return y;
}
__device__ __forceinline__ uint32_t word(const uint4& x, int i) {
  return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
}

template <typename T, int D, bool SHORT_OWN>
__global__ void __launch_bounds__(kJoinWarps * 32, kJoinCtas<D>)
    join_kernel(const __grid_constant__ AttnParams p, Deal deal) {
  constexpr int EL = D / 4;          // dimensions of a lane
  constexpr int NI = D / 64;         // its runs of 16 of the sums
  const int lane = threadIdx.x & 31, gid = lane >> 2, quad = lane & 3;
  // a row per CTA and turn: its warps meet the same lengths, tables and places,
  // which are looked up one turn ahead
  const ssd_attention& a = p.a;
  extern __shared__ float s_sums[];
  const int warp = threadIdx.x >> 5, part = deal.split > 1 ? warp : 0;
  const int step = deal.split > 1 ? a.R : gridDim.x;  // one task and done
  int page_col = p.by_page.quotient(gid);
  if (page_col >= a.cols) page_col = -1;
  auto page_of = [&](int r) {        // of token gid, before the length is known
    return SHORT_OWN && page_col >= 0 && r < a.R ? a.tables[(int64_t)r * a.table_stride + page_col]
                                                 : -1;
  };
  auto length_of = [&](int r) { return r < a.R ? own_len(p, r) : 0; };
  auto items_of = [&](int r) {
    return a.G > 0 && r < a.R ? p.row_items[r] : row_items_of(-1, 0, 0);
  };
  int r = deal.split > 1 ? blockIdx.x / deal.tasks : blockIdx.x;
  int next_len = length_of(r), next_first = page_of(r);
  wait_previous();
  int4 next_row = items_of(r);
  for (; r < a.R; r += step) {
    const int len = next_len, first = next_first;
    const int4 row = next_row;
    next_len = length_of(r + step);
    next_first = page_of(r + step);
    next_row = items_of(r + step);
    const int32_t* table = a.tables + (int64_t)r * a.table_stride;
    if (SHORT_OWN && a.lens && threadIdx.x == 0 && len != a.lens[r]) flag(p, SSD_DEV_BAD_LENGTH);

    // Several heads of a warp add to the sums of their own lanes, and to the others
    // with weights of zero.  Zero times an infinity or NaN is NaN, so if an output is
    // NaN the heads are taken again one by one, which leaves the others' values out.
    // (Sums kept by a select after each product: 256 x 24 branches take 329 us
    // instead of 306.)
    int alone = -1;
    for (int task = deal.split > 1 ? blockIdx.x - r * deal.tasks : warp; task < deal.tasks;) {
      // key/value heads h0 .. of the task, this lane's one and its query head in it
      const int lanes = kJoinHeads / deal.pack;
      const int first_h = deal.pack > 1 ? task * deal.pack : task / deal.blocks;
      const int h0 = first_h + max(alone, 0), h = first_h + gid / lanes, sub = h - h0;
      const int in_h = deal.pack > 1 ? gid % lanes
                                     : (task - h0 * deal.blocks) * kJoinHeads + gid;
      const int packed = alone >= 0 ? 1 : min(deal.pack, a.Hkv - h0);
      const bool mine = in_h < p.gqa && (unsigned)sub < (unsigned)packed;
      const int head = h * p.gqa + in_h;
      if (SHORT_OWN && gid < next_len && (unsigned)next_first < (unsigned)a.num_pages) {
        // the next row's tokens on their way to L2: lines of K and V, two lanes each
        const ssd_paged& c = quad < 2 ? a.k : a.v;
        const T* x = static_cast<const T*>(c.ptr) + (int64_t)next_first * c.page_stride +
                     (int64_t)(gid - page_col * a.page_size) * c.token_stride +
                     (int64_t)h0 * c.head_stride + (quad & 1) * 64;
        for (int z = 0; z < packed; ++z)
#pragma unroll
          for (int d = 0; d < D; d += 128)
            if ((quad & 1) * 64 + d < D)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(x + (int64_t)z * c.head_stride + d));
      }

      // where the partials are, on its way while the own tokens are read
      const Parts s = mine ? parts_of(p, row, h, in_h) : Parts{0, 0, 0};
      if (SHORT_OWN && s.np > 0) {
        // the first partial on its way to L2 meanwhile: four heads share its lines
        const float* x = p.po + part_at<D>(s.slot, p.mt, s.i, quad * 16 + (gid & 3) * 4);
#pragma unroll
        for (int i = 0; i < NI; ++i)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(x + (int64_t)i * 64 * p.mt));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.pml + (int64_t)s.slot * p.mt + s.i));
      }

      float o[NI][16] = {};            // sums at dimensions 64 i + 16 quad + e
      float m = -INFINITY, l = 0.f;
      for (int t0 = 0; SHORT_OWN && part == 0 && t0 < len; t0 += 8) {
        const int t = t0 + gid, col = p.by_page.quotient(t);
        int page = -1, in_page = 0;
        if (t < len) {
          page = t0 == 0 ? first : table[col];
          in_page = t - col * a.page_size;
          if ((unsigned)page >= (unsigned)a.num_pages) {
            flag(p, SSD_DEV_BAD_PAGE);
            page = -1;               // reads as zeros
          }
        }
        float s0 = 0.f, s1 = 0.f;    // scores of tokens t0 + 2 quad, + 1
        {
          const T* kt = static_cast<const T*>(a.k.ptr) + (int64_t)page * a.k.page_stride +
                        (int64_t)in_page * a.k.token_stride + (int64_t)h0 * a.k.head_stride +
                        quad * 8;
          uint4 q[EL / 8];
          load_chunks<4>(q, static_cast<const T*>(a.q) + (int64_t)r * a.q_row_stride +
                                (int64_t)head * a.q_head_stride + quad * 8, mine);
          for (int z = 0; z < packed; z += 2) {  // two key/value heads at a time
            uint4 k0[EL / 8], k1[EL / 8];
            load_chunks<4>(k0, kt + (int64_t)z * a.k.head_stride, page >= 0);
            load_chunks<4>(k1, kt + (int64_t)(z + 1) * a.k.head_stride,
                           page >= 0 && z + 1 < packed);
            float x0 = 0.f, x1 = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
            for (int i = 0; i < EL / 4; ++i)
              mma_k16<T>(x0, x1, word(q[i / 2], i % 2 * 2), word(q[i / 2], i % 2 * 2 + 1),
                         word(k0[i / 2], i % 2 * 2), word(k0[i / 2], i % 2 * 2 + 1));
            if (z + 1 < packed) {
#pragma unroll
              for (int i = 0; i < EL / 4; ++i)
                mma_k16<T>(y0, y1, word(q[i / 2], i % 2 * 2), word(q[i / 2], i % 2 * 2 + 1),
                           word(k1[i / 2], i % 2 * 2), word(k1[i / 2], i % 2 * 2 + 1));
            }
            if (sub == z) {
              s0 = x0;
              s1 = x1;
            }
            if (sub == z + 1) {
              s0 = y0;
              s1 = y1;
            }
          }
        }
        s0 = t0 + quad * 2 < len ? s0 * p.scale_log2 : -INFINITY;
        s1 = t0 + quad * 2 + 1 < len ? s1 * p.scale_log2 : -INFINITY;
        float top = fmaxf(s0, s1);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float m1 = fmaxf(m, top), off = m1 == -INFINITY ? 0.f : m1;
        const float keep = exp2_fast(m - off);
        m = m1;
        s0 = exp2_fast(s0 - off);
        s1 = exp2_fast(s1 - off);
        l = l * keep + s0 + s1;
        const uint32_t pw = pack2<T>(s0, s1);  // rounded to the type of the values, for the product
        const int pg0 = __shfl_sync(0xffffffffu, page, quad * 8);
        const int pg1 = __shfl_sync(0xffffffffu, page, quad * 8 + 4);
        const int ip0 = __shfl_sync(0xffffffffu, in_page, quad * 8);
        const int ip1 = __shfl_sync(0xffffffffu, in_page, quad * 8 + 4);
        const T* vh = static_cast<const T*>(a.v.ptr) + (int64_t)h0 * a.v.head_stride + gid * 8;
        const int64_t at0 = (int64_t)pg0 * a.v.page_stride + (int64_t)ip0 * a.v.token_stride;
        const int64_t at1 = (int64_t)pg1 * a.v.page_stride + (int64_t)ip1 * a.v.token_stride;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[i][e] *= keep;
#pragma unroll 2
        for (int z = 0; z < packed; ++z) {
          uint4 v0[NI], v1[NI];
          load_chunks<8>(v0, vh + at0 + (int64_t)z * a.v.head_stride, pg0 >= 0);
          load_chunks<8>(v1, vh + at1 + (int64_t)z * a.v.head_stride, pg1 >= 0);
          const uint32_t w = sub == z ? pw : 0u;
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              mma_k8<T>(o[i][e], o[i][e + 8], w,
                        __byte_perm(word(v0[i], e / 2), word(v1[i], e / 2),
                                    e & 1 ? 0x7632 : 0x5410));
        }
      }
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);

      // The partials: first the largest maximum, then the sums, 16 dimensions at a
      // time, so that no load waits for another stretch's.
      const int64_t pair = (int64_t)r * a.Hq + head;
      const int per = SHORT_OWN || len == 0 ? 1 : own_stretch(p, len);
      const int ns = SHORT_OWN || !mine ? 0 : (len + per - 1) / per;  // of the own tokens
      const float2* ml_p = p.pml + (int64_t)s.slot * p.mt + s.i;
      const float2* ml_o = p.sml + pair * p.nsplit;
      const int64_t next = (int64_t)p.mt * p.hg;  // rows from one partial to the next
      float top = m;
#pragma unroll 4
      for (int j = part; j < s.np; j += deal.split) top = fmaxf(top, ml_p[j * next].x);
#pragma unroll 4
      for (int j = part; j < ns; j += deal.split) top = fmaxf(top, ml_o[j].x);
      const float off = top == -INFINITY ? 0.f : top, keep = exp2_fast(m - off);
      m = top;
      l *= keep;
      for (int j = part; j < s.np; j += deal.split) {
        const float2 ml = ml_p[j * next];
        l = fmaf(ml.y, exp2_fast(ml.x - off), l);
      }
      for (int j = part; j < ns; j += deal.split) l = fmaf(ml_o[j].y, exp2_fast(ml_o[j].x - off), l);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] *= keep;
        auto add = [&](float g, const float* x, int step) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4 y = *reinterpret_cast<const float4*>(x + c * step);
            o[i][c * 4] = fmaf(y.x, g, o[i][c * 4]);
            o[i][c * 4 + 1] = fmaf(y.y, g, o[i][c * 4 + 1]);
            o[i][c * 4 + 2] = fmaf(y.z, g, o[i][c * 4 + 2]);
            o[i][c * 4 + 3] = fmaf(y.w, g, o[i][c * 4 + 3]);
          }
        };
        const float* po = p.po + part_at<D>(s.slot, p.mt, s.i, quad * 16 + i * 64);
#pragma unroll 4
        for (int j = part; j < s.np; j += deal.split)
          add(exp2_fast(ml_p[j * next].x - off), po + j * next * D, 4 * p.mt);
        const float* so = p.so + pair * p.nsplit * D + quad * 16 + i * 64;
#pragma unroll 4
        for (int j = part; j < ns; j += deal.split) add(exp2_fast(ml_o[j].x - off), so + (int64_t)j * D, 4);
      }
      for (int w = deal.split / 2; w > 0; w /= 2) {  // the warps' sums, by halves
        float* mem = s_sums + (warp % w) * 32 * (D / 4 + 2) + lane;
        if (warp >= w && warp < 2 * w) {
          mem[0] = m;
          mem[32] = l;
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) mem[(2 + i * 16 + e) * 32] = o[i][e];
        }
        __syncthreads();
        if (warp < w) {
          const float m1 = fmaxf(m, mem[0]), off1 = m1 == -INFINITY ? 0.f : m1;
          const float f = exp2_fast(m - off1), g = exp2_fast(mem[0] - off1);
          m = m1;
          l = l * f + mem[32] * g;
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] = o[i][e] * f + mem[(2 + i * 16 + e) * 32] * g;
        }
        __syncthreads();
      }
      uint32_t seen = 0;               // a pair of zeros, or NaN if an output is
      if (mine && part == 0) {
        // no token at all: zeros and -inf
        const float inv = l == 0.f ? 0.f : 1.f / l;
        T* to = static_cast<T*>(a.out) + (int64_t)r * a.out_row_stride +
                (int64_t)head * a.out_head_stride + quad * 16;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int c = 0; c < 16; c += 8) {
            const uint4 x = make_uint4(pack2<T>(o[i][c] * inv, o[i][c + 1] * inv),
                                       pack2<T>(o[i][c + 2] * inv, o[i][c + 3] * inv),
                                       pack2<T>(o[i][c + 4] * inv, o[i][c + 5] * inv),
                                       pack2<T>(o[i][c + 6] * inv, o[i][c + 7] * inv));
            *reinterpret_cast<uint4*>(to + i * 64 + c) = x;
            if (SHORT_OWN)
              seen = zero_or_nan<T>(x.x, zero_or_nan<T>(x.y, zero_or_nan<T>(
                         x.z, zero_or_nan<T>(x.w, seen))));
          }
        if (quad == 0 && a.lse) a.lse[pair] = (m + log2f(l)) * 0.6931471805599453f;
      }
      if (SHORT_OWN && deal.pack > 1 &&
          (alone >= 0 || __any_sync(0xffffffffu, (seen & 0x7fff7fffu) != 0)) &&
          ++alone < min(deal.pack, a.Hkv - first_h))
        continue;
      alone = -1;
      task += deal.split > 1 ? deal.tasks : blockDim.x >> 5;
    }
  }
}

// ---- set-up ---------------------------------------------------------------------------
struct Layout {
  bool tc;                  // the prefixes' kernel is the tensor-core one
  bool short_own;           // the join reads own tokens itself
  int own_blocks;
  size_t po, pml, rows, workers, so, sml, total;
};

bool strides_ok(const void* ptr, std::initializer_list<int64_t> strides) {
  if (!ptr || (uintptr_t)ptr % 16 != 0) return false;
  for (int64_t s : strides)
    if (s < 0 || s % 8 != 0) return false;
  return true;
}

// Tokens and (row, head) pairs are counted in 32 bits, in tiles, blocks and stretches that
// may end after the last one.
constexpr int64_t kMaxCount = 0x7fffffff - (1 << 20);

ssd_status check(const ssd_attention* a) {
  if (!a || (a->dtype != SSD_BF16 && a->dtype != SSD_F16) || a->pad_ != 0)
    return SSD_ERR_INVALID_ARG;
  if (a->R < 1 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv != 0 || a->G < 0 ||
      a->num_pages < 1 || a->page_size < 1 || !std::isfinite(a->scale))
    return SSD_ERR_INVALID_ARG;
  if (a->D != 64 && a->D != 128 && a->D != 256) return SSD_ERR_UNSUPPORTED;
  if (a->prefix_cols < 0 || a->cols < 0) return SSD_ERR_INVALID_ARG;
  // tables of no columns may have no address
  if (a->tables ? !a->lens : a->lens && a->cols > 0) return SSD_ERR_INVALID_ARG;
  if (a->G > 0 && ((!a->prefix_tables && a->prefix_cols > 0) || !a->prefix_len || !a->group_off ||
                   a->prefix_table_stride < a->prefix_cols))
    return SSD_ERR_INVALID_ARG;
  if (a->tables && a->table_stride < a->cols) return SSD_ERR_INVALID_ARG;
  if ((int64_t)a->prefix_cols * a->page_size > kMaxCount ||
      (a->tables && (int64_t)a->cols * a->page_size > kMaxCount) ||
      (int64_t)a->R * a->Hq > kMaxCount)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

int ctas_per_sm(int D) { return D == 256 ? 1 : D == 128 ? 2 : 4; }  // by shared memory

// The split and the workspace of a call; false when its work is beyond 32-bit
// counts.
bool plan(const ssd_attention& a, AttnParams& p, Layout& L) {
  const int sms = std::max(num_sms(), 1);
  p.a = a;
  if (!a.tables) p.a.cols = 0;  // no own tokens whatever cols says: the join looks pages up by it
  p.gqa = a.Hq / a.Hkv;
  p.by_page = divisor(a.page_size);
  p.by_gqa = divisor(p.gqa);
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  L.tc = prefix_tc_fits(a);
  p.mt = L.tc ? kTcBlock : kBlockRows;
  p.tn = L.tc ? kTcTile : kTileTokens;
  p.in_step = L.tc;
  const int warps = sms * ctas_per_sm(a.D) * kWarpsPerCta;  // resident at once
  // sets of up to eight heads where a token's heads lie closer than its neighbour
  p.hg = 1;
  if (L.tc && a.k.head_stride < a.k.token_stride && a.v.head_stride < a.v.token_stride)
    for (int n = 2; n <= std::min(8, sms); ++n)
      if (a.Hkv % n == 0) p.hg = n;
  p.sets = a.Hkv / p.hg;
  p.workers = L.tc ? sms / p.hg : warps;
  const int64_t items =
      a.Hkv * ((int64_t)a.R * p.gqa / p.mt + std::min<int64_t>(a.G, a.R));
  const int64_t tiles = ((int64_t)a.prefix_cols * a.page_size + p.tn - 1) / p.tn;
  if (items * (tiles + 1) > 0x7fffffff) return false;
  p.nslots = a.G > 0 ? (int)(items + (int64_t)p.workers * p.hg) : 0;
  // own tokens: read by the join where they are few; else in stretches of two
  // tiles or more, four for each resident warp, which evens out their lengths.
  // (256 rows with 0 to 900 tokens over a prompt of 16000: 128 us, by eight 135, by two
  // 135; 100 rows with 0 to 6000: 233, 233, 248; 256 with 0 to 3000: 312, 292, 338.)
  const int64_t most = a.lens ? (int64_t)a.cols * a.page_size : 0;
  L.short_own = most <= (a.cols == 1 ? kShortPage : kShortOwn);
  p.own_apart = L.tc && !L.short_own;
  L.own_blocks = (p.gqa + kBlockRows - 1) / kBlockRows;
  const int64_t own = (int64_t)a.R * a.Hkv * L.own_blocks;
  p.nsplit = (int)std::max<int64_t>(
      1, std::min<int64_t>((most + 2 * kTileTokens - 1) / (2 * kTileTokens), 4 * warps / own));
  if (own * p.nsplit / kWarpsPerCta >= 0x7fffffff) return false;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  L.po = take((size_t)p.nslots * p.mt * a.D * 4);
  L.pml = take((size_t)p.nslots * p.mt * 8);
  L.rows = take(a.G > 0 ? (size_t)a.R * 16 : 0);
  L.workers = take((size_t)items * 8);
  const size_t owns = L.short_own ? 0 : (size_t)a.R * a.Hq * p.nsplit;
  L.so = take(owns * a.D * 4);
  L.sml = take(owns * 8);
  L.total = std::max<size_t>(at, 256);
  return true;
}

// The next kernel of a call, which may start before the one before is done.
template <typename N>
cudaError_t launch_next(void (*kernel)(AttnParams, N), int grid, int threads, int smem,
                        cudaStream_t s, bool early_start, const AttnParams& p, N n) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = early_start ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, p, n);
}

template <typename T, int D>
cudaError_t launch(const AttnParams& p, const Layout& L, cudaStream_t s) {
  const int ring = kWarpsPerCta * kRing * step_bytes<D>();
  cudaError_t e;
  bool first = p.a.G == 0;
  if (p.a.G > 0 && L.tc) {
    e = launch_prefix_tc(p, s);
    if (e != cudaSuccess) return e;
  } else if (p.a.G > 0) {
    e = cudaFuncSetAttribute(prefix_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (e != cudaSuccess) return e;
    prefix_kernel<T, D><<<p.workers / kWarpsPerCta, kWarpsPerCta * 32, ring, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!L.short_own) {
    e = cudaFuncSetAttribute(own_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (e != cudaSuccess) return e;
    const int64_t tasks = (int64_t)p.a.R * p.a.Hkv * L.own_blocks * p.nsplit;
    e = launch_next(own_kernel<T, D>, (int)((tasks + kWarpsPerCta - 1) / kWarpsPerCta),
                    kWarpsPerCta * 32, ring, s, !first, p, L.own_blocks);
    if (e != cudaSuccess) return e;
    first = false;
  }
  Deal deal{1, (p.gqa + kJoinHeads - 1) / kJoinHeads, 0, 1};
  // Few rows: every key/value head has its warp (12 branches of one sequence: 28 us, two
  // heads to a warp 38), or several that share its partials (20).  When a warp each takes
  // more than a turn: as many heads to a warp as it has lanes for (32 x 12 branches: 106
  // us instead of 108; 256 x 24: 300 instead of 344).  Times of the kernels alone.
  const int64_t warps = (int64_t)std::max(num_sms(), 1) * kJoinCtas<D> * kJoinWarps;
  // In place a warp takes one: several are taken again where an output is NaN, and
  // would find outputs for their queries.
  while (p.a.out != p.a.q && deal.pack * 2 * p.gqa <= kJoinHeads &&
         (int64_t)p.a.R * p.a.Hkv / deal.pack > warps)
    deal.pack *= 2;
  deal.tasks = deal.pack > 1 ? (p.a.Hkv + deal.pack - 1) / deal.pack : p.a.Hkv * deal.blocks;
  const int64_t tasks = (int64_t)p.a.R * deal.tasks;
  while (deal.split < kJoinWarps && tasks * deal.split * 2 <= warps) deal.split *= 2;
  const int threads = (deal.split > 1 ? deal.split : std::min(kJoinWarps, deal.tasks)) * 32;
  const int resident = (int)warps * 32 / threads;
  const int grid = deal.split > 1 ? (int)tasks : std::min(p.a.R, resident);
  const int smem = join_bytes<D>(deal.split > 1 ? deal.split : 0);
  // Started early, the join finds the shared-memory split of the kernel before on
  // its SM: 256 x 24 branches then take 26 us more (it has many turns, and lives
  // on its cache).  With one turn it makes little difference: uneven groups of a few rows
  // 26.8 us instead of 27.1 called one by one, 24.2 instead of 23.5 in a graph.
  const bool early = !first && (deal.split > 1 || p.a.R <= resident);
  return L.short_own
             ? launch_next(join_kernel<T, D, true>, grid, threads, smem, s, early, p, deal)
             : launch_next(join_kernel<T, D, false>, grid, threads, smem, s, early, p, deal);
}

template <typename T>
cudaError_t launch_d(const AttnParams& p, const Layout& L, cudaStream_t s) {
  switch (p.a.D) {
    case 64: return launch<T, 64>(p, L, s);
    case 128: return launch<T, 128>(p, L, s);
    default: return launch<T, 256>(p, L, s);
  }
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_prefix_attention_workspace_size(const ssd_attention* a) {
  AttnParams p{};
  Layout L;
  if (check(a) != SSD_OK || !plan(*a, p, L)) return 0;
  return L.total;
}

ssd_status ssd_prefix_attention(const ssd_attention* a, void* workspace, size_t workspace_bytes,
                                int32_t* dev_status, void* stream) {
  const ssd_status st = check(a);
  if (st != SSD_OK) return st;
  if (!strides_ok(a->q, {a->q_row_stride, a->q_head_stride}) ||
      !strides_ok(a->out, {a->out_row_stride, a->out_head_stride}) ||
      !strides_ok(a->k.ptr, {a->k.page_stride, a->k.token_stride, a->k.head_stride}) ||
      !strides_ok(a->v.ptr, {a->v.page_stride, a->v.token_stride, a->v.head_stride}))
    return SSD_ERR_INVALID_ARG;
  if (a->out == a->q &&
      (a->out_row_stride != a->q_row_stride || a->out_head_stride != a->q_head_stride))
    return SSD_ERR_INVALID_ARG;
  AttnParams p{};
  Layout L;
  if (!plan(*a, p, L)) return SSD_ERR_UNSUPPORTED;
  if (!workspace || (uintptr_t)workspace % 256 != 0 || workspace_bytes < L.total)
    return SSD_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  p.po = reinterpret_cast<float*>(ws + L.po);
  p.pml = reinterpret_cast<float2*>(ws + L.pml);
  p.row_items = reinterpret_cast<int4*>(ws + L.rows);
  p.item_workers = reinterpret_cast<int2*>(ws + L.workers);
  p.so = reinterpret_cast<float*>(ws + L.so);
  p.sml = reinterpret_cast<float2*>(ws + L.sml);
  p.status = dev_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == SSD_BF16 ? launch_d<__nv_bfloat16>(p, L, s)
                                             : launch_d<__half>(p, L, s);
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return SSD_ERR_CUDA;
}

}  // extern "C"
