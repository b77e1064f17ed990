// ssd_attention.cu -- attention over shared prefixes and own tokens of a
// paged cache (ssd_prefix_attention): the kernel of few rows, the join of
// partial results, and the entry point.
//
// out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), with m the running
// maximum, over any stretch of tokens; two stretches join by weighting each
// with exp(m_i - max m).

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
  __shared__ int2 s_warp[kWarpsPerCta];
  const int w0 = blockIdx.x * kWarpsPerCta, warp = threadIdx.x >> 5, w = w0 + warp;
  const int total = find_starts<kWarpsPerCta * 32, kWarpsPerCta>(p, w0, s_start, s_warp);
  const uint32_t ring = smem_addr(s_ring) + warp * kRing * step_bytes<D>();
  Walk k;
  k.u = first_unit(p, w, total);
  k.u1 = first_unit(p, w + 1, total);
  if (k.u >= k.u1) return;
  k.g = s_start[warp].g;
  k.unit = s_start[warp].unit;
  k.item = s_start[warp].item;
  k.w = w;
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
__global__ void __launch_bounds__(kWarpsPerCta * 32)
    own_kernel(const __grid_constant__ AttnParams p, int blocks) {
  extern __shared__ __align__(128) unsigned char s_ring[];
  const int warp = threadIdx.x >> 5;
  int64_t task = (int64_t)blockIdx.x * kWarpsPerCta + warp;
  if (task >= (int64_t)p.a.R * p.a.Hkv * blocks * p.nsplit) return;
  const int split = (int)(task % p.nsplit);
  task /= p.nsplit;
  const int mb = (int)(task % blocks);
  task /= blocks;
  const int h = (int)(task % p.a.Hkv), r = (int)(task / p.a.Hkv);
  const int len = own_len(p, r), n = own_stretch(p, len);
  const int t0 = min(len, split * n), t1 = min(len, t0 + n);
  if (h == 0 && mb == 0 && split == 0 && (threadIdx.x & 31) == 0 && len != p.a.lens[r])
    flag(p, SSD_DEV_BAD_LENGTH);
  if (t0 >= t1) return;  // the join does not look at it
  const int64_t at = ((int64_t)r * p.a.Hq + h * p.gqa + mb * kBlockRows) * p.nsplit + split;
  const Partial out{p.so + at * D, (int64_t)p.nsplit * D, 4, p.sml + at, p.nsplit};
  warp_stretch<T, D>(p, smem_addr(s_ring) + warp * kRing * step_bytes<D>(), r, mb * kBlockRows,
                     p.gqa, h, p.a.tables + (int64_t)r * p.a.table_stride, t0, t1, out);
}

// ---- the join ------------------------------------------------------------------------
// One warp per (row, key/value head, up to four of its query heads): the row's
// own tokens, or their partials, then the prefix's partials, then the output.
//
// Own tokens are few in the calls that this kernel is made for (a branch's
// drafts), and such a task is a chain of loads: length, page, token beside
// group, sums, partials.  It is bound by that latency, so it has few registers
// and many warps: a token is spread over D / 8 lanes of 16 bytes, and the
// products run on the ordinary units.  Long own caches go through own_kernel,
// split over many warps.
constexpr int kJoinWarps = 8;
constexpr int kJoinHeads = 4;
constexpr int kShortOwn = 64;  // tokens of an own cache up to which the join reads it

// The group of row r: the last one that starts at or before it.
__device__ __forceinline__ int group_of_row(const int32_t* off, int G, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = G;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, i < lo + n && off[i] <= r);
    const int k = le ? 31 - __clz(le) : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// The prefix's partials of a pair: np of them, from `slot` on, at row `i`.
struct Parts {
  int np, slot, i;
};
__device__ __forceinline__ Parts parts_of(const AttnParams& p, const Group& q, int item0, int r,
                                          int h, int head) {
  Parts s{0, 0, 0};
  if (r < q.row0 || r >= q.row0 + q.rows || q.tiles == 0 || item0 < 0) return s;
  const int i = (r - q.row0) * p.gqa + head, mb = p.mt == kTcBlock ? i / kTcBlock : i / kBlockRows;
  const int item = item0 + h * q.blocks + mb;
  const int2 w = p.item_workers[item];
  s.np = w.y - w.x + 1;
  s.slot = item + w.x;
  s.i = i - mb * p.mt;
  return s;
}

template <typename T>
__device__ __forceinline__ void widen(float (&f)[8], const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 y;
    if constexpr (__is_same(T, __half))
      y = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    else
      y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    f[2 * i] = y.x;
    f[2 * i + 1] = y.y;
  }
}

// Weighted sums of one more stretch: o, l at maximum m take x, its weight and
// maximum in ml.
__device__ __forceinline__ void add_part(float (&o)[8], float& m, float& l, float2 ml,
                                         const float4& x0, const float4& x1) {
  const float m1 = fmaxf(m, ml.x), off = m1 == -INFINITY ? 0.f : m1;
  const float a = exp2_fast(m - off), b = exp2_fast(ml.x - off);
  m = m1;
  l = l * a + ml.y * b;
  const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = o[e] * a + x[e] * b;
}

template <typename T, int D, bool SHORT_OWN>
__global__ void __launch_bounds__(kJoinWarps * 32, SHORT_OWN ? 2 : 3)
    join_kernel(const __grid_constant__ AttnParams p, int head_blocks) {
  constexpr int LT = D / 8;          // lanes of a token
  constexpr int TS = 32 / LT;        // tokens at a time
  constexpr int HS = kJoinHeads / TS;  // heads that a lane's share finishes
  static_assert(HS * TS == kJoinHeads, "heads are dealt to the tokens' lanes");
  const int lane = threadIdx.x & 31, sub = lane / LT, d0 = lane % LT * 8;
  // a CTA per row: its warps meet the same lengths, tables and sums
  const int r = blockIdx.x;
  const ssd_attention& a = p.a;
  const int len = own_len(p, r);
  Group q{};
  int item0 = -1;
  if (a.G > 0) {
    const int g = group_of_row(a.group_off, a.G, r);
    q = group_of(p, g);
    item0 = p.item_base[g];
  }
  for (int task = threadIdx.x >> 5; task < a.Hkv * head_blocks; task += blockDim.x >> 5) {
    const int h = head_blocks == 1 ? task : task / head_blocks;
    const int hb = (task - h * head_blocks) * kJoinHeads;
    const int heads = min(kJoinHeads, p.gqa - hb);

    float o[kJoinHeads][8] = {};
    float m[kJoinHeads], l[kJoinHeads];
#pragma unroll
    for (int i = 0; i < kJoinHeads; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    if (SHORT_OWN && a.lens && h == 0 && hb == 0 && lane == 0 && len != a.lens[r])
      flag(p, SSD_DEV_BAD_LENGTH);
    if (SHORT_OWN && len > 0) {
      uint4 qx[kJoinHeads];
#pragma unroll
      for (int i = 0; i < kJoinHeads; ++i)
        qx[i] = i < heads ? *reinterpret_cast<const uint4*>(
                                static_cast<const T*>(a.q) + (int64_t)r * a.q_row_stride +
                                (int64_t)(h * p.gqa + hb + i) * a.q_head_stride + d0)
                          : make_uint4(0u, 0u, 0u, 0u);
      const int32_t* table = a.tables + (int64_t)r * a.table_stride;
      for (int t0 = 0; t0 < len; t0 += 2 * TS) {
        uint4 kx[2], vx[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = t0 + j * TS + sub;
          kx[j] = vx[j] = make_uint4(0u, 0u, 0u, 0u);
          if (t < len) {
            const int col = p.by_page.quotient(t), page = table[col];
            if ((unsigned)page < (unsigned)a.num_pages) {
              const int in_page = t - col * a.page_size;
              kx[j] = *reinterpret_cast<const uint4*>(
                  static_cast<const T*>(a.k.ptr) + (int64_t)page * a.k.page_stride +
                  (int64_t)in_page * a.k.token_stride + (int64_t)h * a.k.head_stride + d0);
              vx[j] = *reinterpret_cast<const uint4*>(
                  static_cast<const T*>(a.v.ptr) + (int64_t)page * a.v.page_stride +
                  (int64_t)in_page * a.v.token_stride + (int64_t)h * a.v.head_stride + d0);
            } else {
              flag(p, SSD_DEV_BAD_PAGE);
            }
          }
        }
        float sc[2][kJoinHeads];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float kf[8];
          widen<T>(kf, kx[j]);
#pragma unroll
          for (int i = 0; i < kJoinHeads; ++i) {
            float qf[8], x = 0.f;
            widen<T>(qf, qx[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) x = fmaf(qf[e], kf[e], x);
#pragma unroll
            for (int d = LT / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            sc[j][i] = t0 + j * TS + sub < len ? x * p.scale_log2 : -INFINITY;
          }
        }
        float vf[2][8];
        widen<T>(vf[0], vx[0]);
        widen<T>(vf[1], vx[1]);
#pragma unroll
        for (int i = 0; i < kJoinHeads; ++i) {
          float top = fmaxf(sc[0][i], sc[1][i]);
#pragma unroll
          for (int d = LT; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          const float m1 = fmaxf(m[i], top), off = m1 == -INFINITY ? 0.f : m1;
          const float keep = exp2_fast(m[i] - off);
          const float w0 = exp2_fast(sc[0][i] - off), w1 = exp2_fast(sc[1][i] - off);
          m[i] = m1;
          l[i] = l[i] * keep + w0 + w1;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            o[i][e] = fmaf(w1, vf[1][e], fmaf(w0, vf[0][e], o[i][e] * keep));
        }
      }
#pragma unroll
      for (int i = 0; i < kJoinHeads; ++i)
#pragma unroll
        for (int d = LT; d < 32; d <<= 1) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[i][e] += __shfl_xor_sync(0xffffffffu, o[i][e], d);
        }
    }

    // each token's lanes finish heads sub, sub + TS, ..
#pragma unroll
    for (int k = 0; k < HS; ++k) {
      const int i = k * TS + sub;
      float y[8], my = m[k * TS], ly = l[k * TS];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = o[k * TS][e];
#pragma unroll
      for (int z = 1; z < TS; ++z)
        if (sub == z) {
          my = m[k * TS + z];
          ly = l[k * TS + z];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = o[k * TS + z][e];
        }
      if (i >= heads) continue;
      const int head = h * p.gqa + hb + i;
      const int64_t pair = (int64_t)r * a.Hq + head;
      if (!SHORT_OWN && len > 0) {
        const int ns = (len + own_stretch(p, len) - 1) / own_stretch(p, len);
        for (int j = 0; j < ns; ++j) {
          const int64_t at = pair * p.nsplit + j;
          const float4* x = reinterpret_cast<const float4*>(p.so + at * D + d0);
          add_part(y, my, ly, p.sml[at], x[0], x[1]);
        }
      }
      const Parts s = parts_of(p, q, item0, r, h, hb + i);
#pragma unroll 2
      for (int j = 0; j < s.np; ++j) {
        const float2 ml = p.pml[(int64_t)(s.slot + j) * p.mt + s.i];
        const float* x = p.po + part_at<D>(s.slot + j, p.mt, s.i, d0);
        add_part(y, my, ly, ml, *reinterpret_cast<const float4*>(x),
                 *reinterpret_cast<const float4*>(x + 4 * p.mt));
      }
      // no token at all: zeros and -inf
      const float inv = ly == 0.f ? 0.f : 1.f / ly;
      uint4 out;
      out.x = pack2<T>(y[0] * inv, y[1] * inv);
      out.y = pack2<T>(y[2] * inv, y[3] * inv);
      out.z = pack2<T>(y[4] * inv, y[5] * inv);
      out.w = pack2<T>(y[6] * inv, y[7] * inv);
      *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (int64_t)r * a.out_row_stride +
                                (int64_t)head * a.out_head_stride + d0) = out;
      if (d0 == 0 && a.lse) a.lse[pair] = (my + log2f(ly)) * 0.6931471805599453f;
    }
  }
}

// ---- set-up ---------------------------------------------------------------------------
struct Layout {
  bool tc;                  // the prefixes' kernel is the tensor-core one
  bool short_own;           // the join reads own tokens itself
  int own_blocks;
  size_t po, pml, item, workers, so, sml, total;
};

bool strides_ok(const void* ptr, std::initializer_list<int64_t> strides) {
  if (!ptr || (uintptr_t)ptr % 16 != 0) return false;
  for (int64_t s : strides)
    if (s < 0 || s % 8 != 0) return false;
  return true;
}

ssd_status check(const ssd_attention* a) {
  if (!a || (a->dtype != SSD_BF16 && a->dtype != SSD_F16) || a->pad_ != 0)
    return SSD_ERR_INVALID_ARG;
  if (a->R < 1 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv != 0 || a->G < 0 ||
      a->num_pages < 1 || a->page_size < 1 || !std::isfinite(a->scale))
    return SSD_ERR_INVALID_ARG;
  if (a->D != 64 && a->D != 128 && a->D != 256) return SSD_ERR_UNSUPPORTED;
  if (a->prefix_cols < 0 || a->cols < 0 || (a->tables == nullptr) != (a->lens == nullptr))
    return SSD_ERR_INVALID_ARG;
  if (a->G > 0 && (!a->prefix_tables || !a->prefix_len || !a->group_off ||
                   a->prefix_table_stride < a->prefix_cols))
    return SSD_ERR_INVALID_ARG;
  if (a->tables && a->table_stride < a->cols) return SSD_ERR_INVALID_ARG;
  if ((int64_t)a->prefix_cols * a->page_size > 0x7fffffff ||
      (int64_t)a->cols * a->page_size > 0x7fffffff || (int64_t)a->R * a->Hq > 0x7fffffff)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

int ctas_per_sm(int D) { return D == 256 ? 1 : D == 128 ? 2 : 4; }  // by shared memory

// The split and the workspace of a call; false when its work is beyond 32-bit
// counts.
bool plan(const ssd_attention& a, AttnParams& p, Layout& L) {
  const int sms = std::max(num_sms(), 1);
  p.a = a;
  p.gqa = a.Hq / a.Hkv;
  p.by_page = divisor(a.page_size);
  p.by_gqa = divisor(p.gqa);
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  L.tc = prefix_tc_fits(a);
  p.mt = L.tc ? kTcBlock : kBlockRows;
  p.tn = L.tc ? kTcTile : kTileTokens;
  const int warps = sms * ctas_per_sm(a.D) * kWarpsPerCta;  // resident at once
  p.workers = L.tc ? sms : warps;
  const int64_t items =
      a.Hkv * ((int64_t)a.R * p.gqa / p.mt + std::min<int64_t>(a.G, a.R));
  const int64_t tiles = ((int64_t)a.prefix_cols * a.page_size + p.tn - 1) / p.tn;
  if (items * (tiles + 1) > 0x7fffffff) return false;
  p.nslots = a.G > 0 ? (int)(items + p.workers) : 0;
  // own tokens: read by the join where they are few; else in stretches of two
  // tiles or more, four for each resident warp, which evens out their lengths
  const int64_t most = a.lens ? (int64_t)a.cols * a.page_size : 0;
  L.short_own = most <= kShortOwn;
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
  L.item = take((size_t)a.G * 4);
  L.workers = take((size_t)items * 8);
  const size_t rows = L.short_own ? 0 : (size_t)a.R * a.Hq * p.nsplit;
  L.so = take(rows * a.D * 4);
  L.sml = take(rows * 8);
  L.total = std::max<size_t>(at, 256);
  return true;
}

template <typename T, int D>
cudaError_t launch(const AttnParams& p, const Layout& L, cudaStream_t s) {
  const int smem = kWarpsPerCta * kRing * step_bytes<D>();
  cudaError_t e;
  if (p.a.G > 0 && L.tc) {
    e = launch_prefix_tc(p, s);
    if (e != cudaSuccess) return e;
  } else if (p.a.G > 0) {
    e = cudaFuncSetAttribute(prefix_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    prefix_kernel<T, D><<<p.workers / kWarpsPerCta, kWarpsPerCta * 32, smem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!L.short_own) {
    e = cudaFuncSetAttribute(own_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t tasks = (int64_t)p.a.R * p.a.Hkv * L.own_blocks * p.nsplit;
    own_kernel<T, D><<<(unsigned)((tasks + kWarpsPerCta - 1) / kWarpsPerCta), kWarpsPerCta * 32,
                       smem, s>>>(p, L.own_blocks);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const int head_blocks = (p.gqa + kJoinHeads - 1) / kJoinHeads;
  const int threads = std::min(kJoinWarps, p.a.Hkv * head_blocks) * 32;
  if (L.short_own)
    join_kernel<T, D, true><<<p.a.R, threads, 0, s>>>(p, head_blocks);
  else
    join_kernel<T, D, false><<<p.a.R, threads, 0, s>>>(p, head_blocks);
  return cudaGetLastError();
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
  AttnParams p{};
  Layout L;
  if (!plan(*a, p, L)) return SSD_ERR_UNSUPPORTED;
  if (!workspace || (uintptr_t)workspace % 256 != 0 || workspace_bytes < L.total)
    return SSD_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  p.po = reinterpret_cast<float*>(ws + L.po);
  p.pml = reinterpret_cast<float2*>(ws + L.pml);
  p.item_base = reinterpret_cast<int*>(ws + L.item);
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
