// ssd_logits.cu -- penalties, biases and grammar masks on the logit rows of
// a round (ssd_process_logits).
//
// Per row (b, u) and token v, with c = occurrences of v in the generated part
// of the history and on the draft path to u:
//   z = seen ? (z > 0 ? z / r : z * r) : z;  z -= c > 0 ? f*c + p : 0;
//   z += bias[v];  z = allowed ? z : fill.
//
// The work is one read and one write of every logit; the rules touch a few
// thousand tokens of a row.  A CTA owns a slice of the vocabulary of one
// sequence: it counts the history's tokens of the slice once in shared
// memory and streams that slice of the sequence's rows past the counts, so
// the history is scanned once for all N rows.  A token that is among the drafts
// has a bit of its own in its count, and the few such tokens walk the path of
// their row when they are met, so that the rows need no counts of their own.
//
// A warp streams its own vectors, 64 in a row of a step, through its own part of
// a ring in shared memory, filled by asynchronous copies.  Which of its tokens
// are touched is the same in every row, so they are listed once; in each row the
// warp first adjusts those in the ring, one per lane (one token in thirty is
// touched after 4096), and then streams the vectors through the mask.  What
// bounds the kernel next to memory is what it issues: 167 instructions per warp
// and vector (241 when touched tokens were looked for in every vector of every row).
// Measured: 64 x 9 x 128256 bf16 with masks 62 us, 4.9 TB/s (0.72 of the issue slots);
// 256 x 9 x 151936 f32 456 us, 6.2 TB/s (92% of a copy); 1 x 5 x 128256 bf16 5 us.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ssd.h"
#include "ssd_device.cuh"
#include "ssd_internal.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlice = 4096;     // tokens of a slice: 16 KB of counts, 8 KB of bias entries
constexpr int kMinSlice = 1024;
constexpr int kMaxRows = 16;        // rows of a CTA: 8 KB of mask bits
constexpr int kStages = 2;          // steps of the ring
constexpr int kBatch = 8;           // history tokens in flight per thread,
constexpr int kBiasBatch = 2;       // biases
static_assert(kMaxTreeNodes <= kThreads, "a draft per thread");
constexpr uint32_t kPromptBit = 0x80000000u;  // counts word: token occurs in the prompt,
constexpr uint32_t kDraftBit = 0x40000000u;   // among the drafts of some row
constexpr uint32_t kCountBits = kDraftBit - 1;

struct LogitParams {
  const void* in;
  int64_t in_stride;
  void* out;
  int64_t out_stride;
  int B, N, V;
  int slice, nslice;        // tokens per slice (a power of two), slices per row
  int rows, ngroup;         // rows per CTA, row groups per sequence
  ssd_logit_rules r;
  int32_t* allowed;
  int32_t* status;
  int16_t parent[kMaxTreeNodes];
};

// A step is a slice of kMaxSlice tokens: kVecs vectors per thread.
template <int DT> struct Elem;
template <> struct Elem<SSD_BF16> {
  static constexpr int kVecs = 2;
  using type = uint16_t;
  static __device__ float load(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
  static __device__ uint16_t store(float z) { return __bfloat16_as_ushort(__float2bfloat16_rn(z)); }
};
template <> struct Elem<SSD_F32> {
  static constexpr int kVecs = 4;
  using type = float;
  static __device__ float load(float x) { return x; }
  static __device__ float store(float z) { return z; }
};

// What a rule needs of its sequence.
struct Rules {
  float rep, freq, pres;
  const float* bias;
  const int* tok;           // draft token of each node
  const int16_t* parent;
};

// Logit z of token v in row u, whose count word and bias entry are given.
__device__ __forceinline__ float adjust(float z, uint32_t word, uint32_t bias_entry,
                                        const Rules& ru, int v, int u) {
  uint32_t c = word & kCountBits;
  if (word & kDraftBit)
    for (int w = u; w > 0; w = ru.parent[w]) c += ru.tok[w] == v;
  // a division: 1 / rep would be infinite for the smallest rep, and one rounding more
  // (it saved 1.5 us of 64.6 in bf16, 4.5 of 458 in f32)
  if (c != 0u || (word & kPromptBit)) z = z > 0.f ? z / ru.rep : z * ru.rep;
  if (c != 0u) z = z - ru.freq * (float)c - ru.pres;
  if (bias_entry != 0u) z += ru.bias[bias_entry - 1];
  return z;
}

// 16 bytes global -> shared, of this thread's own ring.
__device__ __forceinline__ void fetch(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Bits k .. of a bitmap in shared memory with a word to spare.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* map, int k) {
  return __funnelshift_r(map[k >> 5], map[(k >> 5) + 1], k & 31);
}

// The top bits of four bytes, chosen by `which`, each repeated over its byte.
__device__ __forceinline__ uint32_t tops(uint32_t x, uint32_t which) {
  uint32_t y;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(y) : "r"(x), "r"(which));
  return y;
}

// A vector with the tokens whose bit is not set replaced.
template <int DT>
__device__ __forceinline__ uint4 masked(uint4 x, uint32_t ok,
                                        typename Elem<DT>::type fill) {
  if constexpr (DT == SSD_BF16) {
    // four bits to the top of four bytes, then each spread over two bytes
    const uint32_t lo = (ok & 15u) * 0x10204080u & 0x80808080u;
    const uint32_t hi = (ok >> 4) * 0x10204080u & 0x80808080u;
    const uint32_t m0 = tops(lo, 0x9988), m1 = tops(lo, 0xbbaa);
    const uint32_t m2 = tops(hi, 0x9988), m3 = tops(hi, 0xbbaa);
    const uint32_t f = (uint32_t)fill * 0x10001u;
    return make_uint4((x.x & m0) | (f & ~m0), (x.y & m1) | (f & ~m1), (x.z & m2) | (f & ~m2),
                      (x.w & m3) | (f & ~m3));
  } else {
    const uint32_t f = __float_as_uint(fill);
    return make_uint4(ok & 1u ? x.x : f, ok & 2u ? x.y : f, ok & 4u ? x.z : f, ok & 8u ? x.w : f);
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) logits_kernel(const __grid_constant__ LogitParams p) {
  using E = typename Elem<DT>::type;
  constexpr int VE = 16 / (int)sizeof(E);  // tokens of a vector
  constexpr int kVecs = Elem<DT>::kVecs;
  static_assert(kVecs * kThreads * VE == kMaxSlice, "a step per row");
  constexpr uint32_t kAll = (1u << VE) - 1u;
  extern __shared__ uint4 smem4[];
  constexpr int kStep = kVecs * kThreads;                           // vectors of a step
  uint4* ring = smem4;                                              // [kStages][kStep]
  // Touched tokens of each warp: those whose vector is the warp's in a
  // row that starts on a vector, or the one after (rows that do not start on one
  // shift their vectors by less than a vector).
  constexpr int kList = (kVecs * 32 + 1) * VE;
  constexpr int lists = kThreads / 32;
  uint16_t* list = reinterpret_cast<uint16_t*>(ring + kStages * kStep);  // [lists][kList]
  uint32_t* count = reinterpret_cast<uint32_t*>(list + lists * kList);   // [slice]
  uint32_t* touched = count + p.slice;                              // [slice / 32 + 4]
  const int words = p.slice / 32 + 4;
  uint32_t* bits = touched + words;                                 // [rows][words] if a mask
  uint16_t* bias_at = reinterpret_cast<uint16_t*>(bits + (p.r.mask ? p.rows * words : 0));
  __shared__ int s_tok[kMaxTreeNodes];
  __shared__ int16_t s_parent[kMaxTreeNodes];
  __shared__ int s_sum[kThreads / 32];

  const int tid = threadIdx.x;
  const int64_t cta = blockIdx.x;
  const int sl = (int)(cta % p.nslice);
  const int64_t rest = cta / p.nslice;
  const int grp = (int)(rest % p.ngroup);
  const int64_t b = rest / p.ngroup;
  const int u0 = grp * p.rows, u1 = min(p.N, u0 + p.rows);
  const int v0 = sl * p.slice, nv = min(p.slice, p.V - v0);
  const ssd_logit_rules& r = p.r;

  // ---- the rows' vectors: steps of kVecs * kThreads, alike for the whole CTA ----------
  struct Place {
    int u;                  // row
    const E* in;            // the slice of the row
    E* out;
    int head, nvec;         // tokens before its first whole vector, vectors
  };
  auto measure = [&](Place& q) {
    const uint32_t mis = (uint32_t)(uintptr_t)q.in & 15u;
    const bool vec = mis == ((uint32_t)(uintptr_t)q.out & 15u);
    q.head = vec ? min(nv, (int)((16u - mis) & 15u) / (int)sizeof(E)) : nv;
    q.nvec = (nv - q.head) / VE;
  };
  // rows that start alike have the same head and vectors
  const bool alike = ((p.in_stride | p.out_stride) * (int64_t)sizeof(E)) % 16 == 0;
  auto next_row = [&](Place& q) {
    q.in += p.in_stride;
    q.out += p.out_stride;
    ++q.u;
    if (!alike) measure(q);
  };
  auto settle = [&](Place& q) {  // to the next row that has vectors
    while (q.u < u1 && q.nvec == 0) next_row(q);
  };
  Place first;
  first.u = u0;
  first.in = static_cast<const E*>(p.in) + (b * p.N + u0) * p.in_stride + v0;
  first.out = static_cast<E*>(p.out) + (b * p.N + u0) * p.out_stride + v0;
  measure(first);
  Place ahead = first;
  settle(ahead);
  Place at = ahead;
  const int lane = tid & 31, warp = tid >> 5, mine = warp * kVecs * 32;
  const uint32_t my_ring = smem_addr(ring + mine + lane);
  auto fetch_next = [&](int stage) {
    if (ahead.u < u1) {
      const uint4* in = reinterpret_cast<const uint4*>(ahead.in + ahead.head) + mine + lane;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (mine + j * 32 + lane < ahead.nvec)
          fetch(my_ring + (stage * kStep + j * 32) * 16, in + j * 32);
      next_row(ahead);
      settle(ahead);
    }
    fetch_commit();
  };
  // the rows' mask bits, then the first vectors: both arrive while the counts are made
  if (r.mask) {
    const int w0 = v0 >> 5, per = min(p.slice / 32 + 1, ((p.V - 1) >> 5) + 1 - w0);
    for (int u = u0 + warp; u < u1; u += kThreads / 32) {
      const int32_t* m = r.mask + b * r.mask_seq_stride + u * r.mask_row_stride + w0;
      const uint32_t d = smem_addr(bits + (u - u0) * words);
      for (int i = lane; i < per; i += 32) fetch4(d + i * 4, m + i);
    }
  }
  fetch_commit();
#pragma unroll
  for (int d = 0; d < kStages - 1; ++d) fetch_next(d);

  // ---- what the sequence's rules say: all loads first, so that they wait for memory
  // together (a CTA lives for about 20 us) ------------------------------------------
  float rep = 1.f, freq = 0.f, pres = 0.f;
  int len = 0, prompt = 0, tok = 0, h[kBatch], id[kBiasBatch];
  const int32_t* hist = r.history + b * r.history_stride;
  const int32_t* ids = r.bias_ids + b * r.n_bias;
  if (r.repetition) rep = r.repetition[b];
  if (r.frequency) freq = r.frequency[b];
  if (r.presence) pres = r.presence[b];
  if (r.history) {
    len = r.history_len[b];
    if (r.prompt_len) prompt = r.prompt_len[b];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {  // before the length is known
      const int i = tid + j * kThreads;
      h[j] = i < r.history_max ? hist[i] : 0;
    }
  }
  const bool draft = r.draft_tokens && tid > 0 && tid < p.N;  // N <= kThreads
  if (draft) tok = r.draft_tokens[b * r.draft_stride + tid - 1];
#pragma unroll
  for (int j = 0; j < kBiasBatch; ++j) {
    const int i = tid + j * kThreads;
    id[j] = i < r.n_bias ? ids[i] : -1;
  }

  // ---- counts of the slice's tokens ---------------------------------------------
  for (int i = tid; i < (p.slice + words) / 4; i += kThreads)
    reinterpret_cast<uint4*>(count)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (r.n_bias)
    for (int i = tid; i < p.slice / 8; i += kThreads)
      reinterpret_cast<uint4*>(bias_at)[i] = make_uint4(0u, 0u, 0u, 0u);
  int bad = 0;
  if (!(rep > 0.f) || isinf(rep)) { rep = 1.f; bad = SSD_DEV_BAD_PENALTY; }
  if (!isfinite(freq)) { freq = 0.f; bad = SSD_DEV_BAD_PENALTY; }
  if (!isfinite(pres)) { pres = 0.f; bad = SSD_DEV_BAD_PENALTY; }
  const Rules ru{rep, freq, pres, r.bias + b * r.n_bias, s_tok, s_parent};
  if (len < 0 || len > r.history_max) {
    bad |= SSD_DEV_BAD_LENGTH;
    len = min(max(len, 0), r.history_max);
  }
  __syncthreads();

  auto touch = [&](int k) { atomicOr(&touched[k >> 5], 1u << (k & 31)); };
  for (int i0 = tid; i0 < len;) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads, k = h[j] - v0;
      if (i >= len) break;
      if ((unsigned)h[j] >= (unsigned)p.V) {
        bad |= SSD_DEV_BAD_TOKEN;
      } else if ((unsigned)k < (unsigned)nv) {
        if (i < prompt) atomicOr(&count[k], kPromptBit);
        else atomicAdd(&count[k], 1u);
        touch(k);
      }
    }
    i0 += kThreads * kBatch;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads;
      h[j] = i < len ? hist[i] : 0;
    }
  }
  if (draft) {
    const int k = tok - v0;
    s_tok[tid] = tok;
    s_parent[tid] = p.parent[tid];
    if ((unsigned)tok >= (unsigned)p.V) {
      bad |= SSD_DEV_BAD_TOKEN;
    } else if ((unsigned)k < (unsigned)nv) {
      atomicOr(&count[k], kDraftBit);
      touch(k);
    }
  }
  for (int i0 = tid; i0 < r.n_bias;) {
#pragma unroll
    for (int j = 0; j < kBiasBatch; ++j) {
      const int i = i0 + j * kThreads, k = id[j] - v0;
      if (i >= r.n_bias) break;
      if (id[j] >= p.V) {
        bad |= SSD_DEV_BAD_TOKEN;
      } else if (id[j] >= 0 && (unsigned)k < (unsigned)nv) {
        // the latest entry of a token holds: the largest index + 1
        unsigned short* at = &bias_at[k];
        unsigned short old = *at;
        while (old < (unsigned short)(i + 1)) {
          const unsigned short seen = atomicCAS(at, old, (unsigned short)(i + 1));
          if (seen == old) break;
          old = seen;
        }
        touch(k);
      }
    }
    i0 += kThreads * kBiasBatch;
#pragma unroll
    for (int j = 0; j < kBiasBatch; ++j) {
      const int i = i0 + j * kThreads;
      id[j] = i < r.n_bias ? ids[i] : -1;
    }
  }
  if (bad && p.status) atomicOr(p.status, bad);

  const E fill = Elem<DT>::store(r.fill);
  fetch_wait<kStages - 1>();  // the mask bits
  __syncthreads();

  // ---- the touched tokens of each warp ----------------------------------------------------
  uint16_t* my_list = list + warp * kList;
  int n = 0;
  {
    const int from = mine * VE, to = min(from + kList, p.slice);
    for (int w0 = from; w0 < to; w0 += 32 * 32) {  // a word of the bitmap per lane
      const int k = w0 + lane * 32;
      uint32_t m = k < to ? touched[k >> 5] : 0u;
      if (k < to && to - k < 32) m &= (1u << (to - k)) - 1u;
      int before = __popc(m);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += y;
      }
      const int all = __shfl_sync(0xffffffffu, before, 31);
      before += n - __popc(m);
      for (; m != 0u; m &= m - 1u) my_list[before++] = (uint16_t)(k + __ffs(m) - 1);
      n += all;
    }
  }

  for (int stage = 0; at.u < u1; stage = (stage + 1) % kStages) {
    fetch_next((stage + kStages - 1) % kStages);
    fetch_wait<kStages - 1>();
    __syncwarp();  // the warp's copies are there for all its lanes
    const uint32_t* allow = bits + (at.u - u0) * words;
    uint4* mem = ring + stage * kStep + mine;
    for (int t = lane; t < n; t += 32) {
      const int k = my_list[t], d = k - at.head, i = d / VE;
      if (d < 0 || (unsigned)(i - mine) >= (unsigned)(kVecs * 32) || i >= at.nvec) continue;
      if (r.mask && !(allow[k >> 5] >> (k & 31) & 1u)) continue;
      E* z = reinterpret_cast<E*>(mem + (i - mine)) + d % VE;
      *z = Elem<DT>::store(adjust(Elem<DT>::load(*z), count[k], r.n_bias ? bias_at[k] : 0u, ru,
                                  v0 + k, at.u));
    }
    __syncwarp();
    uint4* out = reinterpret_cast<uint4*>(at.out + at.head) + mine + lane;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = mine + j * 32 + lane;
      if (i < at.nvec) {
        uint4 x = mem[j * 32 + lane];
        if (r.mask) {
          uint32_t ok;
          if (at.head != 0)
            ok = bits_at(allow, at.head + i * VE) & kAll;
          else if constexpr (VE == 8)
            ok = reinterpret_cast<const uint8_t*>(allow)[i];
          else
            ok = reinterpret_cast<const uint8_t*>(allow)[i >> 1] >> (i & 1) * 4 & 15u;
          if (ok != kAll) x = masked<DT>(x, ok, fill);
        }
        __stcs(out + j * 32, x);
      }
    }
    __syncwarp();  // the ring is read
    next_row(at);
    settle(at);
  }

  // ---- the ends of rows that do not start or end on a vector, token by token: up to 2 VE
  // of a row, all rows side by side; rows whose vectors lie differently in and out have no
  // vectors, and are taken one after the other ------------------------------------------
  if (!alike || first.head + first.nvec * VE < nv || first.head > 0) {
    const bool whole = first.nvec == 0 && nv >= 2 * VE;
    const int per = whole ? kThreads : 2 * VE;  // threads of a row
    for (int u = u0 + tid / per; u < u1; u += kThreads / per) {
      Place q = first;
      q.in += (u - u0) * p.in_stride;
      q.out += (u - u0) * p.out_stride;
      measure(q);
      const int skip = q.nvec * VE;  // the tokens between the ends
      for (int i = tid % per; i < nv - skip; i += per) {
        const int k = i < q.head ? i : i + skip;
        E e = q.in[k];
        if (touched[k >> 5] >> (k & 31) & 1u)
          e = Elem<DT>::store(adjust(Elem<DT>::load(e), count[k], r.n_bias ? bias_at[k] : 0u, ru,
                                     v0 + k, u));
        if (r.mask && !(bits[(u - u0) * words + (k >> 5)] >> (k & 31) & 1u)) e = fill;
        q.out[k] = e;
      }
    }
  }

  // ---- allowed tokens: each row is counted whole by one of the slices' CTAs --------------
  if (p.allowed) {
    const int last_word = (p.V - 1) >> 5;
    for (int u = u0 + sl; u < u1; u += p.nslice) {
      int n = tid == 0 ? p.V : 0;
      if (r.mask) {
        const int32_t* mask = r.mask + b * r.mask_seq_stride + u * r.mask_row_stride;
        n = 0;
#pragma unroll 4
        for (int i = tid; i <= last_word; i += kThreads) {
          uint32_t m = (uint32_t)mask[i];
          if (i == last_word && (p.V & 31)) m &= (1u << (p.V & 31)) - 1u;
          n += __popc(m);
        }
      }
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) s_sum[warp] = n;
      __syncthreads();
      if (tid == 0) {
        int t = 0;
        for (int i = 0; i < kThreads / 32; ++i) t += s_sum[i];
        p.allowed[b * p.N + u] = t;
      }
      __syncthreads();  // s_sum is read
    }
  }
}

// Bytes of shared memory of a call.
template <int DT>
constexpr size_t smem_bytes(int slice, int rows, bool mask, bool bias) {
  constexpr size_t es = sizeof(typename Elem<DT>::type);
  const size_t words = slice / 32 + 4;
  return (size_t)kStages * kMaxSlice * es +                  // ring
         (kMaxSlice + kThreads / 32 * (16 / es)) * 2 +       // lists
         (slice + words) * 4 + (mask ? rows * words * 4 : 0) + (bias ? (size_t)slice * 2 : 0);
}

template <int DT>
cudaError_t launch(const LogitParams& p, int64_t grid, cudaStream_t s) {
  const size_t smem = smem_bytes<DT>(p.slice, p.rows, p.r.mask != nullptr, p.r.n_bias > 0);
  if (smem > 46 * 1024) {  // more than a kernel may have without asking (48 KB with its static part)
    // the most that any call needs: the limit is the function's, and a call of another
    // thread may come between this and the launch
    const cudaError_t e = cudaFuncSetAttribute(
        logits_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)smem_bytes<DT>(kMaxSlice, kMaxRows, true, true));
    if (e != cudaSuccess) return e;
  }
  logits_kernel<DT><<<(unsigned)grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" ssd_status ssd_process_logits(const ssd_logits* in, const ssd_logits* out, int B, int N,
                                         int V, const ssd_logit_rules* rules, int32_t* allowed,
                                         int32_t* dev_status, void* stream) {
  for (const ssd_logits* l : {in, out}) {
    if (!l || !l->ptr || (l->dtype != SSD_BF16 && l->dtype != SSD_F32) || l->pad_ != 0 ||
        l->row_stride < V || ((uintptr_t)l->ptr) % (l->dtype == SSD_BF16 ? 2 : 4) != 0)
      return SSD_ERR_INVALID_ARG;
  }
  if (in->dtype != out->dtype || !rules || B < 1 || N < 1 || V < 1) return SSD_ERR_INVALID_ARG;
  if (in->ptr == out->ptr && in->row_stride != out->row_stride) return SSD_ERR_INVALID_ARG;
  if (V > SSD_MAX_V || N > kMaxTreeNodes) return SSD_ERR_UNSUPPORTED;
  const ssd_logit_rules& r = *rules;
  if (r.pad_ != 0 || std::isnan(r.fill)) return SSD_ERR_INVALID_ARG;
  if (r.history && (!r.history_len || r.history_max < 0 || r.history_stride < 0))
    return SSD_ERR_INVALID_ARG;
  if (r.n_bias < 0 || r.n_bias > 65535 || (r.n_bias > 0 && (!r.bias_ids || !r.bias)))
    return SSD_ERR_INVALID_ARG;
  if (r.mask && (r.mask_seq_stride < 0 || r.mask_row_stride < 0)) return SSD_ERR_INVALID_ARG;
  if (r.draft_tokens && r.draft_stride < 0) return SSD_ERR_INVALID_ARG;
  LogitParams p{};
  for (int u = 0; u < N; ++u) {
    const int par = r.parent ? r.parent[u] : u - 1;
    if (u == 0 ? par != -1 : (par < 0 || par >= u)) return SSD_ERR_INVALID_ARG;
    p.parent[u] = (int16_t)par;
  }
  p.in = in->ptr;
  p.in_stride = in->row_stride;
  p.out = const_cast<void*>(out->ptr);
  p.out_stride = out->row_stride;
  p.B = B;
  p.N = N;
  p.V = V;
  p.r = r;
  p.allowed = allowed;
  p.status = dev_status;
  // The widest slices with all rows of a sequence per CTA, so that its
  // history is scanned least; where that leaves SMs idle, one row per CTA,
  // then narrower slices.
  const int64_t want = 2 * (int64_t)std::max(num_sms(), 1);
  p.slice = kMaxSlice;
  while (p.slice > kMinSlice && p.slice / 2 >= V) p.slice /= 2;
  p.rows = std::min(N, kMaxRows);
  auto ctas = [&] {
    p.nslice = (V + p.slice - 1) / p.slice;
    p.ngroup = (N + p.rows - 1) / p.rows;
    return (int64_t)B * p.nslice * p.ngroup;
  };
  if (ctas() < want) p.rows = 1;
  while (ctas() < want && p.slice > kMinSlice) p.slice /= 2;
  const int64_t grid = ctas();
  if (grid > 0x7fffffff) return SSD_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = in->dtype == SSD_BF16 ? launch<SSD_BF16>(p, grid, s)
                                              : launch<SSD_F32>(p, grid, s);
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return SSD_ERR_CUDA;
}
