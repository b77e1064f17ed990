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
// A warp streams its own vectors through its own part of a ring in shared
// memory, filled by asynchronous copies, four vectors per thread a step.  A
// bitmap tells which tokens of a vector are touched; the warp lists those of a
// step and shares them out evenly, a token per lane (one in thirty is touched
// after 4096 tokens: each lane by itself would take its hits one after the
// other, with most lanes idle).  No barrier stands between the rows.
//
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
constexpr int kVecs = 2;            // vectors of a thread and step: 8 KB per CTA
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

template <int DT> struct Elem;
template <> struct Elem<SSD_BF16> {
  using type = uint16_t;
  static __device__ float load(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
  static __device__ uint16_t store(float z) { return __bfloat16_as_ushort(__float2bfloat16_rn(z)); }
};
template <> struct Elem<SSD_F32> {
  using type = float;
  static __device__ float load(float x) { return x; }
  static __device__ float store(float z) { return z; }
};

// What a rule needs of its sequence.
struct Rules {
  float rep, inv, freq, pres;  // inv = 1 / rep: one more rounding than a division, 20 instructions less
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
  if (c != 0u || (word & kPromptBit)) z *= z > 0.f ? ru.inv : ru.rep;
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

template <int DT>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitParams p) {
  using E = typename Elem<DT>::type;
  constexpr int VE = 16 / (int)sizeof(E);  // tokens of a vector
  constexpr uint32_t kAll = (1u << VE) - 1u;
  extern __shared__ uint4 smem4[];
  uint4* ring = smem4;                                              // [kStages][kVecs][kThreads]
  constexpr int kHits = kVecs * 32 * VE;                            // tokens of a warp and step
  uint16_t* list = reinterpret_cast<uint16_t*>(ring + kStages * kVecs * kThreads) +
                   (threadIdx.x >> 5) * kHits;
  uint32_t* count =                                                 // [slice]
      reinterpret_cast<uint32_t*>(list + (kThreads / 32 - (threadIdx.x >> 5)) * kHits);
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
  constexpr int kStep = kVecs * kThreads;
  struct Place {
    int u, i;               // row, its first vector of the step
    const E* in;            // the slice of the row
    int head, nvec;         // tokens before its first whole vector, vectors
  };
  auto row_at = [&](Place& q) {
    q.in = static_cast<const E*>(p.in) + (b * p.N + q.u) * p.in_stride + v0;
    const E* out = static_cast<const E*>(p.out) + (b * p.N + q.u) * p.out_stride + v0;
    const uint32_t mis = (uint32_t)(uintptr_t)q.in & 15u;
    const bool vec = mis == ((uint32_t)(uintptr_t)out & 15u);
    q.head = vec ? min(nv, (int)((16u - mis) & 15u) / (int)sizeof(E)) : nv;
    q.nvec = (nv - q.head) / VE;
    q.i = 0;
  };
  auto settle = [&](Place& q) {  // to the next row that has vectors
    while (q.u < u1 && q.i >= q.nvec)
      if (++q.u < u1) row_at(q);
  };
  Place ahead;
  ahead.u = u0;
  row_at(ahead);
  settle(ahead);
  Place at = ahead;
  auto fetch_next = [&](int stage) {
    if (ahead.u < u1) {
      const uint4* in = reinterpret_cast<const uint4*>(ahead.in + ahead.head);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const int i = ahead.i + j * kThreads + tid;
        if (i < ahead.nvec) fetch(smem_addr(ring + stage * kStep + j * kThreads + tid), in + i);
      }
      ahead.i += kStep;
      settle(ahead);
    }
    fetch_commit();
  };
  // the rows' mask bits, then the first vectors: both arrive while the counts are made
  if (r.mask) {
    const int w0 = v0 >> 5, per = min(p.slice / 32 + 1, ((p.V - 1) >> 5) + 1 - w0);
    const int32_t* m = r.mask + b * r.mask_seq_stride + w0;
    for (int i = tid; i < (u1 - u0) * per; i += kThreads) {
      const int u = i / per, w = i - u * per;
      fetch4(smem_addr(bits + u * words + w), m + (u0 + u) * r.mask_row_stride + w);
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
  const Rules ru{rep, 1.f / rep, freq, pres, r.bias + b * r.n_bias, s_tok, s_parent};
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

  const int lane = tid & 31;
  for (int stage = 0; at.u < u1; stage = (stage + 1) % kStages) {
    fetch_next((stage + kStages - 1) % kStages);
    fetch_wait<kStages - 1>();
    __syncwarp();  // the warp's copies are there for all its lanes
    E* out = static_cast<E*>(p.out) + (b * p.N + at.u) * p.out_stride + v0;
    const uint32_t* allow = bits + (at.u - u0) * words;
    const int k0 = at.head + at.i * VE;  // the step's first token
    uint32_t hit[kVecs];
    int n = 0;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = at.i + j * kThreads + tid, k = at.head + i * VE;
      hit[j] = 0u;
      if (i < at.nvec) {
        const uint4 x = ring[stage * kStep + j * kThreads + tid];
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
        const uint32_t ok = r.mask ? bits_at(allow, k) & kAll : kAll;
        hit[j] = bits_at(touched, k) & ok;
        if (ok != kAll) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (DT == SSD_BF16) {
              const uint32_t m = (ok >> (2 * q) & 1u ? 0xffffu : 0u) |
                                 (ok >> (2 * q + 1) & 1u ? 0xffff0000u : 0u);
              w[q] = (w[q] & m) | (((uint32_t)fill * 0x10001u) & ~m);
            } else {
              w[q] = ok >> q & 1u ? w[q] : __float_as_uint(fill);
            }
          }
        }
        __stcs(reinterpret_cast<uint4*>(out + k), make_uint4(w[0], w[1], w[2], w[3]));
        n += __popc(hit[j]);
      }
    }
    // the touched tokens of the warp's vectors, listed and then taken one per lane
    int before = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += y;
    }
    const int total = __shfl_sync(0xffffffffu, before, 31);
    before -= n;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      for (uint32_t h = hit[j]; h != 0u; h &= h - 1u)
        list[before++] = (uint16_t)((j * kThreads + tid) * VE + __ffs(h) - 1);
    __syncwarp();
    const E* raw = reinterpret_cast<const E*>(ring + stage * kStep);
    for (int t = lane; t < total; t += 32) {
      const int e = list[t], k = k0 + e;
      const float z = adjust(Elem<DT>::load(raw[e]), count[k], r.n_bias ? bias_at[k] : 0u, ru,
                             v0 + k, at.u);
      out[k] = Elem<DT>::store(z);
    }
    __syncwarp();  // list and ring are read
    at.i += kStep;
    settle(at);
  }

  const int last_word = (p.V - 1) >> 5;
  for (int u = u0; u < u1; ++u) {
    // ---- the ends of rows that are not aligned, token by token -------------------------
    Place q;
    q.u = u;
    row_at(q);
    E* out = static_cast<E*>(p.out) + (b * p.N + u) * p.out_stride + v0;
    auto single = [&](int k) {
      E e = q.in[k];
      if (touched[k >> 5] >> (k & 31) & 1u)
        e = Elem<DT>::store(adjust(Elem<DT>::load(e), count[k], r.n_bias ? bias_at[k] : 0u, ru,
                                   v0 + k, u));
      if (r.mask && !(bits[(u - u0) * words + (k >> 5)] >> (k & 31) & 1u)) e = fill;
      out[k] = e;
    };
    for (int k = tid; k < q.head; k += kThreads) single(k);
    for (int k = q.head + q.nvec * VE + tid; k < nv; k += kThreads) single(k);

    // ---- allowed tokens: each row is counted whole by one of the slices' CTAs --------
    if (p.allowed && (u - u0) % p.nslice == sl) {
      int n = 0;
      if (r.mask) {
        const int32_t* mask = r.mask + b * r.mask_seq_stride + u * r.mask_row_stride;
        for (int i = tid; i <= last_word; i += kThreads) {
          uint32_t m = (uint32_t)mask[i];
          if (i == last_word && (p.V & 31)) m &= (1u << (p.V & 31)) - 1u;
          n += __popc(m);
        }
      } else {
        n = tid == 0 ? p.V : 0;
      }
      n = __reduce_add_sync(0xffffffffu, n);
      if ((tid & 31) == 0) s_sum[tid >> 5] = n;
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

template <int DT>
cudaError_t launch(const LogitParams& p, int64_t grid, size_t smem, cudaStream_t s) {
  if (smem > 46 * 1024) {  // more than a kernel may have without asking (48 KB with its static part)
    const cudaError_t e = cudaFuncSetAttribute(
        logits_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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
  const size_t words = p.slice / 32 + 4;
  const int ve = in->dtype == SSD_BF16 ? 8 : 4;
  const size_t smem = (size_t)kStages * kVecs * kThreads * 16 + kVecs * kThreads * ve * 2 +
                      (p.slice + words) * 4 +
                      (r.mask ? p.rows * words * 4 : 0) + (r.n_bias ? p.slice * 2 : 0);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = in->dtype == SSD_BF16 ? launch<SSD_BF16>(p, grid, smem, s)
                                              : launch<SSD_F32>(p, grid, smem, s);
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return SSD_ERR_CUDA;
}
