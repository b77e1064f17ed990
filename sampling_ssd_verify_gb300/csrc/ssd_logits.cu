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
// the history is scanned once for all N rows.  From row to row only the
// drafts that differ between the two paths are added or taken out.  A bitmap
// of the touched tokens lets a 16-byte vector of untouched ones pass with one
// look-up.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ssd.h"
#include "ssd_internal.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlice = 8192;     // tokens of a slice: 32 KB of counts, 16 KB of bias entries
constexpr int kMinSlice = 1024;
constexpr int kBatch = 4;           // vectors in flight per thread
constexpr uint32_t kPromptBit = 0x80000000u;  // counts word: token occurs in the prompt

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
  float rep, freq, pres;
  const float* bias;
};

__device__ __forceinline__ float adjust(float z, uint32_t word, uint32_t bias_entry,
                                        const Rules& ru) {
  if (word != 0u) z = z > 0.f ? z / ru.rep : z * ru.rep;
  const uint32_t c = word & ~kPromptBit;
  if (c != 0u) z = z - ru.freq * (float)c - ru.pres;
  if (bias_entry != 0u) z += ru.bias[bias_entry - 1];
  return z;
}

// The 32 mask bits from token v on (bits past the row are whatever the last
// word repeats; callers use only tokens of the row).
__device__ __forceinline__ uint32_t mask_bits(const int32_t* m, int v, int last_word) {
  const int w = v >> 5;
  const uint32_t lo = (uint32_t)m[w];
  if ((v & 31) == 0) return lo;
  const uint32_t hi = (uint32_t)m[min(w + 1, last_word)];
  return __funnelshift_r(lo, hi, v & 31);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitParams p) {
  using E = typename Elem<DT>::type;
  constexpr int VE = 16 / (int)sizeof(E);  // tokens of a vector
  constexpr uint32_t kAll = (1u << VE) - 1u;
  extern __shared__ uint4 smem4[];
  uint32_t* count = reinterpret_cast<uint32_t*>(smem4);             // [slice]
  uint32_t* touched = count + p.slice;                              // [slice / 32 + 2]
  uint16_t* bias_at = reinterpret_cast<uint16_t*>(touched + p.slice / 32 + 4);  // [slice] if biases
  __shared__ int s_tok[kMaxTreeNodes];
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

  // ---- the sequence's rules -----------------------------------------------------
  Rules ru{1.f, 0.f, 0.f, r.bias + b * r.n_bias};
  int bad = 0;
  if (r.repetition) {
    ru.rep = r.repetition[b];
    if (!(ru.rep > 0.f) || isinf(ru.rep)) { ru.rep = 1.f; bad = SSD_DEV_BAD_PENALTY; }
  }
  if (r.frequency) {
    ru.freq = r.frequency[b];
    if (!isfinite(ru.freq)) { ru.freq = 0.f; bad = SSD_DEV_BAD_PENALTY; }
  }
  if (r.presence) {
    ru.pres = r.presence[b];
    if (!isfinite(ru.pres)) { ru.pres = 0.f; bad = SSD_DEV_BAD_PENALTY; }
  }

  // ---- counts of the slice's tokens ---------------------------------------------
  for (int i = tid; i < (p.slice + p.slice / 32 + 4) / 4; i += kThreads)
    smem4[i] = make_uint4(0u, 0u, 0u, 0u);
  if (r.n_bias)
    for (int i = tid; i < p.slice / 8; i += kThreads)
      reinterpret_cast<uint4*>(bias_at)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (r.draft_tokens)
    for (int u = 1 + tid; u < p.N; u += kThreads) {
      const int t = r.draft_tokens[b * r.draft_stride + u - 1];
      s_tok[u] = t;
      if ((unsigned)t >= (unsigned)p.V) bad |= SSD_DEV_BAD_TOKEN;
    }
  __syncthreads();
  if (r.history) {
    int len = r.history_len[b];
    int prompt = r.prompt_len ? r.prompt_len[b] : 0;
    if (len < 0 || len > r.history_max) {
      bad |= SSD_DEV_BAD_LENGTH;
      len = min(max(len, 0), r.history_max);
    }
    const int32_t* h = r.history + b * r.history_stride;
    for (int i = tid; i < len; i += kThreads) {
      const int t = h[i], k = t - v0;
      if ((unsigned)t >= (unsigned)p.V) {
        bad |= SSD_DEV_BAD_TOKEN;
      } else if ((unsigned)k < (unsigned)nv) {
        if (i < prompt) atomicOr(&count[k], kPromptBit);
        else atomicAdd(&count[k], 1u);
        atomicOr(&touched[k >> 5], 1u << (k & 31));
      }
    }
  }
  for (int i = tid; i < r.n_bias; i += kThreads) {
    const int t = r.bias_ids[b * r.n_bias + i], k = t - v0;
    if (t >= p.V) {
      bad |= SSD_DEV_BAD_TOKEN;
    } else if (t >= 0 && (unsigned)k < (unsigned)nv) {
      // the latest entry of a token holds: the largest index + 1
      unsigned short* at = &bias_at[k];
      unsigned short old = *at;
      while (old < (unsigned short)(i + 1)) {
        const unsigned short seen = atomicCAS(at, old, (unsigned short)(i + 1));
        if (seen == old) break;
        old = seen;
      }
      atomicOr(&touched[k >> 5], 1u << (k & 31));
    }
  }
  if (bad && p.status) atomicOr(p.status, bad);

  const int last_word = (p.V - 1) >> 5;
  const E fill = Elem<DT>::store(r.fill);
  int at_node = 0;  // the node whose path the counts hold (thread 0)
  for (int u = u0; u < u1; ++u) {
    // ---- the drafts of this row's path -------------------------------------------
    __syncthreads();
    if (tid == 0 && r.draft_tokens) {
      // from node a's path to node c's: parents have lower indices, so the
      // larger index steps up until both meet
      int a = at_node, c = u;
      while (a != c) {
        const bool drop = a > c;
        const int node = drop ? a : c;
        const int k = s_tok[node] - v0;
        if ((unsigned)s_tok[node] < (unsigned)p.V && (unsigned)k < (unsigned)nv) {
          count[k] += drop ? 0xffffffffu : 1u;
          touched[k >> 5] |= 1u << (k & 31);
        }
        if (drop) a = p.parent[a];
        else c = p.parent[c];
      }
      at_node = u;
    }
    __syncthreads();

    const int32_t* mask =
        r.mask ? r.mask + b * r.mask_seq_stride + u * r.mask_row_stride : nullptr;
    const int64_t row = b * p.N + u;
    const E* in = static_cast<const E*>(p.in) + row * p.in_stride + v0;
    E* out = static_cast<E*>(p.out) + row * p.out_stride + v0;

    // one token, for the ends of rows that are not aligned
    auto single = [&](int k) {
      E e = in[k];
      if ((touched[k >> 5] >> (k & 31)) & 1u)
        e = Elem<DT>::store(adjust(Elem<DT>::load(e), count[k], r.n_bias ? bias_at[k] : 0u, ru));
      if (mask) {
        const int v = v0 + k;
        if (!(((uint32_t)mask[v >> 5] >> (v & 31)) & 1u)) e = fill;
      }
      out[k] = e;
    };
    const uint32_t mis = (uint32_t)(uintptr_t)in & 15u;
    const bool vec = mis == ((uint32_t)(uintptr_t)out & 15u);
    const int head = vec ? min(nv, (int)((16u - mis) & 15u) / (int)sizeof(E)) : nv;
    const int nvec = (nv - head) / VE;
    for (int k = tid; k < head; k += kThreads) single(k);
    for (int k = head + nvec * VE + tid; k < nv; k += kThreads) single(k);

    const uint4* in4 = reinterpret_cast<const uint4*>(in + head);
    uint4* out4 = reinterpret_cast<uint4*>(out + head);
    for (int i0 = tid; i0 < nvec; i0 += kThreads * kBatch) {
      uint4 x[kBatch];
      uint32_t ok[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * kThreads;
        if (i < nvec) {
          x[j] = __ldcs(in4 + i);
          ok[j] = mask ? mask_bits(mask, v0 + head + i * VE, last_word) & kAll : kAll;
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * kThreads;
        if (i >= nvec) break;
        const int k = head + i * VE;
        uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        const uint32_t hit =
            __funnelshift_r(touched[k >> 5], touched[(k >> 5) + 1], k & 31) & ok[j];
        if (ok[j] != kAll) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (DT == SSD_BF16) {
              const uint32_t m = (ok[j] >> (2 * q) & 1u ? 0xffffu : 0u) |
                                 (ok[j] >> (2 * q + 1) & 1u ? 0xffff0000u : 0u);
              w[q] = (w[q] & m) | (((uint32_t)fill * 0x10001u) & ~m);
            } else {
              w[q] = ok[j] >> q & 1u ? w[q] : __float_as_uint(fill);
            }
          }
        }
        __stcs(out4 + i, make_uint4(w[0], w[1], w[2], w[3]));
        // touched tokens: few, and written again by the same thread
        for (uint32_t h = hit & kAll; h != 0u; h &= h - 1u) {
          const int e = __ffs(h) - 1;
          const int q = DT == SSD_BF16 ? e >> 1 : e;
          const uint32_t word = q & 2 ? (q & 1 ? w[3] : w[2]) : (q & 1 ? w[1] : w[0]);
          float z;
          if constexpr (DT == SSD_BF16)
            z = Elem<DT>::load((uint16_t)(word >> (16 * (e & 1))));
          else
            z = __uint_as_float(word);
          z = adjust(z, count[k + e], r.n_bias ? bias_at[k + e] : 0u, ru);
          out[k + e] = Elem<DT>::store(z);
        }
      }
    }

    // ---- allowed tokens: each row is counted whole by one of the slices' CTAs --------
    if (p.allowed && (u - u0) % p.nslice == sl) {
      int n = 0;
      if (mask) {
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
        p.allowed[row] = t;
      }
    }
  }
}

template <int DT>
cudaError_t launch(const LogitParams& p, int64_t grid, size_t smem, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(
      logits_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
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
  p.rows = N;
  auto ctas = [&] {
    p.nslice = (V + p.slice - 1) / p.slice;
    p.ngroup = (N + p.rows - 1) / p.rows;
    return (int64_t)B * p.nslice * p.ngroup;
  };
  if (ctas() < want) p.rows = 1;
  while (ctas() < want && p.slice > kMinSlice) p.slice /= 2;
  const int64_t grid = ctas();
  if (grid > 0x7fffffff) return SSD_ERR_UNSUPPORTED;
  const size_t smem = (size_t)(p.slice + p.slice / 32 + 4) * 4 + (r.n_bias ? p.slice * 2 : 0);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = in->dtype == SSD_BF16 ? launch<SSD_BF16>(p, grid, smem, s)
                                              : launch<SSD_F32>(p, grid, smem, s);
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return SSD_ERR_CUDA;
}
