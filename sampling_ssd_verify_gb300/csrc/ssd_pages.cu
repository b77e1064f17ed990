// ssd_pages.cu -- pages, slots and positions of a paged key/value cache from
// request lengths (ssd_page_plan).
//
// All arithmetic is running sums over the requests: of their new tokens, of
// the pages they give back and of the pages they take.  The i-th page taken
// is entry top - 1 - i of the stack with the returned pages on it, so every
// page and every slot follows from the sums by itself.  Each CTA therefore
// forms the sums of all requests again in its shared memory (a few KB of
// lengths from L2) and writes its share of the outputs; no CTA waits for
// another, and nothing that the launch writes is read by it: table entries
// taken lie at columns >= held, those read below it; stack entries written
// lie at >= *free_count, those read below it.  Bound by the latency of the
// launch, the loads of the lengths and the scan; bytes count from about a
// hundred thousand new tokens on (16 bytes each): 4.1 us for 32 requests, 6.0 for 256,
// 10.5 for 1000 with half a million new tokens.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ssd.h"
#include "ssd_internal.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRequests = 8192;  // five numbers each in shared memory
constexpr int smem_bytes(int B) { return 5 * (B + 1) * (int)sizeof(int); }
constexpr int kBatch = 4;           // new tokens per thread at a time
constexpr int kMaxCount = 1 << 30;
constexpr int kRowsPerCta = 2048;   // new tokens per CTA before another one is added

struct PageParams {
  const int32_t *lens, *add, *held;
  int B;
  int32_t* tables;
  int64_t table_stride;
  int cols;
  int32_t* free_pages;
  int free_cap;
  const int32_t* free_count;
  int page, max_rows;
  Divisor by_page;
  int64_t* slots;
  int32_t *positions, *owner, *cu, *kv_len, *held_out, *served, *free_out, *status;
};

struct Request {
  int len, add, held, need;
  bool ok;  // its lengths are consistent
};

__device__ __forceinline__ Request request(const PageParams& p, int b) {
  Request q;
  q.len = p.lens[b];
  q.add = p.add[b];
  q.held = p.held[b];
  const int64_t end = (int64_t)q.len + q.add;
  q.ok = q.len >= 0 && q.add >= 0 && q.held >= 0 && q.held <= p.cols &&
         end <= min((int64_t)p.cols * p.page, (int64_t)0x7fffffff) &&
         q.len <= (int64_t)q.held * p.page;
  q.need = q.ok ? p.by_page.quotient((int)end) + (p.by_page.quotient((int)end) * p.page < end)
                : q.held;
  if (!q.ok) q.add = 0;
  return q;
}

__device__ __forceinline__ int clamp32(int64_t x) {
  return (int)(x < 0x7fffffff ? x : 0x7fffffff);
}

// The largest b in [0, n) with sum[b] <= i (sum[0] = 0 <= i).
__device__ __forceinline__ int find(const int* sum, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(const PageParams p) {
  extern __shared__ int s_sums[];
  int* s_cu = s_sums;                   // [B + 1] new tokens before request b
  int* s_back = s_cu + p.B + 1;         // [B + 1] pages given back before it
  int* s_ask = s_back + p.B + 1;        // [B + 1] pages asked for before it
  int* s_len = s_ask + p.B + 1;         // [B] its tokens,
  int* s_held = s_len + p.B;            // [B] and pages
  __shared__ int64_t s_warp[3][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n0 = *p.free_count;
  int bad = 0;

  // ---- running sums: consecutive requests per thread, then over the threads ------
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int64_t sum[3] = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const Request q = request(p, b);
    if (!q.ok) bad = SSD_DEV_BAD_LENGTH;
    sum[0] += q.add;
    sum[1] += max(q.held - q.need, 0);
    sum[2] += max(q.need - q.held, 0);
  }
  int64_t inc[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int64_t x = sum[k];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    inc[k] = x;
    if (lane == 31) s_warp[k][warp] = x;
  }
  __syncthreads();
  int64_t run[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += s_warp[k][w];
    run[k] = before + inc[k] - sum[k];
  }
  for (int b = b0; b < b1; ++b) {
    const Request q = request(p, b);
    s_cu[b] = clamp32(run[0]);
    s_back[b] = clamp32(run[1]);
    s_ask[b] = clamp32(run[2]);
    s_len[b] = q.len;
    s_held[b] = q.held;
    run[0] += q.add;
    run[1] += max(q.held - q.need, 0);
    run[2] += max(q.need - q.held, 0);
  }
  if (b1 == p.B && b0 < p.B) {  // the thread of the last request
    s_cu[p.B] = clamp32(run[0]);
    s_back[p.B] = clamp32(run[1]);
    s_ask[p.B] = clamp32(run[2]);
  }
  __syncthreads();

  const int n = min(max(n0, 0), p.free_cap);
  const int total = s_cu[p.B], back = s_back[p.B], ask = s_ask[p.B];
  const int64_t top = (int64_t)n + back;

  // where entry i of the stack with the returned pages on it is, 0 <= i < top
  auto stack_at = [&](int64_t i) -> const int32_t* {
    if (i < n) return p.free_pages + i;
    const int k = (int)(i - n);
    const int b = find(s_back, p.B, k);  // it gives back its last pages
    return p.tables + b * p.table_stride + (s_held[b] - (s_back[b + 1] - k));
  };
  auto is_served = [&](const Request& q, int b) {
    return q.ok && (q.need <= q.held || (int64_t)s_ask[b + 1] <= top);
  };

  const int gtid = blockIdx.x * kThreads + tid, nthreads = gridDim.x * kThreads;
  // ---- rows of the new tokens (of consistent requests only) -------------------------
  for (int t0 = gtid; t0 < p.max_rows; t0 += nthreads * kBatch) {
    const int32_t* from[kBatch];
    int pos[kBatch], own[kBatch], off[kBatch], page[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int t = t0 + j * nthreads;
      from[j] = nullptr;
      pos[j] = own[j] = -1;
      off[j] = 0;
      if (t < p.max_rows && t < total) {
        const int b = find(s_cu, p.B, t), held = s_held[b];
        own[j] = b;
        pos[j] = s_len[b] + (t - s_cu[b]);
        const int col = p.by_page.quotient(pos[j]);
        off[j] = pos[j] - col * p.page;
        if (s_ask[b] == s_ask[b + 1] || (int64_t)s_ask[b + 1] <= top)  // served
          from[j] = col < held ? p.tables + b * p.table_stride + col
                               : stack_at(top - 1 - (s_ask[b] + (col - held)));
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) page[j] = from[j] ? *from[j] : 0;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int t = t0 + j * nthreads;
      if (t >= p.max_rows) break;
      p.slots[t] = from[j] ? (int64_t)page[j] * p.page + off[j] : -1;
      if (p.positions) p.positions[t] = pos[j];
      if (p.owner) p.owner[t] = own[j];
    }
  }
  // ---- pages taken, pages given back ---------------------------------------------
  for (int64_t i = gtid; i < min((int64_t)ask, top); i += nthreads) {
    const int b = find(s_ask, p.B, (int)i);
    if ((int64_t)s_ask[b + 1] <= top)
      p.tables[b * p.table_stride + s_held[b] + ((int)i - s_ask[b])] = *stack_at(top - 1 - i);
  }
  for (int k = gtid; k < back; k += nthreads)
    if (n + (int64_t)k < p.free_cap) p.free_pages[n + k] = *stack_at(n + (int64_t)k);
  // ---- the requests ----------------------------------------------------------------
  // the stack once `taken` pages are off it: what lies past the array then is lost
  auto leave = [&](int taken) {
    *p.free_out = (int)min(top - taken, (int64_t)p.free_cap);
    if (top - taken > p.free_cap) bad |= SSD_DEV_BAD_LENGTH;
  };
  for (int b = gtid; b < p.B; b += nthreads) {
    const Request q = request(p, b);
    const bool ok = is_served(q, b);
    p.cu[b] = s_cu[b];
    p.kv_len[b] = ok ? q.len + q.add : q.len;
    p.held_out[b] = ok ? q.need : q.held;
    p.served[b] = ok;
    if (q.ok && !ok) bad |= SSD_DEV_NO_PAGES;
    // the pages left after the last request that got what it asked for
    if (s_ask[b] < s_ask[b + 1] && s_ask[b] <= top && s_ask[b + 1] > top) leave(s_ask[b]);
  }
  if (gtid == 0) {
    p.cu[p.B] = total;
    if (ask <= top) leave(ask);
    if (n != n0 || total > p.max_rows) bad |= SSD_DEV_BAD_LENGTH;
  }
  if (bad && p.status) atomicOr(p.status, bad);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" ssd_status ssd_page_plan(const int32_t* lens, const int32_t* new_tokens,
                                    const int32_t* held, int B, int32_t* tables,
                                    int64_t table_stride, int cols, int32_t* free_pages,
                                    int free_cap, const int32_t* free_count, int page,
                                    int max_rows, int64_t* slots, int32_t* positions,
                                    int32_t* owner, int32_t* cu, int32_t* kv_len,
                                    int32_t* held_out, int32_t* served, int32_t* free_out,
                                    int32_t* dev_status, void* stream) {
  if (!lens || !new_tokens || !held || !tables || !free_count || !cu || !kv_len || !held_out ||
      !served || !free_out)
    return SSD_ERR_INVALID_ARG;
  if (B < 1 || cols < 1 || page < 1 || free_cap < 0 || max_rows < 0 || table_stride < cols)
    return SSD_ERR_INVALID_ARG;
  if ((free_cap > 0 && !free_pages) || (max_rows > 0 && !slots)) return SSD_ERR_INVALID_ARG;
  // sums of pages and indexes of rows stay below 2^31 with room for a stride
  if (B > kMaxRequests || (int64_t)B * cols > kMaxCount || max_rows > kMaxCount)
    return SSD_ERR_UNSUPPORTED;
  // lengths and pages are read again while outputs are written
  for (const void* out : {(const void*)slots, (const void*)positions, (const void*)owner,
                          (const void*)cu, (const void*)kv_len, (const void*)held_out,
                          (const void*)served, (const void*)free_out})
    for (const int32_t* in : {lens, new_tokens, held, (const int32_t*)tables,
                              (const int32_t*)free_pages, free_count})
      if (out && out == in) return SSD_ERR_INVALID_ARG;
  const PageParams p{lens,     new_tokens, held,  B, tables, table_stride, cols,
                     free_pages, free_cap, free_count, page,    max_rows, divisor(page), slots, positions,
                     owner,    cu,         kv_len, held_out,   served, free_out,     dev_status};
  const int smem = smem_bytes(B);
  const int64_t work = std::max<int64_t>(max_rows / kRowsPerCta, B / kThreads);
  const int grid = work == 0 ? 1 : (int)std::min<int64_t>(std::max(num_sms(), 1), 1 + work);
  cudaError_t e = cudaSuccess;
  if (smem > 46 * 1024)  // more than a kernel may have without asking; the most that any call
    // needs, since the limit is the function's and another thread's call may come between
    e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_bytes(kMaxRequests));
  if (e == cudaSuccess) {
    page_plan_kernel<<<grid, kThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return SSD_ERR_CUDA;
}
