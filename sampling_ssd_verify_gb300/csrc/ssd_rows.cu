// ssd_rows.cu -- rows of a paged key/value cache: the keys and values of
// accepted nodes into their slots (ssd_append_path), and rows of the block
// tables continued, forked and freed (ssd_fork_rows).
//
// Both move whole tokens of all layers: a token of a layer is H rows of
// row_bytes, a few KB that mostly lie side by side, and copying is all there is
// to it.  A warp takes a token (append) or a few tokens (fork) of one layer's
// keys or values, with its loads in flight together before the first store.

#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "ssd_attention_dev.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;  // of a CTA that copies
constexpr int kFlight = 4; // 16-byte loads of a lane in flight

// What the copies of a call share.
struct Geometry {
  int planes;              // layers, times two with values beside the keys
  int pair;                // 1: plane j is layer j / 2, values if j is odd
  int chunks;              // 16-byte chunks of a token
  int head_chunks;         // of a head
  Divisor by_token, by_head;
};

__device__ __forceinline__ const char* plane_of(const ssd_layers& k, const ssd_layers& v,
                                                const Geometry& g, int j, const ssd_layers** at) {
  const ssd_layers& x = g.pair && (j & 1) ? v : k;
  *at = &x;
  return static_cast<const char*>(x.ptr) + (int64_t)(g.pair ? j >> 1 : j) * x.layer_stride;
}
// Chunk c of a token: its place in the token's bytes.
__device__ __forceinline__ int64_t chunk_at(const ssd_layers& x, const Geometry& g, int c) {
  if (g.head_chunks == g.chunks) return (int64_t)c * 16;
  const int h = g.by_head.quotient(c);
  return h * x.head_stride + (int64_t)(c - h * g.head_chunks) * 16;
}

// ---- accepted nodes ------------------------------------------------------------------
struct AppendParams {
  ssd_append a;
  Geometry g;
  Divisor by_page, by_group;
  int groups, per;         // groups of planes of a row, planes of a group
  int64_t warps;
  int32_t* status;
};

__global__ void __launch_bounds__(kWarps * 32)
    append_kernel(const __grid_constant__ AppendParams p) {
  const ssd_append& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w >= p.warps) return;
  const int t = p.by_group.quotient((int)w), group = (int)w - t * p.groups;
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  const int b = a.owner[t];
  int bad = 0, node = 0;
  if (slot >= (int64_t)a.num_pages * a.page_size) bad |= SSD_DEV_BAD_PAGE;
  if ((unsigned)b >= (unsigned)a.B) {
    bad |= SSD_DEV_BAD_LENGTH;
  } else {
    const int i = t - a.cu[b];
    if (i < 0 || (a.path && i > a.path_cols)) bad |= SSD_DEV_BAD_LENGTH;
    else node = i == 0 || !a.path ? i : a.path[b * a.path_stride + i - 1];
    if ((unsigned)node >= (unsigned)a.N) bad |= SSD_DEV_BAD_LENGTH;
  }
  if (bad) {
    if (group == 0 && lane == 0 && p.status) atomicOr(p.status, bad);
    return;
  }
  const int64_t page = slot / a.page_size, in_page = slot - page * a.page_size;
  const int j0 = group * p.per, j1 = min(j0 + p.per, p.g.planes);
  for (int c0 = lane; c0 < p.g.chunks; c0 += 32 * kFlight) {
    for (int j = j0; j < j1; ++j) {
      const ssd_layers *from, *to;
      const char* x = plane_of(a.k, a.v, p.g, j, &from) + b * from->page_stride +
                      node * from->token_stride;
      char* y = const_cast<char*>(plane_of(a.k_cache, a.v_cache, p.g, j, &to)) +
                page * to->page_stride + in_page * to->token_stride;
      uint4 z[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (c0 + i * 32 < p.g.chunks)
          z[i] = __ldcs(reinterpret_cast<const uint4*>(x + chunk_at(*from, p.g, c0 + i * 32)));
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (c0 + i * 32 < p.g.chunks)
          *reinterpret_cast<uint4*>(y + chunk_at(*to, p.g, c0 + i * 32)) = z[i];
    }
  }
}

// ---- rows of the tables ----------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kMaxRows = 8192;
constexpr int kMaxCount = 1 << 30;
constexpr int kNoHeir = INT_MAX;    // an old row that ends
constexpr int kTableCols = 256;     // columns of a table row that a warp writes
constexpr int kGroupBytes = 8192;   // of a last page that a warp copies, about

struct ForkParams {
  ssd_fork f;
  Geometry g;
  Divisor by_page;
  int clusters;            // CTAs of the plan's cluster
  int group, groups;       // tokens of a warp's copy, such groups of a page
  int* last;               // [num_pages] the last place that gives the page back
  int* back;               // [S] pages that an old row gives back for good
  int* freed;              // [num_pages] those pages, in order
  int4* rows;              // [B] what becomes of the new rows
  int4* copies;            // [B] old page, new page, tokens
  int* ncopies;
  int32_t* status;
};

// Exclusive sums over n numbers, consecutive ones per thread, by the whole CTA:
// s_sum[i] for i <= n.
template <typename F>
__device__ __forceinline__ void running_sums(int* s_sum, int n, int* s_warp, F value) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += value(i);
  int x = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int run = x - sum;
  for (int w = 0; w < warp; ++w) run += s_warp[w];
  for (int i = i0; i < i1; ++i) {
    s_sum[i] = run;
    run += value(i);
  }
  if (i1 == n && (i0 < n || tid == 0)) s_sum[n] = run;  // n > 0: its last thread
  __syncthreads();
}

// One cluster: heirs, pages given back, pages taken.  Every CTA finds the heirs
// and the sums again in its own shared memory; what goes through memory (the
// counts of shares, the pages given back) is ordered by the cluster's barriers
// and read from L2.
__global__ void __launch_bounds__(kPlanThreads, 1)
    fork_plan_kernel(const __grid_constant__ ForkParams p) {
  extern __shared__ int s_mem[];
  const ssd_fork& f = p.f;
  int* s_heir = s_mem;               // [S] lowest new row of an old one, -1: inconsistent
  int* s_back = s_heir + f.S;        // [S + 1] pages given back before an old row
  int* s_nth = s_back + f.S + 1;     // [B + 1] pages taken before a new row
  __shared__ int s_warp[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = (int)cluster_rank();
  const int threads = p.clusters * kPlanThreads, gtid = rank * kPlanThreads + tid;
  const int warps = threads / 32, warp = gtid / 32;
  int bad = 0;
  start_next();

  // ---- heirs; shares so far ----------------------------------------------------------
  for (int s = tid; s < f.S; s += kPlanThreads) {
    const int len = f.lens[s], held = f.held[s];
    const bool ok = len >= 0 && held >= 0 && held <= f.cols && len <= (int64_t)held * f.page_size;
    s_heir[s] = ok ? kNoHeir : -1;
    if (!ok) bad |= SSD_DEV_BAD_LENGTH;
  }
  __syncthreads();
  for (int b = tid; b < f.B; b += kPlanThreads) {
    const int s = f.src[b];
    if (s < -1 || s >= f.S) bad |= SSD_DEV_BAD_LENGTH;
    else if (s >= 0 && s_heir[s] >= 0) atomicMin(&s_heir[s], b);
  }
  for (int i = gtid; i < f.num_pages; i += threads) f.shares_out[i] = max(f.shares[i], 0);
  __syncthreads();
  // Old rows by warps; visit(row, place, page, count so far) of those that end by the lanes
  // of its warp, 32 columns at a time (no page: -1), which gives a new count; then
  // after(row, count).
  auto ending = [&](auto visit, auto after) {
    for (int s = warp; s < f.S; s += warps) {
      const int held = s_heir[s] == kNoHeir ? f.held[s] : 0;
      int count = 0;
      for (int c0 = 0; c0 < held; c0 += 32) {
        const int c = c0 + lane;
        int page = c < held ? f.tables[s * f.table_stride + c] : -1;
        if (c < held && (unsigned)page >= (unsigned)f.num_pages) {
          bad |= SSD_DEV_BAD_PAGE;
          page = -1;
        }
        count = visit(s, s * f.cols + c, page, count);
      }
      after(s, count);
    }
  };
  auto nothing = [](int, int) {};
  ending([&](int, int, int page, int) {
    if (page >= 0) p.last[page] = -1;
    return 0;
  }, nothing);
  cluster_barrier();
  ending([&](int, int place, int page, int) {
    if (page >= 0) {
      atomicSub(f.shares_out + page, 1);
      atomicMax(p.last + page, place);
    }
    return 0;
  }, nothing);
  cluster_barrier();
  // ---- pages whose last holder ends ----------------------------------------------------
  auto is_freed = [&](int place, int page) {
    return page >= 0 && __ldcg(f.shares_out + page) < 0 && __ldcg(p.last + page) == place;
  };
  ending([&](int, int place, int page, int count) {
    return count + __popc(__ballot_sync(0xffffffffu, is_freed(place, page)));
  }, [&](int s, int count) {
    if (lane == 0) p.back[s] = count;
  });
  cluster_barrier();
  const int n0 = *f.free_count, n = min(max(n0, 0), f.free_cap);
  running_sums(s_back, f.S, s_warp, [&](int s) { return __ldcg(p.back + s); });
  auto takes = [&](int b) {          // a page for the last tokens
    const int s = f.src[b];
    if (s < 0 || s >= f.S || s_heir[s] < 0 || s_heir[s] == b) return 0;
    const int len = f.lens[s];
    return (int)(p.by_page.quotient(len) * f.page_size < len);
  };
  running_sums(s_nth, f.B, s_warp, takes);
  const int64_t top = (int64_t)n + s_back[f.S];
  ending([&](int s, int place, int page, int count) {
    const bool freed = is_freed(place, page);
    const unsigned all = __ballot_sync(0xffffffffu, freed);
    if (freed) {
      const int k = s_back[s] + count + __popc(all & ((1u << lane) - 1));
      p.freed[k] = page;
      if (n + (int64_t)k < f.free_cap) f.free_pages[n + k] = page;
      if (__ldcg(f.shares_out + page) < -1) bad |= SSD_DEV_BAD_PAGE;
      f.shares_out[page] = 0;
    }
    return count + __popc(all);
  }, nothing);
  cluster_barrier();
  // ---- the new rows ----------------------------------------------------------------------
  const int asked = s_nth[f.B];
  for (int b = gtid; b < f.B; b += threads) {
    const int s = f.src[b];
    int4 row = make_int4(-1, 0, 0, -1);  // 2 * old row + heir; pages; those from its table; a page
    int len = 0, ok = s == -1;
    if (s >= 0 && s < f.S && s_heir[s] >= 0) {
      const int full = p.by_page.quotient(f.lens[s]);
      const bool heir = s_heir[s] == b, take = takes(b) != 0;
      if (!take || s_nth[b] < top) {
        ok = 1;
        len = f.lens[s];
        row.x = 2 * s + heir;
        row.z = heir ? f.held[s] : full;
        row.y = row.z + take;
        if (take) {
          const int64_t i = top - 1 - s_nth[b];
          row.w = i < n ? f.free_pages[i] : __ldcg(p.freed + (i - n));
          p.copies[s_nth[b]] = make_int4(f.tables[s * f.table_stride + full], row.w,
                                         len - full * f.page_size, 0);
        }
      } else {
        bad |= SSD_DEV_NO_PAGES;
      }
    }
    p.rows[b] = row;
    f.lens_out[b] = len;
    f.held_out[b] = row.y;
    f.served[b] = ok;
  }
  if (gtid == 0) {
    const int64_t taken = min((int64_t)asked, top);
    *p.ncopies = (int)taken;
    *f.free_out = (int)min(top - taken, (int64_t)f.free_cap);
    if (n != n0 || top - taken > f.free_cap) bad |= SSD_DEV_BAD_LENGTH;
  }
  if (bad && p.status) atomicOr(p.status, bad);
}

// The tables, the shares that forks add, and the tokens of last pages.
__global__ void __launch_bounds__(kWarps * 32)
    fork_copy_kernel(const __grid_constant__ ForkParams p) {
  const ssd_fork& f = p.f;
  const int lane = threadIdx.x & 31;
  const int64_t first = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * kWarps;
  wait_previous();
  int bad = 0;
  const int64_t copies = (int64_t)*p.ncopies * p.g.planes * p.groups;
  for (int64_t w = first; w < copies; w += step) {
    const int64_t q = w / p.groups;
    const int k = (int)(q / p.g.planes), j = (int)(q - (int64_t)k * p.g.planes);
    const int4 c = p.copies[k];
    const int t0 = (int)(w - q * p.groups) * p.group, n = min(p.group, c.z - t0);
    if (n <= 0) continue;
    if ((unsigned)c.x >= (unsigned)f.num_pages || (unsigned)c.y >= (unsigned)f.num_pages) {
      bad |= SSD_DEV_BAD_PAGE;
      continue;
    }
    const ssd_layers* at;
    char* x = const_cast<char*>(plane_of(f.k_cache, f.v_cache, p.g, j, &at)) +
              t0 * at->token_stride;
    const char* from = x + c.x * at->page_stride;
    char* to = x + c.y * at->page_stride;
    const int total = n * p.g.chunks;
    for (int i0 = lane; i0 < total; i0 += 32 * kFlight) {
      uint4 z[kFlight];
      int64_t where[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (i0 + i * 32 < total) {
          const int e = i0 + i * 32, t = p.g.by_token.quotient(e);
          where[i] = t * at->token_stride + chunk_at(*at, p.g, e - t * p.g.chunks);
          z[i] = *reinterpret_cast<const uint4*>(from + where[i]);
        }
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (i0 + i * 32 < total) *reinterpret_cast<uint4*>(to + where[i]) = z[i];
    }
  }
  const int pieces = (f.cols + kTableCols - 1) / kTableCols;
  for (int64_t w = first; w < (int64_t)f.B * pieces; w += step) {
    const int b = (int)(w / pieces), c0 = (int)(w - (int64_t)b * pieces) * kTableCols;
    const int4 row = p.rows[b];
    const int32_t* table = f.tables + (int64_t)(row.x >> 1) * f.table_stride;
    const int c1 = min(f.cols, c0 + kTableCols);
    for (int c = c0 + lane; c < c1; c += 32) {
      int page = -1;
      if (c < row.z) {
        page = table[c];
        if (!(row.x & 1)) {
          if ((unsigned)page < (unsigned)f.num_pages) atomicAdd(f.shares_out + page, 1);
          else bad |= SSD_DEV_BAD_PAGE;
        }
      } else if (c < row.y) {
        page = row.w;
      }
      f.tables_out[(int64_t)b * f.cols + c] = page;
    }
  }
  if (bad && p.status) atomicOr(p.status, bad);
}

// ---- set-up ------------------------------------------------------------------------------
bool layers_ok(const ssd_layers& x) {
  if (!x.ptr || (uintptr_t)x.ptr % 16 != 0) return false;
  for (int64_t s : {x.layer_stride, x.page_stride, x.token_stride, x.head_stride})
    if (s < 0 || s % 16 != 0) return false;
  return true;
}
// Heads side by side in all of them are one row.
Geometry geometry(int L, int H, int row_bytes, bool pair,
                  std::initializer_list<const ssd_layers*> all) {
  Geometry g{};
  g.pair = pair;
  g.planes = pair ? 2 * L : L;
  g.chunks = H * (row_bytes / 16);
  g.head_chunks = g.chunks;
  if (H > 1)
    for (const ssd_layers* x : all)
      if (x->ptr && x->head_stride != row_bytes) g.head_chunks = row_bytes / 16;
  g.by_token = divisor(g.chunks);
  g.by_head = divisor(g.head_chunks);
  return g;
}
bool rows_fit(int64_t H, int64_t row_bytes, int64_t L) {
  return H * row_bytes <= 1 << 24 && L <= 1 << 20;
}

ssd_status check(const ssd_fork* f) {
  if (!f || f->pad_ != 0 || f->S < 1 || f->B < 1 || f->cols < 1 || f->page_size < 1 ||
      f->num_pages < 1 || f->free_cap < 0 || f->L < 0)
    return SSD_ERR_INVALID_ARG;
  if (f->L > 0 && (f->H < 1 || f->row_bytes < 16 || f->row_bytes % 16 != 0))
    return SSD_ERR_INVALID_ARG;
  if (f->S > kMaxRows || f->B > kMaxRows || (int64_t)f->S * f->cols > kMaxCount ||
      (int64_t)f->B * f->cols > kMaxCount || f->num_pages > kMaxCount ||
      (f->L > 0 && !rows_fit(f->H, f->row_bytes, f->L)))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}
struct ForkLayout {
  size_t last, back, freed, rows, copies, ncopies, total;
};
ForkLayout layout(const ssd_fork& f) {
  ForkLayout L;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  L.last = take((size_t)f.num_pages * 4);
  L.back = take((size_t)f.S * 4);
  L.freed = take((size_t)f.num_pages * 4);
  L.rows = take((size_t)f.B * 16);
  L.copies = take((size_t)f.B * 16);
  L.ncopies = take(4);
  L.total = at;
  return L;
}

ssd_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return SSD_ERR_CUDA;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_append_path(const ssd_append* a, int32_t* dev_status, void* stream) {
  if (!a || a->pad_ != 0 || a->L < 1 || a->B < 1 || a->N < 1 || a->H < 1 || a->rows < 0 ||
      a->row_bytes < 16 || a->row_bytes % 16 != 0 || a->num_pages < 1 || a->page_size < 1 ||
      a->path_cols < 0)
    return SSD_ERR_INVALID_ARG;
  if ((a->rows > 0 && (!a->slots || !a->owner)) || !a->cu) return SSD_ERR_INVALID_ARG;
  if (a->path && a->path_stride < a->path_cols) return SSD_ERR_INVALID_ARG;
  const bool pair = a->v_cache.ptr != nullptr;
  if (!layers_ok(a->k) || !layers_ok(a->k_cache) || (a->v.ptr != nullptr) != pair ||
      (pair && (!layers_ok(a->v) || !layers_ok(a->v_cache))))
    return SSD_ERR_INVALID_ARG;
  for (const void* in : {a->k.ptr, a->v.ptr, a->v_cache.ptr})
    if (in == a->k_cache.ptr) return SSD_ERR_INVALID_ARG;
  if (pair && (a->k.ptr == a->v_cache.ptr || a->v.ptr == a->v_cache.ptr))
    return SSD_ERR_INVALID_ARG;
  if (!rows_fit(a->H, a->row_bytes, a->L)) return SSD_ERR_UNSUPPORTED;
  AppendParams p{};
  p.a = *a;
  p.g = geometry(a->L, a->H, a->row_bytes, pair, {&a->k, &a->v, &a->k_cache, &a->v_cache});
  p.per = 1;
  p.groups = p.g.planes;
  p.by_group = divisor(p.groups);
  p.warps = (int64_t)a->rows * p.groups;
  p.status = dev_status;
  if (p.warps > 0x7fffffff - 64) return SSD_ERR_UNSUPPORTED;
  if (p.warps == 0) return SSD_OK;
  append_kernel<<<(unsigned)((p.warps + kWarps - 1) / kWarps), kWarps * 32, 0,
                  static_cast<cudaStream_t>(stream)>>>(p);
  return status_of(cudaGetLastError());
}

size_t ssd_fork_rows_workspace_size(const ssd_fork* f) {
  return check(f) == SSD_OK ? layout(*f).total : 0;
}

ssd_status ssd_fork_rows(const ssd_fork* f, void* workspace, size_t workspace_bytes,
                         int32_t* dev_status, void* stream) {
  const ssd_status st = check(f);
  if (st != SSD_OK) return st;
  if (!f->src || !f->lens || !f->held || !f->tables || !f->shares || !f->free_count ||
      (f->free_cap > 0 && !f->free_pages) || f->table_stride < f->cols || !f->tables_out ||
      !f->lens_out || !f->held_out || !f->served || !f->shares_out || !f->free_out)
    return SSD_ERR_INVALID_ARG;
  const bool pair = f->v_cache.ptr != nullptr;
  if (f->L > 0 && (!layers_ok(f->k_cache) || (pair && !layers_ok(f->v_cache)) ||
                   f->k_cache.ptr == f->v_cache.ptr))
    return SSD_ERR_INVALID_ARG;
  // inputs are read again while outputs are written
  for (const int32_t* out : {f->tables_out, f->lens_out, f->held_out, f->served, f->shares_out,
                             f->free_out})
    for (const int32_t* in : {f->src, f->lens, f->held, f->tables, f->shares,
                              (const int32_t*)f->free_pages, f->free_count})
      if (out == in) return SSD_ERR_INVALID_ARG;
  const ForkLayout L = layout(*f);
  if (!workspace || (uintptr_t)workspace % 256 != 0 || workspace_bytes < L.total)
    return SSD_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  ForkParams p{};
  p.f = *f;
  p.by_page = divisor(f->page_size);
  p.last = reinterpret_cast<int*>(ws + L.last);
  p.back = reinterpret_cast<int*>(ws + L.back);
  p.freed = reinterpret_cast<int*>(ws + L.freed);
  p.rows = reinterpret_cast<int4*>(ws + L.rows);
  p.copies = reinterpret_cast<int4*>(ws + L.copies);
  p.ncopies = reinterpret_cast<int*>(ws + L.ncopies);
  p.status = dev_status;
  p.group = p.groups = 1;
  if (f->L > 0) {
    p.g = geometry(f->L, f->H, f->row_bytes, pair, {&f->k_cache, &f->v_cache});
    p.group = std::min(f->page_size, std::max(1, kGroupBytes / (f->H * f->row_bytes)));
    p.groups = (f->page_size + p.group - 1) / p.group;
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // 8 CTAs share the tables' rows and the counts of shares when there are many
  p.clusters = (int64_t)f->S * f->cols + f->num_pages > 8192 ? 8 : 1;
  const int smem = (2 * f->S + f->B + 2) * (int)sizeof(int);
  cudaError_t e = cudaSuccess;
  if (smem > 46 * 1024)  // the most that any call needs: the limit is the function's
    e = cudaFuncSetAttribute(fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (3 * kMaxRows + 2) * (int)sizeof(int));
  if (e != cudaSuccess) return status_of(e);
  cudaLaunchAttribute attr{};
  cudaLaunchConfig_t c{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)p.clusters;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  c.gridDim = dim3((unsigned)p.clusters);
  c.blockDim = dim3(kPlanThreads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, fork_plan_kernel, p);
  if (e != cudaSuccess) return status_of(e);
  const int64_t work =
      (int64_t)f->B * ((f->cols + kTableCols - 1) / kTableCols + (int64_t)p.g.planes * p.groups);
  const int grid = (int)std::min<int64_t>((work + kWarps - 1) / kWarps,
                                          (int64_t)std::max(num_sms(), 1) * 8);
  attr = cudaLaunchAttribute{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3(kWarps * 32);
  c.dynamicSmemBytes = 0;
  return status_of(cudaLaunchKernelEx(&c, fork_copy_kernel, p));
}

}  // extern "C"
