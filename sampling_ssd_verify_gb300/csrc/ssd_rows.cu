// ssd_rows.cu -- rows of a paged key/value cache: the keys and values of
// accepted nodes into their slots (ssd_append_path), and rows of the block
// tables continued, forked and freed (ssd_fork_rows).
//
// Both move whole tokens of all layers: a token of a layer is H rows of
// row_bytes, a few KB that mostly lie side by side, and copying is all there is
// to it.  A warp takes a token (append) or a few tokens (fork) of one layer's
// keys or values, with its loads in flight together before the first store.
//
// Measured in a graph, over inputs that together pass L2 (in brackets at a copy's rate):
// accepted nodes of 64 trees of 11 into 32 layers 9.0 us (5.6), of twice as many 15.5 (11.2),
// of one tree 2.4: 6.4 for the bytes beside 2.6 for the launch and the loads of places.  8
// samples of one prompt over 32 layers 12.2 (4.1), 64 beams over 8 layers 16.7 (1.7), 512
// rows over 4 layers 25 (4.4): most of it the plan's chain of loads and barriers.  From L2
// they take 5.5, 10.3, 13.4 and 20.6.

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

// Keys or values of plane j, and their first byte.
__device__ __forceinline__ const ssd_layers& side_of(const ssd_layers& k, const ssd_layers& v,
                                                     const Geometry& g, int j) {
  return g.pair && (j & 1) ? v : k;
}
__device__ __forceinline__ char* plane_of(const ssd_layers& x, const Geometry& g, int j) {
  return static_cast<char*>(x.ptr) + (int64_t)(g.pair ? j >> 1 : j) * x.layer_stride;
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
  Divisor by_group;
  int groups;              // of planes of a row: a warp each
  int64_t warps;
  int32_t* status;
};

template <int PLANES, int FLIGHT>    // of a warp; 16-byte loads of a lane and plane in flight
__global__ void __launch_bounds__(kWarps * 32)
    append_kernel(const __grid_constant__ AppendParams p) {
  const ssd_append& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  wait_previous();
  if (w >= p.warps) return;
  const int t = p.by_group.quotient((int)w), group = (int)w - t * p.groups;
  const int64_t slot = a.slots[t];
  const int b = a.owner[t];
  if (slot < 0) return;
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
  const int page = (int)(slot / a.page_size), in_page = (int)(slot - (int64_t)page * a.page_size);
  const char* from[PLANES];
  char* to[PLANES];
  int side[PLANES];                  // the plane that keys or values are told by
#pragma unroll
  for (int x = 0; x < PLANES; ++x) {
    const int j = min(group * PLANES + x, p.g.planes - 1);
    const ssd_layers& k = side_of(a.k, a.v, p.g, j);
    const ssd_layers& c = side_of(a.k_cache, a.v_cache, p.g, j);
    side[x] = j;
    from[x] = plane_of(k, p.g, j) + b * k.page_stride + node * k.token_stride;
    to[x] = plane_of(c, p.g, j) + page * c.page_stride + in_page * c.token_stride;
  }
  for (int c0 = lane; c0 < p.g.chunks; c0 += 32 * FLIGHT) {
    uint4 z[PLANES][FLIGHT];
#pragma unroll
    for (int x = 0; x < PLANES; ++x)
#pragma unroll
      for (int i = 0; i < FLIGHT; ++i)
        if (c0 + i * 32 < p.g.chunks)
          z[x][i] = __ldcs(reinterpret_cast<const uint4*>(
              from[x] + chunk_at(side_of(a.k, a.v, p.g, side[x]), p.g, c0 + i * 32)));
#pragma unroll
    for (int x = 0; x < PLANES; ++x)
      if (x == 0 || group * PLANES + x < p.g.planes)
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i)
          if (c0 + i * 32 < p.g.chunks)
            *reinterpret_cast<uint4*>(
                to[x] + chunk_at(side_of(a.k_cache, a.v_cache, p.g, side[x]), p.g, c0 + i * 32)) =
                z[x][i];
  }
}

template <int PLANES, int FLIGHT>
cudaError_t launch_append(AppendParams& p, cudaStream_t s) {
  p.groups = (p.g.planes + PLANES - 1) / PLANES;
  p.by_group = divisor(p.groups);
  p.warps = (int64_t)p.a.rows * p.groups;
  // begins while the kernel before it ends, and waits for it
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)((p.warps + kWarps - 1) / kWarps));
  c.blockDim = dim3(kWarps * 32);
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, append_kernel<PLANES, FLIGHT>, p);
}

// ---- rows of the tables ----------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCtas = 8;        // of its cluster, at most
constexpr int kMaxRows = 8192;
constexpr int kMaxCount = 1 << 30;
constexpr int kNoHeir = INT_MAX;    // an old row that ends
constexpr int kBatch = 4;           // pieces of ending rows that a warp has in flight
constexpr int kTableCols = 256;     // columns of a table row that a warp writes
constexpr int kGroupBytes = 8192;   // of a last page that a warp copies, about
__host__ __device__ constexpr int plan_ints(int S, int B) { return 4 * S + 3 * B + 2; }

struct ForkParams {
  ssd_fork f;
  Geometry g;
  Divisor by_page;
  int ctas;                // of the plan's cluster
  int group, groups;       // tokens of a warp's copy, such groups of a page
  int* last;               // [num_pages] the last place that gives the page back
  int4* rows;              // [B] what becomes of the new rows
  int4* copies;            // [B] old page, new page, tokens
  int* ncopies;
  int32_t* status;
};

// Exclusive sums over n numbers, consecutive ones per thread, by the whole CTA:
// s_sum[i] for i <= n.  Ends with a barrier.
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
  int run = x - sum + __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0);
  for (int i = i0; i < i1; ++i) {
    const int v = value(i);
    s_sum[i] = run;
    run += v;
  }
  if (i1 == n && i0 < n) s_sum[n] = run;  // the thread of the last
  __syncthreads();
}

// One cluster, or one CTA.  Every CTA finds the heirs, the pages taken and the
// places of the pages given back again in its own shared memory; only the counts
// of shares and the last places go through memory.  The tables' rows that end, in
// order, are cut into pieces of 32 columns and these divided among the warps, so
// that the pages given back for good have their order by warps and lanes.  It is a
// chain of loads and barriers, not of bytes: what can be is loaded side by side, and
// a page goes from the row that gives it back to the row that takes it without a
// look at the stack.
__global__ void __launch_bounds__(kPlanThreads, 1)
    fork_plan_kernel(const __grid_constant__ ForkParams p) {
  extern __shared__ int s_mem[];
  const ssd_fork& f = p.f;
  int* s_heir = s_mem;               // [S] lowest new row of an old one, -1: inconsistent
  int* s_len = s_heir + f.S;         // [S] an old row's tokens
  int* s_held = s_len + f.S;         // [S] its pages
  int* s_piece = s_held + f.S;       // [S + 1] pieces of ending rows before it
  int* s_src = s_piece + f.S + 1;    // [B]
  int* s_nth = s_src + f.B;          // [B + 1] pages taken before a new row
  int* s_taker = s_nth + f.B + 1;    // [B] the new row that takes the i-th page
  __shared__ int s_warp[kPlanWarps], s_count[kPlanWarps], s_total[kPlanCtas];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = p.ctas > 1 ? (int)cluster_rank() : 0;
  const int threads = p.ctas * kPlanThreads, gtid = rank * kPlanThreads + tid;
  const int warps = threads / 32, warp = gtid / 32;
  int bad = 0;
  start_next();
  wait_previous();
  auto barrier = [&] {
    if (p.ctas > 1) cluster_barrier();
    else __syncthreads();
  };

  // ---- heirs; shares so far ----------------------------------------------------------
  constexpr int kEarly = 4;
  int early[kEarly];                 // shares, on their way while the rows are looked at
#pragma unroll
  for (int j = 0; j < kEarly; ++j) {
    const int i = gtid + j * threads;
    early[j] = i < f.num_pages ? f.shares[i] : 0;
  }
  const int n0 = *f.free_count, n = min(max(n0, 0), f.free_cap);
  for (int s = tid; s < f.S; s += kPlanThreads) {
    const int len = f.lens[s], held = f.held[s];
    const bool ok = len >= 0 && held >= 0 && held <= f.cols && len <= (int64_t)held * f.page_size;
    s_heir[s] = ok ? kNoHeir : -1;
    s_len[s] = len;
    s_held[s] = held;
    if (!ok) bad |= SSD_DEV_BAD_LENGTH;
  }
  for (int b = tid; b < f.B; b += kPlanThreads) {
    int s = f.src[b];
    if (s < -1 || s >= f.S) {
      bad |= SSD_DEV_BAD_LENGTH;
      s = -2;
    }
    s_src[b] = s;
  }
  __syncthreads();
  for (int b = tid; b < f.B; b += kPlanThreads) {
    const int s = s_src[b];
    if (s >= 0 && s_heir[s] >= 0) atomicMin(&s_heir[s], b);
  }
  for (int j = 0; j < kEarly; ++j) {
    const int i = gtid + j * threads;
    if (i < f.num_pages) f.shares_out[i] = max(early[j], 0);
  }
#pragma unroll 4
  for (int i = gtid + kEarly * threads; i < f.num_pages; i += threads)
    f.shares_out[i] = max(f.shares[i], 0);
  __syncthreads();
  running_sums(s_piece, f.S, s_warp,
               [&](int s) { return s_heir[s] == kNoHeir ? (s_held[s] + 31) >> 5 : 0; });
  auto takes = [&](int b) {          // a page for the last tokens
    const int s = s_src[b];
    if (s < 0 || s_heir[s] < 0 || s_heir[s] == b) return 0;
    return (int)(p.by_page.quotient(s_len[s]) * f.page_size < s_len[s]);
  };
  running_sums(s_nth, f.B, s_warp, takes);
  const int asked = s_nth[f.B];
  for (int b = tid; b < f.B; b += kPlanThreads)
    if (s_nth[b] < s_nth[b + 1]) s_taker[s_nth[b]] = b;  // read after the next barriers
  // the page with the last tokens of the row that this thread's first new one forks
  auto last_page = [&](int b) {
    const int s = s_src[b];
    return f.tables[(int64_t)s * f.table_stride + p.by_page.quotient(s_len[s])];
  };
  const int early_page = gtid < f.B && s_nth[gtid] < s_nth[gtid + 1] ? last_page(gtid) : 0;

  // ---- pages given back --------------------------------------------------------------------
  const int pieces = s_piece[f.S];
  const int per = (pieces + warps - 1) / warps;
  const int q0 = min(pieces, warp * per), q1 = min(pieces, q0 + per);
  const bool once = per <= kBatch;   // a warp's pages stay in its registers
  int page[kBatch], place[kBatch];   // -1: none
  int left[kBatch];                  // holders beside the first, if it goes; 0
  auto load = [&](int q) {           // pieces q .. q + kBatch - 1
    int s = 0;
    if (q < q1) {                    // the row of the first: s_piece[s] <= q < s_piece[s + 1]
      int hi = f.S;
      while (hi - s > 1) {
        const int mid = (s + hi) >> 1;
        if (s_piece[mid] <= q) s = mid;
        else hi = mid;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      place[i] = page[i] = -1;
      if (q + i < q1) {
        while (s_piece[s + 1] <= q + i) ++s;  // ends: q + i < s_piece[S]
        const int c = (q + i - s_piece[s]) * 32 + lane;
        if (c < s_held[s]) {
          place[i] = s * f.cols + c;
          page[i] = f.tables[(int64_t)s * f.table_stride + c];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (place[i] >= 0 && (unsigned)page[i] >= (unsigned)f.num_pages) {
        bad |= SSD_DEV_BAD_PAGE;
        page[i] = -1;
      }
  };
  auto each = [&](bool first, auto visit) {  // visit(i) of the batch
    for (int q = q0; q < q1; q += kBatch) {
      if (first || !once) load(q);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) visit(i);
    }
  };
  // Whether a page goes: its last holder ends, and this is the last place that gives it back.
  auto look = [&](int i) {
    const bool there = page[i] >= 0;
    const int x = there ? __ldcg(f.shares_out + page[i]) : 0;
    const int at = there ? __ldcg(p.last + page[i]) : 0;
    left[i] = x < 0 && at == place[i] ? x : 0;
  };
  each(true, [&](int i) {
    if (page[i] >= 0) p.last[page[i]] = -1;
  });
  barrier();
  each(false, [&](int i) {
    if (page[i] >= 0) {
      atomicSub(f.shares_out + page[i], 1);
      atomicMax(p.last + page[i], place[i]);
    }
  });
  barrier();
  int freed = 0;                     // of this warp
  for (int q = q0; q < q1; q += kBatch) {
    if (!once) load(q);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) look(i);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) freed += __popc(__ballot_sync(0xffffffffu, left[i] < 0));
  }
  if (lane == 0) s_count[tid >> 5] = freed;
  __syncthreads();
  const int before_warp =
      __reduce_add_sync(0xffffffffu, lane < (tid >> 5) ? s_count[lane] : 0);
  if (p.ctas > 1) {
    const int total = __reduce_add_sync(0xffffffffu, s_count[lane]);
    if (tid < p.ctas) st_cluster_u32(cluster_addr(&s_total[rank], tid), (uint32_t)total);
  } else if (tid < 32) {
    const int total = __reduce_add_sync(0xffffffffu, s_count[lane]);
    if (tid == 0) s_total[0] = total;
  }
  barrier();
  int before = before_warp, back = 0;
  for (int r = 0; r < p.ctas; ++r) {
    if (r < rank) before += s_total[r];
    back += s_total[r];
  }
  const int64_t top = (int64_t)n + back;
  each(false, [&](int i) {
    if (!once) look(i);
    const unsigned all = __ballot_sync(0xffffffffu, left[i] < 0);
    if (left[i] < 0) {
      const int nth = before + __popc(all & ((1u << lane) - 1));
      if (n + (int64_t)nth < f.free_cap) f.free_pages[n + nth] = page[i];
      if (left[i] < -1) bad |= SSD_DEV_BAD_PAGE;
      f.shares_out[page[i]] = 0;
      const int taken = back - 1 - nth;  // the stack's top goes first
      if (taken < asked) {
        p.rows[s_taker[taken]].w = page[i];
        p.copies[taken].y = page[i];
      }
    }
    before += __popc(all);
  });
  // ---- the new rows ----------------------------------------------------------------------
  for (int b = gtid; b < f.B; b += threads) {
    const int s = s_src[b];
    int4 row = make_int4(-1, 0, 0, -1);  // 2 * old row + heir; pages; those from its table; a page
    int len = 0, ok = s == -1;
    bool given = false;
    if (s >= 0 && s_heir[s] >= 0) {
      const int full = p.by_page.quotient(s_len[s]), nth = s_nth[b];
      const bool heir = s_heir[s] == b, take = nth < s_nth[b + 1];
      if (!take || nth < top) {
        ok = 1;
        len = s_len[s];
        row.x = 2 * s + heir;
        row.z = heir ? s_held[s] : full;
        row.y = row.z + take;
        if (take) {
          given = nth < back;              // its page is put down where it is given back
          if (!given) row.w = f.free_pages[top - 1 - nth];
          const bool none = !given && (unsigned)row.w >= (unsigned)f.num_pages;
          int* copy = reinterpret_cast<int*>(p.copies + nth);
          copy[0] = b == gtid ? early_page : last_page(b);
          if (!given) copy[1] = row.w;
          copy[2] = none ? 0 : len - full * f.page_size;
          if (none) {                      // off the stack, and no page: the row is left empty
            bad |= SSD_DEV_BAD_PAGE;
            ok = len = 0;
            row = make_int4(-1, 0, 0, -1);
          }
        }
      } else {
        bad |= SSD_DEV_NO_PAGES;
      }
    }
    int* to = reinterpret_cast<int*>(p.rows + b);
    to[0] = row.x;
    to[1] = row.y;
    to[2] = row.z;
    if (!given) to[3] = row.w;
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
    const ssd_layers& at = side_of(f.k_cache, f.v_cache, p.g, j);
    char* x = plane_of(at, p.g, j) + t0 * at.token_stride;
    const char* from = x + c.x * at.page_stride;
    char* to = x + c.y * at.page_stride;
    const int total = n * p.g.chunks;
    for (int i0 = lane; i0 < total; i0 += 32 * kFlight) {
      uint4 z[kFlight];
      int64_t where[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (i0 + i * 32 < total) {
          const int e = i0 + i * 32, t = p.g.by_token.quotient(e);
          where[i] = t * at.token_stride + chunk_at(at, p.g, e - t * p.g.chunks);
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
// Whether no two rows of [L, X, Y, H] lie on one another by a stride alone.
bool rows_apart(const ssd_layers& x, int L, int X, int Y, int H, int row_bytes) {
  auto ok = [&](int n, int64_t stride) { return n == 1 || stride >= row_bytes; };
  return ok(L, x.layer_stride) && ok(X, x.page_stride) && ok(Y, x.token_stride) &&
         ok(H, x.head_stride);
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
  size_t last, rows, copies, ncopies, total;
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
  for (const ssd_layers* c : {&a->k_cache, &a->v_cache})
    if (c->ptr && !rows_apart(*c, a->L, a->num_pages, a->page_size, a->H, a->row_bytes))
      return SSD_ERR_INVALID_ARG;
  AppendParams p{};
  p.a = *a;
  p.g = geometry(a->L, a->H, a->row_bytes, pair, {&a->k, &a->v, &a->k_cache, &a->v_cache});
  p.status = dev_status;
  if ((int64_t)a->rows * p.g.planes > 0x7fffffff - 64) return SSD_ERR_UNSUPPORTED;
  if (a->rows == 0) return SSD_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // With more tokens and planes than the GPU has warps a warp takes two planes, and its
  // loads of places serve both.  From memory: 64 x 4 rows of 2 KB in 32 layers 9.1 us instead of
  // 9.5, 256 x 4 of 1.25 KB in 12 layers 8.1 instead of 8.9 (4 loads in flight of each, which
  // short rows leave idle, 8.3; in 6 layers 6.0 instead of 5.3), 256 x 4 of 128 bytes in 32
  // layers 10.1 instead of 17.7; 32 x 4 rows of 2 KB in 32 layers 6.0 instead of 5.9, 5 of them
  // 2.8 instead of 2.3.
  if ((int64_t)a->rows * p.g.planes <= (int64_t)64 * std::max(num_sms(), 1))
    return status_of(launch_append<1, 4>(p, s));
  return status_of(p.g.chunks >= 128 ? launch_append<2, 4>(p, s) : launch_append<2, 2>(p, s));
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
  // Several CTAs share the tables' rows and the counts of shares when there are many.  From
  // memory: 128 rows of 77 pages 18.2 us with 8 instead of 23.2 with one, 512 of 143 25 instead of
  // 91; 64 of 77 16.7 instead of 16.4, 32 of 77 15.9 instead of 14.2, one of 97 13.1 instead of 12.1.
  p.ctas = (int64_t)f->S * f->cols + f->num_pages > 4096 ? kPlanCtas : 1;
  const int smem = plan_ints(f->S, f->B) * (int)sizeof(int);
  cudaError_t e = cudaSuccess;
  if (smem > 46 * 1024)  // the most that any call needs: the limit is the function's
    e = cudaFuncSetAttribute(fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             plan_ints(kMaxRows, kMaxRows) * (int)sizeof(int));
  if (e != cudaSuccess) return status_of(e);
  // both begin while the kernel before them ends, and wait for it
  cudaLaunchAttribute attr[2] = {};
  cudaLaunchConfig_t c{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  c.gridDim = dim3((unsigned)p.ctas);
  c.blockDim = dim3(kPlanThreads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = s;
  c.attrs = attr;
  c.numAttrs = 2;
  e = cudaLaunchKernelEx(&c, fork_plan_kernel, p);
  if (e != cudaSuccess) return status_of(e);
  const int64_t work =
      (int64_t)f->B * ((f->cols + kTableCols - 1) / kTableCols + (int64_t)p.g.planes * p.groups);
  const int grid = (int)std::min<int64_t>((work + kWarps - 1) / kWarps,
                                          (int64_t)std::max(num_sms(), 1) * 8);
  c.numAttrs = 1;
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3(kWarps * 32);
  c.dynamicSmemBytes = 0;
  return status_of(cudaLaunchKernelEx(&c, fork_copy_kernel, p));
}

}  // extern "C"
