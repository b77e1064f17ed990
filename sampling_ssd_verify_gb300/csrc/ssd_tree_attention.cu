// ssd_tree_attention.cu -- attention of drafted nodes over a paged cache and over
// the nodes on their paths (ssd_tree_attention).
//
// out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m) with m the running maximum: one
// warp per (sequence, node, query head), one token at a time.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ssd_attention_dev.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxNodes = 256;

struct TreeAttnParams {
  ssd_tree_attn a;
  Divisor by_page;
  float scale_log2;
  int gqa;
  int64_t rows;
  int32_t* status;
  int16_t parent[kMaxNodes];
};

__device__ __forceinline__ float2 unpack2(uint32_t x, __nv_bfloat16) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
}
__device__ __forceinline__ float2 unpack2(uint32_t x, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
    tree_kernel(const __grid_constant__ TreeAttnParams p) {
  constexpr int E = D / 64;          // pairs of elements of a lane
  const ssd_tree_attn& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  const int head = (int)(row % a.Hq), u = (int)(row / a.Hq % a.N), b = (int)(row / a.Hq / a.N);
  const int h = head / p.gqa;
  const int64_t most = (int64_t)a.cols * a.page_size;
  const int given = a.lens[b], len = given < 0 ? 0 : given > most ? (int)most : given;
  if (len != given && lane == 0 && p.status) atomicOr(p.status, SSD_DEV_BAD_LENGTH);
  float2 q[E], o[E];
  const T* from = static_cast<const T*>(a.q) + b * a.q_seq_stride + u * a.q_node_stride +
                  head * a.q_head_stride + lane * 2;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = unpack2(*reinterpret_cast<const uint32_t*>(from + e * 64), T());
    o[e] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  auto token = [&](const T* k, const T* v) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 x = k ? unpack2(*reinterpret_cast<const uint32_t*>(k + lane * 2 + e * 64), T())
                         : make_float2(0.f, 0.f);
      s = fmaf(q[e].x, x.x, fmaf(q[e].y, x.y, s));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale_log2;
    const float m1 = fmaxf(m, s), off = m1 == -INFINITY ? 0.f : m1;
    const float keep = exp2f(m - off), w = exp2f(s - off);
    m = m1;
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 x = v ? unpack2(*reinterpret_cast<const uint32_t*>(v + lane * 2 + e * 64), T())
                         : make_float2(0.f, 0.f);
      o[e].x = fmaf(w, x.x, o[e].x * keep);
      o[e].y = fmaf(w, x.y, o[e].y * keep);
    }
  };
  for (int t = 0; t < len; ++t) {
    const int col = p.by_page.quotient(t), in_page = t - col * a.page_size;
    const int page = a.tables[b * a.table_stride + col];
    if ((unsigned)page >= (unsigned)a.num_pages) {
      if (lane == 0 && p.status) atomicOr(p.status, SSD_DEV_BAD_PAGE);
      token(nullptr, nullptr);
      continue;
    }
    token(static_cast<const T*>(a.k_cache.ptr) + page * a.k_cache.page_stride +
              in_page * a.k_cache.token_stride + h * a.k_cache.head_stride,
          static_cast<const T*>(a.v_cache.ptr) + page * a.v_cache.page_stride +
              in_page * a.v_cache.token_stride + h * a.v_cache.head_stride);
  }
  for (int n = u; n >= 0; n = p.parent[n])
    token(static_cast<const T*>(a.k.ptr) + b * a.k.page_stride + n * a.k.token_stride +
              h * a.k.head_stride,
          static_cast<const T*>(a.v.ptr) + b * a.v.page_stride + n * a.v.token_stride +
              h * a.v.head_stride);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* to = static_cast<T*>(a.out) + b * a.out_seq_stride + u * a.out_node_stride +
          head * a.out_head_stride + lane * 2;
#pragma unroll
  for (int e = 0; e < E; ++e)
    *reinterpret_cast<uint32_t*>(to + e * 64) = pack2<T>(o[e].x * inv, o[e].y * inv);
  if (lane == 0 && a.lse) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
}

// ---- set-up ---------------------------------------------------------------------------
bool view_ok(const void* ptr, std::initializer_list<int64_t> strides) {
  if (!ptr || (uintptr_t)ptr % 16 != 0) return false;
  for (int64_t s : strides)
    if (s < 0 || s % 8 != 0) return false;
  return true;
}
bool view_ok(const ssd_paged& x) {
  return view_ok(x.ptr, {x.page_stride, x.token_stride, x.head_stride});
}

// Tokens and (node, head) pairs are counted in 32 bits.
constexpr int64_t kMaxCount = 0x7fffffff - (1 << 20);

ssd_status check(const ssd_tree_attn* a) {
  if (!a || (a->dtype != SSD_BF16 && a->dtype != SSD_F16)) return SSD_ERR_INVALID_ARG;
  if (a->B < 1 || a->N < 1 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv != 0 ||
      a->num_pages < 1 || a->page_size < 1 || a->cols < 0 || !std::isfinite(a->scale))
    return SSD_ERR_INVALID_ARG;
  // tables of no columns may have no address
  if ((!a->tables && a->cols > 0) || !a->lens || a->table_stride < a->cols)
    return SSD_ERR_INVALID_ARG;
  if ((a->D != 64 && a->D != 128 && a->D != 256) || a->N > kMaxNodes) return SSD_ERR_UNSUPPORTED;
  if (a->parent)
    for (int u = 0; u < a->N; ++u)
      if (a->parent[u] >= u || a->parent[u] < (u > 0 ? 0 : -1)) return SSD_ERR_INVALID_ARG;
  if ((int64_t)a->cols * a->page_size > kMaxCount || (int64_t)a->B * a->N * a->Hq > kMaxCount)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

template <typename T>
cudaError_t launch(const TreeAttnParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.rows + kWarps - 1) / kWarps);
  switch (p.a.D) {
    case 64: tree_kernel<T, 64><<<grid, kWarps * 32, 0, s>>>(p); break;
    case 128: tree_kernel<T, 128><<<grid, kWarps * 32, 0, s>>>(p); break;
    default: tree_kernel<T, 256><<<grid, kWarps * 32, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_tree_attention_workspace_size(const ssd_tree_attn* a) {
  return check(a) == SSD_OK ? 256 : 0;
}

ssd_status ssd_tree_attention(const ssd_tree_attn* a, void* workspace, size_t workspace_bytes,
                              int32_t* dev_status, void* stream) {
  const ssd_status st = check(a);
  if (st != SSD_OK) return st;
  if (!view_ok(a->q, {a->q_seq_stride, a->q_node_stride, a->q_head_stride}) ||
      !view_ok(a->out, {a->out_seq_stride, a->out_node_stride, a->out_head_stride}) ||
      !view_ok(a->k) || !view_ok(a->v) || !view_ok(a->k_cache) || !view_ok(a->v_cache))
    return SSD_ERR_INVALID_ARG;
  if (a->out == a->q &&
      (a->out_seq_stride != a->q_seq_stride || a->out_node_stride != a->q_node_stride ||
       a->out_head_stride != a->q_head_stride))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || (uintptr_t)workspace % 256 != 0 || workspace_bytes < 256)
    return SSD_ERR_WORKSPACE;
  TreeAttnParams p{};
  p.a = *a;
  p.gqa = a->Hq / a->Hkv;
  p.by_page = divisor(a->page_size);
  p.scale_log2 = (float)((double)a->scale * 1.4426950408889634);
  p.rows = (int64_t)a->B * a->N * a->Hq;
  p.status = dev_status;
  for (int u = 0; u < a->N; ++u) p.parent[u] = (int16_t)(a->parent ? a->parent[u] : u - 1);
  const cudaError_t e = a->dtype == SSD_BF16
                            ? launch<__nv_bfloat16>(p, static_cast<cudaStream_t>(stream))
                            : launch<__half>(p, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return SSD_ERR_CUDA;
}

}  // extern "C"
