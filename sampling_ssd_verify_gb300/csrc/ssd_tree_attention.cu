// ssd_tree_attention.cu -- attention of drafted nodes over a paged cache and over
// the nodes on their paths (ssd_tree_attention): the entry point, the division of the
// work and the workspace.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <numeric>

#include "ssd_tc_dev.cuh"
#include "ssd_tree_attention.cuh"

namespace ssd {
namespace {

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

// Whether rows of D elements that a dimension of n lies apart by a stride are apart.
bool apart(int n, int64_t stride, int D) { return n == 1 || stride >= D; }

// Tokens and (node, head) pairs are counted in 32 bits.
constexpr int64_t kMaxCount = 0x7fffffff - (1 << 20);

// The scale of scores in base 2.
float base_2(float scale) { return (float)((double)scale * 1.4426950408889634); }

ssd_status check(const ssd_tree_attn* a) {
  if (!a || (a->dtype != SSD_BF16 && a->dtype != SSD_F16)) return SSD_ERR_INVALID_ARG;
  if (a->B < 1 || a->N < 1 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv != 0 ||
      a->num_pages < 1 || a->page_size < 1 || a->cols < 0 || !std::isfinite(base_2(a->scale)))
    return SSD_ERR_INVALID_ARG;
  // tables of no columns may have no address
  if ((!a->tables && a->cols > 0) || !a->lens || a->table_stride < a->cols)
    return SSD_ERR_INVALID_ARG;
  if ((a->D != 64 && a->D != 128 && a->D != 256) || a->N > kTreeNodes) return SSD_ERR_UNSUPPORTED;
  if (a->parent)
    for (int u = 0; u < a->N; ++u)
      if (a->parent[u] >= u || a->parent[u] < (u > 0 ? 0 : -1)) return SSD_ERR_INVALID_ARG;
  if ((int64_t)a->cols * a->page_size > kMaxCount || (int64_t)a->B * a->N * a->Hq > kMaxCount)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

struct Layout {
  size_t po, pml, begun, total;
};

// The division of the work and the workspace of a call; false when its work is beyond
// 32-bit counts.
bool plan(const ssd_tree_attn& a, TreeAttnParams& p, Layout& L) {
  const int sms = std::max(num_sms(), 1), tile = tree_tile(a.D);
  p.a = a;
  p.a.parent = nullptr;                // of the host
  p.gqa = a.Hq / a.Hkv;
  p.by_page = divisor(a.page_size);
  p.by_gqa = divisor(p.gqa);
  p.pairs = a.N * p.gqa;
  // Blocks of whole nodes, whose queries TMA brings, where at most an eighth of the rows is
  // left empty for it: 57 nodes of 56 heads on 8 take 232 us instead of 243 with queries row
  // by row (32 sequences of 500 to 8191), 162 instead of 184 (147 of 2 to 5), at D = 256 355
  // instead of 402.
  const int whole = p.gqa <= 128 ? 128 / p.gqa * p.gqa : 0;
  p.block_pairs = whole >= 112 ? whole : 128;
  const int rows = p.block_pairs * tree_blocks(a.D, p.pairs);
  p.blocks = (p.pairs + rows - 1) / rows;
  p.part_rows = (std::min(p.pairs, rows) + 7) / 8 * 8;
  // -q for a negative scale, 0 for none: the maximum is taken before the scale
  p.scale_log2 = std::fabs(base_2(a.scale));
  p.q_and = ~0u;
  p.q_xor = 0u;
  if (p.scale_log2 == 0.f) {
    p.scale_log2 = 1.f;
    p.q_and = 0u;
  } else if (a.scale < 0.f) {
    p.q_xor = 0x80008000u;
  }
  p.q_plain = a.scale > 0.f && p.q_and != 0u;
  // A worker's CTAs go through the same stretches side by side, up to eight of them: for the
  // items of a head, which read the same tiles (32 sequences with two items a head at D = 256
  // 288 us instead of 371, at D = 128 230 instead of 245), and for the heads of a set where a
  // token's heads lie closer than its neighbour (64 x 11 nodes 185 us instead of 188, at D = 64
  // 107 instead of 152; 32 x 64 129 instead of 143; two contexts of 131072 160 instead of 166).
  const int most = std::min(8, sms);
  p.bg = p.hg = 1;
  for (int n = 2; n <= most; ++n)
    if (p.blocks % n == 0) p.bg = n;
  if (a.k_cache.head_stride < a.k_cache.token_stride &&
      a.v_cache.head_stride < a.v_cache.token_stride)
    for (int n = 2; n <= most / p.bg; ++n)
      if (a.Hkv % n == 0) p.hg = n;
  p.sets = a.Hkv / p.hg;
  p.block_sets = p.blocks / p.bg;
  p.side = p.hg * p.bg;
  p.workers = sms / p.side;
  const int64_t items = (int64_t)a.B * p.sets * p.block_sets;
  const int64_t tiles = ((int64_t)a.cols * a.page_size + tile - 1) / tile + (a.N + tile - 1) / tile;
  if (items * p.side > 0x7fffffff || items > 0x7fffffff / (tiles + 1)) return false;
  // A box's tokens are of one page and one tile.  Small boxes take longer than 16-byte copies:
  // 64 x 11 nodes over pages of 20 tokens, so boxes of four, 307 us instead of 350 (D = 128)
  // and 187 instead of 288 (64), but 585 instead of 490 at D = 256, where they are more.
  p.box_rows = std::gcd(a.page_size, tile);
  if (p.box_rows < (a.D == 256 ? 8 : 4) || !box_strides(a.k_cache, a.Hkv, a.page_size, a.num_pages) ||
      !box_strides(a.v_cache, a.Hkv, a.page_size, a.num_pages) ||
      !box_strides(a.k, a.Hkv, a.N, a.B) || !box_strides(a.v, a.Hkv, a.N, a.B))
    p.box_rows = 0;
  p.wide_rows = ((uintptr_t)a.out | 2 * (uintptr_t)(a.out_seq_stride | a.out_node_stride |
                                                    a.out_head_stride)) % 32 == 0;
  p.node_rows = std::min(tile, (a.N + 7) / 8 * 8);
  // Queries by TMA, where a block's are whole nodes, or all there are (32 x 64 nodes 130 us
  // instead of 143 row by row, 256 short sequences of a node each 75 instead of 79).
  const ssd_paged q{a.q, a.q_seq_stride, a.q_node_stride, a.q_head_stride};
  p.q_nodes = p.q_plain && p.gqa <= 128 && (p.pairs <= 128 || p.block_pairs % p.gqa == 0) &&
                      box_strides(q, a.Hq, a.N, a.B)
                  ? std::min(a.N, 128 / p.gqa) : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  const size_t ctas = (size_t)p.workers * p.side;
  L.po = take(2 * ctas * p.part_rows * a.D * 4);
  L.pml = take(2 * ctas * p.part_rows * 8);
  L.begun = take(ctas * 8);
  L.total = at;
  return true;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_tree_attention_workspace_size(const ssd_tree_attn* a) {
  TreeAttnParams p{};
  Layout L;
  return check(a) == SSD_OK && plan(*a, p, L) ? L.total : 0;
}

ssd_status ssd_tree_attention(const ssd_tree_attn* a, void* workspace, size_t workspace_bytes,
                              int32_t* dev_status, void* stream) {
  const ssd_status st = check(a);
  if (st != SSD_OK) return st;
  if (!view_ok(a->q, {a->q_seq_stride, a->q_node_stride, a->q_head_stride}) ||
      !view_ok(a->out, {a->out_seq_stride, a->out_node_stride, a->out_head_stride}) ||
      !view_ok(a->k) || !view_ok(a->v) || !view_ok(a->k_cache) || !view_ok(a->v_cache))
    return SSD_ERR_INVALID_ARG;
  if (!apart(a->B, a->out_seq_stride, a->D) || !apart(a->N, a->out_node_stride, a->D) ||
      !apart(a->Hq, a->out_head_stride, a->D))
    return SSD_ERR_INVALID_ARG;
  if (a->out == a->q &&
      (a->out_seq_stride != a->q_seq_stride || a->out_node_stride != a->q_node_stride ||
       a->out_head_stride != a->q_head_stride))
    return SSD_ERR_INVALID_ARG;
  TreeAttnParams p{};
  Layout L;
  if (!plan(*a, p, L)) return SSD_ERR_UNSUPPORTED;
  if (!workspace || (uintptr_t)workspace % 256 != 0 || workspace_bytes < L.total)
    return SSD_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  p.po = reinterpret_cast<float*>(ws + L.po);
  p.pml = reinterpret_cast<float2*>(ws + L.pml);
  p.begun = reinterpret_cast<int2*>(ws + L.begun);
  p.status = dev_status;
  p.chain = 1;
  for (int u = 1; u < a->N; ++u) {
    const int par = a->parent ? a->parent[u] : u - 1;
    p.parent[u] = (uint8_t)par;
    p.chain &= par == u - 1;
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == SSD_BF16 ? launch_tree_bf16(p, s) : launch_tree_f16(p, s);
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return SSD_ERR_CUDA;
}

}  // extern "C"
