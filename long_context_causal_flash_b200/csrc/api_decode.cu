// C ABI of the decoding entry points: argument validation, views, workspace sizing.  The
// operations, layouts and error conventions are documented in gqa_attn.h.
#include <cmath>

#include "internal.h"
#include "tree.cuh"

namespace gqa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_bytes(int dtype) { return dtype == GQA_F32 ? 4 : dtype == GQA_BF16 ? 2 : 1; }

int check_rows(const gqa_rows_t* r, int B, int64_t L, int dtype) {
  if (!r || !r->data || r->H < 1) return GQA_ERR_INVALID_ARG;
  const int64_t unit = 16 / elem_bytes(dtype);
  if (!aligned16(r->data) || (B > 1 && r->stride_b % unit) || (r->H > 1 && r->stride_h % unit) ||
      (L > 1 && r->stride_l % unit))
    return GQA_ERR_MISALIGNED;
  return GQA_OK;
}

RowsView rows_view(const gqa_rows_t* r) {
  return RowsView{static_cast<char*>(r->data), r->stride_b, r->stride_h, r->stride_l, r->H};
}

int check_rope(const gqa_rope_t* r) {
  if (!r->turns || r->rot < 16 || r->rot > kHeadDim || r->rot % 16) return GQA_ERR_INVALID_ARG;
  if (r->layout != GQA_ROPE_HALF && r->layout != GQA_ROPE_INTERLEAVED) return GQA_ERR_INVALID_ARG;
  return GQA_OK;
}

RopeView rope_view(const gqa_rope_t* r) {
  if (!r) return RopeView{nullptr, nullptr, 0, 0, 1.f, 0, 0};
  return RopeView{r->turns, r->positions, r->positions_stride_b, r->pos_offset, r->magnitude, r->rot,
                  r->layout == GQA_ROPE_INTERLEAVED};
}

bool page_size_ok(int n) { return n >= 8 && n <= 1024 && (n & (n - 1)) == 0; }

int check_cache(const gqa_cache_t* c, int64_t max_pages) {
  if (!c || !c->k || !c->v || c->Hkv < 1 || c->n_pages < 1 || c->n_pages > 0x7fffffff) return GQA_ERR_INVALID_ARG;
  if (c->dtype != GQA_F32 && c->dtype != GQA_BF16 && c->dtype != GQA_E4M3) return GQA_ERR_INVALID_ARG;
  const bool quantised = c->dtype == GQA_E4M3;
  if ((c->k_scale != nullptr) != quantised || (c->v_scale != nullptr) != quantised) return GQA_ERR_INVALID_ARG;
  if (!page_size_ok(c->page_size) || max_pages < 1 || max_pages > 0x7fffffff) return GQA_ERR_INVALID_ARG;
  const int64_t unit = 16 / elem_bytes(c->dtype);
  if (!aligned16(c->k) || !aligned16(c->v) || c->stride_token % unit || (c->Hkv > 1 && c->stride_head % unit) ||
      (c->n_pages > 1 && c->stride_page % unit))
    return GQA_ERR_MISALIGNED;
  return GQA_OK;
}

CacheView cache_view(const gqa_cache_t* c) {
  CacheView v;
  v.k = static_cast<char*>(c->k);
  v.v = static_cast<char*>(c->v);
  v.ks = c->k_scale;
  v.vs = c->v_scale;
  v.status = c->status;
  v.sp = c->stride_page;
  v.sh = c->stride_head;
  v.st = c->stride_token;
  v.n_pages = c->n_pages;
  v.Hkv = c->Hkv;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c->page_size) ++v.page_shift;
  v.dtype = c->dtype;
  return v;
}

bool float_dtype(int dtype) { return dtype == GQA_F32 || dtype == GQA_BF16; }

int check_tree(int B, int Hq, int Hkv, int64_t T, int64_t max_pages, int page_size, int d, int dtype, int cache_dtype) {
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || max_pages < 1 || max_pages > 0x7fffffff || Hq % Hkv)
    return GQA_ERR_INVALID_ARG;
  if (!page_size_ok(page_size) || !float_dtype(dtype)) return GQA_ERR_INVALID_ARG;
  if (cache_dtype != GQA_F32 && cache_dtype != GQA_BF16 && cache_dtype != GQA_E4M3) return GQA_ERR_INVALID_ARG;
  if (d != kHeadDim || T > 1024 || int64_t(B) * Hq > 0x7fffffff) return GQA_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8 && G != 16) return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

// Workspace: per worker two slots of row_tiles x rows partial outputs, then log-sum-exps.
struct TreeWs {
  size_t lse = 0, total = 0;
};

TreeWs tree_ws(const TreeShape& s) {
  TreeWs w;
  const size_t rows = size_t(s.workers) * 2 * s.row_tiles * s.rows;
  w.lse = rows * kHeadDim * sizeof(float);
  w.total = w.lse + round_up(rows * sizeof(float), 256);
  return w;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

int gqa_attn_rope(const gqa_rows_t* x, const gqa_rows_t* out, const gqa_rows_t* x2, const gqa_rows_t* out2, int B,
                  int64_t L, int d, int dtype, const gqa_rope_t* rope, int inverse, gqa_stream_t stream) {
  if (!rope || !x || !out || (x2 == nullptr) != (out2 == nullptr) || B < 0 || L < 0) return GQA_ERR_INVALID_ARG;
  if (!float_dtype(dtype)) return GQA_ERR_INVALID_ARG;
  if (d != kHeadDim) return GQA_ERR_UNSUPPORTED;
  int rc = check_rope(rope);
  if (rc != GQA_OK) return rc;
  if (B == 0 || L == 0) return GQA_OK;
  for (const gqa_rows_t* r : {x, out, x2, out2})
    if (r && (rc = check_rows(r, B, L, dtype)) != GQA_OK) return rc;
  if (x->H != out->H || (x2 && x2->H != out2->H)) return GQA_ERR_INVALID_ARG;
  const RowsView none{nullptr, 0, 0, 0, 0};
  return launch_rope(rows_view(x), rows_view(out), x2 ? rows_view(x2) : none, x2 ? rows_view(out2) : none, B, L,
                     dtype == GQA_BF16, rope_view(rope), inverse != 0, reinterpret_cast<cudaStream_t>(stream));
}

int gqa_attn_cache_write(const gqa_cache_t* cache, const gqa_rows_t* k, const gqa_rows_t* v,
                         const int32_t* page_table, int64_t max_pages, const int32_t* start, const int32_t* lens,
                         int B, int64_t L, int d, int dtype, const gqa_rope_t* rope, gqa_stream_t stream) {
  if (!k || !v || B < 0 || L < 0 || !float_dtype(dtype)) return GQA_ERR_INVALID_ARG;
  if (d != kHeadDim) return GQA_ERR_UNSUPPORTED;
  int rc = check_cache(cache, max_pages);
  if (rc == GQA_OK && rope) rc = check_rope(rope);
  if (rc != GQA_OK) return rc;
  if (B == 0 || L == 0) return GQA_OK;  // empty tensors may have no address
  if (!page_table || !start) return GQA_ERR_INVALID_ARG;
  if ((rc = check_rows(k, B, L, dtype)) != GQA_OK || (rc = check_rows(v, B, L, dtype)) != GQA_OK) return rc;
  if (k->H != cache->Hkv || v->H != cache->Hkv) return GQA_ERR_INVALID_ARG;
  return launch_cache_write(cache_view(cache), rows_view(k), rows_view(v), page_table, max_pages, start, lens, B, L,
                            dtype == GQA_BF16, rope_view(rope), reinterpret_cast<cudaStream_t>(stream));
}

int gqa_attn_cache_read(const gqa_cache_t* cache, const int32_t* page_table, int64_t max_pages, const int32_t* lens,
                        void* k_out, void* v_out, int B, int64_t max_len, int d, int dtype_out,
                        gqa_stream_t stream) {
  if (B < 0 || max_len < 0 || !float_dtype(dtype_out)) return GQA_ERR_INVALID_ARG;
  if (d != kHeadDim) return GQA_ERR_UNSUPPORTED;
  const int rc = check_cache(cache, max_pages);
  if (rc != GQA_OK) return rc;
  if (B == 0 || max_len == 0) return GQA_OK;
  if (!page_table || !lens || !k_out || !v_out) return GQA_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out)) return GQA_ERR_MISALIGNED;
  return launch_cache_read(cache_view(cache), page_table, max_pages, lens, k_out, v_out, B, max_len,
                           dtype_out == GQA_BF16, reinterpret_cast<cudaStream_t>(stream));
}

size_t gqa_attn_tree_workspace_bytes(int B, int Hq, int Hkv, int64_t T, int64_t max_pages, int page_size, int d,
                                     int dtype, int cache_dtype) {
  if (check_tree(B, Hq, Hkv, T, max_pages, page_size, d, dtype, cache_dtype) != GQA_OK) return 0;
  return tree_ws(tree_shape(B, Hkv, Hq / Hkv, T, max_pages, page_size, dtype == GQA_BF16, cache_dtype)).total;
}

int gqa_attn_fwd_tree(const gqa_rows_t* q, const gqa_cache_t* cache, const int32_t* page_table, int64_t max_pages,
                      const int32_t* context_lens, const int32_t* tree_lens, const uint8_t* tree_mask,
                      int64_t mask_stride_b, void* out, float* lse, int B, int64_t T, int d, int dtype,
                      void* workspace, size_t workspace_bytes, gqa_stream_t stream) {
  if (!q || !cache || !page_table || !context_lens || !out || !lse || mask_stride_b < 0) return GQA_ERR_INVALID_ARG;
  int rc = check_tree(B, q->H, cache->Hkv, T, max_pages, cache->page_size, d, dtype, cache->dtype);
  if (rc == GQA_OK) rc = check_cache(cache, max_pages);
  if (rc == GQA_OK) rc = check_rows(q, B, T, dtype);
  if (rc != GQA_OK) return rc;
  if (!aligned16(out) || !aligned16(lse)) return GQA_ERR_MISALIGNED;
  const int G = q->H / cache->Hkv;
  const TreeShape s = tree_shape(B, cache->Hkv, G, T, max_pages, cache->page_size, dtype == GQA_BF16, cache->dtype);
  const TreeWs w = tree_ws(s);
  if (!workspace || workspace_bytes < w.total) return GQA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GQA_ERR_MISALIGNED;
  TreeParams p;
  p.q = rows_view(q);
  p.c = cache_view(cache);
  p.table = page_table;
  p.ctx = context_lens;
  p.tree_lens = tree_lens;
  p.mask = tree_mask;
  p.max_pages = max_pages;
  p.mask_sb = mask_stride_b;
  p.out = out;
  p.lse = lse;
  p.o_part = static_cast<float*>(workspace);
  p.lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.lse);
  p.B = B;
  p.T = int(T);
  p.G = G;
  p.tile_shift = s.tile_shift;
  p.workers = s.workers;
  p.row_tiles = s.row_tiles;
  p.out_bf16 = dtype == GQA_BF16;
  p.scale_log2 = float(1.0 / std::sqrt(double(d)) * 1.4426950408889634);
  p.wait_budget_ns = wait_budget_ns();
  p.test_skip_fill = test_skip_fill();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = s.tensor ? launch_tree_tc(p, s.rows, st) : launch_tree_f32(p, s.rows, dtype == GQA_BF16, st);
  return rc != GQA_OK ? rc : launch_tree_merge(p, s.rows, st);
}

}  // extern "C"
