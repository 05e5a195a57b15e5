// k_attn.cu - the C entry points of mt_paged_attention and mt_tree_attention:
// argument checks and the choice of kernel.
#include <math.h>

#include <algorithm>

#include "k_attn.cuh"

using namespace mt;

namespace {

size_t attn_ws(int head_dim, const DeviceInfo* di) {
  const int sms = di ? di->sm_count : 152;
  return std::max(attn_rows_ws(head_dim, sms), attn_tile_ws(head_dim, sms));
}

// Trees: `visible` has T rows.
struct TreeRows {
  const uint32_t* visible;
  int64_t ld;
  int words;
};

mt_status attention(const void* q, int64_t q_stride, int q_heads, const mt_paged_cache* cache, const mt_paged_batch* batch,
                    const TreeRows* tree, float scale, int window, int sinks, void* out, int64_t out_stride,
                    mt_dtype out_dtype, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  AttnArgs a = {};
  if (const mt_status st = paged_args(cache, batch, &a.pg)) return st;
  if (batch->T > 0 && (!q || !out || !workspace || (tree && !tree->visible))) return MT_ERR_NULL;
  if (out_dtype != MT_BF16 && out_dtype != MT_F32) return MT_ERR_FORMAT;
  const int D = cache->head_dim, Hk = cache->kv_heads, T = batch->T;
  if (q_heads < 1 || q_heads > 1024 || q_heads % Hk || q_heads / Hk > 128 || q_stride < (int64_t)q_heads * D ||
      out_stride < (int64_t)q_heads * D || q_stride > ((int64_t)1 << 38) || out_stride > ((int64_t)1 << 38) ||
      !(scale > 0.f) || !(scale < INFINITY) || window < 0 || sinks < 0)
    return MT_ERR_SHAPE;
  if (tree && (tree->words < 1 || tree->words > MT_TREE_WORDS || tree->ld < tree->words || tree->ld > ((int64_t)1 << 38)))
    return MT_ERR_SHAPE;
  if (q_stride % 8 || out_stride % 8 || !aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(workspace, 16) ||
      !aligned_to(lse, 4) || (tree && !aligned_to(tree->visible, 4)))
    return MT_ERR_ALIGN;
  int derr = 0;
  const DeviceInfo* di = device_info(&derr);
  const size_t need = attn_ws(D, di);
  if (workspace_bytes < need) return MT_ERR_SHAPE;
  const ByteRange iq = byte_range(q, rows_bytes(T, q_stride, (int64_t)q_heads * D, 2));
  const ByteRange ro = byte_range(out, rows_bytes(T, out_stride, (int64_t)q_heads * D, out_dtype == MT_F32 ? 4 : 2));
  const ByteRange rl = byte_range(lse, (size_t)T * q_heads * 4), rw = byte_range(workspace, need);
  const ByteRange ins[] = {iq, byte_range(cache->k, paged_cache_bytes(cache)), byte_range(cache->v, paged_cache_bytes(cache)),
                           byte_range(batch->q_start, (size_t)(batch->B + 1) * 4), byte_range(batch->kv_len, (size_t)batch->B * 4),
                           byte_range(batch->pages, (size_t)((batch->B - 1) * batch->pages_ld + batch->max_pages) * 4),
                           tree ? byte_range(tree->visible, rows_bytes(T, tree->ld, tree->words, 4)) : ByteRange{0, 0}};
  for (const ByteRange& i : ins)
    if (ranges_overlap(i, ro) || ranges_overlap(i, rl) || ranges_overlap(i, rw)) return MT_ERR_ALIAS;
  if (ranges_overlap(ro, rl) || ranges_overlap(ro, rw) || ranges_overlap(rl, rw)) return MT_ERR_ALIAS;
  if (T == 0) return MT_OK;
  if (!di) return cuda_fail((cudaError_t)derr);
  a.pg.err = device_error_ptr();
  if (!a.pg.err) return MT_ERR_CUDA;
  a.q = (const uint16_t*)q;
  a.q_stride = q_stride;
  a.out = out;
  a.out_stride = out_stride;
  a.lse = lse;
  a.out_f32 = out_dtype == MT_F32;
  a.q_heads = q_heads;
  a.group = q_heads / Hk;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  // a window that no text here outgrows is none (and a position less it stays
  // within 32 bits)
  a.window = window < a.pg.max_kv ? window : 0;
  a.sinks = sinks;
  if (tree) {
    a.visible = tree->visible;
    a.visible_ld = tree->ld;
    a.words = tree->words;
  }
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  a.max_q = batch->max_q;
  if (attn_tile_takes(a)) return launch_attn_tile(a, workspace, l, di);
  return launch_attn_rows(a, workspace, l, di);
}

}  // namespace

extern "C" {

size_t mt_paged_attention_workspace_bytes(int T, int B, int q_heads, int kv_heads, int head_dim) {
  if (T < 0 || B < 1 || q_heads < 1 || kv_heads < 1 || head_dim < 16 || head_dim > 256) return 0;
  int derr = 0;
  const DeviceInfo* di = device_info(&derr);
  return attn_ws(head_dim, di);
}

mt_status mt_paged_attention(const void* q, int64_t q_stride, int q_heads, const mt_paged_cache* cache,
                             const mt_paged_batch* batch, float scale, int window, int sinks, void* out,
                             int64_t out_stride, mt_dtype out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return attention(q, q_stride, q_heads, cache, batch, nullptr, scale, window, sinks, out, out_stride, out_dtype, lse,
                   workspace, workspace_bytes, stream);
}

mt_status mt_tree_attention(const void* q, int64_t q_stride, int q_heads, const mt_paged_cache* cache,
                            const mt_paged_batch* batch, const uint32_t* visible, int64_t visible_ld, int words,
                            float scale, int window, int sinks, void* out, int64_t out_stride, mt_dtype out_dtype,
                            float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const TreeRows tree = {visible, visible_ld, words};
  return attention(q, q_stride, q_heads, cache, batch, &tree, scale, window, sinks, out, out_stride, out_dtype, lse,
                   workspace, workspace_bytes, stream);
}

}  // extern "C"
