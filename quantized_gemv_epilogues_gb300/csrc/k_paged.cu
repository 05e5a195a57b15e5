// k_paged.cu - host checks of the cache and batch arguments that the
// paged-cache calls of include/mt.h share.
#include "k_paged.cuh"

#include <algorithm>

namespace mt {

size_t paged_cache_bytes(const mt_paged_cache* c) {
  return (size_t)((int64_t)(c->num_pages - 1) * c->page_stride + (int64_t)(c->page_size - 1) * c->token_stride +
                  (int64_t)(c->kv_heads - 1) * c->head_stride + c->head_dim) *
         2;
}

namespace {

struct Dim {
  int64_t stride, n;
};

// The cache's dimensions of more than one entry, smallest stride first.
int cache_dims(const mt_paged_cache* c, Dim (&d)[3]) {
  const Dim all[3] = {{c->token_stride, c->page_size}, {c->head_stride, c->kv_heads}, {c->page_stride, c->num_pages}};
  int n = 0;
  for (const Dim& x : all)
    if (x.n > 1) d[n++] = x;
  std::sort(d, d + n, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  return n;
}

// Whether two rows of `row` elements, `delta` elements apart but for whole
// steps along the dimensions d[0 .. n), can share an element.  The rows below a
// dimension span at most its stride (paged_rows_apart), so only the two steps
// around delta come into question.
bool rows_meet(int64_t delta, const Dim* d, int n, int row) {
  if (n == 0) return delta < row && delta > -row;
  const Dim& x = d[n - 1];
  int64_t q = delta / x.stride;
  if (delta < q * x.stride) --q;  // towards minus infinity
  for (int i = 0; i < 2; ++i, ++q)
    if (q < x.n && q > -x.n && rows_meet(delta - q * x.stride, d, n - 1, row)) return true;
  return false;
}

}  // namespace

bool paged_rows_apart(const mt_paged_cache* c) {
  Dim d[3];
  const int n = cache_dims(c, d);
  int64_t extent = c->head_dim;  // elements that the dimensions so far span
  for (int i = 0; i < n; ++i) {
    if (d[i].stride < extent) return false;
    const int64_t steps = d[i].n - 1;
    extent = steps > ((int64_t)1 << 60) / d[i].stride ? (int64_t)1 << 60 : steps * d[i].stride + extent;
  }
  return true;
}

bool paged_kv_apart(const mt_paged_cache* c) {
  Dim d[3];
  const int n = cache_dims(c, d);
  return !rows_meet(((int64_t)(uintptr_t)c->v - (int64_t)(uintptr_t)c->k) / 2, d, n, c->head_dim);
}

bool paged_layers_apart(const mt_paged_cache* c, void* const* layers, int L) {
  const int64_t bytes = (int64_t)paged_cache_bytes(c);
  int64_t at[2 * PG_MAX_LAYERS];
  for (int i = 0; i < 2 * L; ++i) at[i] = (int64_t)(uintptr_t)layers[i];
  std::sort(at, at + 2 * L);
  // Most caches lie one behind the other.
  bool behind = true;
  for (int i = 1; i < 2 * L; ++i) behind &= at[i] - at[i - 1] >= bytes;
  if (behind) return true;
  Dim d[3];
  const int n = cache_dims(c, d);
  // Layers side by side within each page (or token, or head), where every cache
  // spans all others: what a cache has in one step of a dimension repeats with its
  // stride, so places in that step that are apart are apart everywhere.  (36
  // layers: 60 us by the comparison of all pairs below, 1024: 35 ms.)
  for (int k = n - 1; k >= 0; --k) {
    if (k < n - 1 && d[k + 1].stride % d[k].stride) break;
    int64_t in[2 * PG_MAX_LAYERS], span = c->head_dim;
    for (int i = 0; i < k; ++i) span += (d[i].n - 1) * d[i].stride;
    for (int i = 0; i < 2 * L; ++i) in[i] = (at[i] - at[0]) / 2 % d[k].stride;
    std::sort(in, in + 2 * L);
    bool apart = in[2 * L - 1] + span <= in[0] + d[k].stride;
    for (int i = 1; apart && i < 2 * L; ++i) apart = in[i] - in[i - 1] >= span;
    if (apart) return true;
  }
  // otherwise the rows of each pair whose spans meet
  for (int i = 0; i < 2 * L; ++i)
    for (int j = i + 1; j < 2 * L && at[j] - at[i] < bytes; ++j)
      if (rows_meet((at[j] - at[i]) / 2, d, n, c->head_dim)) return false;
  return true;
}

mt_status paged_args(const mt_paged_cache* c, const mt_paged_batch* b, PagedArgs* a) {
  if (!c || !b || !c->k || !c->v || !b->q_start || !b->kv_len || !b->pages) return MT_ERR_NULL;
  if (c->num_pages < 1 || c->page_size < 1 || c->page_size > 65536 || c->kv_heads < 1 || c->kv_heads > 1024 ||
      c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 8)
    return MT_ERR_SHAPE;
  if (b->B < 1 || b->B > PG_MAX_B || b->T < 0 || b->T > (1 << 22) || b->max_pages < 1 ||
      (int64_t)b->max_pages * c->page_size > (1 << 30) || b->pages_ld < b->max_pages)
    return MT_ERR_SHAPE;
  const int64_t st[3] = {c->page_stride, c->token_stride, c->head_stride};
  for (int64_t s : st) {
    if (s < 0 || s > ((int64_t)1 << 38)) return MT_ERR_SHAPE;
    if (s % 8) return MT_ERR_ALIGN;
  }
  // neighbours along each dimension may not share elements (whether any two
  // rows do matters only to a call that writes: paged_rows_apart)
  if ((c->page_size > 1 && c->token_stride < c->head_dim) || (c->kv_heads > 1 && c->head_stride < c->head_dim) ||
      (c->num_pages > 1 && c->page_stride < c->head_dim))
    return MT_ERR_SHAPE;
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(b->q_start, 4) || !aligned_to(b->kv_len, 4) ||
      !aligned_to(b->pages, 4))
    return MT_ERR_ALIGN;
  *a = PagedArgs{};
  a->k = (uint16_t*)c->k;
  a->v = (uint16_t*)c->v;
  a->page_stride = c->page_stride;
  a->token_stride = c->token_stride;
  a->head_stride = c->head_stride;
  a->num_pages = c->num_pages;
  a->page_size = c->page_size;
  a->kv_heads = c->kv_heads;
  a->head_dim = c->head_dim;
  a->q_start = b->q_start;
  a->kv_len = b->kv_len;
  a->pages = b->pages;
  a->pages_ld = b->pages_ld;
  a->B = b->B;
  a->T = b->T;
  a->max_pages = b->max_pages;
  a->max_kv = b->max_pages * c->page_size;
  return MT_OK;
}

}  // namespace mt
