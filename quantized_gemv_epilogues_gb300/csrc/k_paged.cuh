// k_paged.cuh - what the paged-cache calls share: the cache and batch
// arguments as the kernels take them, the host's checks of them, and the
// device's reads of lengths and page indices, which are clamped and checked
// there because only the device sees their values.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "mt_device.cuh"
#include "mt_internal.h"

namespace mt {

constexpr int PG_MAX_B = 1024;

struct PagedArgs {
  uint16_t* k;
  uint16_t* v;
  int64_t page_stride, token_stride, head_stride;  // elements
  int num_pages, page_size, kv_heads, head_dim;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* pages;
  int64_t pages_ld;
  int B, T, max_pages;
  int max_kv;  // max_pages * page_size
  int* err;    // device error word
};

// New tokens [row0, row0 + n) of a sequence and its kv tokens in the cache
// (the new ones among them).  Whatever the arrays hold, the rows are within
// [0, T) and kv within the page table's row.
struct PagedSeq {
  int row0, n, kv;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int b) {
  const int s = min(max(__ldg(a.q_start + b), 0), a.T);
  const int e = min(max(__ldg(a.q_start + b + 1), s), a.T);
  return PagedSeq{s, e - s, min(max(__ldg(a.kv_len + b), 0), a.max_kv)};
}

// Records a page out of range, unless the word already holds an error: a
// timeout stays until it is cleared.
__device__ __forceinline__ void page_error(const PagedArgs& a) { atomicCAS(a.err, 0, (int)MT_ERR_PAGE); }

// Page index of entry i of sequence b, or -1 (with the error word set) if it
// is out of range.  i < max_pages.
__device__ __forceinline__ int paged_entry(const PagedArgs& a, int b, int i) {
  const int p = __ldg(a.pages + (int64_t)b * a.pages_ld + i);
  if ((unsigned)p < (unsigned)a.num_pages) return p;
  page_error(a);
  return -1;
}

// ---- host side (k_paged.cu)
// Checks of the cache and batch arguments; fills `a` (without the error word).
mt_status paged_args(const mt_paged_cache* c, const mt_paged_batch* b, PagedArgs* a);
// Whether no two (page, token, head) rows of K (or of V) share an element, for
// checked arguments: each stride spans the dimensions of smaller strides.
bool paged_rows_apart(const mt_paged_cache* c);
// Whether no row of K shares an element with one of V; rows apart only.
bool paged_kv_apart(const mt_paged_cache* c);
// Bytes from a cache pointer to the end of its last element.
size_t paged_cache_bytes(const mt_paged_cache* c);

struct ByteRange {
  uintptr_t lo, hi;
};
inline ByteRange byte_range(const void* p, size_t n) { return ByteRange{(uintptr_t)p, (uintptr_t)p + (p ? n : 0)}; }
inline bool ranges_overlap(ByteRange a, ByteRange b) { return a.lo < b.hi && b.lo < a.hi; }
// Bytes that rows of `row` elements, `stride` elements apart, span.
inline size_t rows_bytes(int64_t rows, int64_t stride, int64_t row, int elem) {
  return rows < 1 ? 0 : (size_t)((rows - 1) * stride + row) * elem;
}
inline bool aligned_to(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace mt
