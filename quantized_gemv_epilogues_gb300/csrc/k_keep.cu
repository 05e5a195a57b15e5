// k_keep.cu - mt_cache_keep: the keys and values of a drafted path moved
// together, in every layer's cache.
//
// Bound: latency for few texts, then memory: a token's K and V of every layer
// read and written once.  A thread owns 16 bytes of a token's K or V (one
// layer, head and column) and moves them for every token of the path, in order:
// the path's indices increase and each is at least its place in the path, so a
// place is written only after the token that lay there was read, and no thread
// waits for another.  36 layers of 8 heads of 128: one text's three moved tokens
// 3.1 us, 64 texts' 234 (69 MB read and written) 15.2, where the bytes take 10.2; the
// four loads one after another before a token moves (lengths, path, page, row) are
// what is left.
#include <algorithm>

#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int CK_THREADS = 256, CK_LAYERS = 64, CK_MANY = 4;

struct KeepArgs {
  PagedArgs pg;  // of the first cache
  const int32_t* path;
  const int32_t* count;
  int cols;
  int32_t* new_len;
  int layers;
  uint16_t* kv[CK_LAYERS][2];
};

// LAYERS layers a block, whose pages and places are looked up once.
template <int LAYERS>
__global__ void __launch_bounds__(CK_THREADS, LAYERS > 1 ? 4 : 1) cache_keep_kernel(const __grid_constant__ KeepArgs a) {
  constexpr int MOVES = LAYERS > 1 ? 2 : 4;  // tokens whose loads are in flight together
  const PagedArgs& pg = a.pg;
  const int b = blockIdx.x, layer = blockIdx.y * LAYERS;
  pdl_wait();
  pdl_trigger();
  const PagedSeq s = paged_seq(pg, b);
  const int base = s.kv - s.n, most = min(max(__ldg(a.count + b), 0), a.cols);
  const int32_t* path = a.path + (int64_t)b * a.cols;
  const int chunks = pg.head_dim / 8, units = 2 * pg.kv_heads * chunks;
  for (int u = blockIdx.z * CK_THREADS + threadIdx.x; u < units; u += gridDim.z * CK_THREADS) {
    const int side = u / (pg.kv_heads * chunks), rest = u - side * pg.kv_heads * chunks, h = rest / chunks;
    const int64_t column = (int64_t)h * pg.head_stride + 8 * (rest - h * chunks);
    uint16_t* kv[LAYERS];
#pragma unroll
    for (int l = 0; l < LAYERS; ++l) kv[l] = a.kv[min(layer + l, a.layers - 1)][side] + column;
    auto place = [&](int pos) -> int64_t {  // of a token's row in the cache, or -1
      if (pos < 0) return -1;
      const int e = pos / pg.page_size, page = paged_entry(pg, b, e);
      return page < 0 ? -1 : (int64_t)page * pg.page_stride + (int64_t)(pos - e * pg.page_size) * pg.token_stride;
    };
    int before = -1;
    for (int i0 = 0; i0 < most; i0 += MOVES) {
      uint4 x[MOVES][LAYERS];
      int64_t to[MOVES];
      bool end = false;
      int at[MOVES];
#pragma unroll
      for (int q = 0; q < MOVES; ++q) at[q] = i0 + q < most ? __ldg(path + i0 + q) : -1;
#pragma unroll
      for (int q = 0; q < MOVES; ++q) {
        to[q] = -1;
        end |= at[q] <= before || at[q] >= s.n;
        if (end) continue;
        before = at[q];
        if (at[q] == i0 + q) continue;
        const int64_t from = place(base + at[q]);
        to[q] = from < 0 ? -1 : place(base + i0 + q);
        if (to[q] < 0) continue;
#pragma unroll
        for (int l = 0; l < LAYERS; ++l) x[q][l] = *reinterpret_cast<const uint4*>(kv[l] + from);
      }
#pragma unroll
      for (int q = 0; q < MOVES; ++q) {
        if (to[q] < 0) continue;
#pragma unroll
        for (int l = 0; l < LAYERS; ++l)
          if (layer + l < a.layers) *reinterpret_cast<uint4*>(kv[l] + to[q]) = x[q][l];
      }
      if (end) break;
    }
  }
  if (a.new_len && layer == 0 && blockIdx.z == 0 && threadIdx.x == 0) {
    int i = 0, before = -1;
    for (; i < most; ++i) {
      const int at = __ldg(path + i);
      if (at <= before || at >= s.n) break;
      before = at;
    }
    a.new_len[b] = base + i;
  }
}

}  // namespace

}  // namespace mt

using namespace mt;

extern "C" mt_status mt_cache_keep(const mt_paged_cache* cache, void* const* layers, int L, const mt_paged_batch* batch,
                                   const int32_t* path, const int32_t* count, int cols, int32_t* new_len, void* stream) {
  if (!cache || !layers || !batch || !path || !count) return MT_ERR_NULL;
  if (L < 1 || L > PG_MAX_LAYERS || cols < 1 || cols > (1 << 20)) return MT_ERR_SHAPE;
  for (int i = 0; i < 2 * L; ++i)
    if (!layers[i]) return MT_ERR_NULL;
  mt_paged_cache c = *cache;
  c.k = layers[0];
  c.v = layers[1];
  KeepArgs a = {};
  if (const mt_status st = paged_args(&c, batch, &a.pg)) return st;
  for (int i = 0; i < 2 * L; ++i)
    if (!aligned_to(layers[i], 16)) return MT_ERR_ALIGN;
  if (!aligned_to(path, 4) || !aligned_to(count, 4) || !aligned_to(new_len, 4)) return MT_ERR_ALIGN;
  if (!paged_rows_apart(&c)) return MT_ERR_SHAPE;
  if (!paged_layers_apart(&c, layers, L)) return MT_ERR_ALIAS;
  const size_t bytes = paged_cache_bytes(&c);
  const ByteRange ins[] = {byte_range(batch->q_start, (size_t)(batch->B + 1) * 4), byte_range(batch->kv_len, (size_t)batch->B * 4),
                           byte_range(batch->pages, (size_t)((batch->B - 1) * batch->pages_ld + batch->max_pages) * 4),
                           byte_range(path, (size_t)batch->B * cols * 4), byte_range(count, (size_t)batch->B * 4)};
  const ByteRange rn = byte_range(new_len, (size_t)batch->B * 4);
  for (const ByteRange& r : ins)
    if (ranges_overlap(r, rn)) return MT_ERR_ALIAS;
  for (int i = 0; i < 2 * L; ++i) {
    const ByteRange rc = byte_range(layers[i], bytes);
    if (ranges_overlap(rc, rn)) return MT_ERR_ALIAS;
    for (const ByteRange& r : ins)
      if (ranges_overlap(r, rc)) return MT_ERR_ALIAS;
  }
  int derr = 0;
  const DeviceInfo* di = device_info(&derr);
  if (!di) return cuda_fail((cudaError_t)derr);
  a.pg.err = device_error_ptr();
  if (!a.pg.err) return MT_ERR_CUDA;
  a.path = path;
  a.count = count;
  a.cols = cols;
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  const int units = 2 * a.pg.kv_heads * (a.pg.head_dim / 8);
  for (int i = 0; i < L; i += CK_LAYERS) {
    a.layers = std::min(CK_LAYERS, L - i);
    a.new_len = i == 0 ? new_len : nullptr;
    for (int j = 0; j < a.layers; ++j) {
      a.kv[j][0] = (uint16_t*)layers[2 * (i + j)];
      a.kv[j][1] = (uint16_t*)layers[2 * (i + j) + 1];
    }
    // one layer a block for few texts, several where there are blocks enough (64
    // texts, 36 layers: 18.8 us with one, 15.2 with four)
    const int parts = (units + CK_THREADS - 1) / CK_THREADS;
    const bool many = (int64_t)batch->B * a.layers * parts > 8 * (int64_t)di->sm_count;
    const dim3 grid(batch->B, many ? (a.layers + CK_MANY - 1) / CK_MANY : a.layers, parts);
    const mt_status st = many ? launch(cache_keep_kernel<CK_MANY>, grid, dim3(CK_THREADS), 0, l, a)
                              : launch(cache_keep_kernel<1>, grid, dim3(CK_THREADS), 0, l, a);
    if (st) return st;
  }
  return MT_OK;
}
