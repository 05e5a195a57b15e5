// k_tree.cu - mt_tree_layout: positions and visibility bits of drafted trees
// from their parents.
//
// Mathematics.  anc(i) = {i} + anc(parent of i); position = kv - n + |anc(i)| - 1;
// bit j of i's row is set for j in anc(i).
//
// Bound: latency (a tree of 60 tokens is 240 bytes; 2.0 us).  A token's ancestors have
// lower indices, so a row is built word by word downwards: within a block of 32
// tokens (a warp) five rounds of pointer doubling over shuffles give each token
// its ancestors in the block and the parent through which it leaves the block;
// then every token hops from block to block through shared memory, at most 31
// hops in a chunk of 1024 tokens.  A token that leaves its chunk takes the rest
// of its row, and of its depth, from that ancestor's, which the block wrote
// before.  One block a sequence, two an SM (32 registers, 16 bytes of them spilled).
#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int TL_THREADS = 1024;

struct LayoutArgs {
  const int32_t* parent;
  const int32_t* q_start;
  const int32_t* kv_len;  // or nullptr
  int T;
  int32_t* positions;  // or nullptr
  uint32_t* visible;   // or nullptr
  int64_t ld;
  int words;
  int fours;  // a row's words are whole groups of four, each on a 16-byte boundary
};

__global__ void __launch_bounds__(TL_THREADS) tree_layout_kernel(const LayoutArgs a) {
  __shared__ uint32_t bits[TL_THREADS];  // a token's ancestors in its block of 32, itself among them
  __shared__ int out[TL_THREADS];        // the parent of the first of them: outside the block, or -1
  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int row0 = min(max(__ldg(a.q_start + b), 0), a.T);
  const int n = min(max(__ldg(a.q_start + b + 1), row0), a.T) - row0;
  const int base = a.kv_len ? __ldg(a.kv_len + b) - n : 0;
  for (int c0 = 0; c0 < n; c0 += TL_THREADS) {  // a chunk of the sequence's tokens
    const int i = c0 + tid;
    int up = i < n ? __ldg(a.parent + row0 + i) : -1;
    if (up < 0 || up >= i) up = -1;
    // doubling: `in` is the lane of the 2^k-th ancestor while that is in the block
    uint32_t m = 1u << lane;
    int leave = up >= (i & ~31) ? -1 : up, in = up >= (i & ~31) ? up & 31 : -1;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const uint32_t m2 = __shfl_sync(0xffffffffu, m, in & 31);
      const int leave2 = __shfl_sync(0xffffffffu, leave, in & 31), in2 = __shfl_sync(0xffffffffu, in, in & 31);
      if (in >= 0) {
        m |= m2;
        leave = leave2;
        in = in2;
      }
    }
    __syncthreads();  // the last chunk's words have been read
    bits[tid] = m;
    out[tid] = leave;
    __syncthreads();
    if (i < n) {
      int depth = -1, at = i;
      uint32_t* row = a.visible ? a.visible + (int64_t)(row0 + i) * a.ld : nullptr;
      int w = a.words - 1;  // words above are done
      // the row's words from the last on, four to a store where rows lie on
      // 16-byte boundaries (128 trees of up to 500 tokens: 6.6 -> 4.7 us)
      uint4 four = make_uint4(0, 0, 0, 0);
      auto put = [&](uint32_t x) {
        if (a.fours) {
          four = make_uint4(x, four.x, four.y, four.z);
          if ((w & 3) == 0) *reinterpret_cast<uint4*>(row + w) = four;
        } else {
          row[w] = x;
        }
        --w;
      };
      while (at >= c0) {
        const uint32_t x = bits[at - c0];
        depth += __popc(x);
        if (row) {
          while (w > at >> 5) put(0u);
          if (w == at >> 5) put(x);
        }
        at = out[at - c0];
      }
      if (at >= 0) {  // an ancestor in an earlier chunk
        if (row) {
          while (w > at >> 5) put(0u);
          const uint32_t* rest = a.visible + (int64_t)(row0 + at) * a.ld;
          while (w >= 0) put(rest[w]);
        }
        if (a.positions) depth += a.positions[row0 + at] - base + 1;
      } else if (row) {
        while (w >= 0) put(0u);
      }
      if (a.positions) a.positions[row0 + i] = base + depth;
    }
    __syncthreads();  // this chunk's rows are there for the next
  }
}

}  // namespace

}  // namespace mt

using namespace mt;

extern "C" mt_status mt_tree_layout(const int32_t* parent, const int32_t* q_start, const int32_t* kv_len, int B, int T,
                                    int32_t* positions, uint32_t* visible, int64_t visible_ld, int words, void* stream) {
  if (!q_start || (T > 0 && (!parent || (!positions && !visible)))) return MT_ERR_NULL;
  if (B < 1 || B > PG_MAX_B || T < 0 || T > (1 << 22)) return MT_ERR_SHAPE;
  if (visible && (words < 1 || words > MT_TREE_WORDS || visible_ld < words || visible_ld > ((int64_t)1 << 38))) return MT_ERR_SHAPE;
  const void* all[] = {parent, q_start, kv_len, positions, visible};
  for (const void* p : all)
    if (!aligned_to(p, 4)) return MT_ERR_ALIGN;
  const ByteRange rp = byte_range(positions, (size_t)T * 4), rv = byte_range(visible, rows_bytes(T, visible_ld, words, 4));
  const ByteRange ins[] = {byte_range(parent, (size_t)T * 4), byte_range(q_start, (size_t)(B + 1) * 4), byte_range(kv_len, (size_t)B * 4)};
  for (const ByteRange& i : ins)
    if (ranges_overlap(i, rp) || ranges_overlap(i, rv)) return MT_ERR_ALIAS;
  if (ranges_overlap(rp, rv)) return MT_ERR_ALIAS;
  if (T == 0) return MT_OK;
  const int fours = aligned_to(visible, 16) && visible_ld % 4 == 0 && words % 4 == 0;
  const LayoutArgs a = {parent, q_start, kv_len, T, positions, visible, visible_ld, words, fours};
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  return launch(tree_layout_kernel, dim3(B), dim3(TL_THREADS), 0, l, a);
}
