// k_attn_tile.cu - attention over a paged cache for chunks of new tokens, on
// the fifth-generation tensor cores.
//
// Bound: the tensor cores, 4 D flops per visible (row, key).  A CTA holds two
// tiles of 128 rows (packed (token, query head) pairs of one key/value head)
// and streams blocks of 128 keys past both: S = Q K^T and O += P V are
// tcgen05.mma with M = 128 and fp32 accumulators in tensor memory.
//  * Tensor memory (512 columns): S of tile 0 and of tile 1 (128 each), O of
//    both (DP each).  P overwrites the first 64 columns of its S as bf16
//    pairs and is the second product's A operand there: P never passes
//    through shared memory.
//  * Shared memory: both Q tiles, and one ring of stages that K and V blocks
//    enter in the order they are used (K0 V0 K1 V1 ...), by TMA with the
//    128-byte swizzle.  K's rows are the K-major operand of S, V's rows the
//    MN-major operand of O: V is used as stored.
//  * A block comes as boxes of the largest power of two of tokens that divides
//    the page size (at most 128), one lane of the producer warp each, with the
//    page's index from the table as a TMA coordinate; boxes that no row sees,
//    or whose entry is out of range, are asked for at a page beyond the cache,
//    which TMA fills with zeros.  Keys of a box that no row sees (beyond the
//    sequence's end in its last page, before the window in its first) may hold
//    anything: the producer zeroes their V before handing it on (a weight of
//    zero times NaN is NaN).
//  * One softmax warpgroup per tile, one row per thread, so that maxima and
//    sums need no exchange and no warp waits for another.  (Two warpgroups a
//    tile, half a row per thread, cost more in the exchange than the shorter
//    rows gained: 521 against 426 us for a prompt of 8000, all else as it then
//    was.)  The row's reference maximum moves only when a
//    score exceeds it by more than 2^8 (8 in log2 units): fp32 sums and bf16
//    weights lose nothing by weights up to 2^8, and O is rescaled in tensor
//    memory only then - once or twice a row, typically.  When S of block j is
//    complete so is every earlier product of the tile (one thread issues them
//    and they complete in order), so the softmax warps may rescale O without
//    another barrier.
//  * While one tile's softmax runs, the tensor cores work on the other tile:
//    PV0(j) S0(j+1) PV1(j) S1(j+1) is the issue order.  A piece with rows in
//    one tile only (single tokens beside a chunk) uses both buffers of S in
//    turn, and S runs a block ahead.
// Weights are rounded to bf16 (2^-8 of each) because the MMA takes one type
// for both operands and V is bf16; the sum l is of the unrounded weights.
// Every mbarrier wait is bounded (~1 s): on expiry the error word gets
// MT_ERR_TIMEOUT, the CTA's other roles stop at their own next wait, copies
// and MMAs in flight are waited for, and tensor memory is freed.
#include <math.h>

#include <atomic>

#include "k_attn.cuh"
#include "k_prefill.cuh"

namespace mt {

namespace {

constexpr int AT_BK = 128, AT_R = 256, AT_THREADS = 384;
constexpr int AT_EXTRA = 6;  // units of a tile beside its blocks' 3 or 2
constexpr int AT_SOFT = 8;  // warps 0-7: softmax; tile warp / 4, rows 32 (warp % 4) on
constexpr int AT_MMA = 8, AT_WALK = 9, AT_LOAD = 10;  // AT_LOAD: Q and K, and the next warp V

template <int DP>
struct AtShape {
  static constexpr int CH = DP / 64;                 // 64-element column halves (one 128-byte swizzle row each)
  static constexpr int HALF = 128 * 128;             // 128 rows of 128 bytes
  static constexpr int TILE = CH * HALF;             // a Q tile, or a K or V block
  static constexpr int NS = DP == 128 ? 4 : 8;       // ring stages
  static constexpr size_t OFF_KV = 2 * (size_t)TILE;
  static constexpr size_t OFF_OUT = OFF_KV + (size_t)NS * TILE;  // 128 bytes of each softmax thread's row, on their way out
  static_assert((size_t)NS * TILE >= sizeof(PlanShared), "the plan uses the ring's memory");
};

// 32 consecutive 32-bit columns of this thread's tensor-memory lane; at_ld_done
// must follow before a register is used.
__device__ __forceinline__ void at_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                 "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                 "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                 "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(taddr)
               : "memory");
}
// Waits for this thread's tensor-memory loads; names the registers so that no
// use of them is scheduled before the wait.
__device__ __forceinline__ void at_ld_done32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) : : "memory");
}
__device__ __forceinline__ void at_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::
               "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                 "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
                 "r"(r[15]) : "memory");
}

__device__ __forceinline__ void at_st_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Descriptor of V as the MN-major B operand: 64 elements of a key's row are
// 128 contiguous bytes (128-byte swizzle), 8 keys 1024 bytes; the next 64
// elements start HALF bytes on.
__device__ __forceinline__ uint64_t at_desc_mn(uint32_t saddr, uint32_t half_bytes) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(half_bytes >> 4) << 16;  // leading offset: between 64-element columns
  d |= (uint64_t)(1024 >> 4) << 32;        // stride offset: between groups of 8 keys
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// bf16 A and B, fp32 accumulator, M = 128; B MN-major for V.
constexpr uint32_t at_idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void at_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A from tensor memory.
__device__ __forceinline__ void at_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One thread's bulk copy shared -> global (16-byte aligned, a multiple of 16
// bytes), the wait until its copies have read their sources, and until they
// are done.
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, int bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y), "r"(z),
               "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_reads_done() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Bits [0, n), n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// A piece of a tile: the part of its blocks that lies in this CTA's stretch.
// One warp walks the stretch and puts the pieces into a small ring in shared
// memory for the others (each walking for itself cost them registers and, at
// every piece, two thousand cycles of index arithmetic).
struct Piece {
  int n[2];       // blocks for each of the two 128-row tiles (0: it has no rows, or sees none of them)
  int first;      // the piece's first block within the tile's
  int sink, win;  // as TileSpan
  int key_end, win_lo;
  int kv, base;   // the sequence's tokens; the position of its first new one
  int b, h, row0, i0, i1, p0;
  int whole;      // the tile's only piece: its rows are written, not its parts
  int stop;       // no piece: the stretch has ended
};
constexpr int AT_PIECES = 4;

// What follows the tiles in shared memory (all of it is dynamic, so that the
// tiles start where it starts, on a 1024-byte boundary).
struct AtShared {
  uint64_t bars[2 * 10 + 6 + 4 + 2 + 2 * AT_PIECES + 2 + AT_PIECES];
  uint32_t tmem;
  int abort;
  Piece piece[AT_PIECES];
};
template <int DP>
constexpr size_t at_smem() {
  return AtShape<DP>::OFF_OUT + 256 * 128 + sizeof(AtShared);
}
static_assert(at_smem<128>() <= 227 * 1024 && at_smem<64>() <= 227 * 1024, "shared memory plan");

template <int DP>
__global__ void __launch_bounds__(AT_THREADS, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap, const AttnArgs a,
                     const int box_rows) {
  using S = AtShape<DP>;
  constexpr int NS = S::NS;
  extern __shared__ __align__(1024) unsigned char smem[];
  AtShared& sh = *reinterpret_cast<AtShared*>(smem + S::OFF_OUT + 256 * 128);
  uint64_t* bars = sh.bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto kv_full = [&](int i) { return smem_u32(&bars[i]); };
  auto kv_free = [&](int i) { return smem_u32(&bars[NS + i]); };
  auto s_full = [&](int s) { return smem_u32(&bars[2 * NS + s]); };      // S of a block is in tensor memory
  auto p_full = [&](int s) { return smem_u32(&bars[2 * NS + 2 + s]); };  // P is (and O rescaled)
  // o_full(0): the first tile's O of the piece is complete; o_full(1): O of a
  // block, in pieces with rows in the first tile only
  auto o_full = [&](int s) { return smem_u32(&bars[2 * NS + 4 + s]); };
  auto p_half = [&](int s) { return smem_u32(&bars[2 * NS + 12 + 2 * AT_PIECES + s]); };  // P of the block's first 64 keys is
  auto q_full = [&](int s) { return smem_u32(&bars[2 * NS + 6 + s]); };
  auto q_free = [&](int s) { return smem_u32(&bars[2 * NS + 8 + s]); };
  const uint32_t tail_bar = smem_u32(&bars[2 * NS + 10]), mma_done = smem_u32(&bars[2 * NS + 11]);
  auto piece_full = [&](int k) { return smem_u32(&bars[2 * NS + 12 + k % AT_PIECES]); };
  auto piece_free = [&](int k) { return smem_u32(&bars[2 * NS + 12 + AT_PIECES + k % AT_PIECES]); };
  // every product of the piece is complete: a barrier per place in the ring of
  // pieces, which is not used again before every warp has left the piece, so
  // that a warp that waits for it is never two phases behind (a parity would
  // not tell it)
  auto piece_done = [&](int k) { return smem_u32(&bars[2 * NS + 14 + 2 * AT_PIECES + k % AT_PIECES]); };
  auto q_tile = [&](int s) { return smem_u32(smem + (size_t)s * S::TILE); };
  auto stage = [&](int i) { return smem_u32(smem + S::OFF_KV + (size_t)i * S::TILE); };

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(kv_full(i), 1);
      mbar_init(kv_free(i), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(p_half(s), 4);  // one arrival per softmax warp
      mbar_init(p_full(s), 4);
      mbar_init(o_full(s), 1);
      mbar_init(q_full(s), 1);
      mbar_init(q_free(s), 1);
    }
    for (int k = 0; k < AT_PIECES; ++k) {
      mbar_init(piece_full(k), 1);
      mbar_init(piece_free(k), AT_SOFT + 3);  // one arrival per warp that reads it
      mbar_init(piece_done(k), 1);
    }
    mbar_init(tail_bar, 1);
    mbar_init(mma_done, 1);
    sh.abort = 0;
    mbar_fence_init();
  }
  if (warp == AT_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid < 4) {  // the maps' descriptors, on their way while the plan is made
    const CUtensorMap* m = tid == 0 ? &qmap : tid == 1 ? &kmap : tid == 2 ? &vmap : &omap;
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
  }
  pdl_wait();
  pdl_trigger();
  long long u0, u1, per;
  Cursor c;
  plan<AT_R, AT_BK, AT_THREADS, AT_EXTRA>(a, reinterpret_cast<PlanShared*>(smem + S::OFF_KV), blockIdx.x, gridDim.x, &u0, &u1, &per, &c);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the plan's accesses before TMA's to the same memory
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sh.tmem;
  volatile int* abort_flag = &sh.abort;
  auto fail = [&]() {
    atomicExch(a.pg.err, (int)MT_ERR_TIMEOUT);
    *abort_flag = 1;
  };
  // This thread's bounded wait; false after an abort, or if it expires.
  auto wait1 = [&](uint32_t bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
      for (int i = 0; i < 32; ++i)
        if (mbar_try_wait(bar, parity)) return true;
      if (*abort_flag) return false;
      if (clock64() - t0 > (1ll << 31)) {
        fail();
        return false;
      }
    }
  };
  // a warp's, one answer for all its lanes
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait1(bar, parity)); };

  // a softmax thread holds a row of S, the other warps need fewer registers:
  // 256 x 216 + 128 x 72 of the launch's 384 x 168
  if (warp >= AT_SOFT) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == AT_WALK) {
      // ---- the stretch's pieces
      if (lane == 0) {
        const int tps = a.tile_tokens >> 1;
        a.cut[2 * blockIdx.x].x = -1;
        long long left = u1 - u0;  // units of the stretch from unit c.i of the tile on
        for (int k = 0;; ++k) {
          if (k >= AT_PIECES && !wait1(piece_free(k), ((k / AT_PIECES) + 1) & 1)) break;
          Piece& p = sh.piece[k % AT_PIECES];
          // blocks [i0, i1) of the tile
          const int w = block_units<AT_EXTRA>(a, c.r), all_units = AT_EXTRA + w * c.t.n;
          const int end = (int)min((long long)all_units, c.i + left);
          const int i0 = max(c.i - AT_EXTRA, 0) / w, i1 = (end - AT_EXTRA) / w;
          // (a stretch that ends before a tile's first block does leaves the tile to the next)
          const bool stop = left <= 0 || end < AT_EXTRA + w;
          p.stop = stop;
          if (!stop) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int first = c.r.i0 + s * tps, last = min(first + tps - 1, c.r.i1);
              const int to = (max(c.s.kv - c.s.n + last + 1, 0) + AT_BK - 1) / AT_BK;
              const int all = min(c.t.sink, to) + max(0, to - c.t.win);  // of the tile's blocks, those up to the last token
              p.n[s] = first > c.r.i1 ? 0 : min(max(all - i0, 0), i1 - i0);
            }
            p.first = i0;
            p.sink = c.t.sink;
            p.win = c.t.win;
            p.key_end = c.t.key_end;
            p.win_lo = c.t.win_lo;
            p.kv = c.s.kv;
            p.base = c.s.kv - c.s.n;
            p.b = c.b;
            p.h = c.h;
            p.row0 = c.s.row0;
            p.i0 = c.r.i0;
            p.i1 = c.r.i1;
            p.p0 = c.r.p0;
            p.whole = i0 == 0 && i1 == c.t.n;
            if (i0 == 0 && i1 < c.t.n) put_cut(a, blockIdx.x, (int)div_count(u1 - left + all_units - c.i - 1, per), c);
          }
          mbar_arrive(piece_full(k));
          if (stop) break;
          left -= end - c.i;
          if (left > 0) {
            c.i = c.t.n - 1;
            cursor_next<AT_R, AT_BK>(a, c);
          }
        }
      }
    } else if (warp >= AT_LOAD) {
      // ---- K blocks (stages 0, 2, ... of the ring) and V blocks (1, 3, ...),
      // a warp each: a lane's copy takes its warp some 70 cycles to ask for, and
      // pages of 16 tokens make 16 copies a block.  (Four warps in place of two
      // cost the softmax 5 %.)  The K warp also fetches Q at a piece's start,
      // once the last piece's S products are done with it.
      const int kv = warp - AT_LOAD;
      const CUtensorMap* map = kv ? &vmap : &kmap;
      const int boxes = AT_BK / box_rows;
      int st = kv;  // the next block's stage
      uint32_t tails = 0, asked[2] = {0, 0};
      bool ok = true;
      for (int k = 0; ok; ++k) {
        ok = wait(piece_full(k), (k / AT_PIECES) & 1);
        const Piece& p = sh.piece[k % AT_PIECES];
        if (!ok || p.stop) break;
        const int n = max(p.n[0], p.n[1]), h = p.h;
        // Entries of the sequence's row of the table: the lane's own of the 32
        // from e0 on and of the next 32.  (A load per block, even one block
        // ahead, held the warp to a block in 1300 cycles.)
        const int32_t* const table = a.pg.pages + (int64_t)p.b * a.pg.pages_ld;
        auto entries = [&](int e) -> int { return e + lane < a.pg.max_pages ? __ldg(table + e + lane) : -1; };
        int e0 = -(1 << 30), here = -1, there = -1;
        if (kv == 0 && lane == 0) {
          const int tps = a.tile_tokens >> 1;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || p.n[s] == 0) continue;
            if (asked[s] > 0) ok = wait1(q_free(s), (asked[s] + 1) & 1);
            if (!ok) continue;
            mbar_arrive_expect_tx(q_full(s), (uint32_t)(S::CH * 128 * a.group * tps));
            for (int c = 0; c < S::CH; ++c)
              tma_load_3d(q_tile(s) + c * S::HALF, &qmap, 64 * c, h * a.group, p.row0 + p.i0 + s * tps, q_full(s));
            ++asked[s];
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        for (int j = 0; ok && j < n; ++j) {
          const int i = p.first + j, blk0 = (i < p.sink ? i : i - p.sink + p.win) * AT_BK;
          // The block's keys that no row sees start at the sequence's (or the
          // last token's) end, and lie between the sinks and the first window.
          // Where such a border falls within a box, V's rows beyond it are
          // zeroed below: a weight of zero times what lies there may be NaN.
          const int end = p.key_end - blk0, gap0 = a.sinks - blk0, gap1 = p.win_lo - blk0;
          auto within = [&](int x) -> bool { return x > 0 && x < AT_BK && (x & (box_rows - 1)); };
          const bool patch = kv && (within(end) || (gap1 > gap0 && (within(gap1) || within(gap0))));
          // this lane's box: the table's entry and the row in the page
          const int k0 = blk0 + lane * box_rows, e = k0 / a.pg.page_size;
          const int first = __shfl_sync(0xffffffffu, e, 0), last = __shfl_sync(0xffffffffu, e, boxes - 1);
          if (first < e0 || last >= e0 + 64) {
            e0 = first;
            here = entries(e0);
            there = entries(e0 + 32);
          } else if (first >= e0 + 32) {
            e0 += 32;
            here = there;
            there = entries(e0 + 32);
          }
          const int p_here = __shfl_sync(0xffffffffu, here, (e - e0) & 31), p_there = __shfl_sync(0xffffffffu, there, (e - e0) & 31);
          int page = a.pg.num_pages, row = 0;  // beyond the cache: zeros, for a box that no row sees
          if (lane < boxes && k0 < p.key_end && (k0 + box_rows > p.win_lo || k0 < a.sinks)) {
            const int x = e - e0 < 32 ? p_here : p_there;
            row = k0 - e * a.pg.page_size;
            if ((unsigned)x < (unsigned)a.pg.num_pages) page = x;
            else page_error(a.pg);
          }
          const int q = st % NS;
          if (st >= NS) ok = wait(kv_free(q), ((st / NS) + 1) & 1);
          if (!ok) break;
          const uint32_t bar = patch ? tail_bar : kv_full(q), dst = stage(q);
          if (lane == 0) mbar_arrive_expect_tx(bar, S::TILE);
          __syncwarp();
          if (lane < boxes) {
#pragma unroll
            for (int c = 0; c < S::CH; ++c)
              tma_load_4d(dst + c * S::HALF + lane * box_rows * 128, map, 64 * c, row, h, page, bar);
          }
          st += 2;
          if (patch) {
            ok = wait(tail_bar, tails & 1);
            ++tails;
            unsigned char* v = smem + S::OFF_KV + (size_t)q * S::TILE;
            for (int r = lane; r < AT_BK; r += 32)
              if (r >= end || (r >= gap0 && r < gap1))
                for (int c = 0; c < 8 * S::CH; ++c)  // 16 bytes each
                  *reinterpret_cast<uint4*>(v + (c >> 3) * S::HALF + r * 128 + 16 * ((c + r) & 7)) = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(kv_full(q));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(piece_free(k));
      }
      // copies still in flight (only after an abort) land before the CTA ends
      for (int i = max(kv, st - NS); !ok && i < st; i += 2) (void)mbar_wait_bounded(kv_full(i % NS), (i / NS) & 1);
      for (int s = 0; s < 2; ++s)
        if (!ok && lane == 0 && asked[s] > 0) (void)mbar_wait_bounded(q_full(s), (asked[s] - 1) & 1);
    } else if (warp == AT_MMA) {
      // ---- the products, all issued by one lane
      if (elect_one()) {
        int st = 0;
        uint32_t pp[2] = {0, 0}, qq[2] = {0, 0};  // p_full and q_full phases passed
        auto qk = [&](int s, int i, int buf) {  // S = Q_s K^T into buffer buf, K in stage i
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            const uint32_t o = (uint32_t)((ks >> 2) * S::HALF + (ks & 3) * 32);
            at_mma_ss(tbase + 128 * buf, pf_desc_sw128(q_tile(s) + o), pf_desc_sw128(stage(i) + o), at_idesc(128, false), ks > 0);
          }
          tc_commit(s_full(buf));
        };
        // O_s (+)= P V, P in buffer buf, V in stage i; the first 64 keys as soon as their weights are there
        auto pv = [&](int s, int i, int buf, bool add) -> bool {
#pragma unroll
          for (int ks = 0; ks < AT_BK / 16; ++ks) {
            if (ks == 0 || ks == AT_BK / 32) {
              if (!wait1(ks ? p_full(buf) : p_half(buf), pp[buf] & 1)) return false;
              tc_fence_after();
            }
            at_mma_ts(tbase + 256 + DP * s, tbase + 128 * buf + 8 * ks, at_desc_mn(stage(i) + ks * 2048, S::HALF), at_idesc(DP, true),
                      add || ks > 0);
          }
          ++pp[buf];
          return true;
        };
        // a piece with rows in one tile only: S of the next block goes into the
        // other tile's buffer (and uses its barriers), so that the softmax has
        // it when it has finished a block
        auto single = [&](int n) -> bool {
          if (!wait1(q_full(0), qq[0] & 1)) return false;
          ++qq[0];
          for (int j = -1; j < n; ++j) {
            if (j + 1 < n) {
              const int k = st + 2 * (j + 1);
              if (!wait1(kv_full(k % NS), (k / NS) & 1)) return false;
              tc_fence_after();
              qk(0, k % NS, (j + 1) & 1);
              tc_commit(kv_free(k % NS));
              if (j + 2 == n) tc_commit(q_free(0));
            }
            if (j < 0) continue;
            const int v = st + 2 * j + 1;
            if (!wait1(kv_full(v % NS), (v / NS) & 1)) return false;
            tc_fence_after();
            if (!((j & 1) ? pv(0, v % NS, 1, j > 0) : pv(0, v % NS, 0, j > 0))) return false;
            tc_commit(j + 1 == n ? o_full(0) : o_full(1));
            tc_commit(kv_free(v % NS));
          }
          st += 2 * n;
          return true;
        };
        auto products = [&](int n0, int n1) -> bool {  // one piece's
          if (n1 == 0) return single(n0);
          const int nb = max(n0, n1);
          if (!wait1(kv_full(st % NS), (st / NS) & 1)) return false;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int n = s ? n1 : n0;
            if (n == 0) continue;
            if (!wait1(q_full(s), qq[s] & 1)) return false;
            ++qq[s];
            tc_fence_after();
            qk(s, st % NS, s);
            if (n == 1) tc_commit(q_free(s));
          }
          tc_commit(kv_free(st % NS));
          ++st;
          for (int j = 0; j < nb; ++j) {
            const int iv = st % NS, ik = (st + 1) % NS;
            if (!wait1(kv_full(iv), (st / NS) & 1)) return false;
            bool have_k = false;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int n = s ? n1 : n0;
              if (j >= n) continue;
              if (!pv(s, iv, s, j > 0)) return false;
              if (j + 1 == n) {
                if (s == 0) tc_commit(o_full(0));  // the second tile's last block is the piece's (n1 >= n0)
              } else {
                if (!have_k && !wait1(kv_full(ik), ((st + 1) / NS) & 1)) return false;
                have_k = true;
                tc_fence_after();
                qk(s, ik, s);
                if (j + 2 == n) tc_commit(q_free(s));
              }
            }
            tc_commit(kv_free(iv));
            ++st;
            if (j + 1 < nb) {
              tc_commit(kv_free(ik));
              ++st;
            }
          }
          return true;
        };
        for (int k = 0;; ++k) {
          if (!wait1(piece_full(k), (k / AT_PIECES) & 1)) break;
          const Piece& p = sh.piece[k % AT_PIECES];
          if (p.stop) break;
          const int n0 = p.n[0], n1 = p.n[1];
          mbar_arrive(piece_free(k));
          if ((n0 > 0 || n1 > 0) && !products(n0, n1)) break;
          tc_commit(piece_done(k));
        }
        tc_commit(mma_done);  // completes when every MMA issued above has
      }
      __syncwarp();
      (void)mbar_wait_bounded(mma_done, 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---- softmax of tile s, row r
    const int s = warp >> 2, r = tid & 127, G = a.group, tps = a.tile_tokens >> 1;
    const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_o = lanes + 256 + DP * s;
    const float cl = a.scale_log2;
    const int r_tok = r / G, r_head = r - r_tok * G;
    uint32_t sp0 = 0, sp1 = 0, op0 = 0, op1 = 0;  // phases of s_full and o_full that have been (here, or by the other tile's warps)
    for (int k = 0;; ++k) {
      if (!wait(piece_full(k), (k / AT_PIECES) & 1)) break;
      const Piece& p = sh.piece[k % AT_PIECES];
      if (p.stop) break;
      const int tok0 = p.i0 + s * tps, n = p.n[s];
      const int n_first = p.n[0], n_second = p.n[1];
      const bool single = n_second == 0;  // the first tile's blocks alternate between both tiles' buffers of S
      if (tok0 <= p.i1) {  // the tile has rows
        const int tok = tok0 + r_tok;
        const bool row = r < tps * G && tok <= p.i1;
        const int pos = row ? p.base + tok : -1;
        const int pos_first = p.base + tok0, pos_last = p.base + min(tok0 + tps - 1, p.i1);
        float m = -INFINITY;  // reference maximum, in units of scores
        float l = 0.f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
          const int i0 = p.first + j, k0 = (i0 < p.sink ? i0 : i0 - p.sink + p.win) * AT_BK;
          const int buf = single ? j & 1 : s;
          const uint32_t t_s = lanes + 128 * buf;
          ok = wait(s_full(buf), ((buf ? sp1 : sp0) + (single ? j >> 1 : j)) & 1);
          if (!ok) break;
          tc_fence_after();
          uint32_t x[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) at_ld32(t_s + 32 * q, x + 32 * q);
#pragma unroll
          for (int q = 0; q < 4; ++q) at_ld_done32(x + 32 * q);
          // every row sees the whole block, unless it reaches past the first row or out of the last row's window
          const bool clear = k0 + AT_BK - 1 <= pos_first && (a.window == 0 || k0 > pos_last - a.window || k0 + AT_BK <= a.sinks);
          if (!clear) {
            // a bit for each key that the row sees: [lo, hi) and the sinks [0, sk).
            // The empty statement keeps the selects inside the branch (without it
            // every block paid for them: 2200 of a block's 5800 cycles)
            asm volatile("");
            const int hi = pos - k0 + 1, lo = a.window ? hi - a.window : 0, sk = min(a.sinks - k0, hi);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t w = (low_bits(hi - 32 * q) & ~low_bits(lo - 32 * q)) | low_bits(sk - 32 * q);
              if (__all_sync(0xffffffffu, w == 0xFFFFFFFFu)) continue;
              asm volatile("");
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((w >> i) & 1u)) x[32 * q + i] = 0xFF800000u;
            }
          }
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = __uint_as_float(x[q]);
#pragma unroll
          for (int i = 4; i < 124; i += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], __uint_as_float(x[i + q]), __uint_as_float(x[i + 4 + q]));
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], __uint_as_float(x[124 + q]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          if (j == 0) {
            m = top;
          } else if (__any_sync(0xffffffffu, (top - m) * cl > 8.f)) {
            const float mn = fmaxf(m, top);
            const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * cl);
            m = mn;
            l *= f;
            // O is complete up to the last block: with S, unless S runs ahead
            if (single) {
              ok = wait(o_full(1), (op1 + j - 1) & 1);
              if (!ok) break;
              tc_fence_after();
            }
#pragma unroll 1
            for (int q = 0; q < DP / 16; ++q) {
              float v[16];
              uint32_t o[16];
              tc_ld16_wait(t_o + 16 * q, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(v[i] * f);
              at_st16(t_o + 16 * q, o);
            }
          }
          const float b = m == -INFINITY ? 0.f : -m * cl;
          const uint64_t b2 = pair(b, b), c2 = pair(cl, cl);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float u, v;
              unpair(fma2(pair(__uint_as_float(x[32 * q + 2 * i]), __uint_as_float(x[32 * q + 2 * i + 1])), c2, b2), u, v);
              u = ex2(u);
              v = ex2(v);
              sum[i & 1] = add2(sum[i & 1], pair(u, v));
              w[i] = bf16x2(u, v);
            }
            at_st16(t_s + 16 * q, w);
            if (q == 1) {  // half of the second product can start
              at_st_done();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(p_half(buf));
            }
          }
          at_st_done();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(buf));
          float u, v;
          unpair(add2(sum[0], sum[1]), u, v);
          l += u + v;
        }
        if (!ok) break;
        // ---- the piece's rows
        if (n > 0) {
          ok = s ? wait(piece_done(k), (k / AT_PIECES) & 1) : wait(o_full(0), op0 & 1);
          if (!ok) break;
          tc_fence_after();
        }
        const bool whole = p.whole;
        const float f = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
        const int D = a.pg.head_dim, h = p.h * G + r_head;
        const int64_t t = p.row0 + tok;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (p.first == 0 ? 1 : 0);
        // A row's columns lie in one thread; stored from there, 16 bytes of 32
        // rows at a time, they cost the warps 7000 cycles a piece.  A warp's 32
        // rows go through shared memory, 128 bytes of each at a time, as the
        // 128-byte swizzle lays them out (no bank conflicts), and leave in one
        // piece: parts as 4 KB in one bulk copy (the joining kernel undoes the
        // swizzle), full rows of 32 / G whole tokens as one TMA store, others
        // as 16 bytes a lane, 8 lanes a row.
        const int w_tok = tok0 + (warp & 3) * (32 / G);  // the warp's first token, where 32 % G == 0
        const bool tma = whole && 32 % G == 0 && w_tok + 32 / G - 1 <= p.i1;
        unsigned char* const buf = smem + S::OFF_OUT + warp * 4096;
        const int64_t at = t * a.out_stride + (int64_t)h * D;
        const unsigned rows_here = __ballot_sync(0xffffffffu, row);
        auto send = [&](const uint32_t* v, int c0) {  // v: the row's 128 bytes from column c0 on
          if (lane == 0) bulk_reads_done();            // the last ones have left
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (!whole) {
            if (lane == 0) bulk_s2g(a.part_o + (slot * (DP / 32) + c0 / 32) * (AT_R * 32) + warp * (32 * 32), smem_u32(buf), 4096);
          } else if (tma) {
            if (lane == 0) tma_store_3d(&omap, c0, p.h * G, p.row0 + w_tok, smem_u32(buf));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int src = 4 * i + (lane >> 3), col = c0 + 8 * (lane & 7);
              const int64_t to = __shfl_sync(0xffffffffu, at, src) + col;
              if (((rows_here >> src) & 1u) && col < D)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + to) = *reinterpret_cast<const uint4*>(buf + src * 128 + (((lane & 7) ^ (src & 7)) << 4));
            }
          }
        };
        // A decode step's few rows are stored from where they are: the copies
        // above take 1200 cycles each, four of them for a part.
        const bool few = __popc(rows_here) <= 8;
#pragma unroll
        for (int c0 = 0; c0 < DP; c0 += 64) {
          if (rows_here == 0) break;
          uint32_t o[64];
          if (n > 0) {
            at_ld32(t_o + c0, o);
            at_ld32(t_o + c0 + 32, o + 32);
            at_ld_done32(o);
            at_ld_done32(o + 32);
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) o[i] = 0;
          }
          if (whole) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = bf16x2(__uint_as_float(o[2 * i]) * f, __uint_as_float(o[2 * i + 1]) * f);
            if (!few) {
              send(w, c0);
            } else if (row) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (c0 + 8 * i < D)
                  *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at + c0 + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
          } else if (few) {
            if (row) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                *reinterpret_cast<uint4*>(a.part_o + part_at<AT_R, DP>(slot, 128 * s + r, c0 + 4 * i)) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          } else {
            send(o, c0);
            send(o + 32, c0 + 32);
          }
          __syncwarp();
        }
        if (row) {
          const float ml = m == -INFINITY ? m : m * cl;
          if (!whole) a.part_ml[slot * AT_R + 128 * s + r] = make_float2(ml, l);
          else if (a.lse) a.lse[t * a.q_heads + h] = l > 0.f || l != l ? ((m == -INFINITY ? 0.f : ml) + log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
        // the reads of O above come before the next piece's products, which this tile's P allows
        tc_fence_before();
      }
      // The second tile's warps keep to the first one's pieces, which may need
      // nothing of them: the phases of s_full(1) that those use have passed when
      // the piece is done.  (The first tile's warps are kept by S of a piece's
      // first block, which completes after everything before it.)
      if (s == 1 && !wait(piece_done(k), (k / AT_PIECES) & 1)) break;
      sp0 += single ? (n_first + 1) >> 1 : n_first;
      sp1 += single ? n_first >> 1 : n_second;
      op0 += n_first > 0;
      op1 += single ? max(n_first - 1, 0) : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(piece_free(k));
    }
    bulk_done();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == AT_MMA) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tbase));
}

// The tensor map of a cache or of q: `dims` and byte strides from the second
// dimension on, boxes of 64 elements.
bool at_map(CUtensorMap* m, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
            CUtensorMapL2promotion fetch = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, fetch,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens of a box: the largest power of two that divides the page size, at most a block.
int at_box(int page_size) { return std::min(page_size & -page_size, AT_BK); }

template <int DP>
mt_status run_tile(AttnArgs a, void* ws, const Launch& l, const DeviceInfo* di) {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev >= 0 && dev < 64 && !set[dev].load()) {
    e = cudaFuncSetAttribute(attn_tile_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)at_smem<DP>());
    if (e != cudaSuccess) return cuda_fail(e);
    set[dev].store(true);
  }
  const PagedArgs& pg = a.pg;
  const int tps = 128 / a.group, box = at_box(pg.page_size);
  a.tile_tokens = 2 * tps;
  a.min_units = 3;  // no stretch without a block
  CUtensorMap qmap, kmap, vmap, omap;
  const cuuint64_t row = (cuuint64_t)pg.head_dim * 2;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)pg.head_dim, (cuuint64_t)a.q_heads, (cuuint64_t)pg.T};
    const cuuint64_t st[2] = {row, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t bx[3] = {64, (cuuint32_t)a.group, (cuuint32_t)tps};
    if (!at_map(&qmap, a.q, 3, dims, st, bx)) return cuda_fail(cudaErrorInvalidValue);
    // a warp's 32 rows of the output (used where they are whole tokens)
    const cuuint64_t so[2] = {row, (cuuint64_t)a.out_stride * 2};
    const cuuint32_t bo[3] = {64, (cuuint32_t)a.group, (cuuint32_t)std::max(1, 32 / a.group)};
    if (!at_map(&omap, a.out, 3, dims, so, bo)) return cuda_fail(cudaErrorInvalidValue);
  }
  {
    const cuuint64_t dims[4] = {(cuuint64_t)pg.head_dim, (cuuint64_t)pg.page_size, (cuuint64_t)pg.kv_heads, (cuuint64_t)pg.num_pages};
    // a dimension of one entry may have stride 0
    const cuuint64_t st[3] = {pg.token_stride ? (cuuint64_t)pg.token_stride * 2 : row, pg.head_stride ? (cuuint64_t)pg.head_stride * 2 : row,
                              pg.page_stride ? (cuuint64_t)pg.page_stride * 2 : row};
    const cuuint32_t bx[4] = {64, (cuuint32_t)box, 1, 1};
    // A head's rows of 128 bytes that do not follow one another (a token's heads
    // side by side, D = 64): L2 fetches 128 bytes, as 256 would bring another
    // head's row too early (window of 4096 over 32 texts: 65 against 78 us; rows of
    // 256 bytes: 184 against 181 us the other way).
    const auto fetch = pg.head_dim <= 64 && pg.token_stride > 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    if (!at_map(&kmap, pg.k, 4, dims, st, bx, fetch) || !at_map(&vmap, pg.v, 4, dims, st, bx, fetch)) return cuda_fail(cudaErrorInvalidValue);
  }
  const int ctas = di->sm_count;
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.cut = reinterpret_cast<int4*>(w);
  w += (size_t)ctas * 2 * sizeof(int4);
  a.part_ml = reinterpret_cast<float2*>(w);
  w += (size_t)ctas * 2 * AT_R * sizeof(float2);
  a.part_o = reinterpret_cast<float*>(w);
  if (const mt_status st = launch(attn_tile_kernel<DP>, dim3(ctas), dim3(AT_THREADS), at_smem<DP>(), l, qmap, kmap, vmap, omap, a, box)) return st;
  return launch(attn_join_kernel<AT_R, DP>, dim3(ctas, join_blocks(a)), dim3(32 * JOIN_WARPS), 0, l, a);
}

}  // namespace

// This kernel takes every layout that it can, single tokens too: against
// k_attn_rows.cu 176 and 209 us for 48 ragged texts of 32 / 8 heads of 128, 27
// and 37 for 2 of 100 000 with 14 / 2 of 64, 28 and 30 for 8 of 2000 with 16 / 16
// of 128, 12.3 and 12.2 for one of 777, 17 and 36 for a prompt of 300, 77 and 449
// for a chunk beside single tokens.  It cannot take fp32 outputs (weights of one
// bf16), head sizes below 64 or above 128 (its tensor memory's columns), and
// pages that are no multiple of 8 tokens (a box is whole 8-row swizzle atoms).
bool attn_tile_takes(const AttnArgs& a) {
  return !a.out_f32 && a.pg.head_dim >= 64 && a.pg.head_dim <= 128 && at_box(a.pg.page_size) >= 8;
}

size_t attn_tile_ws(int head_dim, int sms) {
  if (head_dim < 64 || head_dim > 128) return 0;
  return (size_t)sms * 2 * (sizeof(int4) + AT_R * (sizeof(float2) + (size_t)(head_dim <= 64 ? 64 : 128) * 4));
}

mt_status launch_attn_tile(AttnArgs a, void* ws, const Launch& l, const DeviceInfo* di) {
  return a.pg.head_dim <= 64 ? run_tile<64>(a, ws, l, di) : run_tile<128>(a, ws, l, di);
}

}  // namespace mt
