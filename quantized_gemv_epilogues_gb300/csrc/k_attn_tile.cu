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
//    which TMA fills with zeros.  Rows beyond the sequence's end in its last
//    page may hold anything: the producer zeroes V's before handing it on (a
//    weight of zero times NaN is NaN).
//  * One softmax warpgroup per tile, one row per thread, so that maxima and
//    sums need no exchange.  The row's reference maximum moves only when a
//    score exceeds it by more than 2^8 (8 in log2 units): fp32 sums and bf16
//    weights lose nothing by weights up to 2^8, and O is rescaled in tensor
//    memory only then - once or twice a row, typically.  When S of block j is
//    complete so is every earlier product of the tile (one thread issues them
//    and they complete in order), so the softmax warps may rescale O without
//    another barrier.
//  * While one tile's softmax runs, the tensor cores work on the other tile:
//    PV0(j) S0(j+1) PV1(j) S1(j+1) is the issue order.
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
constexpr int AT_TMA = 8, AT_MMA = 9, AT_Q = 10;  // warps 0-3 and 4-7: softmax of tile 0 and 1

template <int DP>
struct AtShape {
  static constexpr int CH = DP / 64;                 // 64-element column halves (one 128-byte swizzle row each)
  static constexpr int HALF = 128 * 128;             // 128 rows of 128 bytes
  static constexpr int TILE = CH * HALF;             // a Q tile, or a K or V block
  static constexpr int NS = DP == 128 ? 5 : 10;      // ring stages
  static constexpr size_t OFF_KV = 2 * (size_t)TILE;
  static constexpr size_t SMEM = 1024 + OFF_KV + (size_t)NS * TILE;
  static_assert(SMEM <= 226 * 1024, "shared memory plan");
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
__device__ __forceinline__ void at_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::
               "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                 "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                 "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                 "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
                 "r"(r[31]) : "memory");
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

// Bits [0, n), n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// The piece of a tile that this CTA works on next, as every role sees it.
struct Segment {
  Cursor c;        // c.i: its first block
  long long left;  // units of the CTA's stretch from here on
};
// Blocks of the piece for 128-row tile s of the two (0: none, or no rows).
__device__ __forceinline__ int seg_blocks(const AttnArgs& a, const Segment& g, int s) {
  const int tps = a.tile_tokens >> 1, first = g.c.r.i0 + s * tps;
  if (first > g.c.r.i1) return 0;
  const int last = min(first + tps - 1, g.c.r.i1);
  const int end = (max(g.c.s.kv - g.c.s.n + last + 1, 0) + AT_BK - 1) / AT_BK;
  const int all = min(g.c.t.sink, end) + max(0, end - g.c.t.win);
  return min(max(all - g.c.i, 0), (int)min((long long)(g.c.t.n - g.c.i), g.left));
}
// To the next piece; false at the stretch's end.
__device__ __forceinline__ bool seg_next(const AttnArgs& a, Segment& g) {
  g.left -= g.c.t.n - g.c.i;
  if (g.left <= 0) return false;
  g.c.i = g.c.t.n - 1;
  cursor_next<AT_R, AT_BK>(a, g.c);
  return true;
}

template <int DP>
__global__ void __launch_bounds__(AT_THREADS, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const AttnArgs a, const int box_rows) {
  using S = AtShape<DP>;
  constexpr int NS = S::NS;
  extern __shared__ unsigned char at_raw[];
  unsigned char* smem = at_raw + ((1024u - (smem_u32(at_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bars[2 * NS + 11];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  __shared__ Segment seg_sh[2];  // the softmax warpgroups' pieces (in registers they would displace parts of S)
  __shared__ int more_sh[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto kv_full = [&](int i) { return smem_u32(&bars[i]); };
  auto kv_free = [&](int i) { return smem_u32(&bars[NS + i]); };
  auto s_full = [&](int s) { return smem_u32(&bars[2 * NS + s]); };      // S of a block is in tensor memory
  auto p_full = [&](int s) { return smem_u32(&bars[2 * NS + 2 + s]); };  // P is (and O rescaled)
  auto o_full = [&](int s) { return smem_u32(&bars[2 * NS + 4 + s]); };  // O of the piece is complete
  const uint32_t q_full = smem_u32(&bars[2 * NS + 6]), q_free = smem_u32(&bars[2 * NS + 7]);
  const uint32_t tail_bar = smem_u32(&bars[2 * NS + 8]), mma_done = smem_u32(&bars[2 * NS + 9]);
  auto q_tile = [&](int s) { return smem_u32(smem + (size_t)s * S::TILE); };
  auto stage = [&](int i) { return smem_u32(smem + S::OFF_KV + (size_t)i * S::TILE); };

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(kv_full(i), 1);
      mbar_init(kv_free(i), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 4);  // one arrival per softmax warp
      mbar_init(o_full(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(tail_bar, 1);
    mbar_init(mma_done, 1);
    abort_sh = 0;
    mbar_fence_init();
  }
  if (warp == AT_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_sh)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();
  long long u0, u1, per;
  Segment g;
  plan<AT_R, AT_BK, AT_THREADS>(a, reinterpret_cast<PlanShared*>(smem + S::OFF_KV), blockIdx.x, gridDim.x, &u0, &u1, &per, &g.c);
  g.left = u1 - u0;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the plan's accesses before TMA's to the same memory
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_sh;
  if (tid == 0) a.cut[2 * blockIdx.x].x = -1;
  volatile int* abort_flag = &abort_sh;
  auto fail = [&]() {
    atomicExch(a.pg.err, (int)MT_ERR_TIMEOUT);
    *abort_flag = 1;
  };
  // a warp's bounded wait, one answer for all its lanes
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    const bool ok = mbar_wait_bounded(bar, parity);
    if (__all_sync(0xffffffffu, ok) && !__any_sync(0xffffffffu, *abort_flag)) return true;
    fail();
    return false;
  };

  // a softmax thread holds a row of S, the other warps need few registers:
  // 2 x 128 x 208 + 128 x 80 of the launch's 384 x 168
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (u0 >= u1) {
    } else if (warp == AT_TMA) {
      // ---- K and V blocks
      const int boxes = AT_BK / box_rows;
      int st = 0;             // blocks asked for (K and V each count)
      uint32_t tails = 0;
      bool ok = true;
      do {
        const int n = max(seg_blocks(a, g, 0), seg_blocks(a, g, 1));
        for (int j = 0; ok && j < n; ++j) {
          const int blk = span_block(g.c.t, g.c.i + j);
          // this lane's box
          int page = a.pg.num_pages, row = 0;
          if (lane < boxes) {
            const int k0 = blk * AT_BK + lane * box_rows, k1 = k0 + box_rows;
            if (k0 < g.c.t.key_end && (k1 > g.c.t.win_lo || k0 < a.sinks)) {
              const int e = k0 / a.pg.page_size, p = paged_entry(a.pg, g.c.b, e);
              if (p >= 0) page = p;
              row = k0 - e * a.pg.page_size;
            }
          }
          // rows of the block beyond the sequence's end that a box still reads
          const int tail0 = g.c.s.kv - blk * AT_BK, tail1 = min((tail0 + box_rows - 1) / box_rows * box_rows, AT_BK);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int i = st % NS;
            if (st >= NS) ok = wait(kv_free(i), ((st / NS) + 1) & 1);
            if (!ok) break;
            const bool patch = kv == 1 && tail0 < AT_BK && tail0 > 0 && tail1 > tail0;
            const uint32_t bar = patch ? tail_bar : kv_full(i), dst = stage(i);
            if (lane == 0) mbar_arrive_expect_tx(bar, S::TILE);
            __syncwarp();
            if (lane < boxes) {
#pragma unroll
              for (int c = 0; c < S::CH; ++c)
                tma_load_4d(dst + c * S::HALF + lane * box_rows * 128, kv ? &vmap : &kmap, 64 * c, row, g.c.h, page, bar);
            }
            ++st;
            if (patch) {
              ok = wait(tail_bar, tails & 1);
              ++tails;
              unsigned char* v = smem + S::OFF_KV + (size_t)i * S::TILE;
              for (int x = lane; x < (tail1 - tail0) * 8 * S::CH; x += 32) {
                const int c = x & 7, r = (x >> 3) % (tail1 - tail0), h = (x >> 3) / (tail1 - tail0);
                *reinterpret_cast<uint4*>(v + h * S::HALF + (tail0 + r) * 128 + 16 * c) = make_uint4(0, 0, 0, 0);
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
              if (lane == 0) mbar_arrive(kv_full(i));
              if (!ok) break;
            }
          }
        }
      } while (ok && seg_next(a, g));
      // copies still in flight (only after an abort) land before the CTA ends
      for (int k = max(0, st - NS); !ok && k < st; ++k) (void)mbar_wait_bounded(kv_full(k % NS), (k / NS) & 1);
    } else if (warp == AT_Q) {
      // ---- Q tiles, once the last piece's S products are done with them
      int k = 0;
      bool ok = true;
      do {
        const int n0 = seg_blocks(a, g, 0), n1 = seg_blocks(a, g, 1);
        if (n0 == 0 && n1 == 0) continue;
        if (k > 0) ok = wait(q_free, (k + 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          const int tps = a.tile_tokens >> 1;
          const uint32_t bytes = (uint32_t)(S::CH * 128 * a.group * tps);
          mbar_arrive_expect_tx(q_full, bytes * ((n0 > 0) + (n1 > 0)));
          for (int s = 0; s < 2; ++s)
            if ((s ? n1 : n0) > 0)
              for (int c = 0; c < S::CH; ++c)
                tma_load_3d(q_tile(s) + c * S::HALF, &qmap, 64 * c, g.c.h * a.group, g.c.s.row0 + g.c.r.i0 + s * tps, q_full);
        }
        __syncwarp();
        ++k;
      } while (seg_next(a, g));
      if (!ok && k > 0) (void)mbar_wait_bounded(q_full, (k - 1) & 1);
    } else if (warp == AT_MMA) {
      // ---- the products; the whole warp walks, one elected lane issues
      int st = 0, k = 0;
      uint32_t pp[2] = {0, 0};  // p_full phases passed
      bool ok = true;
      auto qk = [&](int s, int i) {  // S_s = Q_s K^T, K in stage i
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            const uint32_t o = (uint32_t)((ks >> 2) * S::HALF + (ks & 3) * 32);
            at_mma_ss(tbase + 128 * s, pf_desc_sw128(q_tile(s) + o), pf_desc_sw128(stage(i) + o), at_idesc(128, false), ks > 0);
          }
          tc_commit(s_full(s));
        }
        __syncwarp();
      };
      auto commit = [&](uint32_t bar) {
        if (elect_one()) tc_commit(bar);
        __syncwarp();
      };
      do {
        const int n[2] = {seg_blocks(a, g, 0), seg_blocks(a, g, 1)};
        const int nb = max(n[0], n[1]);
        if (nb == 0) continue;
        ok = wait(q_full, k & 1) && wait(kv_full(st % NS), (st / NS) & 1);
        ++k;
        if (!ok) break;
        tc_fence_after();
        for (int s = 0; s < 2; ++s)
          if (n[s] > 0) qk(s, st % NS);
        commit(kv_free(st % NS));
        if (nb == 1) commit(q_free);
        ++st;
        for (int j = 0; ok && j < nb; ++j) {
          const int iv = st % NS, ik = (st + 1) % NS;
          ok = wait(kv_full(iv), (st / NS) & 1);
          bool have_k = false;
          for (int s = 0; ok && s < 2; ++s) {
            if (j >= n[s]) continue;
            ok = wait(p_full(s), pp[s] & 1);
            ++pp[s];
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < AT_BK / 16; ++ks)
                at_mma_ts(tbase + 256 + DP * s, tbase + 128 * s + 8 * ks, at_desc_mn(stage(iv) + ks * 2048, S::HALF),
                          at_idesc(DP, true), j > 0 || ks > 0);
              if (j + 1 == n[s]) tc_commit(o_full(s));
            }
            __syncwarp();
            if (j + 1 < n[s]) {
              if (!have_k) ok = wait(kv_full(ik), ((st + 1) / NS) & 1);
              have_k = true;
              if (!ok) break;
              tc_fence_after();
              qk(s, ik);
            }
          }
          if (!ok) break;
          commit(kv_free(iv));
          ++st;
          if (j + 1 < nb) {
            commit(kv_free(ik));
            ++st;
            if (j + 2 == nb) commit(q_free);
          }
        }
      } while (ok && seg_next(a, g));
      commit(mma_done);  // completes when every MMA issued above has
      (void)mbar_wait_bounded(mma_done, 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if (u0 < u1) {
      // ---- softmax of tile s, row r
      const int s = warp >> 2, r = tid & 127, G = a.group, tps = a.tile_tokens >> 1;
      const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t t_s = lanes + 128 * s, t_o = lanes + 256 + DP * s;
      const float c = a.scale_log2;
      const uint64_t c2 = pair(c, c);
      uint32_t sp = 0, op = 0;  // s_full and o_full phases passed
      bool ok = true;
      const Segment& sg = seg_sh[s];
      if (r == 0) seg_sh[s] = g;
      auto wg_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + s) : "memory"); };
      // the next piece, for the whole warpgroup; false at the end (or after an abort of any of its warps)
      auto advance = [&]() -> bool {
        wg_sync();
        if (r == 0) more_sh[s] = !*abort_flag && seg_next(a, seg_sh[s]);
        wg_sync();
        return more_sh[s] != 0;
      };
      wg_sync();
      do {
        if (!ok) continue;
        const int n = seg_blocks(a, sg, s);
        const int tok0 = sg.c.r.i0 + s * tps;
        if (tok0 > sg.c.r.i1) continue;  // no rows of this tile
        const int tok = tok0 + r / G;
        const bool row = r < tps * G && tok <= sg.c.r.i1;
        const int base = sg.c.s.kv - sg.c.s.n;  // position of the sequence's first new token
        const int pos = row ? base + tok : -1;
        const int pos_first = base + tok0, pos_last = base + min(tok0 + tps - 1, sg.c.r.i1);
        float m = -INFINITY;  // reference maximum, in units of scores
        float l = 0.f;
        for (int j = 0; j < n; ++j) {
          const int k0 = span_block(sg.c.t, sg.c.i + j) * AT_BK;
          ok = wait(s_full(s), sp & 1);
          ++sp;
          if (!ok) break;
          tc_fence_after();
          __syncwarp();
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
          } else if (__any_sync(0xffffffffu, (top - m) * c > 8.f)) {
            const float mn = fmaxf(m, top);
            const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * c);
            m = mn;
            l *= f;
#pragma unroll
            for (int q = 0; q < DP / 32; ++q) {
              uint32_t o[32];
              at_ld32(t_o + 32 * q, o);
              at_ld_done32(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              at_st32(t_o + 32 * q, o);
            }
          }
          const float b = m == -INFINITY ? 0.f : -m * c;
          const uint64_t b2 = pair(b, b);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float u, v;
              unpair(fma2(pair(__uint_as_float(x[32 * q + 2 * i]), __uint_as_float(x[32 * q + 2 * i + 1])), c2, b2), u, v);
              u = ex2(u);
              v = ex2(v);
              sum[i & 1] = add2(sum[i & 1], pair(u, v));
              p[i] = bf16x2(u, v);
            }
            at_st16(t_s + 16 * q, p);
          }
          float u0_, u1_;
          unpair(add2(sum[0], sum[1]), u0_, u1_);
          l += u0_ + u1_;
          at_st_done();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(s));
        }
        if (!ok) continue;
        // ---- the piece's rows
        const bool whole = sg.c.i == 0 && sg.left >= sg.c.t.n;
        if (n > 0) {
          ok = wait(o_full(s), op & 1);
          ++op;
          if (!ok) continue;
          tc_fence_after();
        }
        const float f = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
        const int D = a.pg.head_dim, h = sg.c.h * G + r % G;
        const int64_t t = sg.c.s.row0 + tok;
        const int64_t slot = (2 * (int64_t)blockIdx.x + (sg.c.i == 0 ? 1 : 0)) * AT_R + s * tps * G + r;
#pragma unroll
        for (int q = 0; q < DP / 32; ++q) {
          uint32_t o[32];
          __syncwarp();
          if (n > 0) {
            at_ld32(t_o + 32 * q, o);
            at_ld_done32(o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
          }
          if (row && !whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.part_o + slot * DP + 32 * q);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          } else if (row) {
            uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + t * a.out_stride + (int64_t)h * D + 32 * q;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (32 * q + 8 * i < D) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(o[8 * i + e]) * f;
                *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(bf16x2(y[0], y[1]), bf16x2(y[2], y[3]), bf16x2(y[4], y[5]), bf16x2(y[6], y[7]));
              }
            }
          }
        }
        if (row) {
          const float ml = m == -INFINITY ? m : m * c;
          if (!whole) a.part_ml[slot] = make_float2(ml, l);
          else if (a.lse) a.lse[t * a.q_heads + h] = l > 0.f || l != l ? ((m == -INFINITY ? 0.f : ml) + log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
        if (!whole && sg.c.i == 0 && tid == 0) put_cut(a, blockIdx.x, (int)((u1 - sg.left + sg.c.t.n - 1) / per), sg.c);
        // the reads of O above come before the next piece's products, which this warpgroup's P allows
        tc_fence_before();
      } while (advance());
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == AT_MMA) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tbase));
}

// The tensor map of a cache or of q: `dims` and byte strides from the second
// dimension on, boxes of 64 elements.
bool at_map(CUtensorMap* m, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens of a box: the largest power of two that divides the page size, at most a block.
int at_box(int page_size) { return std::min(page_size & -page_size, AT_BK); }

template <int DP>
mt_status run_tile(AttnArgs a, void* ws, const Launch& l, const DeviceInfo* di) {
  using S = AtShape<DP>;
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev >= 0 && dev < 64 && !set[dev].load()) {
    e = cudaFuncSetAttribute(attn_tile_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM);
    if (e != cudaSuccess) return cuda_fail(e);
    set[dev].store(true);
  }
  const PagedArgs& pg = a.pg;
  const int tps = 128 / a.group, box = at_box(pg.page_size);
  a.tile_tokens = 2 * tps;
  a.min_units = 1;
  CUtensorMap qmap, kmap, vmap;
  const cuuint64_t row = (cuuint64_t)pg.head_dim * 2;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)pg.head_dim, (cuuint64_t)a.q_heads, (cuuint64_t)pg.T};
    const cuuint64_t st[2] = {row, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t bx[3] = {64, (cuuint32_t)a.group, (cuuint32_t)tps};
    if (!at_map(&qmap, a.q, 3, dims, st, bx)) return cuda_fail(cudaErrorInvalidValue);
  }
  {
    const cuuint64_t dims[4] = {(cuuint64_t)pg.head_dim, (cuuint64_t)pg.page_size, (cuuint64_t)pg.kv_heads, (cuuint64_t)pg.num_pages};
    // a dimension of one entry may have stride 0
    const cuuint64_t st[3] = {pg.token_stride ? (cuuint64_t)pg.token_stride * 2 : row, pg.head_stride ? (cuuint64_t)pg.head_stride * 2 : row,
                              pg.page_stride ? (cuuint64_t)pg.page_stride * 2 : row};
    const cuuint32_t bx[4] = {64, (cuuint32_t)box, 1, 1};
    if (!at_map(&kmap, pg.k, 4, dims, st, bx) || !at_map(&vmap, pg.v, 4, dims, st, bx)) return cuda_fail(cudaErrorInvalidValue);
  }
  const int ctas = di->sm_count;
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.cut = reinterpret_cast<int4*>(w);
  w += (size_t)ctas * 2 * sizeof(int4);
  a.part_ml = reinterpret_cast<float2*>(w);
  w += (size_t)ctas * 2 * AT_R * sizeof(float2);
  a.part_o = reinterpret_cast<float*>(w);
  if (const mt_status st = launch(attn_tile_kernel<DP>, dim3(ctas), dim3(AT_THREADS), S::SMEM, l, qmap, kmap, vmap, a, box)) return st;
  return launch(attn_join_kernel<AT_R, DP>, dim3(ctas, 32), dim3(128), 0, l, a);
}

}  // namespace

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
