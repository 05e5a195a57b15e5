// k_attn_rows.cu - attention over a paged cache for the layouts that the chunk
// kernel (k_attn_tile.cu) does not take: fp32 outputs, head sizes below 64 or
// above 128, pages that are no multiple of 8 tokens.
//
// Bound: memory for single tokens.  A key and its value (4 D bytes) are read
// once for 16 rows, so a CTA does 16 * 4 D flops for 4 D bytes: 48 ragged texts
// of 32 / 8 heads of 128, 209 us (5.2 TB/s) where the chunk kernel takes 176.
// Prompts read the keys again for every 16 rows and are bound by mma.sync: one
// of 3000 tokens 1029 us, 78 in the chunk kernel.  The products run on
// mma.sync m16n8k16 (16 rows is its whole M, and rows of any head size and
// pages of any length reach its fragments), each of the
// four warps over its own 16 of a block's 64 keys with its own running
// maximum and sum, joined through shared memory at the tile's end.  K and V
// blocks come by 16-byte cp.async into a ring of ST stages, which runs on
// across tiles; page indices are fetched a block ahead of the copies that
// need them.  (Head size 256: 255 registers and 84 bytes of spills.)  P enters the second product as bf16 hi + lo (2^-16 of each
// weight; the tensor pipe has the time).
#include <math.h>

#include <atomic>

#include "k_attn.cuh"

namespace mt {

namespace {

constexpr int AR_R = 16, AR_BK = 64, AR_THREADS = 128;

template <int DP>
struct ArShape {
  static constexpr int ROWB = DP * 2;               // bytes of a key's row in shared memory
  static constexpr int HALF = AR_BK * ROWB;         // K (or V) of a block
  static constexpr int ST = DP == 64 ? 4 : 3;       // ring stages
  static constexpr int PER_SM = DP == 64 ? 3 : DP == 128 ? 2 : 1;  // CTAs an SM holds
  static constexpr size_t RING = (size_t)ST * 2 * HALF;
  static constexpr size_t RED = 4 * 16 * 32 * 4;    // four warps' 32 columns of 16 rows
  static constexpr size_t SMEM = 128 + RING + RED;
  static_assert(RING >= sizeof(PlanShared), "the plan uses the ring's memory");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// Two floats as bf16x2 (round to nearest), and what rounding left of them.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const uint16_t hx = f2bf(x), hy = f2bf(y);
  hi = (uint32_t)hx | ((uint32_t)hy << 16);
  lo = (uint32_t)f2bf(x - bf16f(hx)) | ((uint32_t)f2bf(y - bf16f(hy)) << 16);
}

template <int DP>
__global__ void __launch_bounds__(AR_THREADS, ArShape<DP>::PER_SM) attn_rows_kernel(const AttnArgs a) {
  using S = ArShape<DP>;
  constexpr int ST = S::ST, CPR = DP / 8, NT8 = DP / 8;
  extern __shared__ __align__(128) unsigned char ar_smem[];
  __shared__ int64_t off_sh[2][AR_BK];  // element offset of each key's row in the cache, -1: zeros
  __shared__ float2 ml_sh[4][AR_R];
  unsigned char* ring = ar_smem;
  float* red = reinterpret_cast<float*>(ar_smem + S::RING);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int cta = blockIdx.x, ctas = gridDim.x, D = a.pg.head_dim, G = a.group;

  pdl_wait();
  pdl_trigger();
  long long u0, u1, per;
  Cursor ld;  // of the block whose page indices are fetched next
  plan<AR_R, AR_BK, AR_THREADS, 0>(a, reinterpret_cast<PlanShared*>(ring), cta, ctas, &u0, &u1, &per, &ld);
  if (tid == 0) a.cut[2 * cta].x = -1;
  if (u0 >= u1) return;
  const int units = (int)(u1 - u0);

  // key `tid` (< 64) of the cursor's block: its row's offset, or -1 if no row of the tile sees it
  auto fetch = [&](const Cursor& c) -> int64_t {
    const int key = span_block(c.t, c.i) * AR_BK + tid;
    if (tid >= AR_BK || key >= c.t.key_end || (key < c.t.win_lo && key >= a.sinks)) return -1;
    const int e = key / a.pg.page_size, page = paged_entry(a.pg, c.b, e);
    if (page < 0) return -1;
    return (int64_t)page * a.pg.page_stride + (int64_t)(key - e * a.pg.page_size) * a.pg.token_stride +
           (int64_t)c.h * a.pg.head_stride;
  };
  auto issue = [&](int u) {  // copies of block u, whose offsets are in off_sh[u & 1]
    unsigned char* kb = ring + (size_t)(u % ST) * 2 * S::HALF;
    const uint32_t kd = smem_u32(kb);
#pragma unroll
    for (int j = 0; j < AR_BK * CPR / AR_THREADS; ++j) {
      const int x = j * AR_THREADS + tid, row = x / CPR, ch = x % CPR;
      const int64_t off = off_sh[u & 1][row];
      const bool there = off >= 0 && 8 * ch < D;
      const int64_t at = there ? off + 8 * ch : 0;
      const uint32_t d = kd + (uint32_t)(row * S::ROWB + ((ch ^ (row & 7)) << 4));
      cp_async16_zfill(d, a.pg.k + at, there);
      cp_async16_zfill(d + S::HALF, a.pg.v + at, there);
    }
  };

  Cursor cc = ld;  // of the block that is computed
  // blocks 0 .. ST - 2 on their way, the offsets of block ST - 1 stored
  for (int u = 0; u < ST; ++u) {
    if (u < units) {
      const int64_t off = fetch(ld);
      if (tid < AR_BK) off_sh[u & 1][tid] = off;
      if (u + 1 < units) cursor_next<AR_R, AR_BK>(a, ld);
    }
    __syncthreads();
    if (u < ST - 1) {
      if (u < units) issue(u);
      cp_async_commit();
    }
    // the next store goes to the other half; the one after it is ordered by
    // the barrier of the next round
  }

  uint32_t qf[DP / 16][4];
  float o[NT8][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // of rows g and g + 8
  int i_first = cc.i;
  bool fresh = true;
  int pos0 = 0, pos1 = 0;
  for (int u = 0; u < units; ++u) {
    if (fresh) {  // a new tile: its rows of Q
      fresh = false;
      i_first = cc.i;
      const int r0 = cc.r.p0 + g, r1 = r0 + 8;
      const bool h0 = g < cc.r.rows, h1 = g + 8 < cc.r.rows;
      const uint16_t* q0 = a.q + (int64_t)(cc.s.row0 + (h0 ? r0 / G : 0)) * a.q_stride + (int64_t)(cc.h * G + (h0 ? r0 % G : 0)) * D;
      const uint16_t* q1 = a.q + (int64_t)(cc.s.row0 + (h1 ? r1 / G : 0)) * a.q_stride + (int64_t)(cc.h * G + (h1 ? r1 % G : 0)) * D;
      pos0 = h0 ? cc.s.kv - cc.s.n + r0 / G : -1;
      pos1 = h1 ? cc.s.kv - cc.s.n + r1 / G : -1;
#pragma unroll
      for (int ks = 0; ks < DP / 16; ++ks) {
        const int c = ks * 16 + 2 * tq;
        qf[ks][0] = h0 && c < D ? *reinterpret_cast<const uint32_t*>(q0 + c) : 0u;
        qf[ks][1] = h1 && c < D ? *reinterpret_cast<const uint32_t*>(q1 + c) : 0u;
        qf[ks][2] = h0 && c + 8 < D ? *reinterpret_cast<const uint32_t*>(q0 + c + 8) : 0u;
        qf[ks][3] = h1 && c + 8 < D ? *reinterpret_cast<const uint32_t*>(q1 + c + 8) : 0u;
      }
#pragma unroll
      for (int n = 0; n < NT8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
    __syncthreads();  // block u is in shared memory, and every warp is done with block u - 1
    if (u + ST - 1 < units) issue(u + ST - 1);
    cp_async_commit();
    int64_t off_next = -1;
    const bool more = u + ST < units;
    if (more) {
      off_next = fetch(ld);
      if (u + ST + 1 < units) cursor_next<AR_R, AR_BK>(a, ld);
    }

    const uint32_t kb = smem_u32(ring + (size_t)(u % ST) * 2 * S::HALF), vb = kb + S::HALF;
    const int mi = lane >> 3, lr = lane & 7;
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    {
      const int row = warp * 16 + (mi >> 1) * 8 + lr;
      const uint32_t base = kb + (uint32_t)(row * S::ROWB);
#pragma unroll
      for (int ks = 0; ks < DP / 16; ++ks) {
        uint32_t b[4];
        ldsm4(base + (((ks * 2 + (mi & 1)) ^ lr) << 4), b);
        mma_bf16(s[0], qf[ks], b[0], b[1]);
        mma_bf16(s[1], qf[ks], b[2], b[3]);
      }
    }
    const int key0 = span_block(cc.t, cc.i) * AR_BK + warp * 16 + 2 * tq;
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = key0 + 8 * n + e;
        const bool v0 = key <= pos0 && (a.window == 0 || key > pos0 - a.window || key < a.sinks);
        const bool v1 = key <= pos1 && (a.window == 0 || key > pos1 - a.window || key < a.sinks);
        s[n][e] = v0 ? s[n][e] * a.scale_log2 : -INFINITY;
        s[n][2 + e] = v1 ? s[n][2 + e] * a.scale_log2 : -INFINITY;
        x0 = fmaxf(x0, s[n][e]);
        x1 = fmaxf(x1, s[n][2 + e]);
      }
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
    }
    const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
    if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1)) {
      const float f0 = n0 == -INFINITY ? 1.f : exp2_(m0 - n0), f1 = n1 == -INFINITY ? 1.f : exp2_(m1 - n1);
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int n = 0; n < NT8; ++n) {
        o[n][0] *= f0;
        o[n][1] *= f0;
        o[n][2] *= f1;
        o[n][3] *= f1;
      }
      m0 = n0;
      m1 = n1;
    }
    const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        p[e] = exp2_(s[n][e] - b0);
        p[2 + e] = exp2_(s[n][2 + e] - b1);
      }
      l0 += p[0] + p[1];
      l1 += p[2] + p[3];
      split2(p[0], p[1], ph[2 * n], pl[2 * n]);
      split2(p[2], p[3], ph[2 * n + 1], pl[2 * n + 1]);
    }
    {
      const int row = warp * 16 + (mi & 1) * 8 + lr;
      const uint32_t base = vb + (uint32_t)(row * S::ROWB);
#pragma unroll
      for (int n = 0; n < NT8 / 2; ++n) {
        uint32_t b[4];
        ldsm4t(base + (((2 * n + (mi >> 1)) ^ lr) << 4), b);
        mma_bf16(o[2 * n], ph, b[0], b[1]);
        mma_bf16(o[2 * n], pl, b[0], b[1]);
        mma_bf16(o[2 * n + 1], ph, b[2], b[3]);
        mma_bf16(o[2 * n + 1], pl, b[2], b[3]);
      }
    }
    // offsets of block u + ST into the half that block u + ST - 2 used: its
    // copies were issued before this step's barrier
    if (more && tid < AR_BK) off_sh[(u + ST) & 1][tid] = off_next;

    const bool tile_done = cc.i + 1 == cc.t.n;
    if (tile_done || u + 1 == units) {
      // join the warps: maxima and sums first, then 32 columns at a time
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, w);
        l1 += __shfl_xor_sync(0xffffffffu, l1, w);
      }
      if (tq == 0) {
        ml_sh[warp][g] = make_float2(m0, l0);
        ml_sh[warp][g + 8] = make_float2(m1, l1);
      }
      __syncthreads();
      auto joined = [&](int r, float* l) -> float {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, ml_sh[w][r].x);
        const float ms = M == -INFINITY ? 0.f : M;
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) L += ml_sh[w][r].y * exp2_(ml_sh[w][r].x - ms);
        *l = L;
        return M;
      };
      float La, Lb;
      const float Ma = joined(g, &La), Mb = joined(g + 8, &Lb);
      const float fa = Ma == -INFINITY ? 0.f : exp2_(m0 - Ma), fb = Mb == -INFINITY ? 0.f : exp2_(m1 - Mb);
      const bool whole = tile_done && i_first == 0;
      const int rr = tid >> 3, cq = tid & 7;  // this thread's row and column quad of the joined 32 columns
      float Lr;
      const float Mr = joined(rr, &Lr);
      const float inv = whole ? (Lr > 0.f || Lr != Lr ? 1.f / Lr : 0.f) : 1.f;
      const int pr = cc.r.p0 + rr, t = cc.s.row0 + pr / G, h = cc.h * G + pr % G;
      const int64_t slot = 2 * (int64_t)cta + (i_first == 0 ? 1 : 0);
#pragma unroll
      for (int cb = 0; cb < DP / 32; ++cb) {
        __syncthreads();
        float* w = red + warp * 16 * 32;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int col = 8 * n + 2 * tq;
          const float(&x)[4] = o[4 * cb + n];
          // columns rotated by the row: rows g and g + 4 share banks otherwise
          *reinterpret_cast<float2*>(w + g * 32 + ((col + 4 * g) & 31)) = make_float2(x[0] * fa, x[1] * fa);
          *reinterpret_cast<float2*>(w + (g + 8) * 32 + ((col + 4 * g) & 31)) = make_float2(x[2] * fb, x[3] * fb);
        }
        __syncthreads();
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 y = *reinterpret_cast<const float4*>(red + (k * 16 + rr) * 32 + ((4 * cq + 4 * (rr & 7)) & 31));
          v.x += y.x;
          v.y += y.y;
          v.z += y.z;
          v.w += y.w;
        }
        const int d = cb * 32 + 4 * cq;
        if (rr < cc.r.rows) {
          if (!whole) {
            *reinterpret_cast<float4*>(a.part_o + (slot * AR_R + rr) * DP + d) = v;
          } else if (d < D) {
            const int64_t at = (int64_t)t * a.out_stride + (int64_t)h * D + d;
            if (a.out_f32)
              *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            else
              *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
                  make_uint2((uint32_t)f2bf(v.x * inv) | ((uint32_t)f2bf(v.y * inv) << 16),
                             (uint32_t)f2bf(v.z * inv) | ((uint32_t)f2bf(v.w * inv) << 16));
          }
        }
      }
      if (cq == 0 && rr < cc.r.rows) {
        if (!whole) a.part_ml[slot * AR_R + rr] = make_float2(Mr, Lr);
        else if (a.lse)
          a.lse[(int64_t)t * a.q_heads + h] =
              Lr > 0.f || Lr != Lr ? ((Mr == -INFINITY ? 0.f : Mr) + log2f(Lr)) * 0.6931471805599453f : -INFINITY;
      }
      if (!tile_done && i_first == 0 && tid == 0)
        put_cut(a, cta, (int)div_count(u0 + u + (cc.t.n - 1 - cc.i), per), cc);
      fresh = true;
    }
    if (u + 1 < units) cursor_next<AR_R, AR_BK>(a, cc);
  }
  cp_async_wait_all();
}

int ar_ctas(int dp, int sms) { return sms * (dp == 64 ? 3 : dp == 128 ? 2 : 1); }
int ar_dp(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

template <int DP>
mt_status run_rows(AttnArgs a, void* ws, const Launch& l, const DeviceInfo* di) {
  using S = ArShape<DP>;
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev >= 0 && dev < 64 && !set[dev].load()) {
    e = cudaFuncSetAttribute(attn_rows_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM);
    if (e != cudaSuccess) return cuda_fail(e);
    set[dev].store(true);
  }
  const int ctas = ar_ctas(DP, di->sm_count);
  a.tile_tokens = 0;
  a.min_units = 2;
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.cut = reinterpret_cast<int4*>(w);
  w += (size_t)ctas * 2 * sizeof(int4);
  a.part_ml = reinterpret_cast<float2*>(w);
  w += (size_t)ctas * 2 * AR_R * sizeof(float2);
  a.part_o = reinterpret_cast<float*>(w);
  if (const mt_status st = launch(attn_rows_kernel<DP>, dim3(ctas), dim3(AR_THREADS), S::SMEM, l, a)) return st;
  return launch(attn_join_kernel<AR_R, DP>, dim3(ctas, join_blocks(a)), dim3(32 * JOIN_WARPS), 0, l, a);
}

}  // namespace

size_t attn_rows_ws(int head_dim, int sms) {
  const int dp = ar_dp(head_dim);
  return (size_t)ar_ctas(dp, sms) * 2 * (sizeof(int4) + AR_R * (sizeof(float2) + (size_t)dp * 4));
}

mt_status launch_attn_rows(AttnArgs a, void* ws, const Launch& l, const DeviceInfo* di) {
  switch (ar_dp(a.pg.head_dim)) {
    case 64: return run_rows<64>(a, ws, l, di);
    case 128: return run_rows<128>(a, ws, l, di);
    default: return run_rows<256>(a, ws, l, di);
  }
}

}  // namespace mt
