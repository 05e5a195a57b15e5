// k_attn.cuh - mt_paged_attention: how the work of a batch is shared out over
// the GPU, and the joining of the parts.
//
// Mathematics.  Row r of a tile is one (new token, query head) pair; with
// s_j = scale * q_r . k_j over the visible keys, any set of keys gives a part
// (m, l, o) = (max s_j, sum exp(s_j - m), sum exp(s_j - m) v_j), and parts
// join by (m, sum l_i e^(m_i - m), sum o_i e^(m_i - m)).  The kernels keep m
// in units of log2 e, so that every exponential is an exp2.
//
// Sharing out.  The query heads of one key/value head and the new tokens of
// one sequence are packed into tiles of R rows, which read each key and value
// once for all of their rows.  A tile's visible keys are blocks of BK: those
// with sinks, then those from the first row's window to the last row's
// position.  All (sequence, key/value head, tile, block) units form one line,
// and CTA c of a persistent grid takes the c-th equal stretch of it: lengths
// are only known on the device, sequences differ by orders of magnitude, and
// this balances every mixture to one block.  A tile that a stretch boundary
// cuts leaves parts in the workspace (at most two per CTA), which a second
// kernel joins in key order; the sum's order depends only on the lengths.
// The kernel for chunks weighs its tiles (EXTRA > 0): a tile has EXTRA units
// before its blocks, which stand for the time that its start and its output
// take (a stretch that begins or ends among them begins or ends at the tile's
// first block), and a block is 3 units, or 2 where only one of the two 128-row
// tiles has rows.  (A chunk of 384 beside 15 single tokens: 78 us, and 85 with
// equal blocks, 94 with 3 and 4; a prompt of 8000: 338, 343 and 341 us.)  A
// stretch border within a block leaves the block to the later stretch.
#pragma once
#include <float.h>

#include "k_paged.cuh"

namespace mt {

struct AttnArgs {
  PagedArgs pg;
  const uint16_t* q;
  int64_t q_stride;
  void* out;
  int64_t out_stride;
  float* lse;  // or nullptr
  int out_f32;
  int q_heads, group;
  float scale_log2;  // scale * log2 e
  int window, sinks;
  int tile_tokens;  // tokens of a tile, 0: tiles of packed rows that may start within a token
  int max_q;        // the host's hint
  int min_units;    // fewest blocks of a CTA's stretch
  float* part_o;    // [2 * CTAs][R][DP], or as part_at() says
  float2* part_ml;  // [2 * CTAs][R]
  int4* cut;        // [CTAs][2]: the tile that begins in CTA c's stretch and ends in a later one
};

// The blocks of a tile: block i of n is key block i < sink ? i : i - sink + win.
struct TileSpan {
  int first_pos, last_pos;  // positions of the tile's first and last token
  int key_end;              // keys [0, key_end) reach the last token
  int win_lo;               // first key of the first token's window
  int sink, win, n;
};
template <int BK>
__device__ __forceinline__ TileSpan tile_span(const PagedSeq& s, int i0, int i1, int window, int sinks) {
  TileSpan t;
  t.first_pos = s.kv - s.n + i0;
  t.last_pos = s.kv - s.n + i1;
  t.key_end = max(t.last_pos + 1, 0);
  t.win_lo = window > 0 ? max(t.first_pos - window + 1, 0) : 0;
  const int end = (t.key_end + BK - 1) / BK;
  t.win = min(t.win_lo / BK, end);
  t.sink = (min(sinks, t.key_end) + BK - 1) / BK;
  if (t.win <= t.sink) t.win = t.sink = 0;
  t.n = max(t.sink + end - t.win, 1);  // a tile that sees no key still has its output to write
  return t;
}
__device__ __forceinline__ int span_block(const TileSpan& t, int i) { return i < t.sink ? i : i - t.sink + t.win; }

// Tile rt of a sequence: its first packed row, its rows and its tokens.
struct TileRows {
  int p0, rows, i0, i1;
};
template <int R>
__device__ __forceinline__ TileRows tile_rows(const AttnArgs& a, const PagedSeq& s, int rt) {
  const int per = a.tile_tokens ? a.tile_tokens * a.group : R;
  TileRows t;
  t.p0 = rt * per;
  t.rows = min(per, s.n * a.group - t.p0);
  t.i0 = t.p0 / a.group;
  t.i1 = (t.p0 + t.rows - 1) / a.group;
  return t;
}
template <int R>
__device__ __forceinline__ int tile_count(const AttnArgs& a, const PagedSeq& s) {
  const int per = a.tile_tokens ? a.tile_tokens * a.group : R;
  return (s.n * a.group + per - 1) / per;  // n <= 2^22, group <= 128: within 31 bits
}

template <int EXTRA>
__device__ __forceinline__ int block_units(const AttnArgs& a, const TileRows& r) {
  return EXTRA == 0 ? 1 : r.rows > a.tile_tokens / 2 * a.group ? 3 : 2;
}
template <int R, int BK, int EXTRA>
__device__ __forceinline__ int tile_units(const AttnArgs& a, const PagedSeq& s, int rt) {
  const TileRows r = tile_rows<R>(a, s, rt);
  return EXTRA + block_units<EXTRA>(a, r) * tile_span<BK>(s, r.i0, r.i1, a.window, a.sinks).n;
}

// A position in the line of units.
struct Cursor {
  int b, h, rt, i, tiles;
  PagedSeq s;
  TileSpan t;
  TileRows r;
};

template <int R, int BK>
__device__ __forceinline__ void cursor_tile(const AttnArgs& a, Cursor& c) {
  c.r = tile_rows<R>(a, c.s, c.rt);
  c.t = tile_span<BK>(c.s, c.r.i0, c.r.i1, a.window, a.sinks);
}
// The next unit (there is one).
template <int R, int BK>
__device__ __forceinline__ void cursor_next(const AttnArgs& a, Cursor& c) {
  if (++c.i < c.t.n) return;
  c.i = 0;
  if (++c.rt == c.tiles) {
    c.rt = 0;
    if (++c.h == a.pg.kv_heads) {
      c.h = 0;
      do {
        if (++c.b >= a.pg.B) { c.b = a.pg.B - 1; break; }  // past the end: never used
        c.s = paged_seq(a.pg, c.b);
      } while (c.s.n == 0);
      c.tiles = tile_count<R>(a, c.s);
      if (c.s.n == 0) return;
    }
  }
  cursor_tile<R, BK>(a, c);
}

// a / b for counts: by the 32-bit divider where both fit (a 64-bit division takes
// about a thousand cycles, and the plan needs three of them one after the other).
__device__ __forceinline__ long long div_count(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The plan's shared memory: may overlap what the kernel uses after it.
struct PlanShared {
  long long pre[PG_MAX_B + 1];  // units before each sequence
  long long sum[32];
  int big[PG_MAX_B];
  int n_big;
};

// The head, tile and unit of a sequence's unit `at`, of `each` to a head: by
// every warp for itself, 32 tiles at a time.
template <int R, int BK, int EXTRA>
__device__ __forceinline__ void plan_tile(const AttnArgs& a, Cursor& c, long long each, long long at, int lane) {
  c.tiles = tile_count<R>(a, c.s);
  c.h = (int)div_count(at, each);
  long long rest = at - (long long)c.h * each;
  for (int rt0 = 0; rt0 < c.tiles; rt0 += 32) {
    const int rt = rt0 + lane;
    long long n = 0;
    if (rt < c.tiles) n = tile_units<R, BK, EXTRA>(a, c.s, rt);
    long long in = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, in > rest);
    if (past) {
      const int l = __ffs(past) - 1;
      c.rt = rt0 + l;
      c.i = (int)(rest - __shfl_sync(0xffffffffu, in - n, l));
      break;
    }
    rest -= __shfl_sync(0xffffffffu, in, 31);
  }
  cursor_tile<R, BK>(a, c);
}

// The plan for up to 32 sequences, a lane each, by every warp for itself: no
// barrier and no shared memory.  (A kernel's first instructions run cold, and
// the general plan below takes 6000 cycles, half of a short decode step.)
template <int R, int BK, int EXTRA>
__device__ __forceinline__ void plan_small(const AttnArgs& a, int cta, int ctas, long long* u0, long long* u1, long long* per, Cursor* cur) {
  const PagedArgs& pg = a.pg;
  const int lane = threadIdx.x & 31;
  PagedSeq s = {0, 0, 0};
  if (lane < pg.B) s = paged_seq(pg, lane);
  const int tiles = tile_count<R>(a, s);
  long long n = 0;  // units a head
  if (tiles == 1) n = tile_units<R, BK, EXTRA>(a, s, 0);
  for (unsigned big = __ballot_sync(0xffffffffu, tiles > 1); big; big &= big - 1) {
    const int l = __ffs(big) - 1;
    const PagedSeq x = {__shfl_sync(0xffffffffu, s.row0, l), __shfl_sync(0xffffffffu, s.n, l), __shfl_sync(0xffffffffu, s.kv, l)};
    const int count = __shfl_sync(0xffffffffu, tiles, l);
    long long m = 0;
    for (int rt = lane; rt < count; rt += 32) m += tile_units<R, BK, EXTRA>(a, x, rt);
#pragma unroll
    for (int o = 16; o; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if (lane == l) n = m;
  }
  const long long units = n * pg.kv_heads;
  long long inc = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  const long long total = __shfl_sync(0xffffffffu, inc, 31);
  *per = max(div_count(total + ctas - 1, ctas), (long long)a.min_units);
  *u0 = min((long long)cta * *per, total);
  *u1 = min(*u0 + *per, total);
  Cursor c = {};
  if (*u0 < *u1) {
    const int lo = __ffs(__ballot_sync(0xffffffffu, inc > *u0)) - 1;
    c.b = lo;
    c.s = PagedSeq{__shfl_sync(0xffffffffu, s.row0, lo), __shfl_sync(0xffffffffu, s.n, lo), __shfl_sync(0xffffffffu, s.kv, lo)};
    plan_tile<R, BK, EXTRA>(a, c, __shfl_sync(0xffffffffu, n, lo), *u0 - __shfl_sync(0xffffffffu, inc - units, lo), lane);
  }
  *cur = c;
}

// Units of every sequence, their running sums, and the start of this CTA's
// stretch: [u0, u1) of all units, `per` to a CTA; cur->i counts the tile's
// units, the EXTRA ones first.  Every thread of the block
// (NT of them) calls it and gets the same answers; ends with a barrier.
template <int R, int BK, int NT, int EXTRA>
__device__ void plan(const AttnArgs& a, PlanShared* sh, int cta, int ctas, long long* u0, long long* u1, long long* per,
                     Cursor* cur) {
  const PagedArgs& pg = a.pg;
  if (pg.B <= 32) {
    plan_small<R, BK, EXTRA>(a, cta, ctas, u0, u1, per, cur);
    __syncthreads();
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) sh->n_big = 0;
  __syncthreads();
  // a sequence's units, one thread each; those of many tiles go to the whole block
  for (int b = tid; b < pg.B; b += NT) {
    const PagedSeq s = paged_seq(pg, b);
    const int tiles = tile_count<R>(a, s);
    long long n = 0;
    if (tiles <= 4) {
      for (int rt = 0; rt < tiles; ++rt) n += tile_units<R, BK, EXTRA>(a, s, rt);
    } else {
      sh->big[atomicAdd(&sh->n_big, 1)] = b;
    }
    sh->pre[b + 1] = n * pg.kv_heads;
  }
  __syncthreads();
  for (int k = 0; k < sh->n_big; ++k) {
    const int b = sh->big[k];
    const PagedSeq s = paged_seq(pg, b);
    const int tiles = tile_count<R>(a, s);
    long long n = 0;
    for (int rt = tid; rt < tiles; rt += NT) n += tile_units<R, BK, EXTRA>(a, s, rt);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    // (one per warp: a 64-bit addition to one word by every thread took 13000 cycles)
    if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long*>(&sh->pre[b + 1]), (unsigned long long)(n * pg.kv_heads));
  }
  __syncthreads();
  // running sums: a run of sequences per thread, then over the threads
  const int run = (pg.B + NT - 1) / NT, b0 = min(tid * run, pg.B), b1 = min(b0 + run, pg.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += sh->pre[b + 1];
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh->sum[warp] = inc;
  __syncthreads();
  long long base = inc - mine;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) base += w < warp ? sh->sum[w] : 0;
  for (int b = b0; b < b1; ++b) {
    base += sh->pre[b + 1];
    sh->pre[b + 1] = base;
  }
  if (tid == 0) sh->pre[0] = 0;
  __syncthreads();
  const long long total = sh->pre[pg.B];
  *per = max(div_count(total + ctas - 1, ctas), (long long)a.min_units);
  *u0 = min((long long)cta * *per, total);
  *u1 = min(*u0 + *per, total);
  Cursor c = {};
  if (*u0 < *u1) {
    int lo = 0, hi = pg.B;  // the sequence with pre[lo] <= u0 < pre[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh->pre[mid] <= *u0) lo = mid;
      else hi = mid;
    }
    c.b = lo;
    c.s = paged_seq(pg, lo);
    plan_tile<R, BK, EXTRA>(a, c, div_count(sh->pre[lo + 1] - sh->pre[lo], pg.kv_heads), *u0 - sh->pre[lo], lane);
  }
  *cur = c;
  __syncthreads();
}

// Records the tile that begins in CTA `cta`'s stretch and ends in CTA `last`'s
// (or none): what the joining kernel needs to write its rows.
__device__ __forceinline__ void put_cut(const AttnArgs& a, int cta, int last, const Cursor& c) {
  a.cut[2 * cta] = make_int4(last, c.s.row0, c.h, c.r.p0);
  a.cut[2 * cta + 1] = make_int4(c.r.rows, 0, 0, 0);
}

__device__ __forceinline__ float exp2_(float x) { return exp2f(x); }

// Where column d of row r of a part lies, in floats.  The kernel for chunks
// (R = 256) writes 32 columns of 32 rows at a time, as 128-byte rows whose
// 16-byte chunks are swizzled, and its second tile's rows from 128 on.
template <int R, int DP>
__device__ __forceinline__ int64_t part_at(int64_t slot, int r, int d) {
  if (R == 16) return (slot * R + r) * DP + d;
  return (slot * (DP / 32) + d / 32) * (R * 32) + r * 32 + ((((d >> 2) & 7) ^ (r & 7)) << 2) + (d & 3);
}

// Joins the tile cut at the end of CTA x's stretch.  A warp takes two rows at a
// time, V columns a lane: the loads of both rows' parts are in flight
// together.  Where a tile has more than eight parts, the block's eight warps
// share out those of one row, and add up in order.
constexpr int JOIN_WARPS = 8;
template <int R, int DP>
__global__ void __launch_bounds__(32 * JOIN_WARPS) attn_join_kernel(const AttnArgs a) {
  constexpr int V = DP / 32;
  __shared__ float o_sh[JOIN_WARPS][DP];
  __shared__ float2 ml_sh[JOIN_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.pg.head_dim, c0 = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int4 k0 = a.cut[2 * c0];
  const int rows = a.cut[2 * c0 + 1].x;
  const int c1 = k0.x;
  if (c1 <= c0) return;
  const int parts = c1 - c0 + 1;
  const int half = a.tile_tokens / 2 * a.group;
  struct Row {
    float m, l, o[V];
  };
  auto clear = [&](Row& x) {
    x.m = -INFINITY;
    x.l = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) x.o[i] = 0.f;
  };
  auto load = [&](int p, int r, float2& ml, float (&v)[V]) {
    const int64_t slot = 2 * (int64_t)(c0 + p) + (p == 0 ? 1 : 0);
    const int at = R != 16 && r >= half ? r - half + R / 2 : r;  // the row's place in the parts
    ml = a.part_ml[slot * R + at];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float* src = a.part_o + part_at<R, DP>(slot, at, V * lane + i);
      if (V == 2) {
        *reinterpret_cast<float2*>(&v[0]) = *reinterpret_cast<const float2*>(src);
      } else {
        const float4 q = *reinterpret_cast<const float4*>(src);
        v[i] = q.x;
        v[i + 1] = q.y;
        v[(i + 2) % V] = q.z;
        v[(i + 3) % V] = q.w;
      }
    }
  };
  auto add = [&](Row& x, const float2 ml, const float (&v)[V]) {
    const float mn = fmaxf(x.m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
    const float f0 = exp2_(x.m - ms), f1 = exp2_(ml.x - ms);
    x.l = x.l * f0 + ml.y * f1;
#pragma unroll
    for (int i = 0; i < V; ++i) x.o[i] = x.o[i] * f0 + v[i] * f1;
    x.m = mn;
  };
  auto write = [&](int r, const Row& x) {
    const bool any = x.l > 0.f || x.l != x.l;
    const float inv = any ? 1.f / x.l : 0.f;
    const int pr = k0.w + r, t = k0.y + pr / a.group, h = k0.z * a.group + pr % a.group;
    const int64_t at = (int64_t)t * a.out_stride + (int64_t)h * D;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const int d = V * lane + i;  // D is even
      if (d < D) {
        const float y0 = x.o[i] * inv, y1 = x.o[i + 1] * inv;
        if (a.out_f32) *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at + d) = make_float2(y0, y1);
        else *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out) + at + d) = (uint32_t)f2bf(y0) | ((uint32_t)f2bf(y1) << 16);
      }
    }
    if (lane == 0 && a.lse) a.lse[(int64_t)t * a.q_heads + h] = any ? ((x.m == -INFINITY ? 0.f : x.m) + log2f(x.l)) * 0.6931471805599453f : -INFINITY;
  };
  if (parts <= 8) {
    const int step = JOIN_WARPS * gridDim.y;
    for (int r = blockIdx.y * JOIN_WARPS + warp; r < rows; r += 2 * step) {
      const bool two = r + step < rows;
      const int r2 = two ? r + step : r;
      Row x, y;
      clear(x);
      clear(y);
#pragma unroll 2
      for (int p = 0; p < parts; ++p) {
        float2 ma, mb;
        float va[V], vb[V];
        load(p, r, ma, va);
        load(p, r2, mb, vb);
        add(x, ma, va);
        add(y, mb, vb);
      }
      write(r, x);
      if (two) write(r2, y);
    }
    return;
  }
  const int per = (parts + JOIN_WARPS - 1) / JOIN_WARPS, p0 = min(parts, warp * per), p1 = min(parts, p0 + per);
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    Row x;
    clear(x);
#pragma unroll 8
    for (int p = p0; p < p1; ++p) {
      float2 ml;
      float v[V];
      load(p, r, ml, v);
      add(x, ml, v);
    }
    __syncthreads();
    if (lane == 0) ml_sh[warp] = make_float2(x.m, x.l);
#pragma unroll
    for (int i = 0; i < V; ++i) o_sh[warp][V * lane + i] = x.o[i];
    __syncthreads();
    if (warp) continue;
    clear(x);
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) {
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = o_sh[w][V * lane + i];
      add(x, ml_sh[w], v);
    }
    write(r, x);
  }
}

// Blocks of the joining kernel for each cut: as many as a tile has rows, as far
// as the host knows (each block strides over them), but at most 16: blocks that
// find nothing to join still cost their launch.
inline int join_blocks(const AttnArgs& a) {
  const int64_t rows = (int64_t)(a.max_q > 0 ? a.max_q : 1) * a.group;
  return (int)(rows < 8 ? rows : rows < 64 ? 8 : 16);
}

// Launchers (k_attn_rows.cu, k_attn_tile.cu): the main kernel and the join.
mt_status launch_attn_rows(AttnArgs a, void* ws, const Launch& l, const DeviceInfo* di);
size_t attn_rows_ws(int head_dim, int sms);
mt_status launch_attn_tile(AttnArgs a, void* ws, const Launch& l, const DeviceInfo* di);
size_t attn_tile_ws(int head_dim, int sms);
bool attn_tile_takes(const AttnArgs& a);

}  // namespace mt
