// k_probs.cu - mt_token_probs: probabilities of rows of logits under a
// temperature.
//
//   p = e / sum e,  e = exp((x - max x) / t);  t <= 0: 1 at the first largest.
//
// Bound: memory, each logit read and each probability written once; the
// instructions come near it, so that everything is done on two floats at a time.
// A cluster of up to eight blocks shares out a row; its blocks' largest logits,
// sums and first places meet in one exchange through distributed shared memory.
//  * Few rows (token_probs_kernel): the row lies in the blocks' registers, 8 K
//    logits a thread.  9 rows of 151 936 fp32 logits take 5.9 us.
//  * Many (token_probs_loop_kernel): a block passes over its share with a running
//    maximum and sum, and over it again, from L2, for the output: nothing but one
//    exchange stands between the loads and the stores.  448 rows of 128 256 bf16
//    logits: 70 us, 4.9 TB/s; some 5 more without the next vectors on their way.
//    (The first kernel: 100; with clusters that stay and the next row's logits on
//    their way 76, most of it waiting between the steps of a row.)
#include <math.h>

#include <algorithm>

#include "k_cluster.cuh"
#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int PB_THREADS = 512, PB_WARPS = PB_THREADS / 32, PB_MOST = 5;  // most vectors of 8 logits of a thread's registers

struct ProbArgs {
  const char* in;
  float* out;
  int64_t in_ld, out_ld;
  int V;
  const float* temperature;
  int R, blocks;  // blocks of a row
};

// 1 / t in units of log2 e, as a sum of two floats: the exponent's argument, (x -
// base) / t with the difference as fp32 gives it, is off by 2^-40 of itself, not by
// the 2^-23 that would be 2^-17 of a small p.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
struct Scale {
  float hi, lo;
  bool flat;  // a temperature above 2^100: all alike
};
__device__ __forceinline__ Scale log2_scale(float t) {
  constexpr float TOP = 1.2676506e30f;  // 2^100
  Scale s;
  s.flat = t > TOP;
  t = fminf(fmaxf(t, 1.f / TOP), TOP);  // products stay finite
  const float l_hi = 1.44269502f, l_lo = 1.92596303e-8f, r = rcp(t);  // log2 e
  s.hi = l_hi * r;
  s.lo = (fmaf(-s.hi, t, l_hi) + l_lo) * r;  // what is off in r and the product
  return s;
}
// 2^((x - top) c) for x <= top.
__device__ __forceinline__ float exp_scaled(float x, float top, Scale c) {
  if (c.flat) return x > -INFINITY ? 1.f : 0.f;
  const float d = x - top;
  const float y = d * c.hi;
  const float rest = fmaf(d, c.hi, -y) + d * c.lo;  // what y's rounding left
  return y < -160.f ? 0.f : exp2f(y) * fmaf(rest, 0.693147182f, 1.f);
}

template <bool F32>
__device__ __forceinline__ float logit_at(const char* p, int i) {
  return F32 ? reinterpret_cast<const float*>(p)[i] : bf16f(reinterpret_cast<const uint16_t*>(p)[i]);
}
// The larger, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two floats at a time: the kernel would be bound by its instructions.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// The larger of each half, NaN if either is; and not NaN where one is not.
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// Both halves of w plus c, as floats.
__device__ __forceinline__ uint64_t add_bf16x2(uint32_t w, float c) {
  float u, v;
  asm("{\n\t.reg .b16 a0, a1;\n\tmov.b32 {a0, a1}, %2;\n\t"
      "fma.rn.f32.bf16 %0, a0, %3, %4;\n\tfma.rn.f32.bf16 %1, a1, %3, %4;\n\t}"
      : "=f"(u), "=f"(v)
      : "r"(w), "h"((uint16_t)0x3F80), "f"(c));
  return pack2(u, v);
}
// Eight consecutive floats to a 32-byte boundary.
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
               "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Eight consecutive probabilities; `mis`: floats past a 32-byte boundary.
__device__ __forceinline__ void put8(float* to, int mis, const float (&y)[8]) {
  if (mis == 0) {
    store8(to, y);
  } else if (mis == 4) {
    reinterpret_cast<float4*>(to)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) to[i] = y[i];
  }
}

// Pairs of 2^(40 + (x - base) c), x <= base: so that what lies below 2^-126 of the
// largest stays normal.  The argument d c + 40 is y + rest.  y is a multiple of 2^-16
// (d hi + 384 is in [184, 384], where floats are 2^-15 or 2^-16 apart), so that y, 40
// - y and what d hi is beyond them are without a rounding but the last's, which is
// 2^-40 or less; a y rounded to its own step, which is smaller where it is near 0,
// would be lost in 40 - y by up to 2^-17.  (One more addition for two logits: 448
// rows of 128 256 bf16 logits 68 -> 70 us, fp32 ones no change.)
struct Exp2 {
  uint64_t hi, lo;
  float low, c_hi;  // d as small as 2^-200 needs stands for all that is less, -inf too
  __device__ __forceinline__ explicit Exp2(const Scale& c) : hi(pack2(c.hi, c.hi)), lo(pack2(c.lo, c.lo)), low(-200.f * rcp(c.hi)), c_hi(c.hi) {}
  __device__ __forceinline__ uint64_t of(uint64_t d) const {
    const uint64_t y = add2(fma2(d, hi, pack2(384.f, 384.f)), pack2(-344.f, -344.f));
    const uint64_t rest = fma2(d, lo, fma2(d, hi, fma2(y, pack2(-1.f, -1.f), pack2(40.f, 40.f))));
    float u, v;
    unpack2(y, u, v);
    return mul2(pack2(ex2_ftz(u), ex2_ftz(v)), fma2(rest, pack2(0.693147182f, 0.693147182f), pack2(1.f, 1.f)));
  }
  __device__ __forceinline__ uint64_t of(float u, float v, float base) const { return of(pack2(fmaxf(u - base, low), fmaxf(v - base, low))); }
  // Two bf16 logits: the least d stands in bf16, rounded down (least()), which
  // does not do where it would overflow (tame()).
  __device__ __forceinline__ bool tame(float base) const { return fabsf(base) < 1e30f && fabsf(base) * c_hi < 1e37f; }
  __device__ __forceinline__ uint32_t least(float base) const {
    const float x = base + low;
    const uint16_t h = f2bf(x - 0.0078125f * fabsf(x));
    return h | (uint32_t)h << 16;
  }
  __device__ __forceinline__ uint64_t of(uint32_t w, uint32_t least, float base) const { return of(add_bf16x2(max_bf16x2(w, least), -base)); }
};
__device__ __forceinline__ float finite_or_0(float x) { return fabsf(x) < INFINITY ? x : 0.f; }
__device__ __forceinline__ float is_there(float x) { return x > -INFINITY ? 1.f : 0.f; }

// The vectors of a row start at its first 16-byte boundary.  The logits before it,
// and those after the last whole vector, are single ones of the first block.
struct Span {
  int e0, v0, v1, one;
};
template <bool F32>
__device__ __forceinline__ Span span_of(const char* in, int V, int C, int rank) {
  const int tid = threadIdx.x;
  Span s;
  s.e0 = min(V, (int)((16u - ((uint32_t)(uintptr_t)in & 15u)) & 15u) / (F32 ? 4 : 2));
  const int nvec = (V - s.e0) / 8, per = (nvec + C - 1) / C, rest = s.e0 + 8 * nvec;
  s.v0 = min(rank * per, nvec);
  s.v1 = min(s.v0 + per, nvec);
  s.one = rank ? -1 : tid < s.e0 ? tid : tid >= 32 && tid - 32 < V - rest ? rest + tid - 32 : -1;
  return s;
}

// What the blocks of a row, and the warps of a block, come to together.  `sum` is
// of 2^(40 + ..) from the same thread's, warp's or block's `top`; cold rows have
// none, but the first place of the largest.
struct Meeting {
  float top[PB_WARPS], sum[PB_WARPS];
  int first[PB_WARPS];
  __align__(16) uint64_t share[8][2];
};
struct Total {
  float top, sum;
  int first;
};
// From every thread's own (the cluster's first arrival is behind it).
__device__ __forceinline__ Total meet(Meeting& m, float top, float sum, int first, bool warm, const Scale& c, int C, int rank) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto join = [&](int n) {  // over the first n lanes, a power of two
    float all = top;
    for (int o = n / 2; o; o >>= 1) all = max_nan(all, __shfl_xor_sync(0xffffffffu, all, o));
    if (warm) {
      sum *= exp_scaled(top, all, c);
      if (top == -INFINITY) sum = 0.f;
      for (int o = n / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    } else {
      if (top != all) first = 1 << 30;
      for (int o = n / 2; o; o >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
    }
    top = all;
  };
  join(32);
  if (lane == 0) {
    m.top[warp] = top;
    m.sum[warp] = sum;
    m.first[warp] = first;
  }
  __syncthreads();
  if (C > 1) cluster_wait();
  if (warp == 0) {
    top = m.top[lane % PB_WARPS];
    sum = m.sum[lane % PB_WARPS];
    first = m.first[lane % PB_WARPS];
    join(PB_WARPS);
    if (lane < C) {
      const uint64_t lo = (uint64_t)__float_as_uint(top) | ((uint64_t)__float_as_uint(sum) << 32), hi = (uint32_t)first;
      if (C > 1) {
        cluster_put(&m.share[rank][0], lane, lo);
        cluster_put(&m.share[rank][1], lane, hi);
      } else {
        m.share[0][0] = lo;
        m.share[0][1] = hi;
      }
    }
    __syncwarp();
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  const uint64_t lo = m.share[lane % C][0];  // C is a power of two
  top = __uint_as_float((uint32_t)lo);
  sum = __uint_as_float((uint32_t)(lo >> 32));
  first = (int)m.share[lane % C][1];
  join(C);
  return Total{top, sum, first};
}

template <bool F32, int K>
__global__ void __launch_bounds__(PB_THREADS, 2) token_probs_kernel(const ProbArgs a) {
  constexpr int T = PB_THREADS, ES = F32 ? 4 : 2;
  __shared__ Meeting m;
  const int tid = threadIdx.x, C = a.blocks;
  const int rank = C > 1 ? (int)cluster_rank() : 0, r = blockIdx.x / C;
  if (C > 1) cluster_arrive();  // this block runs: the others may write to it
  pdl_wait();
  pdl_trigger();
  const char* in = a.in + (int64_t)r * a.in_ld * ES;
  const float t = a.temperature ? __ldg(a.temperature + r) : 1.f;
  const Span s = span_of<F32>(in, a.V, C, rank);
  float x[K][8], x1 = -INFINITY;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int v = s.v0 + k * T + tid;
    if (v < s.v1) {
      const uint4* src = reinterpret_cast<const uint4*>(in + ((int64_t)s.e0 + 8 * (int64_t)v) * ES);
      const uint4 p = src[0], q = src[F32 ? 1 : 0];
      const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = F32 ? __uint_as_float(w[i]) : i & 1 ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = -INFINITY;
    }
  }
  if (s.one >= 0) x1 = logit_at<F32>(in, s.one);
  const bool warm = t > 0.f;
  const Scale c = log2_scale(t);
  const Exp2 ex(c);

  float top = x1;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; i += 2) top = max_nan(top, x[k][i], x[k][i + 1]);
  // exponentials from the warp's largest, which the output takes a scale from
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f;
  int first = 1 << 30;
  if (!warm) {
    if (x1 == top && s.one >= 0) first = s.one;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 7; i >= 0; --i)
        if (x[k][i] == top) first = min(first, s.e0 + 8 * (s.v0 + k * T + tid) + i);
  } else if (c.flat) {
    sum = x1 = is_there(x1);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[k][i] = is_there(x[k][i]);
  } else {
    const float base = finite_or_0(top);
    uint64_t sums[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint64_t e = ex.of(x[k][i], x[k][i + 1], base);
        sums[i / 2 & 1] = add2(sums[i / 2 & 1], e);
        unpack2(e, x[k][i], x[k][i + 1]);
      }
    float u, v;
    unpack2(ex.of(x1, -INFINITY, base), x1, v);
    unpack2(add2(sums[0], sums[1]), u, v);
    sum = x1 + (u + v);
  }
  const Total all = meet(m, top, sum, first, warm, c, C, rank);

  // a row with NaN or +inf, one with nothing but -inf, one of a single token
  float* out = a.out + (int64_t)r * a.out_ld;
  const int mis = (int)(((uintptr_t)out / 4 + s.e0) & 7);
  const bool bad = !(all.top < INFINITY), some = !bad && all.top > -INFINITY;
  if (warm && some) {
    // in two steps where the scale would be subnormal
    const float f = top > -INFINITY ? exp_scaled(top, all.top, c) : 0.f, inv = __frcp_rn(all.sum);
    const bool whole = f * inv > 1e-37f;
    const float f1 = whole ? f * inv : f, f2 = whole ? 1.f : inv;
    const uint64_t g = pack2(f1, f1), h = pack2(f2, f2);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; i += 2) unpack2(mul2(mul2(pack2(x[k][i], x[k][i + 1]), g), h), x[k][i], x[k][i + 1]);
    x1 = x1 * f1 * f2;
  } else {
    const float fill = bad ? __int_as_float(0x7FFFFFFF) : 0.f;
    const int is = !warm && some ? all.first : -2;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = s.e0 + 8 * (s.v0 + k * T + tid) + i == is ? 1.f : fill;
    x1 = s.one == is ? 1.f : fill;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int v = s.v0 + k * T + tid;
    if (v < s.v1) put8(out + s.e0 + 8 * (int64_t)v, mis, x[k]);
  }
  if (s.one >= 0) out[s.one] = x1;
}

template <bool F32>
__global__ void __launch_bounds__(PB_THREADS, 2) token_probs_loop_kernel(const ProbArgs a) {
  constexpr int T = PB_THREADS, ES = F32 ? 4 : 2, F = F32 ? 2 : 4, Q = F32 ? 8 : 4;  // F vectors of Q words at a time
  __shared__ Meeting m;
  const int tid = threadIdx.x, C = a.blocks;
  const int rank = C > 1 ? (int)cluster_rank() : 0, r = blockIdx.x / C;
  if (C > 1) cluster_arrive();  // this block runs: the others may write to it
  pdl_wait();
  pdl_trigger();
  const char* in = a.in + (int64_t)r * a.in_ld * ES;
  const float t = a.temperature ? __ldg(a.temperature + r) : 1.f;
  const Span s = span_of<F32>(in, a.V, C, rank);
  const bool warm = t > 0.f;
  const Scale c = log2_scale(t);
  const Exp2 ex(c);
  auto load = [&](uint32_t (&w)[F][Q], int v) {
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int q = 0; q < Q / 4; ++q) {
        uint4 p = F32 ? make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u) : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
        if (v + f * T < s.v1) p = *reinterpret_cast<const uint4*>(in + ((int64_t)s.e0 + 8 * (int64_t)(v + f * T)) * ES + 16 * q);
        w[f][4 * q] = p.x;
        w[f][4 * q + 1] = p.y;
        w[f][4 * q + 2] = p.z;
        w[f][4 * q + 3] = p.w;
      }
  };
  auto take = [](uint32_t (&w)[F][Q], const uint32_t (&from)[F][Q]) {
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int q = 0; q < Q; ++q) w[f][q] = from[f][q];
  };
  auto logit = [](const uint32_t (&w)[Q], int i) { return F32 ? __uint_as_float(w[i % Q]) : i & 1 ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]); };

  // ---- the share's largest logit and its sum, a thread's own
  float x1 = s.one >= 0 ? logit_at<F32>(in, s.one) : -INFINITY;
  float top = warm ? x1 : -INFINITY, base = finite_or_0(top), sum = 0.f;
  int first = 1 << 30;
  bool tame = ex.tame(base);
  uint32_t least = ex.least(base);
  if (warm) {
    float none;
    if (c.flat) sum = is_there(x1);
    else unpack2(ex.of(x1, -INFINITY, base), sum, none);
  }
  uint32_t ahead[F][Q];  // the next vectors, on their way
  load(ahead, s.v0 + tid);
#pragma unroll 1
  for (int v = s.v0 + tid; v < s.v1; v += F * T) {
    uint32_t w[F][Q];
    take(w, ahead);
    load(ahead, v + F * T);
    float most = -INFINITY;
    if (F32) {
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int i = 0; i < 8; i += 2) most = max_nan(most, logit(w[f], i), logit(w[f], i + 1));
    } else {
      uint32_t b = w[0][0];
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int i = f ? 0 : 1; i < 4; ++i) b = max_nan_bf16x2(b, w[f][i]);
      most = max_nan(bf16lo(b), bf16hi(b));
    }
    if (!(most <= top)) {
      if (!warm) {
#pragma unroll
        for (int f = F - 1; f >= 0; --f)
#pragma unroll
          for (int i = 7; i >= 0; --i)
            if (logit(w[f], i) == most) first = s.e0 + 8 * (v + f * T) + i;
      } else if (!c.flat) {
        sum = top > -INFINITY ? sum * exp_scaled(top, most, c) : 0.f;
      }
      top = max_nan(top, most);
      base = finite_or_0(top);
      tame = ex.tame(base);
      least = ex.least(base);
    }
    if (!warm) continue;
    if (c.flat) {
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += is_there(logit(w[f], i));
      continue;
    }
    uint64_t sums[2] = {0, 0};
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint64_t e = !F32 && tame ? ex.of(w[f][i / 2 % Q], least, base) : ex.of(logit(w[f], i), logit(w[f], i + 1), base);
        sums[i / 2 & 1] = add2(sums[i / 2 & 1], e);
      }
    float y, z;
    unpack2(add2(sums[0], sums[1]), y, z);
    sum += y + z;
  }
  if (!warm && s.one >= 0) {  // before or behind the vectors
    if (!(x1 < top)) first = x1 == top ? min(first, s.one) : s.one;
    top = max_nan(top, x1);
  }
  const Total all = meet(m, top, sum, first, warm, c, C, rank);

  // ---- the output
  float* out = a.out + (int64_t)r * a.out_ld;
  const int mis = (int)(((uintptr_t)out / 4 + s.e0) & 7);
  const bool bad = !(all.top < INFINITY), some = !bad && all.top > -INFINITY;
  if (!warm || !some) {
    // a row with NaN or +inf, one with nothing but -inf, one of a single token
    const float fill = bad ? __int_as_float(0x7FFFFFFF) : 0.f;
    const int is = !warm && some ? all.first : -2;
#pragma unroll 1
    for (int v = s.v0 + tid; v < s.v1; v += T) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = s.e0 + 8 * v + i == is ? 1.f : fill;
      put8(out + s.e0 + 8 * (int64_t)v, mis, y);
    }
    if (s.one >= 0) out[s.one] = s.one == is ? 1.f : fill;
    return;
  }
  base = all.top;
  tame = ex.tame(base);
  least = ex.least(base);
  const float inv = __frcp_rn(all.sum);
  const uint64_t g = pack2(inv, inv);
  load(ahead, s.v0 + tid);
#pragma unroll 1
  for (int v = s.v0 + tid; v < s.v1; v += F * T) {
    uint32_t w[F][Q];
    take(w, ahead);
    load(ahead, v + F * T);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        if (c.flat) {
          y[i] = is_there(logit(w[f], i)) * inv;
          y[i + 1] = is_there(logit(w[f], i + 1)) * inv;
        } else {
          const uint64_t e = !F32 && tame ? ex.of(w[f][i / 2 % Q], least, base) : ex.of(logit(w[f], i), logit(w[f], i + 1), base);
          unpack2(mul2(e, g), y[i], y[i + 1]);
        }
      }
      if (v + f * T < s.v1) put8(out + s.e0 + 8 * (int64_t)(v + f * T), mis, y);
    }
  }
  if (s.one >= 0) {
    float none;
    if (c.flat) x1 = is_there(x1) * inv;
    else unpack2(mul2(ex.of(x1, -INFINITY, base), g), x1, none);
    out[s.one] = x1;
  }
}

template <bool F32>
mt_status probs_run(ProbArgs a, const Launch& l, int sms) {
  const int nvec = a.V / 8;
  auto per = [&](int C) { return std::max(1, ((nvec + C - 1) / C + PB_THREADS - 1) / PB_THREADS); };  // vectors of a thread
  auto go = [&](auto kernel) {
    const dim3 grid((unsigned)a.R * a.blocks);
    return a.blocks > 1 ? launch_cluster(kernel, a.blocks, grid, dim3(PB_THREADS), 0, l, a) : launch(kernel, grid, dim3(PB_THREADS), 0, l, a);
  };
  // the fewest blocks a row that hold it, more where the rows are few
  a.blocks = 1;
  while (a.blocks < 8 && (per(a.blocks) > PB_MOST || ((int64_t)a.R * a.blocks < sms && per(a.blocks) > 1))) a.blocks *= 2;
  // (64 rows of 50 257 bf16 logits: 7.7 us in registers, 8.6 in two passes; of
  // 128 256, 512 blocks: 16.7 and 15.4; 448 of 4000, a block each: 5.5 and 11.6)
  if (per(a.blocks) <= PB_MOST && (a.blocks == 1 || (int64_t)a.R * a.blocks <= 2 * sms)) {
    switch (per(a.blocks)) {
      case 1: return go(token_probs_kernel<F32, 1>);
      case 2: return go(token_probs_kernel<F32, 2>);
      case 3: return go(token_probs_kernel<F32, 3>);
      case 4: return go(token_probs_kernel<F32, 4>);
      default: return go(token_probs_kernel<F32, PB_MOST>);
    }
  }
  // A share costs as much as its logits and 12 000 more; an SM does two at a time,
  // and one alone is not twice as fast.  (448 rows of 128 256 bf16 logits by 1, 2,
  // 4 and 8 blocks: 74, 70, 83 and 109 us; of 50 257: 32, 39, 53 and 98; 100 rows of
  // 151 936: 30, 29, 28 and 37; 64 of 128 256: 24, 15, 15 and 19.)
  double least = 0;
  for (int C = 1; C <= 8; C *= 2) {
    const int64_t n = ((int64_t)a.R * C + sms - 1) / sms;
    const double cost = (n + (n % 2 ? 0.4 : 0.0)) * (12000.0 + (double)a.V / C);
    if (C == 1 || cost < least) {
      least = cost;
      a.blocks = C;
    }
  }
  return go(token_probs_loop_kernel<F32>);
}

}  // namespace

}  // namespace mt

using namespace mt;

extern "C" mt_status mt_token_probs(const void* logits, int64_t logits_ld, mt_dtype dtype, int R, int V,
                                    const float* temperature, float* probs, int64_t probs_ld, void* stream) {
  if (R != 0 && (!logits || !probs)) return MT_ERR_NULL;
  if (dtype != MT_BF16 && dtype != MT_F32) return MT_ERR_FORMAT;
  if (R < 0 || R > (1 << 22) || V < 1 || V > (1 << 24) || logits_ld < V || probs_ld < V || logits_ld > ((int64_t)1 << 38) ||
      probs_ld > ((int64_t)1 << 38))
    return MT_ERR_SHAPE;
  const int es = dtype == MT_F32 ? 4 : 2;
  if (!aligned_to(logits, es) || !aligned_to(probs, 4) || !aligned_to(temperature, 4)) return MT_ERR_ALIGN;
  const ByteRange ri = byte_range(logits, rows_bytes(R, logits_ld, V, es)), ro = byte_range(probs, rows_bytes(R, probs_ld, V, 4));
  if (ranges_overlap(ri, ro) && !(dtype == MT_F32 && (const void*)probs == logits && (probs_ld == logits_ld || R == 1))) return MT_ERR_ALIAS;
  if (ranges_overlap(byte_range(temperature, (size_t)R * 4), ro)) return MT_ERR_ALIAS;
  if (R == 0) return MT_OK;
  int derr = 0;
  const DeviceInfo* di = device_info(&derr);
  if (!di) return cuda_fail((cudaError_t)derr);
  const ProbArgs a = {(const char*)logits, probs, logits_ld, probs_ld, V, temperature, R, 1};
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  return dtype == MT_F32 ? probs_run<true>(a, l, di->sm_count) : probs_run<false>(a, l, di->sm_count);
}
