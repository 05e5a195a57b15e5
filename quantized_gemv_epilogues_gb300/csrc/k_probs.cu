// k_probs.cu - mt_token_probs: probabilities of rows of logits under a
// temperature.
//
//   p = e / sum e,  e = exp((x - max x) / t);  t <= 0: 1 at the first largest.
//
// Bound: memory, each logit read and each probability written once.  A row lies
// in the registers of a cluster of up to eight blocks, 8 K logits a thread, so
// that it is read once; each block takes its exponentials from its own largest
// logit, and the blocks' largest logits, sums and first places meet in one
// exchange through distributed shared memory, after which a block's share is
// scaled by 2^((its largest - the row's) c).
#include <math.h>

#include <algorithm>
#include <atomic>

#include "k_cluster.cuh"
#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int PB_THREADS = 512, PB_MOST = 5;  // threads of a block, most vectors of 8 logits of one

struct ProbArgs {
  const char* in;
  float* out;
  int64_t in_ld, out_ld;
  int V;
  const float* temperature;
  int R;
  int blocks, log2_blocks;  // of a row
};

// 1 / t in units of log2 e, as a sum of two floats: the exponent's argument is
// off by 2^-40 of itself, not by the 2^-23 that would be 2^-17 of a small p.
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

// The same without results below 2^-126, for parts of a row: 2^((x - top) c) for
// x <= top, 0 for x = -inf.
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_part(float x, float top, Scale c) {
  if (c.flat) return x > -INFINITY ? 1.f : 0.f;
  const float d = x - top, y = d * c.hi, rest = fmaf(d, c.lo, fmaf(d, c.hi, -y));
  return y > -126.f ? ex2_ftz(y) * fmaf(rest, 0.693147182f, 1.f) : 0.f;
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

template <bool F32, int K, int T>
__global__ void __launch_bounds__(T, T <= 512 ? 2 : 1) token_probs_kernel(const ProbArgs a) {
  constexpr int W = T / 32, ES = F32 ? 4 : 2, Q = F32 ? 2 : 1;  // Q: 16-byte pieces of a vector
  extern __shared__ __align__(16) uint4 next[];                  // [K][Q][T]: each thread's vectors of the next row
  __shared__ uint64_t tell[2][8 * W];  // of each warp of the row, in turn: its largest logit, and its sum or that logit's place
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = a.blocks, V = a.V;
  const int rank = C > 1 ? (int)cluster_rank() : 0, clusters = gridDim.x / C;
  if (C > 1) cluster_arrive();  // this block runs: the others may write to it
  pdl_wait();
  pdl_trigger();
  // A row's vectors start at its first 16-byte boundary.  The logits before it,
  // and those after the last whole vector, are single ones of the first block.
  struct Row {
    int r, e0, v0, v1, one;
    float x1, t;
  };
  auto fetch = [&](int r) {
    Row w = {r, 0, 0, 0, -1, -INFINITY, 1.f};
    if (r >= a.R) return w;
    const char* in = a.in + (int64_t)r * a.in_ld * ES;
    w.e0 = min(V, (int)((16u - ((uint32_t)(uintptr_t)in & 15u)) & 15u) / ES);
    const int nvec = (V - w.e0) / 8, per = (nvec + C - 1) >> a.log2_blocks, rest = w.e0 + 8 * nvec;
    w.v0 = min(rank * per, nvec);
    w.v1 = min(w.v0 + per, nvec);
    w.one = rank ? -1 : tid < w.e0 ? tid : tid >= 32 && tid - 32 < V - rest ? rest + tid - 32 : -1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = w.v0 + k * T + tid;
      constexpr uint32_t NONE = F32 ? 0xFF800000u : 0xFF80FF80u;  // -inf
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        uint4* to = &next[(k * Q + q) * T + tid];
        if (v < w.v1) cp_async16(to, in + ((int64_t)w.e0 + 8 * (int64_t)v) * ES + 16 * q);
        else *to = make_uint4(NONE, NONE, NONE, NONE);
      }
    }
    cp_async_commit();
    if (w.one >= 0) w.x1 = logit_at<F32>(in, w.one);
    if (a.temperature) w.t = __ldg(a.temperature + r);
    return w;
  };
  Row w = fetch(blockIdx.x / C);
  if (C > 1) cluster_wait();
  for (int turn = 0; w.r < a.R; turn ^= 1) {
    float x1 = w.x1;
    cp_async_wait_all();  // a thread reads what it fetched itself
    // 8 logits a vector: fp32 ones where their exponentials will be, bf16 ones as they come
    float x[K][8];
    uint32_t u[K][4];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const uint4 p = next[(k * Q + q) * T + tid];
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (F32) x[k][4 * q + i] = __uint_as_float(w[i]);
          else u[k][i] = w[i];
        }
      }
    auto logit = [&](int k, int i) { return F32 ? x[k][i] : i & 1 ? bf16hi(u[k][i / 2]) : bf16lo(u[k][i / 2]); };
    const bool warm = w.t > 0.f;
    const Scale c = log2_scale(w.t);

    float top = x1;
    if (F32) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; i += 2) top = max_nan(top, logit(k, i), logit(k, i + 1));
    } else {
      uint32_t most = u[0][0];
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = k ? 0 : 1; i < 4; ++i) most = max_nan_bf16x2(most, u[k][i]);
      top = max_nan(top, bf16lo(most), bf16hi(most));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));

    float sum = 0.f;
    if (!warm) {
      int first = V;
      if (x1 == top) first = w.one;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 7; i >= 0; --i)
          if (logit(k, i) == top) first = min(first, w.e0 + 8 * (w.v0 + k * T + tid) + i);
      sum = __int_as_float(__reduce_min_sync(0xffffffffu, first));
    } else {
      if (c.flat) {
        auto e = [](float v) { return v > -INFINITY ? 1.f : 0.f; };
        sum = x1 = e(x1);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += x[k][i] = e(logit(k, i));
      } else {
        // 2^(40 + (x - top) c): what lies below 2^-126 of the largest stays normal
        // (d as small as 2^-200 needs stands for all that is less, -inf too: in
        // bf16 the logit of that d, rounded down, unless that would overflow)
        const float base = top > -INFINITY ? top : 0.f, low = -200.f * rcp(c.hi), edge = base + low;
        const bool tame = fabsf(base) < 1e30f && fabsf(base) * c.hi < 1e37f;
        const uint16_t edge16 = f2bf(edge - 0.0078125f * fabsf(edge));
        const uint32_t edge2 = edge16 | (uint32_t)edge16 << 16;
        const uint64_t base2 = pack2(-base, -base), hi2 = pack2(c.hi, c.hi), lo2 = pack2(c.lo, c.lo), ln2 = pack2(0.693147182f, 0.693147182f);
        const uint64_t c40 = pack2(40.f, 40.f), one2 = pack2(1.f, 1.f), minus2 = pack2(-1.f, -1.f);
        auto e2 = [&](uint64_t d, float& u, float& v) {
          const uint64_t y = fma2(d, hi2, c40);
          const uint64_t rest = fma2(d, lo2, fma2(d, hi2, fma2(y, minus2, c40)));  // what y's rounding left
          unpack2(y, u, v);
          const uint64_t e = mul2(pack2(ex2_ftz(u), ex2_ftz(v)), fma2(rest, ln2, one2));
          unpack2(e, u, v);
          return e;
        };
        auto diff = [&](float u, float v) {
          unpack2(add2(pack2(u, v), base2), u, v);
          return pack2(fmaxf(u, low), fmaxf(v, low));
        };
        uint64_t sums[2] = {0, 0};
        if (F32 || !tame) {
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 8; i += 2) sums[i / 2 & 1] = add2(sums[i / 2 & 1], e2(diff(logit(k, i), logit(k, i + 1)), x[k][i], x[k][i + 1]));
        } else {
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              sums[i / 2 & 1] = add2(sums[i / 2 & 1], e2(add_bf16x2(max_bf16x2(u[k][i / 2], edge2), -base), x[k][i], x[k][i + 1]));
        }
        float y, z;
        e2(diff(x1, -INFINITY), x1, z);
        unpack2(add2(sums[0], sums[1]), y, z);
        sum = x1 + (y + z);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    // one exchange: every warp tells all blocks of the row.  (A block that is a
    // row ahead writes to the other half, and cannot be two ahead.)
    if (lane < C) {
      const uint64_t v = (uint64_t)__float_as_uint(top) | ((uint64_t)__float_as_uint(sum) << 32);
      if (C > 1) cluster_put(&tell[turn][rank * W + warp], lane, v);
      else tell[turn][warp] = v;
    }
    __syncwarp();
    if (C > 1) cluster_arrive();
    else __syncthreads();
    // the next row's vectors come in meanwhile (this one's have left shared
    // memory: top depends on all of them)
    const Row after = fetch(w.r + clusters);
    if (C > 1) cluster_wait();
    float all = -INFINITY, total = 0.f;
    int first = V;
    {
      float tops[8 * W / 32], sums[8 * W / 32];
#pragma unroll
      for (int j = 0; j < 8 * W / 32; ++j) {
        const bool in = 32 * j + lane < C * W;
        const uint64_t v = in ? tell[turn][32 * j + lane] : 0;
        tops[j] = in ? __uint_as_float((uint32_t)v) : -INFINITY;
        sums[j] = __uint_as_float((uint32_t)(v >> 32));
        all = max_nan(all, tops[j]);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) all = max_nan(all, __shfl_xor_sync(0xffffffffu, all, o));
#pragma unroll
      for (int j = 0; j < 8 * W / 32; ++j) {
        if (32 * j >= C * W) continue;
        if (warm) total += sums[j] * exp_part(tops[j], all, c);
        else if (tops[j] == all) first = min(first, __float_as_int(sums[j]));
      }
      if (warm) {
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      } else {
        first = __reduce_min_sync(0xffffffffu, first);
      }
    }
    // a row with NaN or +inf, one with nothing but -inf, one of a single token
    const bool bad = !(all < INFINITY);
    if (warm && !bad && all > -INFINITY) {
      const float f = top > -INFINITY ? exp_scaled(top, all, c) : 0.f, inv = __frcp_rn(total);
      // in two steps where the scale would be subnormal
      const bool whole = f * inv > 1e-37f;
      const float f1 = whole ? f * inv : f, f2 = whole ? 1.f : inv;
      const uint64_t g = pack2(f1, f1), h = pack2(f2, f2);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          uint64_t y = mul2(pack2(x[k][i], x[k][i + 1]), g);
          if (!whole) y = mul2(y, h);
          unpack2(y, x[k][i], x[k][i + 1]);
        }
      x1 = x1 * f1 * f2;
    } else {
      const float fill = bad ? __int_as_float(0x7FFFFFFF) : 0.f;
      const int is = !warm && !bad && all > -INFINITY ? first : -1;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = w.e0 + 8 * (w.v0 + k * T + tid) + i == is ? 1.f : fill;
      x1 = w.one == is ? 1.f : fill;
    }
    float* out = a.out + (int64_t)w.r * a.out_ld;
    const int mis = (int)(((uintptr_t)out / 4 + w.e0) & 7);  // floats of the vectors past a 32-byte boundary
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = w.v0 + k * T + tid;
      if (v >= w.v1) continue;
      float* to = out + w.e0 + 8 * v;
      if (mis == 0) {
        store8(to, x[k]);
      } else if ((mis & 3) == 0) {
        reinterpret_cast<float4*>(to)[0] = make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(x[k][4], x[k][5], x[k][6], x[k][7]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i] = x[k][i];
      }
    }
    if (w.one >= 0) out[w.one] = x1;
    w = after;
  }
}

// Rows that no cluster holds (more than 327 680 logits): a block a row, which
// reads it three times, from L2 the second and third.
template <bool F32>
__global__ void __launch_bounds__(1024) token_probs_loop_kernel(const ProbArgs a) {
  __shared__ float top_sh[32], sum_sh[32];
  __shared__ int first_sh[32], bad_sh[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.x, V = a.V;
  pdl_wait();
  pdl_trigger();
  const char* in = a.in + (int64_t)r * a.in_ld * (F32 ? 4 : 2);
  float* out = a.out + (int64_t)r * a.out_ld;
  const float t = a.temperature ? __ldg(a.temperature + r) : 1.f;
  float top = -INFINITY;
  int first = V;
  bool bad = false;
  for (int i = tid; i < V; i += 1024) {
    const float x = logit_at<F32>(in, i);
    bad |= !(x < INFINITY);
    if (x > top) {
      top = x;
      first = i;
    }
  }
  auto better = [](float& top, int& first, float x, int i) {
    if (x > top || (x == top && i < first)) {
      top = x;
      first = i;
    }
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) better(top, first, __shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, first, o));
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    top_sh[warp] = top;
    first_sh[warp] = first;
    bad_sh[warp] = bad;
  }
  __syncthreads();
  for (int w = 0; w < 1024 / 32; ++w) {
    better(top, first, top_sh[w], first_sh[w]);
    bad |= bad_sh[w] != 0;
  }
  const bool none = top == -INFINITY;  // and no NaN
  const Scale c = log2_scale(t);
  float sum = 0.f;
  if (t > 0.f && !none)
    for (int i = tid; i < V; i += 1024) sum += exp_scaled(logit_at<F32>(in, i), top, c);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sum_sh[warp] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < 1024 / 32; ++w) sum += sum_sh[w];
  for (int i = tid; i < V; i += 1024) {
    float p;
    if (bad) p = __int_as_float(0x7FFFFFFF);
    else if (none) p = 0.f;
    else if (t > 0.f) p = __fdiv_rn(exp_scaled(logit_at<F32>(in, i), top, c), sum);
    else p = i == first ? 1.f : 0.f;
    out[i] = p;
  }
}

template <bool F32, int K, int T>
mt_status probs_launch(ProbArgs a, const Launch& l, const DeviceInfo* di) {
  constexpr int smem = K * T * (F32 ? 32 : 16);
  const auto kernel = token_probs_kernel<F32, K, T>;
  static std::atomic<int> fit[64][4];  // clusters of 1, 2, 4, 8 blocks that the device holds at a time
  int dev = 0, size = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  while (1 << size < a.blocks) ++size;
  a.log2_blocks = size;
  int clusters = dev >= 0 && dev < 64 ? fit[dev][size].load() : 0;
  if (clusters < 1) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_fail(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.blocks);
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)a.blocks, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return cuda_fail(e);
    if (clusters < 1) clusters = 1;
    if (dev >= 0 && dev < 64) fit[dev][size].store(clusters);
  }
  // as many rows to each cluster, in one round of clusters
  const int rows = (a.R + clusters - 1) / clusters;
  const dim3 grid((unsigned)((a.R + rows - 1) / rows) * a.blocks);
  return a.blocks > 1 ? launch_cluster(kernel, a.blocks, grid, dim3(T), smem, l, a) : launch(kernel, grid, dim3(T), smem, l, a);
}

// The fewest blocks a row that hold it (their number costs little, but the last
// vectors of their threads lie idle), more where the rows are few.
template <bool F32>
mt_status probs_run(ProbArgs a, const Launch& l, const DeviceInfo* di) {
  const int nvec = a.V / 8;
  auto per = [&](int C, int T) { return std::max(1, ((nvec + C - 1) / C + T - 1) / T); };  // vectors of a thread
  if (per(8, PB_THREADS) > PB_MOST) {
    a.blocks = 8;
    if (per(8, 1024) <= PB_MOST) return probs_launch<F32, PB_MOST, 1024>(a, l, di);
    return launch(token_probs_loop_kernel<F32>, dim3(a.R), dim3(1024), 0, l, a);
  }
  a.blocks = 1;
  while (a.blocks < 8 && (per(a.blocks, PB_THREADS) > 4 || ((int64_t)a.R * a.blocks < di->sm_count && per(a.blocks, PB_THREADS) > 1))) a.blocks *= 2;
  // many rows: blocks of half as many threads with twice the logits each, as
  // what a warp does once a row then counts half
  if ((int64_t)a.R * a.blocks >= 4 * di->sm_count) {
    switch ((per(a.blocks, 256) + 1) / 2) {
      case 1: return probs_launch<F32, 2, 256>(a, l, di);
      case 2: return probs_launch<F32, 4, 256>(a, l, di);
      case 3: return probs_launch<F32, 6, 256>(a, l, di);
      case 4: return probs_launch<F32, 8, 256>(a, l, di);
      default: return probs_launch<F32, 2 * PB_MOST, 256>(a, l, di);
    }
  }
  switch (per(a.blocks, PB_THREADS)) {
    case 1: return probs_launch<F32, 1, PB_THREADS>(a, l, di);
    case 2: return probs_launch<F32, 2, PB_THREADS>(a, l, di);
    case 3: return probs_launch<F32, 3, PB_THREADS>(a, l, di);
    case 4: return probs_launch<F32, 4, PB_THREADS>(a, l, di);
    default: return probs_launch<F32, PB_MOST, PB_THREADS>(a, l, di);
  }
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
  const ProbArgs a = {(const char*)logits, probs, logits_ld, probs_ld, V, temperature, R, 1, 0};
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  return dtype == MT_F32 ? probs_run<true>(a, l, di) : probs_run<false>(a, l, di);
}
