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
  int blocks;  // of a row
};

// 1 / t in units of log2 e, as a sum of two floats: the exponent's argument is
// off by 2^-40 of itself, not by the 2^-23 that would be 2^-17 of a small p.
struct Scale {
  float hi, lo;
  bool flat;  // a temperature above 2^100: all alike
};
__device__ __forceinline__ Scale log2_scale(float t) {
  constexpr float TOP = 1.2676506e30f;  // 2^100
  Scale s;
  s.flat = t > TOP;
  t = fminf(fmaxf(t, 1.f / TOP), TOP);  // products stay finite
  const float l_hi = 1.44269502f, l_lo = 1.92596303e-8f;  // log2 e
  s.hi = __fdiv_rn(l_hi, t);
  s.lo = __fdiv_rn(fmaf(-s.hi, t, l_hi) + l_lo, t);
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
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Eight consecutive floats to a 32-byte boundary.
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
               "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// What a block of a row tells the others: its largest logit and its sum, and the
// first place of the former.
__device__ __forceinline__ float share_top(const uint64_t (&s)[2]) { return __uint_as_float((uint32_t)s[0]); }

template <bool F32, int K, int T>
__global__ void __launch_bounds__(T, T == 512 ? 2 : 1) token_probs_kernel(const ProbArgs a) {
  constexpr int W = T / 32, ES = F32 ? 4 : 2;
  __shared__ float top_sh[W], sum_sh[W];
  __shared__ int first_sh[W];
  __shared__ __align__(16) uint64_t share[8][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = a.blocks, V = a.V;
  const int rank = C > 1 ? (int)cluster_rank() : 0, r = blockIdx.x / C;
  if (C > 1) cluster_arrive();  // this block runs: the others may write to it
  pdl_wait();
  pdl_trigger();
  const char* in = a.in + (int64_t)r * a.in_ld * ES;
  float* out = a.out + (int64_t)r * a.out_ld;
  const float t = a.temperature ? __ldg(a.temperature + r) : 1.f;
  // The row's vectors start at its first 16-byte boundary.  The logits before
  // it, and those after the last whole vector, are single ones of the first block.
  const int e0 = min(V, (int)((16u - ((uint32_t)(uintptr_t)in & 15u)) & 15u) / ES);
  const int nvec = (V - e0) / 8, per = (nvec + C - 1) / C, v0 = min(rank * per, nvec), v1 = min(v0 + per, nvec);
  const int rest = e0 + 8 * nvec;
  const int one = rank ? -1 : tid < e0 ? tid : tid >= 32 && tid - 32 < V - rest ? rest + tid - 32 : -1;
  float x[K][8], x1 = -INFINITY;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int v = v0 + k * T + tid;
    if (v < v1) {
      const uint4* src = reinterpret_cast<const uint4*>(in + ((int64_t)e0 + 8 * (int64_t)v) * ES);
      if (F32) {
        const uint4 p = src[0], q = src[1];
        const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = __uint_as_float(w[i]);
      } else {
        const uint4 p = src[0];
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[k][2 * i] = bf16lo(w[i]);
          x[k][2 * i + 1] = bf16hi(w[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = -INFINITY;
    }
  }
  if (one >= 0) x1 = logit_at<F32>(in, one);
  const bool warm = t > 0.f;
  const Scale c = log2_scale(t);

  float top = x1;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max_nan(top, x[k][i]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) top_sh[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) top = max_nan(top, top_sh[w]);

  float sum = 0.f;
  int first = V;
  if (!warm) {
    if (x1 == top) first = one;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 7; i >= 0; --i)
        if (x[k][i] == top) first = min(first, e0 + 8 * (v0 + k * T + tid) + i);
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) first_sh[warp] = first;
  } else if (c.flat) {
    auto e = [](float v) { return v > -INFINITY ? 1.f : 0.f; };
    sum = x1 = e(x1);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[k][i] = e(x[k][i]);
  } else {
    // 2^(40 + (x - top) c): what lies below 2^-126 of the largest stays normal
    const float base = top > -INFINITY ? top : 0.f, low = -200.f / c.hi;
    auto e = [&](float v) {
      const float d = fmaxf(v - base, low), y = fmaf(d, c.hi, 40.f);
      const float rest = fmaf(d, c.lo, fmaf(d, c.hi, 40.f - y));  // what y's rounding left
      return ex2_ftz(y) * fmaf(rest, 0.693147182f, 1.f);
    };
    sum = x1 = e(x1);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i & 3] += x[k][i] = e(x[k][i]);
    sum += (s[0] + s[1]) + (s[2] + s[3]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sum_sh[warp] = sum;
  __syncthreads();
  if (C > 1) cluster_wait();
  if (tid < C) {
    sum = 0.f;
    first = V;
    for (int w = 0; w < W; ++w) {
      sum += sum_sh[w];
      if (!warm) first = min(first, first_sh[w]);
    }
    const uint64_t lo = (uint64_t)__float_as_uint(top) | ((uint64_t)__float_as_uint(sum) << 32), hi = (uint32_t)first;
    if (C > 1) {
      cluster_put(&share[rank][0], tid, lo);
      cluster_put(&share[rank][1], tid, hi);
    } else {
      share[0][0] = lo;
      share[0][1] = hi;
    }
  }
  __syncwarp();
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  float all = share_top(share[0]), total = 0.f;
  for (int b = 1; b < C; ++b) all = max_nan(all, share_top(share[b]));
  first = V;
  for (int b = 0; b < C; ++b) {
    const float tb = share_top(share[b]);
    if (warm) total += __uint_as_float((uint32_t)(share[b][0] >> 32)) * exp_scaled(tb, all, c);
    else if (tb == all) first = min(first, (int)share[b][1]);
  }
  const float f = exp_scaled(top, all, c), inv = __fdiv_rn(1.f, total);
  // a row with NaN or +inf, one with nothing but -inf, one of a single token
  const bool bad = !(all < INFINITY), plain = warm && !bad && all > -INFINITY;
  auto p = [&](float e, int i) {
    if (plain) return e * f * inv;
    return bad ? __int_as_float(0x7FFFFFFF) : !warm && i == first && all > -INFINITY ? 1.f : 0.f;
  };
  const int mis = (int)(((uintptr_t)out / 4 + e0) & 7);  // floats of the vectors past a 32-byte boundary
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int v = v0 + k * T + tid;
    if (v >= v1) continue;
    const int i0 = e0 + 8 * v;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[k][i] = p(x[k][i], i0 + i);
    float* to = out + i0;
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
  if (one >= 0) out[one] = p(x1, one);
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

template <bool F32, int T>
mt_status probs_launch(const ProbArgs& a, int K, int R, const Launch& l) {
  const dim3 grid((unsigned)R * a.blocks);
  auto go = [&](auto kernel) {
    return a.blocks > 1 ? launch_cluster(kernel, a.blocks, grid, dim3(T), 0, l, a) : launch(kernel, grid, dim3(T), 0, l, a);
  };
  switch (T == 512 ? K : PB_MOST) {
    case 1: return go(token_probs_kernel<F32, T == 512 ? 1 : PB_MOST, T>);
    case 2: return go(token_probs_kernel<F32, T == 512 ? 2 : PB_MOST, T>);
    case 3: return go(token_probs_kernel<F32, T == 512 ? 3 : PB_MOST, T>);
    case 4: return go(token_probs_kernel<F32, T == 512 ? 4 : PB_MOST, T>);
    default: return go(token_probs_kernel<F32, PB_MOST, T>);
  }
}

// The fewest blocks a row that hold it (their number costs little, but the last
// vectors of their threads lie idle), more where the rows are few.
template <bool F32>
mt_status probs_run(ProbArgs a, int R, int sms, const Launch& l) {
  const int nvec = a.V / 8;
  auto per = [&](int C, int T) { return std::max(1, ((nvec + C - 1) / C + T - 1) / T); };  // vectors of a thread
  if (per(8, PB_THREADS) > PB_MOST) {
    a.blocks = 8;
    if (per(8, 1024) <= PB_MOST) return probs_launch<F32, 1024>(a, PB_MOST, R, l);
    return launch(token_probs_loop_kernel<F32>, dim3(R), dim3(1024), 0, l, a);
  }
  a.blocks = 1;
  while (a.blocks < 8 && (per(a.blocks, PB_THREADS) > 4 || ((int64_t)R * a.blocks < sms && per(a.blocks, PB_THREADS) > 1))) a.blocks *= 2;
  return probs_launch<F32, PB_THREADS>(a, per(a.blocks, PB_THREADS), R, l);
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
  const ProbArgs a = {(const char*)logits, probs, logits_ld, probs_ld, V, temperature, 1};
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  return dtype == MT_F32 ? probs_run<true>(a, R, di->sm_count, l) : probs_run<false>(a, R, di->sm_count, l);
}
