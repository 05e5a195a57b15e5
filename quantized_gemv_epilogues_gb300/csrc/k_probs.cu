// k_probs.cu - mt_token_probs: probabilities of rows of logits under a
// temperature.
//
//   p = e / sum e,  e = exp((x - max x) / t);  t <= 0: 1 at the first largest.
//
// Bound: memory, each logit read and each probability written once.
#include <math.h>

#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int PB_THREADS = 1024;

struct ProbArgs {
  const char* in;
  float* out;
  int64_t in_ld, out_ld;
  int V;
  const float* temperature;
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

template <bool F32>
__global__ void __launch_bounds__(PB_THREADS) token_probs_kernel(const ProbArgs a) {
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
  for (int i = tid; i < V; i += PB_THREADS) {
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
  for (int w = 0; w < PB_THREADS / 32; ++w) {
    better(top, first, top_sh[w], first_sh[w]);
    bad |= bad_sh[w] != 0;
  }
  const bool none = top == -INFINITY;  // and no NaN
  const Scale c = log2_scale(t);
  float sum = 0.f;
  if (t > 0.f && !none)
    for (int i = tid; i < V; i += PB_THREADS) sum += exp_scaled(logit_at<F32>(in, i), top, c);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sum_sh[warp] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < PB_THREADS / 32; ++w) sum += sum_sh[w];
  for (int i = tid; i < V; i += PB_THREADS) {
    float p;
    if (bad) p = __int_as_float(0x7FFFFFFF);
    else if (none) p = 0.f;
    else if (t > 0.f) p = __fdiv_rn(exp_scaled(logit_at<F32>(in, i), top, c), sum);
    else p = i == first ? 1.f : 0.f;
    out[i] = p;
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
  const ProbArgs a = {(const char*)logits, probs, logits_ld, probs_ld, V, temperature};
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  return dtype == MT_F32 ? launch(token_probs_kernel<true>, dim3(R), dim3(PB_THREADS), 0, l, a)
                         : launch(token_probs_kernel<false>, dim3(R), dim3(PB_THREADS), 0, l, a);
}
