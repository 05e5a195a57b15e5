// k_logits.cu - mt_logit_penalties: biases, penalties for repeated tokens and
// allowed-token masks in one pass over the vocabulary's logits.
//
//   x = logit + bias;  seen: x > 0 ? x / r : x * r;
//   generated n > 0 times: x - f n - p;  not allowed: -inf
//
// Bound: memory, each logit read and written once (and one mask bit).  A block
// takes CH consecutive logits of one sequence and issues all of its loads at
// once; while they are on their way it counts its sequence's tokens.  Counting
// needs no clearing of CH words: a first walk over the history marks each of
// the block's tokens in a bitmap and zeroes its word, a second walk (the ids
// are in L1 then) adds, and the pass over the logits looks at words only
// where the bitmap has a bit: one byte of shared memory per eight logits
// otherwise.  Every block of a sequence reads its whole history, which L2
// serves: 4 bytes a token against 2 CH (bf16) or 4 CH bytes of logits.
// Counts are integers and a repeated bias entry is resolved by its index, so
// no result depends on the order of the atomics.
#include <math.h>

#include <atomic>

#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int LG_THREADS = 256;

struct LogitArgs {
  const char* in;
  char* out;
  int64_t in_ld, out_ld;  // elements
  int V;
  const int32_t* history;
  const int32_t* history_start;
  const int32_t* prompt_len;
  int n_history;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_ids;
  const float* bias_values;
  const int32_t* bias_start;
  int n_bias;
  const uint32_t* allowed;
  int64_t allowed_ld;
};

// NV 16-byte vectors of logits a thread; CH = logits a block.
template <bool F32, int NV>
struct LogitShape {
  static constexpr int VE = F32 ? 4 : 8;
  static constexpr int CH = NV * LG_THREADS * VE;
  static constexpr int CAP = CH + 32;  // the first block also takes up to VE - 1 logits before the aligned ones
};

template <bool F32>
__device__ __forceinline__ float logit_get(const char* p, int i) {
  return F32 ? reinterpret_cast<const float*>(p)[i] : bf16f(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void logit_put(char* p, int i, float x) {
  if (F32) reinterpret_cast<float*>(p)[i] = x;
  else reinterpret_cast<uint16_t*>(p)[i] = f2bf(x);
}

template <bool F32, int NV>
__global__ void __launch_bounds__(LG_THREADS) logit_penalties_kernel(const LogitArgs a) {
  using S = LogitShape<F32, NV>;
  constexpr int VE = S::VE, CH = S::CH, ES = F32 ? 4 : 2;
  extern __shared__ __align__(16) uint32_t lg_smem[];
  uint32_t* marked = lg_smem;                   // bit per logit: seen
  uint32_t* biased = marked + S::CAP / 32;      // bit per logit: has a bias
  uint32_t* count = biased + S::CAP / 32;       // times generated, where marked
  uint32_t* slot = count + S::CAP;              // 1 + index of the bias entry, where biased (only with biases)
  const int tid = threadIdx.x, b = blockIdx.y, V = a.V;
  pdl_wait();
  pdl_trigger();
  const char* in = a.in + (int64_t)b * a.in_ld * ES;
  char* out = a.out + (int64_t)b * a.out_ld * ES;
  // logits before the row's first 16-byte boundary; vectors need it to be the
  // output's too
  const int e0 = min(V, (int)((16u - ((uint32_t)(uintptr_t)in & 15u)) & 15u) / ES);
  const bool vec = (((uintptr_t)in ^ (uintptr_t)out) & 15u) == 0;
  const int c0 = e0 + blockIdx.x * CH;         // first aligned logit
  const int lo = blockIdx.x ? c0 : 0;          // first logit of the block
  const int hi = min(V, c0 + CH);
  if (lo >= hi) return;

  uint4 raw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int t = c0 + (v * LG_THREADS + tid) * VE;
    if (vec && t + VE <= V) raw[v] = *reinterpret_cast<const uint4*>(in + (int64_t)t * ES);
  }
  for (int i = tid; i < 2 * (S::CAP / 32); i += LG_THREADS) marked[i] = 0;
  __syncthreads();

  const int span = hi - lo;
  int h0 = 0, h1 = 0, hp = 0;
  if (a.history) {
    h0 = min(max(__ldg(a.history_start + b), 0), a.n_history);
    h1 = min(max(__ldg(a.history_start + b + 1), h0), a.n_history);
    hp = a.prompt_len ? min(max(__ldg(a.prompt_len + b), 0), h1 - h0) : 0;  // prompt tokens
    hp += h0;
#pragma unroll 4
    for (int i = h0 + tid; i < h1; i += LG_THREADS) {
      const int id = __ldg(a.history + i);
      const unsigned at = (unsigned)(id - lo);
      if (id >= 0 && at < (unsigned)span) {
        count[at] = 0;
        atomicOr(&marked[at >> 5], 1u << (at & 31));
      }
    }
  }
  int b0 = 0, b1 = 0;
  if (a.bias_ids) {
    b0 = min(max(__ldg(a.bias_start + b), 0), a.n_bias);
    b1 = min(max(__ldg(a.bias_start + b + 1), b0), a.n_bias);
    for (int i = b0 + tid; i < b1; i += LG_THREADS) {
      const int id = __ldg(a.bias_ids + i);
      const unsigned at = (unsigned)(id - lo);
      if (id >= 0 && at < (unsigned)span) {
        slot[at] = 0;
        atomicOr(&biased[at >> 5], 1u << (at & 31));
      }
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int i = hp + tid; i < h1; i += LG_THREADS) {
    const int id = __ldg(a.history + i);
    const unsigned at = (unsigned)(id - lo);
    if (id >= 0 && at < (unsigned)span) atomicAdd(&count[at], 1u);
  }
  for (int i = b0 + tid; i < b1; i += LG_THREADS) {
    const int id = __ldg(a.bias_ids + i);
    const unsigned at = (unsigned)(id - lo);
    if (id >= 0 && at < (unsigned)span) atomicMax(&slot[at], (uint32_t)(i - b0 + 1));
  }
  __syncthreads();

  const float rep = a.repetition ? __ldg(a.repetition + b) : 1.f;
  const float pres = a.presence ? __ldg(a.presence + b) : 0.f;
  const float freq = a.frequency ? __ldg(a.frequency + b) : 0.f;
  const uint32_t* allowed = a.allowed ? a.allowed + (int64_t)b * a.allowed_ld : nullptr;
  auto touched = [&](float x, unsigned at) -> float {  // a logit with a bias or in the history
    if ((biased[at >> 5] >> (at & 31)) & 1u) x += __ldg(a.bias_values + b0 + (int)slot[at] - 1);
    if ((marked[at >> 5] >> (at & 31)) & 1u) {
      x = x > 0.f ? x / rep : x * rep;
      const uint32_t n = count[at];
      if (n) x = x - freq * (float)n - pres;
    }
    return x;
  };
  auto single = [&](int t) {
    float x = touched(logit_get<F32>(in, t), (unsigned)(t - lo));
    if (allowed && !((__ldg(allowed + (t >> 5)) >> (t & 31)) & 1u)) x = -INFINITY;
    logit_put<F32>(out, t, x);
  };
  if (!vec) {  // rows of input and output that are not aligned alike
    for (int t = lo + tid; t < hi; t += LG_THREADS) single(t);
    return;
  }
  if (lo + tid < c0) single(lo + tid);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int t = c0 + (v * LG_THREADS + tid) * VE;
    if (t + VE > V) {
      for (int i = t; i < V; ++i) single(i);
      continue;
    }
    const unsigned at = (unsigned)(t - lo);
    // the VE bits from bit t (at) on, of the mask (the bitmaps)
    uint32_t ok = 0xFFFFFFFFu;
    if (allowed) ok = __funnelshift_r(__ldg(allowed + (t >> 5)), __ldg(allowed + ((t + VE - 1) >> 5)), t & 31);
    const unsigned w0 = at >> 5, w1 = (at + VE - 1) >> 5;
    const uint32_t hit = __funnelshift_r(marked[w0] | biased[w0], marked[w1] | biased[w1], at & 31) & ((1u << VE) - 1);
    uint4 r = raw[v];
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
    if (hit || (~ok & ((1u << VE) - 1))) {
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        float x = F32 ? __uint_as_float(w[F32 ? i : 0]) : ((i & 1) ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]));
        if ((hit >> i) & 1u) x = touched(x, at + i);
        if (!((ok >> i) & 1u)) x = -INFINITY;
        if (F32) w[F32 ? i : 0] = __float_as_uint(x);
        else if (((hit | ~ok) >> i) & 1u)
          w[i >> 1] = (i & 1) ? (w[i >> 1] & 0x0000FFFFu) | ((uint32_t)f2bf(x) << 16)
                              : (w[i >> 1] & 0xFFFF0000u) | (uint32_t)f2bf(x);
      }
    }
    *reinterpret_cast<uint4*>(out + (int64_t)t * ES) = r;
  }
}

template <bool F32, int NV>
mt_status logit_launch(const LogitArgs& a, int B, const Launch& l) {
  using S = LogitShape<F32, NV>;
  const size_t smem = (size_t)(2 * (S::CAP / 32) + S::CAP * (a.bias_ids ? 2 : 1)) * 4;
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev >= 0 && dev < 64 && !set[dev].load()) {
    e = cudaFuncSetAttribute(logit_penalties_kernel<F32, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)((2 * (S::CAP / 32) + S::CAP * 2) * 4));
    if (e != cudaSuccess) return cuda_fail(e);
    set[dev].store(true);
  }
  // one block more where a row's unaligned first logits push its last ones over
  const int blocks = (a.V + S::CH - 1) / S::CH;
  return launch(logit_penalties_kernel<F32, NV>, dim3(blocks, B), dim3(LG_THREADS), smem, l, a);
}

}  // namespace

}  // namespace mt

using namespace mt;

extern "C" mt_status mt_logit_penalties(const void* logits, int64_t logits_ld, void* out, int64_t out_ld, mt_dtype dtype,
                                        int B, int V, const int32_t* history, const int32_t* history_start,
                                        const int32_t* prompt_len, int n_history, const float* repetition,
                                        const float* presence, const float* frequency, const int32_t* bias_ids,
                                        const float* bias_values, const int32_t* bias_start, int n_bias,
                                        const uint32_t* allowed, int64_t allowed_ld, void* stream) {
  if (B != 0 && (!logits || !out)) return MT_ERR_NULL;
  if (dtype != MT_BF16 && dtype != MT_F32) return MT_ERR_FORMAT;
  if ((history != nullptr) != (history_start != nullptr) || (prompt_len && !history)) return MT_ERR_NULL;
  if ((bias_ids != nullptr) != (bias_values != nullptr) || (bias_ids != nullptr) != (bias_start != nullptr))
    return MT_ERR_NULL;
  if (B < 0 || B > 65535 || V < 1 || V > (1 << 24) || logits_ld < V || out_ld < V || n_history < 0 || n_bias < 0 ||
      logits_ld > ((int64_t)1 << 38) || out_ld > ((int64_t)1 << 38) || allowed_ld > ((int64_t)1 << 38) ||
      (allowed && allowed_ld < (V + 31) / 32))
    return MT_ERR_SHAPE;
  const int es = dtype == MT_F32 ? 4 : 2;
  if (!aligned_to(logits, es) || !aligned_to(out, es)) return MT_ERR_ALIGN;
  const void* words[] = {history, history_start, prompt_len, repetition, presence, frequency, bias_ids, bias_values, bias_start, allowed};
  for (const void* p : words)
    if (!aligned_to(p, 4)) return MT_ERR_ALIGN;
  const ByteRange ri = byte_range(logits, rows_bytes(B, logits_ld, V, es)), ro = byte_range(out, rows_bytes(B, out_ld, V, es));
  if (ranges_overlap(ri, ro) && !(out == logits && (out_ld == logits_ld || B == 1))) return MT_ERR_ALIAS;
  const ByteRange others[] = {byte_range(history, (size_t)n_history * 4), byte_range(history_start, (size_t)(B + 1) * 4),
                              byte_range(prompt_len, (size_t)B * 4), byte_range(repetition, (size_t)B * 4),
                              byte_range(presence, (size_t)B * 4), byte_range(frequency, (size_t)B * 4),
                              byte_range(bias_ids, (size_t)n_bias * 4), byte_range(bias_values, (size_t)n_bias * 4),
                              byte_range(bias_start, (size_t)(B + 1) * 4),
                              byte_range(allowed, rows_bytes(B, allowed_ld, (V + 31) / 32, 4))};
  for (const ByteRange& o : others)
    if (ranges_overlap(o, ro)) return MT_ERR_ALIAS;
  if (B == 0) return MT_OK;
  int derr = 0;
  const DeviceInfo* di = device_info(&derr);
  if (!di) return cuda_fail((cudaError_t)derr);
  LogitArgs a = {};
  a.in = (const char*)logits;
  a.out = (char*)out;
  a.in_ld = logits_ld;
  a.out_ld = out_ld;
  a.V = V;
  a.history = history;
  a.history_start = history_start;
  a.prompt_len = prompt_len;
  a.n_history = n_history;
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.bias_ids = bias_ids;
  a.bias_values = bias_values;
  a.bias_start = bias_start;
  a.n_bias = n_bias;
  a.allowed = allowed;
  a.allowed_ld = allowed_ld;
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  // few sequences: 2048 logits a block, so that a vocabulary fills the GPU;
  // many: 8192, which read the history a quarter as often
  if (dtype == MT_F32)
    return (long)B * V < 4L * 8192 * di->sm_count ? logit_launch<true, 2>(a, B, l) : logit_launch<true, 8>(a, B, l);
  return (long)B * V < 4L * 8192 * di->sm_count ? logit_launch<false, 1>(a, B, l) : logit_launch<false, 4>(a, B, l);
}
