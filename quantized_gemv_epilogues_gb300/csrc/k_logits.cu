// k_logits.cu - mt_logit_penalties: biases, penalties for repeated tokens and
// allowed-token masks in one pass over the vocabulary's logits.
//
//   x = logit + bias;  seen: x > 0 ? x / r : x * r;
//   generated n > 0 times: x - (f n + p);  not allowed: -inf
//
// Bound: memory, each logit read and written once (and one mask bit); a
// sequence's history touches a few thousand of its 10^5 logits.  Two kernels:
//  * mask_kernel passes all logits to the output under the mask, 16 bytes a
//    load, NV of them in flight a thread.  In place and without a mask there is
//    nothing to do, and it is not launched.
//  * token_kernel, a block per sequence (several, for few), counts the tokens in a hash table in
//    shared memory, then does their logits, reading each from the input.  It
//    counts while mask_kernel still runs, and waits for it (programmatic
//    dependent launch) before it writes.
// (One kernel, whose blocks each took a chunk of the vocabulary and counted
// the tokens that fell there, read every history 16 times and spent its time
// on those loads' latency: 50 us where this takes 34 for 200
// texts.)
// Counts are integers and a repeated bias entry is resolved by its index, so no
// result depends on the order of the atomics.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int LM_THREADS = 256;  // mask_kernel
constexpr int LT_THREADS = 1024;  // token_kernel

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
  int slots;   // of token_kernel's table, a power of two
  bool in_order;  // token_kernel follows mask_kernel
};

// A token's word: the times it was generated, and
constexpr uint32_t LG_PROMPT = 1u << 31;  // it is in the prompt
constexpr uint32_t LG_BIASED = 1u << 30;  // it has a bias
constexpr uint32_t LG_TIMES = LG_BIASED - 1;
constexpr uint32_t LG_EMPTY = 0xFFFFFFFFu;  // a slot's key without a token

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
__global__ void __launch_bounds__(LM_THREADS) mask_kernel(const LogitArgs a) {
  constexpr int VE = F32 ? 4 : 8, CH = NV * LM_THREADS * VE, ES = F32 ? 4 : 2;
  const int tid = threadIdx.x, b = blockIdx.y, V = a.V;
  pdl_wait();
  pdl_trigger();  // after the wait: what token_kernel reads before its own is complete
  const char* in = a.in + (int64_t)b * a.in_ld * ES;
  char* out = a.out + (int64_t)b * a.out_ld * ES;
  const uint32_t* allowed = a.allowed ? a.allowed + (int64_t)b * a.allowed_ld : nullptr;
  auto one = [&](int t) {
    float x = logit_get<F32>(in, t);
    if (!allowed || ((__ldg(allowed + (t >> 5)) >> (t & 31)) & 1u)) {
      if (F32) reinterpret_cast<uint32_t*>(out)[t] = reinterpret_cast<const uint32_t*>(in)[t];  // as it is, NaN or not
      else reinterpret_cast<uint16_t*>(out)[t] = reinterpret_cast<const uint16_t*>(in)[t];
    } else {
      x = -INFINITY;
      logit_put<F32>(out, t, x);
    }
  };
  // logits before the row's first 16-byte boundary; vectors need it to be the
  // output's too (200 rows of 128 256 bf16 logits, an output one logit off: 88 us,
  // 18 where the boundaries agree)
  const int e0 = min(V, (int)((16u - ((uint32_t)(uintptr_t)in & 15u)) & 15u) / ES);
  const int c0 = e0 + blockIdx.x * CH;
  if ((((uintptr_t)in ^ (uintptr_t)out) & 15u) != 0) {
#pragma unroll 1
    for (int t = (blockIdx.x ? c0 : 0) + tid; t < min(V, c0 + CH); t += LM_THREADS) one(t);
    return;
  }
  uint4 raw[NV];
  uint32_t ok[NV];  // the mask's VE bits from each vector's first logit on
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int t = c0 + (v * LM_THREADS + tid) * VE;
    if (t + VE <= V) {
      raw[v] = *reinterpret_cast<const uint4*>(in + (int64_t)t * ES);
      ok[v] = allowed ? __funnelshift_r(__ldg(allowed + (t >> 5)), __ldg(allowed + ((t + VE - 1) >> 5)), t & 31) : 0xFFFFFFFFu;
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int t = c0 + (v * LM_THREADS + tid) * VE;
    if (t + VE > V) {
#pragma unroll 1
      for (int i = t; i < V; ++i) one(i);  // the row's last logits
      continue;
    }
    uint32_t* w = reinterpret_cast<uint32_t*>(&raw[v]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (F32) {
        w[i] = (ok[v] >> i) & 1u ? w[i] : 0xFF800000u;
      } else {
        const uint32_t keep = ((ok[v] >> (2 * i)) & 1u ? 0x0000FFFFu : 0u) | ((ok[v] >> (2 * i)) & 2u ? 0xFFFF0000u : 0u);
        w[i] = (w[i] & keep) | (0xFF80FF80u & ~keep);
      }
    }
    *reinterpret_cast<uint4*>(out + (int64_t)t * ES) = raw[v];
  }
  if (blockIdx.x == 0 && tid < e0) one(tid);
}

// Table of `slots` entries: key, word, with biases 1 + the bias entry's index;
// and a list of the entries in use.  A sequence whose history and biases could fill it by more than three
// quarters is done in passes over ranges of `slots` tokens instead, the word at
// a token's place in the range.
template <bool F32>
__global__ void __launch_bounds__(LT_THREADS) token_kernel(const LogitArgs a) {
  constexpr int ES = F32 ? 4 : 2, N = 8;
  extern __shared__ __align__(16) uint32_t lt_smem[];
  const int tid = threadIdx.x, b = blockIdx.y, V = a.V, slots = a.slots;
  const int share = blockIdx.x, shares = gridDim.x;  // of the sequence's tokens
  uint32_t* key = lt_smem;
  uint32_t* word = key + slots;
  uint32_t* slot = word + slots;
  uint16_t* list = reinterpret_cast<uint16_t*>(slot + (a.bias_ids ? slots : 0));
  __shared__ int used;
  // alone, the kernel waits for what comes before it now; after mask_kernel it
  // waits for that later
  if (!a.in_order) pdl_wait();
  int h0 = 0, h1 = 0, hp = 0, b0 = 0, b1 = 0;
  if (a.history) {
    h0 = min(max(__ldg(a.history_start + b), 0), a.n_history);
    h1 = min(max(__ldg(a.history_start + b + 1), h0), a.n_history);
    if (h1 - h0 > (int)LG_TIMES) h1 = h0 + (int)LG_TIMES;  // a count stays within its bits
    hp = h0 + (a.prompt_len ? min(max(__ldg(a.prompt_len + b), 0), h1 - h0) : 0);  // the end of the prompt
  }
  if (a.bias_ids) {
    b0 = min(max(__ldg(a.bias_start + b), 0), a.n_bias);
    b1 = min(max(__ldg(a.bias_start + b + 1), b0), a.n_bias);
  }
  const float rep = a.repetition ? __ldg(a.repetition + b) : 1.f;
  const float freq = a.frequency ? __ldg(a.frequency + b) : 0.f, pres = a.presence ? __ldg(a.presence + b) : 0.f;
  const char* in = a.in + (int64_t)b * a.in_ld * ES;
  char* out = a.out + (int64_t)b * a.out_ld * ES;
  const uint32_t* allowed = a.allowed ? a.allowed + (int64_t)b * a.allowed_ld : nullptr;
  const bool hashed = (int64_t)(h1 - h0) + (b1 - b0) <= slots / 4 * 3;
  const int passes = hashed ? 1 : (V + slots - 1) / slots;
  int shift = 32;  // the hash's upper bits: a slot's index
  for (int n = slots; n > 1; n >>= 1) --shift;

  bool first_pass = true;
  for (int p = hashed ? 0 : share; p < passes; p += shares) {
    const int base = hashed ? 0 : p * slots, top = hashed ? V : min(V, base + slots);
    if (tid == 0) used = 0;
    for (int i = tid; i < slots / 4; i += LT_THREADS) {
      if (hashed) reinterpret_cast<uint4*>(key)[i] = make_uint4(LG_EMPTY, LG_EMPTY, LG_EMPTY, LG_EMPTY);
      reinterpret_cast<uint4*>(word)[i] = make_uint4(0, 0, 0, 0);
      if (a.bias_ids) reinterpret_cast<uint4*>(slot)[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    auto mine = [&](int t) -> bool { return hashed ? t >= 0 && t < V && t % shares == share : t >= base && t < top; };
    auto place = [&](int t) -> int {  // of token t in the table, which has room
      if (!hashed) return t - base;
      uint32_t at = (uint32_t)t * 2654435761u >> shift;
      for (;;) {
        uint32_t k = *const_cast<volatile uint32_t*>(&key[at]);
        if (k == LG_EMPTY) k = atomicCAS(&key[at], LG_EMPTY, (uint32_t)t);
        if (k == LG_EMPTY || k == (uint32_t)t) return (int)at;
        at = (at + 1) & (slots - 1);
      }
    };
    // by whole warps: the entries that some lanes are the first to touch join the list
    auto enlist = [&](bool first, int at) {
      const unsigned who = __ballot_sync(0xffffffffu, first);
      if (!who) return;
      int n = 0;
      if ((tid & 31) == 0) n = atomicAdd(&used, __popc(who));
      n = __shfl_sync(0xffffffffu, n, 0);
      if (first) list[n + __popc(who & ((1u << (tid & 31)) - 1u))] = (uint16_t)at;
    };
    // indices past the end of a list of nearly 2^31 entries need the 32nd bit
    for (uint32_t i0 = h0; i0 < (uint32_t)h1; i0 += N * LT_THREADS) {
      int id[N];
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const uint32_t i = i0 + q * LT_THREADS + tid;
        id[q] = i < (uint32_t)h1 ? __ldg(a.history + i) : -1;
      }
#pragma unroll
      for (int q = 0; q < N; ++q) {
        if (i0 + q * LT_THREADS >= (uint32_t)h1) break;
        const int t = id[q];
        bool first = false;
        int at = 0;
        if (mine(t)) {
          at = place(t);
          // (a prompt's token is marked once: frequent ones would queue up at their word)
          if (i0 + q * LT_THREADS + tid >= (uint32_t)hp) first = atomicAdd(&word[at], 1u) == 0;
          else if (!(*const_cast<volatile uint32_t*>(&word[at]) & LG_PROMPT)) first = atomicOr(&word[at], LG_PROMPT) == 0;
        }
        enlist(first, at);
      }
    }
    for (uint32_t i0 = b0; i0 < (uint32_t)b1; i0 += LT_THREADS) {
      const uint32_t i = i0 + tid;
      const int t = i < (uint32_t)b1 ? __ldg(a.bias_ids + i) : -1;
      bool first = false;
      int at = 0;
      if (mine(t)) {
        at = place(t);
        first = atomicOr(&word[at], LG_BIASED) == 0;
        atomicMax(&slot[at], i - (uint32_t)b0 + 1u);
      }
      enlist(first, at);
    }
    if (first_pass && a.in_order) pdl_wait();
    first_pass = false;
    __syncthreads();
    // M entries of a thread's at a time, so that their loads are in flight
    // together.  In place, a logit that was not masked still is what it was,
    // and a masked one is masked again.
    constexpr int M = 4;
    const int n = used;
    for (int i0 = tid; i0 < n; i0 += M * LT_THREADS) {
      uint32_t w[M], m[M];
      int t[M];
      float x[M], add[M];
#pragma unroll
      for (int q = 0; q < M; ++q) {
        const int at = list[min(i0 + q * LT_THREADS, n - 1)];  // past the end: the last one, not written
        w[q] = word[at];
        t[q] = hashed ? (int)key[at] : base + at;
        x[q] = logit_get<F32>(in, t[q]);
        m[q] = allowed ? __ldg(allowed + (t[q] >> 5)) : 0xFFFFFFFFu;
        add[q] = w[q] & LG_BIASED ? __ldg(a.bias_values + b0 + (int)slot[at] - 1) : 0.f;
      }
#pragma unroll
      for (int q = 0; q < M; ++q) {
        float y = x[q];
        if (w[q] & LG_BIASED) y += add[q];
        if (w[q] & (LG_PROMPT | LG_TIMES)) y = y > 0.f ? __fdiv_rn(y, rep) : y * rep;
        if (w[q] & LG_TIMES) y -= fmaf(freq, (float)(w[q] & LG_TIMES), pres);
        if (!((m[q] >> (t[q] & 31)) & 1u)) y = -INFINITY;
        if (i0 + q * LT_THREADS < n) logit_put<F32>(out, t[q], y);
      }
    }
    __syncthreads();  // the next pass's table is this one
  }
  // a share without a pass must not end before mask_kernel either: what follows
  // takes this kernel's end for both
  if (first_pass && a.in_order) pdl_wait();
  pdl_trigger();
}

template <bool F32>
mt_status logit_launch(LogitArgs a, int B, const Launch& l, int sms) {
  const bool tokens = (a.history && a.n_history) || (a.bias_ids && a.n_bias);
  const bool masks = a.in != a.out || a.allowed;
  if (masks) {
    constexpr int VE = F32 ? 4 : 8;
    // few logits: one vector a thread, so that they spread over the GPU
    const bool few = (long)B * a.V < 4L * 4 * LM_THREADS * VE * sms;
    const int ch = (few ? 1 : 4) * LM_THREADS * VE;
    const dim3 grid((a.V + ch - 1) / ch, B);
    const mt_status st = few ? launch(mask_kernel<F32, 1>, grid, dim3(LM_THREADS), 0, l, a)
                             : launch(mask_kernel<F32, 4>, grid, dim3(LM_THREADS), 0, l, a);
    if (st) return st;
  }
  if (!tokens) return MT_OK;
  a.in_order = masks;
  // four slots for a sequence's average token, so that its table is at most
  // half full unless it is twice the average.  One that outgrows three quarters
  // of the table pays for it: 200 texts of 200 tokens take 26 us, and 212 if one
  // of them has 6000 (75 ranges of 2048 slots in one block); 32 of 30 000, 45.
  const int bytes = a.bias_ids ? 14 : 10;  // of a slot
  const long want = 4 * (((long)a.n_history + a.n_bias) / B + 1);
  a.slots = 2048;
  while (a.slots < want && a.slots < 16384) a.slots *= 2;
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev >= 0 && dev < 64 && !set[dev].load()) {
    e = cudaFuncSetAttribute(token_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, 16384 * 14);
    if (e != cudaSuccess) return cuda_fail(e);
    set[dev].store(true);
  }
  // few sequences: several blocks each, as one SM's scattered loads and stores
  // (some two cycles each) would be the bound
  const int shares = std::max(1, std::min(16, 2 * sms / B));
  return launch(token_kernel<F32>, dim3(shares, B), dim3(LT_THREADS), (size_t)a.slots * bytes, l, a);
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
  return dtype == MT_F32 ? logit_launch<true>(a, B, l, di->sm_count) : logit_launch<false>(a, B, l, di->sm_count);
}
