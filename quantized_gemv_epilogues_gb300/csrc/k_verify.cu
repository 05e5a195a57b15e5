// k_verify.cu - mt_tree_verify: drafted tokens accepted against the target's
// probabilities from given random numbers, and the token after them.
//
// Mathematics (recursive rejection sampling).  At a token with target row p and
// draft row q, of whose children k have been refused, what is left to draw from
// is r_k = max(p - S_k q, 0), with S_0 = 0, R_0 = 1, S_{k+1} = S_k + R_k and R_k
// the sum of r_k: max(max(p / R - q, 0) .. - q, 0) over and over, without the
// divisions.  A child drawn from q is accepted with probability min(1, r_k / (R_k
// q)).  Without q a child stands for itself alone (q is 1 at its token): refused
// tokens leave p, and R goes down by theirs.
//
// Every probability is taken in steps of 2^-56 (exact above 2^-33, where a float's
// own step is larger; 2^-57 off below) and all sums are 64-bit integers: a
// distribution function summed in fp32 over 10^5 tokens is off by some 2^-24,
// which is as much as a rare token's share, and would draw other tokens in
// another order of the sum.
//
// Bound: latency, then memory: a float for each child that is tried and one row
// of p (and of q) for the token that is drawn.  A block a sequence.
#include <math.h>

#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int VF_THREADS = 512, VF_WARPS = VF_THREADS / 32;
constexpr uint64_t VF_ONE = 1ull << 56;

struct VerifyArgs {
  const float* target;
  const float* draft;
  int64_t target_ld, draft_ld;
  int V;
  const int32_t* tokens;
  const int32_t* parent;
  const float* random;
  const int32_t* q_start;
  int T;
  int32_t* out_tokens;
  int32_t* out_path;
  int32_t* out_count;
  int cols;
};

// A probability in steps of 2^-56: above 1 as 1, below 0 and NaN as 0.
__device__ __forceinline__ uint64_t steps(float p) {
  p = fminf(fmaxf(p, 0.f), 1.f);  // NaN: 0
  return __float2ull_rn(p * 72057594037927936.f);
}
// A random number in steps of 2^-64, below 1.
__device__ __forceinline__ uint64_t chance(float u) {
  u = fminf(fmaxf(u, 0.f), 0.99999994f);
  return __float2ull_rz(u * 9223372036854775808.f) << 1;
}
// a b for numbers in steps of 2^-56, cut to a step.
__device__ __forceinline__ uint64_t times(uint64_t a, uint64_t b) { return (__umul64hi(a, b) << 8) | ((a * b) >> 56); }
__device__ __forceinline__ uint64_t less(uint64_t a, uint64_t b) { return a > b ? a - b : 0; }

template <bool DRAFT>
__device__ __forceinline__ uint64_t left_of(const float* p, const float* q, int v, uint64_t S) {
  const uint64_t x = steps(__ldg(p + v));
  return DRAFT && S ? less(x, times(S, steps(__ldg(q + v)))) : x;
}

template <bool DRAFT>
__global__ void __launch_bounds__(VF_THREADS) tree_verify_kernel(const VerifyArgs a) {
  __shared__ uint64_t part[VF_WARPS];  // sums of each warp's stretch of the vocabulary
  __shared__ uint64_t s_S, s_U;
  __shared__ int s_node, s_more, s_refused, s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x, V = a.V;
  pdl_wait();
  pdl_trigger();
  const int row0 = min(max(__ldg(a.q_start + b), 0), a.T);
  const int n = min(max(__ldg(a.q_start + b + 1), row0), a.T) - row0;
  int32_t* out_tokens = a.out_tokens + (int64_t)b * a.cols;
  int32_t* out_path = a.out_path + (int64_t)b * a.cols;
  if (n == 0) {
    for (int i = tid; i < a.cols; i += VF_THREADS) out_tokens[i] = out_path[i] = -1;
    if (tid == 0) a.out_count[b] = 0;
    return;
  }
  const int per = ((V + VF_WARPS - 1) / VF_WARPS + 31) & ~31;  // tokens of a warp's stretch
  const int v0 = min(warp * per, V), v1 = min(v0 + per, V);
  auto target = [&](int node) { return a.target + (int64_t)(row0 + node) * a.target_ld; };
  auto draft = [&](int node) { return DRAFT ? a.draft + (int64_t)(row0 + node) * a.draft_ld : nullptr; };
  auto sum_stretch = [&](int node, uint64_t S) {
    const float* p = target(node);
    const float* q = draft(node);
    uint64_t sum = 0;
#pragma unroll 8
    for (int v = v0 + lane; v < v1; v += 32) sum += left_of<DRAFT>(p, q, v, S);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp] = sum;
  };
  // is token c a child of `node`?
  auto child_at = [&](int node, int c) { return c > node && c < n && __ldg(a.parent + row0 + c) == node; };

  if (warp == 0) {
    // ---- the walk; the other warps add up rows for it
    int node = 0, count = 0;
    bool refused = false;
    uint64_t S = 0, R = VF_ONE;
    for (;;) {
      if (lane == 0) out_path[count] = node;
      ++count;
      S = 0;
      R = VF_ONE;
      refused = false;
      if (count == a.cols) break;
      int next = -1;
      for (int c0 = node + 1; c0 < n && next < 0; c0 += 32) {
        for (unsigned kids = __ballot_sync(0xffffffffu, child_at(node, c0 + lane)); kids; kids &= kids - 1) {
          const int c = c0 + __ffs(kids) - 1, x = __ldg(a.tokens + row0 + c);
          const bool in = x >= 0 && x < V;
          const uint64_t U = chance(__ldg(a.random + row0 + c));
          uint64_t r = in ? left_of<DRAFT>(target(node), draft(node), x, S) : 0;
          bool take;
          if (DRAFT) {
            const uint64_t q = in ? steps(__ldg(draft(node) + x)) : 0;
            take = __umul64hi(times(R, q), U) < r;
          } else {
            // a token that was refused here before has nothing left
            for (int d0 = node + 1; d0 < c && r; d0 += 32) {
              const int d = d0 + lane;
              if (__any_sync(0xffffffffu, d < c && child_at(node, d) && __ldg(a.tokens + row0 + d) == x)) r = 0;
            }
            take = __umul64hi(R, U) < r;
          }
          if (take) {
            next = c;
            break;
          }
          refused = true;
          if (DRAFT) {
            S += R;
            if (lane == 0) {
              s_S = S;
              s_node = node;
              s_more = 1;
            }
            __syncthreads();
            sum_stretch(node, S);
            __syncthreads();
            R = 0;
            for (int w = 0; w < VF_WARPS; ++w) R += part[w];
          } else {
            R = less(R, r);
          }
        }
      }
      if (next < 0) break;
      if (lane == 0) out_tokens[count - 1] = __ldg(a.tokens + row0 + next);
      node = next;
    }
    if (lane == 0) {
      s_S = S;
      s_node = node;
      s_more = 0;
      s_refused = refused;
      s_count = count;
      s_U = chance(__ldg(a.random + row0));
      a.out_count[b] = count;
    }
    for (int i = count + lane; i < a.cols; i += 32) out_tokens[i] = out_path[i] = -1;
    __syncthreads();
  } else {
    for (;;) {
      __syncthreads();
      if (!s_more) break;
      sum_stretch(s_node, s_S);
      __syncthreads();
    }
  }
  // ---- the draw
  const int node = s_node;
  uint64_t S = s_S;
  bool without = !DRAFT && s_refused;  // the refused tokens are out
  for (int round = 0; round < 2; ++round) {
    sum_stretch(node, S);
    __syncthreads();
    if (without) {
      // each refused token once: the first child that has it
      for (int c0 = node + 1 + warp * 32; c0 < n; c0 += VF_THREADS) {
        for (unsigned kids = __ballot_sync(0xffffffffu, child_at(node, c0 + lane)); kids; kids &= kids - 1) {
          const int c = c0 + __ffs(kids) - 1, x = __ldg(a.tokens + row0 + c);
          bool again = x < 0 || x >= V;
          for (int d0 = node + 1; d0 < c && !again; d0 += 32) {
            const int d = d0 + lane;
            again = __any_sync(0xffffffffu, d < c && child_at(node, d) && __ldg(a.tokens + row0 + d) == x);
          }
          if (!again && lane == 0)
            atomicAdd(reinterpret_cast<unsigned long long*>(&part[x / per]), (unsigned long long)(0ull - steps(__ldg(target(node) + x))));
        }
      }
      __syncthreads();
    }
    uint64_t total = 0;
    for (int w = 0; w < VF_WARPS; ++w) total += part[w];
    if (total > 0) {
      // the first token whose running sum is above random * total
      uint64_t rest = __umul64hi(total, s_U);
      int w = 0;
      while (rest >= part[w]) rest -= part[w++];
      if (w != warp) return;
      const float* p = target(node);
      const float* q = draft(node);
      for (int v = v0; v < v1; v += 32) {
        uint64_t x = v + lane < v1 ? left_of<DRAFT>(p, q, v + lane, S) : 0;
        if (without) {
          for (int c0 = node + 1; c0 < n; c0 += 32) {
            int t = child_at(node, c0 + lane) ? __ldg(a.tokens + row0 + c0 + lane) : -1;
            t = t >= v && t < v + 32 ? t : -1;
            for (unsigned who = __ballot_sync(0xffffffffu, t >= 0); who; who &= who - 1)
              if (__shfl_sync(0xffffffffu, t, __ffs(who) - 1) == v + lane) x = 0;
          }
        }
        uint64_t upto = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        const unsigned over = __ballot_sync(0xffffffffu, upto > rest);
        if (over) {
          if (lane == 0) out_tokens[s_count - 1] = v + __ffs(over) - 1;
          return;
        }
        rest -= __shfl_sync(0xffffffffu, upto, 31);
      }
      return;
    }
    // nothing left: from the target's row itself
    __syncthreads();
    if (!without && S == 0) break;
    without = false;
    S = 0;
  }
  if (tid == 0) out_tokens[s_count - 1] = -1;
}

}  // namespace

}  // namespace mt

using namespace mt;

extern "C" mt_status mt_tree_verify(const float* target, int64_t target_ld, const float* draft, int64_t draft_ld, int V,
                                    const int32_t* tokens, const int32_t* parent, const float* random, const int32_t* q_start,
                                    int B, int T, int32_t* out_tokens, int32_t* out_path, int32_t* out_count, int cols,
                                    void* stream) {
  if (!q_start || !out_tokens || !out_path || !out_count || (T > 0 && (!target || !tokens || !parent || !random))) return MT_ERR_NULL;
  if (B < 1 || B > PG_MAX_B || T < 0 || T > (1 << 22) || V < 1 || V > (1 << 24) || cols < 1 || cols > (1 << 20) || target_ld < V ||
      target_ld > ((int64_t)1 << 38) || (draft && (draft_ld < V || draft_ld > ((int64_t)1 << 38))))
    return MT_ERR_SHAPE;
  const void* all[] = {target, draft, tokens, parent, random, q_start, out_tokens, out_path, out_count};
  for (const void* p : all)
    if (!aligned_to(p, 4)) return MT_ERR_ALIGN;
  const ByteRange ins[] = {byte_range(target, rows_bytes(T, target_ld, V, 4)), byte_range(draft, rows_bytes(T, draft_ld, V, 4)),
                           byte_range(tokens, (size_t)T * 4), byte_range(parent, (size_t)T * 4), byte_range(random, (size_t)T * 4),
                           byte_range(q_start, (size_t)(B + 1) * 4)};
  const ByteRange outs[] = {byte_range(out_tokens, (size_t)B * cols * 4), byte_range(out_path, (size_t)B * cols * 4),
                            byte_range(out_count, (size_t)B * 4)};
  for (int i = 0; i < 3; ++i) {
    for (const ByteRange& r : ins)
      if (ranges_overlap(r, outs[i])) return MT_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(outs[i], outs[j])) return MT_ERR_ALIAS;
  }
  if (T == 0) return MT_OK;
  const VerifyArgs a = {target, draft, target_ld, draft_ld, V, tokens, parent, random, q_start, T, out_tokens, out_path, out_count, cols};
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  return draft ? launch(tree_verify_kernel<true>, dim3(B), dim3(VF_THREADS), 0, l, a)
               : launch(tree_verify_kernel<false>, dim3(B), dim3(VF_THREADS), 0, l, a);
}
