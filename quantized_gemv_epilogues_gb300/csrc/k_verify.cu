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
// another order of the sum.  R is at most a row's sum, below 256; S, which grows by
// R with every refused child of a token, has a second word (children that the
// target does not have leave R as it is, so that 256 of them take S past 2^64).
//
// Bound: latency, then memory: a float for each child that is tried and one row
// of p (and of q) for the token that is drawn.  A cluster of blocks shares out a
// sequence's vocabulary.  The parents, tokens, numbers and probabilities of all
// of its children are fetched at the start, in one round of loads; every block
// walks the tree for itself in shared memory, all children of a token in a warp
// at a time; sums over the vocabulary meet through distributed shared memory.
// R is summed up only where another child comes: not in chains.
// Measured: 4.5 us for one token and 1000 words, of which the launch and three
// loads one after the other (starts, parents, probabilities) are most; 0.5 us more
// a level of the walk; one tree of 25 over 151 936 tokens 9.1 us; 64 chains over
// 128 256 23 us, 8.7 of them the rows' bytes.
#include <math.h>

#include <algorithm>

#include "k_cluster.cuh"
#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int VF_THREADS = 512, VF_WARPS = VF_THREADS / 32;
constexpr int VF_TREE = 512;  // tokens of a sequence that are kept in shared memory
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
  int blocks;  // of a sequence
};

// Two floats p in [-1, 1] as integers of steps: p = A 2^-20 + B 2^-40 + C 2^-56,
// each the nearest integer to what the ones before leave (exactly, as p has 24
// bits).  In [8, 16) floats are 2^-20 apart, so that p + 12 rounds p to such steps
// and their number is the difference of the sum's bits and 12's; likewise B from
// [2^-17, 2^-16) and C from [2^-33, 2^-32).  (A conversion to 64 bits runs on the
// FP64 pipe, which kept 64 chains at 43 us; with these 23.)
struct Steps {
  uint32_t a, b, c;  // sums of A, B and C
};
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) { return add2(a, b ^ 0x8000000080000000ull); }
// The sum of the two words' integers, less the magic number's bits twice.
__device__ __forceinline__ uint32_t bits2(uint64_t y, uint32_t magic) { return (uint32_t)y + (uint32_t)(y >> 32) - 2u * magic; }
__device__ __forceinline__ void add_steps(Steps& s, float p0, float p1) {
  constexpr uint32_t M1 = 0x41400000u, M2 = 0x37400000u, M3 = 0x2F400000u;  // 12, 1.5 2^-17, 1.5 2^-33
  constexpr uint64_t TWO = 0x100000001ull;
  const uint64_t p = pack2(p0, p1);
  const uint64_t y1 = add2(p, M1 * TWO), r1 = sub2(p, sub2(y1, M1 * TWO));
  const uint64_t y2 = add2(r1, M2 * TWO), r2 = sub2(r1, sub2(y2, M2 * TWO));
  const uint64_t y3 = add2(r2, M3 * TWO);
  s.a += bits2(y1, M1);
  s.b += bits2(y2, M2);
  s.c += bits2(y3, M3);
}
__device__ __forceinline__ uint64_t whole(const Steps& s) {
  return (uint64_t)((int64_t)(int32_t)s.a << 36) + (uint64_t)((int64_t)(int32_t)s.b << 16) + (uint64_t)(int64_t)(int32_t)s.c;
}
// A probability in steps of 2^-56: above 1 as 1, below 0 and NaN as 0.
__device__ __forceinline__ uint64_t steps(float p) {
  Steps s = {0, 0, 0};
  add_steps(s, __saturatef(p), 0.f);
  return whole(s);
}
// A random number in steps of 2^-64 (whole ones of 2^-56), below 1.
__device__ __forceinline__ uint64_t chance(float u) { return steps(fminf(__saturatef(u), 0.99999994f)) << 8; }
// a b for numbers in steps of 2^-56, cut to a step.
__device__ __forceinline__ uint64_t times(uint64_t a, uint64_t b) { return (__umul64hi(a, b) << 8) | ((a * b) >> 56); }
__device__ __forceinline__ uint64_t less(uint64_t a, uint64_t b) { return a > b ? a - b : 0; }

// S: 0 before a child is refused, then the sum of R over the refused ones, of which
// there are at most 2^22: hi stays below 2^22.
struct Cut {
  uint64_t lo;
  uint32_t hi;
  __device__ __forceinline__ bool none() const { return (lo | hi) == 0; }
  __device__ __forceinline__ bool one() const { return hi == 0 && lo == VF_ONE; }
  __device__ __forceinline__ void add(uint64_t R) {
    lo += R;
    hi += lo < R;
  }
  // S q, cut to a step; from 2^56 steps on as those (p has no more).
  __device__ __forceinline__ uint64_t of(uint64_t q) const {
    const uint64_t low = times(lo, q);
    if (hi == 0) return low;
    const uint64_t high = hi * q;
    if ((__umul64hi(hi, q) | high >> 48) != 0) return VF_ONE;
    return (high << 8) + low;  // q < 2^48, so that low < 2^56
  }
};

template <bool DRAFT>
__device__ __forceinline__ uint64_t left_of(const float* p, const float* q, int v, const Cut& S) {
  const uint64_t x = steps(__ldg(p + v));
  return DRAFT && !S.none() ? less(x, S.of(steps(__ldg(q + v)))) : x;
}

// The sum of x over a warp.
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// The sum of x over the lanes up to and with this one.
__device__ __forceinline__ uint64_t warp_upto(uint64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Two blocks an SM: 64 registers, 20 bytes of them spilled with a draft (98 without
// the bound, and one block).
template <bool DRAFT>
__global__ void __launch_bounds__(VF_THREADS, 2) tree_verify_kernel(const VerifyArgs a) {
  __shared__ int32_t t_parent[VF_TREE], t_token[VF_TREE];
  __shared__ uint64_t t_random[VF_TREE], t_p[VF_TREE], t_q[DRAFT ? VF_TREE : 1];  // in steps
  __shared__ uint64_t part[VF_WARPS];  // sums of each warp's stretch of this block's share of the vocabulary
  __shared__ uint64_t share[2][16];    // of each block's share, in turn
  __shared__ uint64_t s_U;
  __shared__ Cut s_S;
  __shared__ int s_node, s_more, s_refused, s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = a.blocks, V = a.V;
  const int rank = C > 1 ? (int)cluster_rank() : 0, b = blockIdx.x / C;
  if (C > 1) cluster_arrive();  // this block runs: the others may write to it
  pdl_wait();
  pdl_trigger();
  const int row0 = min(max(__ldg(a.q_start + b), 0), a.T);
  const int n = min(max(__ldg(a.q_start + b + 1), row0), a.T) - row0;
  int32_t* out_tokens = a.out_tokens + (int64_t)b * a.cols;
  int32_t* out_path = a.out_path + (int64_t)b * a.cols;
  const bool writes = rank == 0;
  if (n == 0) {
    if (writes) {
      for (int i = tid; i < a.cols; i += VF_THREADS) out_tokens[i] = out_path[i] = -1;
      if (tid == 0) a.out_count[b] = 0;
    }
    __syncwarp();
    if (C > 1) cluster_wait();
    return;
  }
  auto target = [&](int node) { return a.target + (int64_t)(row0 + node) * a.target_ld; };
  auto draft = [&](int node) { return DRAFT ? a.draft + (int64_t)(row0 + node) * a.draft_ld : nullptr; };
  for (int i = tid; i < min(n, VF_TREE); i += VF_THREADS) {
    const int up = __ldg(a.parent + row0 + i), x = __ldg(a.tokens + row0 + i);
    const bool in = up >= 0 && up < i && x >= 0 && x < V;
    t_random[i] = chance(__ldg(a.random + row0 + i));
    t_parent[i] = up;
    t_token[i] = x;
    t_p[i] = in ? steps(__ldg(target(up) + x)) : 0;
    if (DRAFT) t_q[i] = in ? steps(__ldg(draft(up) + x)) : 0;
  }
  __syncthreads();
  auto parent = [&](int i) { return i < VF_TREE ? t_parent[i] : __ldg(a.parent + row0 + i); };
  auto token = [&](int i) { return i < VF_TREE ? t_token[i] : __ldg(a.tokens + row0 + i); };
  // is token c a child of `node`?
  auto child_at = [&](int node, int c) { return c > node && c < n && parent(c) == node; };
  // (whole warps) has a child of `node` before this lane's, c0 + lane, its token x?
  auto said_before = [&](int node, int c0, bool child, int x) {
    const unsigned kids = __ballot_sync(0xffffffffu, child);
    const unsigned same = __match_any_sync(0xffffffffu, x) & kids & ((1u << lane) - 1u);
    bool again = same != 0;
    for (int d0 = node + 1; d0 < c0; d0 += 32) {
      const bool early = child_at(node, d0 + lane);
      const int y = early ? token(d0 + lane) : 0;
      for (unsigned who = __ballot_sync(0xffffffffu, early); who; who &= who - 1) again |= __shfl_sync(0xffffffffu, y, __ffs(who) - 1) == x;
    }
    return child && again;
  };

  // This block's share of the vocabulary, and each warp's stretch of it.  Rows
  // are read four floats at a time where they all lie on 16-byte boundaries.
  const int per_block = ((V + C - 1) / C + 31) & ~31, b0 = min(rank * per_block, V), b1 = min(b0 + per_block, V);
  const int per = ((b1 - b0 + VF_WARPS - 1) / VF_WARPS + 31) & ~31;
  const int v0 = min(b0 + warp * per, b1), v1 = min(v0 + per, b1);
  const bool fours = ((uintptr_t)a.target & 15) == 0 && a.target_ld % 4 == 0 && (!DRAFT || (((uintptr_t)a.draft & 15) == 0 && a.draft_ld % 4 == 0));
  // The sum of a stretch's fours: of p, or of what q leaves of it.  (64 chains with
  // two of p and of q in flight a thread 23.2 us, three 24.4, four 25.4.)
  auto sum_fours = [&](const float* p, const float* q, auto add) {
    uint64_t sum = 0;
    constexpr int F = DRAFT ? 2 : 8;
#pragma unroll 1
    for (int v = v0 + 4 * lane; v + 4 <= v1; v += 128 * F) {
      float4 x[F], y[F];
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const bool in = v + 128 * i + 4 <= v1;
        x[i] = in ? __ldg(reinterpret_cast<const float4*>(p + v + 128 * i)) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (DRAFT) y[i] = in && q ? __ldg(reinterpret_cast<const float4*>(q + v + 128 * i)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      sum += add(x, y);
    }
    return sum;
  };
  auto sum_stretch = [&](int node, const Cut& S) {
    const float* p = target(node);
    const float* q = draft(node);
    uint64_t sum = 0;
    int v = v0 + lane;
    if (fours) {
      if (!DRAFT || S.none()) {
        sum = sum_fours(p, nullptr, [](const auto& x, const auto&) {
          Steps s = {0, 0, 0};
#pragma unroll
          for (const float4& f : x) {
            add_steps(s, __saturatef(f.x), __saturatef(f.y));
            add_steps(s, __saturatef(f.z), __saturatef(f.w));
          }
          return whole(s);
        });
      } else if (S.one()) {
        // one refused, as in every chain: p - q where that is positive
        sum = sum_fours(p, q, [](const auto& x, const auto& y) {
          Steps s = {0, 0, 0};
          auto one = [&](float x, float y) {
            x = __saturatef(x);
            y = __saturatef(y);
            add_steps(s, x > y ? x : 0.f, x > y ? -y : 0.f);
          };
#pragma unroll
          for (int i = 0; i < (int)(sizeof(x) / sizeof(x[0])); ++i) {
            one(x[i].x, y[i].x);
            one(x[i].y, y[i].y);
            one(x[i].z, y[i].z);
            one(x[i].w, y[i].w);
          }
          return whole(s);
        });
      } else {
        sum = sum_fours(p, q, [&](const auto& x, const auto& y) {
          uint64_t s = 0;
          auto one = [&](float x, float y) { s += less(steps(x), S.of(steps(y))); };
#pragma unroll
          for (int i = 0; i < (int)(sizeof(x) / sizeof(x[0])); ++i) {
            one(x[i].x, y[i].x);
            one(x[i].y, y[i].y);
            one(x[i].z, y[i].z);
            one(x[i].w, y[i].w);
          }
          return s;
        });
      }
      v = v1 - (v1 - v0) % 4 + lane;  // a stretch starts on a multiple of 32
    }
#pragma unroll 4
    for (; v < v1; v += 32) sum += left_of<DRAFT>(p, q, v, S);
    sum = warp_sum(sum);
    if (lane == 0) part[warp] = sum;
  };
  // (the whole block, part[] written and a barrier passed) the blocks' sums, in share[turn]
  int turn = 0;
  bool met = C == 1;
  auto meet = [&]() {
    if (!met) cluster_wait();  // every block runs
    met = true;
    turn ^= 1;
    if (tid < C) {
      uint64_t sum = 0;
      for (int w = 0; w < VF_WARPS; ++w) sum += part[w];
      if (C > 1) cluster_put(&share[turn][rank], tid, sum);
      else share[turn][0] = sum;
    }
    __syncwarp();
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };
  auto shared_sum = [&]() {
    uint64_t sum = 0;
    for (int r = 0; r < C; ++r) sum += share[turn][r];
    return sum;
  };

  if (warp == 0) {
    // ---- the walk; the other warps add up rows for it
    int node = 0, count = 0;
    bool refused = false, known = true;  // is R?
    Cut S = {0, 0};
    uint64_t R = VF_ONE;
    for (;;) {
      if (lane == 0 && writes) out_path[count] = node;
      ++count;
      S = {0, 0};
      R = VF_ONE;
      refused = false;
      known = true;
      if (count == a.cols) break;
      int next = -1;
      for (int c0 = node + 1; c0 < n && next < 0; c0 += 32) {
        const int c = c0 + lane;
        const bool child = child_at(node, c);
        unsigned kids = __ballot_sync(0xffffffffu, child);
        if (!kids) continue;
        const int x = child ? token(c) : -1;
        const bool in = x >= 0 && x < V;
        const uint64_t U = !child ? 0 : c < VF_TREE ? t_random[c] : chance(__ldg(a.random + row0 + c));
        const uint64_t p = !in ? 0 : c < VF_TREE ? t_p[c] : steps(__ldg(target(node) + x));
        if (!DRAFT) {
          // all of them at once: R is down by the earlier ones' shares
          const bool several = refused || (kids & (kids - 1)) != 0;
          const uint64_t r = several && said_before(node, c0, child, x) ? 0 : p;
          const uint64_t upto = several ? warp_upto(r, lane) : r;
          const unsigned taken = __ballot_sync(0xffffffffu, child && __umul64hi(less(R, upto - r), U) < r);
          if (taken) {
            next = c0 + __ffs(taken) - 1;
          } else {
            R = less(R, __shfl_sync(0xffffffffu, upto, 31 - __clz(kids)));  // upto the last of them
            refused = true;
          }
          continue;
        }
        const uint64_t q = !in ? 0 : c < VF_TREE ? t_q[DRAFT ? c : 0] : steps(__ldg(draft(node) + x));
        for (; kids; kids &= kids - 1) {
          if (!known) {
            if (lane == 0) {
              s_S = S;
              s_node = node;
              s_more = 1;
            }
            __syncthreads();
            sum_stretch(node, S);
            __syncthreads();
            meet();
            R = shared_sum();
            known = true;
          }
          const int who = __ffs(kids) - 1;
          const uint64_t left = S.none() ? p : less(p, S.of(q));
          if (__shfl_sync(0xffffffffu, (int)(__umul64hi(times(R, q), U) < left), who)) {
            next = c0 + who;
            break;
          }
          S.add(R);
          known = false;
        }
      }
      if (next < 0) break;
      if (lane == 0 && writes) out_tokens[count - 1] = token(next);
      node = next;
    }
    if (lane == 0) {
      s_S = S;
      s_node = node;
      s_more = 0;
      s_refused = refused;
      s_count = count;
      s_U = t_random[0];
      if (writes) a.out_count[b] = count;
    }
    if (writes)
      for (int i = count + lane; i < a.cols; i += 32) out_tokens[i] = out_path[i] = -1;
    __syncthreads();
  } else {
    for (;;) {
      __syncthreads();
      if (!s_more) break;
      sum_stretch(s_node, s_S);
      __syncthreads();
      meet();
    }
  }
  // ---- the draw
  const int node = s_node;
  Cut S = s_S;
  bool without = !DRAFT && s_refused;  // the refused tokens are out
  for (int round = 0; round < 2; ++round) {
    sum_stretch(node, S);
    __syncthreads();
    if (without) {
      // each refused token once: the first child that has it
      for (int c0 = node + 1 + warp * 32; c0 < n; c0 += VF_THREADS) {
        const int c = c0 + lane;
        const bool child = child_at(node, c);
        const int x = child ? token(c) : -1;
        const bool again = said_before(node, c0, child, x);
        if (child && !again && x >= b0 && x < b1) {
          const uint64_t p = c < VF_TREE ? t_p[c] : steps(__ldg(target(node) + x));
          atomicAdd(reinterpret_cast<unsigned long long*>(&part[(x - b0) / per]), (unsigned long long)(0ull - p));
        }
      }
      __syncthreads();
    }
    meet();
    const uint64_t total = shared_sum();
    if (total > 0) {
      // the first token whose running sum is above random * total: its block,
      uint64_t rest = __umul64hi(total, s_U);
      int r = 0;
      while (rest >= share[turn][r]) rest -= share[turn][r++];
      if (r != rank) return;
      // its stretch,
      int w = 0;
      while (rest >= part[w]) rest -= part[w++];
      const int w0 = min(b0 + w * per, b1), w1 = min(w0 + per, b1);
      // and there a few tokens a thread
      const float* p = target(node);
      const float* q = draft(node);
      const int each = (w1 - w0 + VF_THREADS - 1) / VF_THREADS, i0 = min(w0 + tid * each, w1), i1 = min(i0 + each, w1);
      const int lo = min(w0 + (tid & ~31) * each, w1), hi = min(lo + 32 * each, w1);  // of the warp
      auto gone = [&](int v) {  // (whole warps) is v, within [lo, hi), a refused token?
        bool is = false;
        for (int c0 = node + 1; c0 < n; c0 += 32) {
          int t = child_at(node, c0 + lane) ? token(c0 + lane) : -1;
          t = t >= lo && t < hi ? t : -1;
          for (unsigned who = __ballot_sync(0xffffffffu, t >= 0); who; who &= who - 1) is |= __shfl_sync(0xffffffffu, t, __ffs(who) - 1) == v;
        }
        return is;
      };
      uint64_t mine = 0;
      for (int i = 0; i < each; ++i) {
        const int v = i0 + i;
        const bool out = without && gone(v);
        if (v < i1 && !out) mine += left_of<DRAFT>(p, q, v, S);
      }
      const uint64_t upto = warp_upto(mine, lane);
      __syncthreads();  // part[] has been read
      if (lane == 31) part[warp] = upto;
      __syncthreads();
      uint64_t before = upto - mine;
      for (int k = 0; k < warp; ++k) before += part[k];
      const bool here = rest >= before && rest - before < mine;
      if (__any_sync(0xffffffffu, here)) {
        rest -= before;
        bool open = here;
        for (int i = 0; i < each; ++i) {
          const int v = i0 + i;
          const bool out = without && gone(v);
          const uint64_t x = v < i1 && !out ? left_of<DRAFT>(p, q, v, S) : 0;
          if (open && rest < x) {
            out_tokens[s_count - 1] = v;
            open = false;
          }
          rest -= x;
        }
      }
      return;
    }
    // nothing left: from the target's row itself
    __syncthreads();
    if (!without && S.none()) break;
    without = false;
    S = {0, 0};
  }
  if (writes && tid == 0) out_tokens[s_count - 1] = -1;
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
  int derr = 0;
  const DeviceInfo* di = device_info(&derr);
  if (!di) return cuda_fail((cudaError_t)derr);
  VerifyArgs a = {target, draft, target_ld, draft_ld, V, tokens, parent, random, q_start, T, out_tokens, out_path, out_count, cols, 1};
  // as many blocks a sequence as the GPU holds at a time, two an SM, but no fewer
  // than 2048 tokens each (64 chains over 128 256 tokens by 4 blocks 23 us, by 8,
  // two rounds of blocks, 28)
  while (a.blocks < 8 && B * a.blocks * 2 <= 2 * di->sm_count && V / (a.blocks * 2) >= 2048) a.blocks *= 2;
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  const dim3 grid(B * a.blocks);
  auto go = [&](auto kernel) {
    return a.blocks > 1 ? launch_cluster(kernel, a.blocks, grid, dim3(VF_THREADS), 0, l, a) : launch(kernel, grid, dim3(VF_THREADS), 0, l, a);
  };
  return draft ? go(tree_verify_kernel<true>) : go(tree_verify_kernel<false>);
}
