// k_rope.cu - mt_rope_append: per-head RMSNorm, rotary positions with several
// axes, and the write of K and V into the paged cache, in one pass over a
// projection's rows.
//
// Mathematics.  Pair i of a head turns by angle t_i = pos[axis[i]] * f_i:
//   a' = a cos t - b sin t,  b' = b cos t + a sin t.
// Positions are integers, so the angle is taken modulo one turn in integers:
// F_i = f_i / 2 pi as a 64-bit binary fraction (from a 128-bit expansion of
// 1 / 2 pi), and pos * F_i modulo 2^64 is the fraction of a turn, off by at
// most 2^-33 turns at any 31-bit position.  What is left after the nearest
// quarter of a turn goes to sincospif.
//
// Bound: memory, 4 bytes an element (bf16 in, bf16 out), 5.3 TB/s on 11 000
// tokens of 32 + 8 + 8 heads of 128.  A block takes TOK
// tokens (one when there are few) and a range of their heads, computes each
// token's rot/2 sines and cosines once into shared memory, and then L lanes
// take one head's row at a time: each lane holds the 16-byte chunks of both
// halves of its pairs (or two whole chunks), so the rotation needs no
// exchange between lanes and the norm one butterfly over L lanes.
#include "k_paged.cuh"

namespace mt {

namespace {

constexpr int RP_THREADS = 128;

struct RopeArgs {
  PagedArgs pg;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride, qo_stride;
  uint16_t* q_out;
  int q_heads;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  float eps;
  const int32_t* positions;
  int n_axes;
  const float* inv_freq;
  const uint8_t* axis;
  int rot;
  int heads_per_block;
};

// Fraction of a turn that one step of position adds, f / 2 pi modulo 1, as a
// 64-bit binary fraction (truncated).  f = m 2^e with a 24-bit m; the product
// of m with the first 128 fraction bits of 1 / 2 pi is shifted into place.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int ex = (int)((bits >> 23) & 255u);
  const uint64_t m = (bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  const int sh = 64 - ((ex ? ex : 1) - 150);  // right shift of the product that leaves 64 fraction bits
  constexpr uint64_t C_HI = 0x28BE60DB9391054Aull, C_LO = 0x7F09D5F47D4D3770ull;  // 2^128 / 2 pi
  const uint64_t p0 = m * C_LO;
  const uint64_t c0 = __umul64hi(m, C_LO);
  uint64_t p1 = m * C_HI;
  uint64_t p2 = __umul64hi(m, C_HI);
  p1 += c0;
  p2 += p1 < c0 ? 1u : 0u;
  uint64_t r = 0;
  if (sh >= 0 && sh < 64) r = sh ? (p0 >> sh) | (p1 << (64 - sh)) : p0;
  else if (sh < 128 && sh >= 64) r = sh > 64 ? (p1 >> (sh - 64)) | (p2 << (128 - sh)) : p1;
  else if (sh < 192 && sh >= 128) r = p2 >> (sh - 128);
  return (bits >> 31) ? 0ull - r : r;
}

// Cosine and sine of a fraction of a turn.  The nearest quarter is taken off in
// integers, so that what becomes a float is an angle of at most an eighth of a
// turn with all of its bits: both are exact to fp32 relative to their own size,
// next to their zeros too.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t turns) {
  const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(turns - ((uint64_t)quarter << 62));
  float s, c;
  sincospif((float)rest * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
  const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
  return quarter & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

// Where pair i's cosine and sine lie: two neighbouring pairs together, and the
// pairs that neighbouring lanes read at once (8, or 4, apart) side by side.
template <bool ADJ>
__device__ __forceinline__ int cs_at(int i) {
  return ADJ ? (((i >> 1) & 1) * 32 + (i >> 2)) * 2 + (i & 1) : (((i >> 1) & 3) * 16 + (i >> 3)) * 2 + (i & 1);
}

struct Chunk {
  float x[8];
};
__device__ __forceinline__ Chunk chunk_load(const uint16_t* p) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  return Chunk{{bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y), bf16lo(v.z), bf16hi(v.z), bf16lo(v.w), bf16hi(v.w)}};
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ void chunk_store(uint16_t* p, const Chunk& c) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(c.x[0], c.x[1]), pack2(c.x[2], c.x[3]), pack2(c.x[4], c.x[5]), pack2(c.x[6], c.x[7]));
}

template <int L, bool ADJ, int TOK, int BLOCKS>
__global__ void __launch_bounds__(RP_THREADS, BLOCKS) rope_append_kernel(const RopeArgs a) {
  __shared__ __align__(16) float2 cs[TOK][128];  // cosine and sine of each token's pairs, at cs_at()
  __shared__ int seq_sh[TOK];                    // the token's sequence, -1 for none
  __shared__ int64_t at_sh[TOK];                 // its row's first element in the cache, -1 if it has none
  const PagedArgs& pg = a.pg;
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * TOK;
  if (tid < TOK) {
    seq_sh[tid] = -1;
    at_sh[tid] = -1;
  }
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  // which sequence: every thread looks at its share of them (one load's
  // latency for up to 128, where a search would take one per halving)
  for (int b = tid; b < pg.B; b += RP_THREADS) {
    const PagedSeq s = paged_seq(pg, b);
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      const int at = t0 + i - s.row0;
      if (at >= 0 && at < s.n) {
        seq_sh[i] = b;
        const int pl = s.kv - s.n + at;
        if (pl >= 0) {
          const int e = pl / pg.page_size, page = paged_entry(pg, b, e);
          if (page >= 0) at_sh[i] = (int64_t)page * pg.page_stride + (int64_t)(pl - e * pg.page_size) * pg.token_stride;
        }
      }
    }
  }
  const int half = a.rot >> 1;
  for (int i = tid; i < half; i += RP_THREADS) {
    const uint64_t F = turn_fraction(__ldg(a.inv_freq + i));
    const int ax = a.axis ? min((int)__ldg(a.axis + i), a.n_axes - 1) : 0;
    const int32_t* pos = a.positions + (int64_t)ax * pg.T;
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
      if (t0 + k >= pg.T) break;
      cs[k][cs_at<ADJ>(i)] = turn_cos_sin((uint64_t)(int64_t)__ldg(pos + t0 + k) * F);
    }
  }
  __syncthreads();

  const int D = pg.head_dim, chunks = D >> 3, pairs = a.rot >> 4;  // 8-element chunks; chunks of a rotated half
  const int lane = tid % L, grp = tid / L;
  // this lane's chunks of a row: A, and B (-1: none)
  int ca, cb;
  if (ADJ) {
    const int n = (chunks + 1) >> 1;
    ca = lane < n ? lane : -1;
    cb = lane < n && lane + n < chunks ? lane + n : -1;
  } else if (lane < pairs) {
    ca = lane;
    cb = lane + pairs;
  } else {
    ca = lane + pairs < chunks ? lane + pairs : -1;
    cb = -1;
  }
  const int rows = a.q_heads + 2 * pg.kv_heads;
  const int r_lo = blockIdx.y * a.heads_per_block, r_hi = min(rows, r_lo + a.heads_per_block);
  const int per = r_hi - r_lo;
  // the group's rows: token-major; the butterfly below needs whole warps, so
  // every group walks the same number of steps
  const int steps = (TOK * per + RP_THREADS / L - 1) / (RP_THREADS / L);
  for (int s = 0; s < steps; ++s) {
    const int w = s * (RP_THREADS / L) + grp;
    static_assert(TOK <= 2, "w / per");
    const int k = TOK == 2 && w >= per ? 1 : 0, r = r_lo + w - k * per, t = t0 + k;
    const bool is_q = r < a.q_heads, is_v = r >= a.q_heads + pg.kv_heads;
    const int h = is_q ? r : (is_v ? r - a.q_heads - pg.kv_heads : r - a.q_heads);
    const int b = seq_sh[k];
    const bool live = w < TOK * per && b >= 0 && (is_q || at_sh[k] >= 0);
    uint16_t* dst = nullptr;
    Chunk A = {}, Bc = {};
    if (live) {
      const uint16_t* src = (is_q ? a.q + (int64_t)t * a.q_stride : is_v ? a.v + (int64_t)t * a.v_stride : a.k + (int64_t)t * a.k_stride) + h * D;
      if (ca >= 0) A = chunk_load(src + 8 * ca);
      if (cb >= 0) Bc = chunk_load(src + 8 * cb);
      if (is_q) {
        dst = a.q_out + (int64_t)t * a.qo_stride + h * D;
      } else {
        dst = (is_v ? pg.v : pg.k) + at_sh[k] + (int64_t)h * pg.head_stride;
      }
    }
    const uint16_t* gain = is_q ? a.q_norm : is_v ? nullptr : a.k_norm;
    if (a.q_norm || a.k_norm) {  // uniform over the block: the shuffles need every lane
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(A.x[i], A.x[i], fmaf(Bc.x[i], Bc.x[i], ss));
#pragma unroll
      for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (gain && live) {
        const float inv = rsqrtf(ss / (float)D + a.eps);
        if (ca >= 0) {
          const Chunk g = chunk_load(gain + 8 * ca);
#pragma unroll
          for (int i = 0; i < 8; ++i) A.x[i] *= inv * g.x[i];
        }
        if (cb >= 0) {
          const Chunk g = chunk_load(gain + 8 * cb);
#pragma unroll
          for (int i = 0; i < 8; ++i) Bc.x[i] *= inv * g.x[i];
        }
      }
    }
    if (!dst) continue;
    if (!is_v) {
      // two neighbouring pairs' cosines and sines a load
      auto pairs2 = [&](int i) -> float4 { return *reinterpret_cast<const float4*>(&cs[k][cs_at<ADJ>(i)]); };
      if (ADJ) {
        auto turn = [&](Chunk& c, int ch) {
          if (8 * ch < a.rot) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const float4 u = pairs2(4 * ch + i);
              const float x = c.x[2 * i], y = c.x[2 * i + 1], z = c.x[2 * i + 2], v = c.x[2 * i + 3];
              c.x[2 * i] = x * u.x - y * u.y;
              c.x[2 * i + 1] = y * u.x + x * u.y;
              c.x[2 * i + 2] = z * u.z - v * u.w;
              c.x[2 * i + 3] = v * u.z + z * u.w;
            }
          }
        };
        if (ca >= 0) turn(A, ca);
        if (cb >= 0) turn(Bc, cb);
      } else if (lane < pairs) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float4 u = pairs2(8 * lane + i);
          const float x = A.x[i], y = Bc.x[i], z = A.x[i + 1], v = Bc.x[i + 1];
          A.x[i] = x * u.x - y * u.y;
          Bc.x[i] = y * u.x + x * u.y;
          A.x[i + 1] = z * u.z - v * u.w;
          Bc.x[i + 1] = v * u.z + z * u.w;
        }
      }
    }
    if (ca >= 0) chunk_store(dst + 8 * ca, A);
    if (cb >= 0) chunk_store(dst + 8 * cb, Bc);
  }
}

template <int L, bool ADJ>
mt_status rope_launch(const RopeArgs& a0, const Launch& l, int sms) {
  RopeArgs a = a0;
  const int rows = a.q_heads + 2 * a.pg.kv_heads, groups = RP_THREADS / L;
  const int T = a.pg.T;
  // Two tokens a block (11 000 tokens: 61 us as it then was; one: 66, four: 62;
  // 2900 tokens: 21, 21 and 26).  Where the blocks come to several rounds, 32
  // registers a thread (20 to 24 bytes of them spilled) and 16 blocks an SM: 54
  // against 58 us for 11 000 tokens, 33 and 32 for 5800, 24 and 18 for 2900.
  if (T >= 8 * sms) {
    a.heads_per_block = rows;
    const dim3 grid((T + 1) / 2);
    return T >= 48 * sms ? launch(rope_append_kernel<L, ADJ, 2, 16>, grid, dim3(RP_THREADS), 0, l, a)
                         : launch(rope_append_kernel<L, ADJ, 2, 10>, grid, dim3(RP_THREADS), 0, l, a);
  }
  // few tokens: their heads over several blocks, one row per lane group, until
  // the blocks fill the GPU
  int parts = (rows + groups - 1) / groups;
  while (parts > 1 && (long)T * parts > 8L * sms) parts = (parts + 1) / 2;
  a.heads_per_block = (rows + parts - 1) / parts;
  parts = (rows + a.heads_per_block - 1) / a.heads_per_block;
  return launch(rope_append_kernel<L, ADJ, 1, 10>, dim3(T, parts), dim3(RP_THREADS), 0, l, a);
}

}  // namespace

}  // namespace mt

using namespace mt;

extern "C" mt_status mt_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                    int64_t v_stride, int q_heads, const void* q_norm, const void* k_norm, float eps,
                                    const int32_t* positions, int n_axes, const float* inv_freq, const uint8_t* axis,
                                    int rot, mt_rope_pairing pairing, void* q_out, int64_t q_out_stride,
                                    const mt_paged_cache* cache, const mt_paged_batch* batch, void* stream) {
  RopeArgs a = {};
  if (const mt_status st = paged_args(cache, batch, &a.pg)) return st;
  if (!inv_freq || (batch->T > 0 && (!q || !k || !v || !positions || !q_out))) return MT_ERR_NULL;
  if (pairing != MT_ROPE_HALF && pairing != MT_ROPE_ADJACENT) return MT_ERR_FORMAT;
  const int D = cache->head_dim, Hk = cache->kv_heads, T = batch->T;
  if (q_heads < 1 || q_heads > 1024 || n_axes < 1 || n_axes > 8 || rot < 16 || rot > D || rot % 16) return MT_ERR_SHAPE;
  if (q_stride < (int64_t)q_heads * D || k_stride < (int64_t)Hk * D || v_stride < (int64_t)Hk * D ||
      q_out_stride < (int64_t)q_heads * D)
    return MT_ERR_SHAPE;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return MT_ERR_SHAPE;
  if (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_out_stride % 8) return MT_ERR_ALIGN;
  const void* al[] = {q, k, v, q_norm, k_norm, q_out};
  for (const void* p : al)
    if (!aligned_to(p, 16)) return MT_ERR_ALIGN;
  if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 4)) return MT_ERR_ALIGN;
  // tokens are written by blocks that run at the same time
  if (!paged_rows_apart(cache)) return MT_ERR_SHAPE;
  if (!paged_kv_apart(cache)) return MT_ERR_ALIAS;
  const ByteRange iq = byte_range(q, rows_bytes(T, q_stride, (int64_t)q_heads * D, 2));
  const ByteRange oq = byte_range(q_out, rows_bytes(T, q_out_stride, (int64_t)q_heads * D, 2));
  const ByteRange ik = byte_range(k, rows_bytes(T, k_stride, (int64_t)Hk * D, 2));
  const ByteRange iv = byte_range(v, rows_bytes(T, v_stride, (int64_t)Hk * D, 2));
  const ByteRange ck = byte_range(cache->k, paged_cache_bytes(cache)), cv = byte_range(cache->v, paged_cache_bytes(cache));
  const bool in_place = q_out == q && q_out_stride == q_stride;
  if (!in_place && ranges_overlap(oq, iq)) return MT_ERR_ALIAS;
  // in place, k and v may be other columns of the same rows
  const auto beside = [&](const void* p, int64_t stride) {
    if (T < 2 || stride % q_stride) return false;
    int64_t col = ((int64_t)(uintptr_t)p - (int64_t)(uintptr_t)q) / 2 % q_stride;
    if (col < 0) col += q_stride;
    return col >= (int64_t)q_heads * D && col + (int64_t)Hk * D <= q_stride;
  };
  if (ranges_overlap(oq, ik) && !(in_place && beside(k, k_stride))) return MT_ERR_ALIAS;
  if (ranges_overlap(oq, iv) && !(in_place && beside(v, v_stride))) return MT_ERR_ALIAS;
  const ByteRange others[] = {byte_range(positions, (size_t)n_axes * T * 4), byte_range(inv_freq, (size_t)rot * 2),
                              byte_range(axis, rot / 2), byte_range(q_norm, D * 2), byte_range(k_norm, D * 2),
                              byte_range(batch->q_start, (size_t)(batch->B + 1) * 4), byte_range(batch->kv_len, (size_t)batch->B * 4),
                              byte_range(batch->pages, (size_t)((batch->B - 1) * batch->pages_ld + batch->max_pages) * 4)};
  for (const ByteRange& o : others)
    if (ranges_overlap(o, oq) || ranges_overlap(o, ck) || ranges_overlap(o, cv)) return MT_ERR_ALIAS;
  const ByteRange ins[] = {iq, ik, iv, oq};
  for (const ByteRange& o : ins)
    if (ranges_overlap(o, ck) || ranges_overlap(o, cv)) return MT_ERR_ALIAS;
  if (T == 0) return MT_OK;
  int derr = 0;
  const DeviceInfo* di = device_info(&derr);
  if (!di) return cuda_fail((cudaError_t)derr);
  a.pg.err = device_error_ptr();
  if (!a.pg.err) return MT_ERR_CUDA;
  a.q = (const uint16_t*)q;
  a.k = (const uint16_t*)k;
  a.v = (const uint16_t*)v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.qo_stride = q_out_stride;
  a.q_out = (uint16_t*)q_out;
  a.q_heads = q_heads;
  a.q_norm = (const uint16_t*)q_norm;
  a.k_norm = (const uint16_t*)k_norm;
  a.eps = eps;
  a.positions = positions;
  a.n_axes = n_axes;
  a.inv_freq = inv_freq;
  a.axis = axis;
  a.rot = rot;
  const Launch l{(cudaStream_t)stream, mt_get_option(MT_OPT_PDL) != 0};
  // lanes a row needs: one per pair of rotated chunks and one per other chunk
  // (half pairing), or one per two chunks
  const int need = pairing == MT_ROPE_ADJACENT ? (D / 8 + 1) / 2 : D / 8 - rot / 16;
  if (pairing == MT_ROPE_ADJACENT)
    return need <= 8 ? rope_launch<8, true>(a, l, di->sm_count) : rope_launch<16, true>(a, l, di->sm_count);
  return need <= 8    ? rope_launch<8, false>(a, l, di->sm_count)
         : need <= 16 ? rope_launch<16, false>(a, l, di->sm_count)
                      : rope_launch<32, false>(a, l, di->sm_count);
}
