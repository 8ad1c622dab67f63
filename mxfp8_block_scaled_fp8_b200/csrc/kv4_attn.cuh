// kv4_attn.cuh -- attention of a few query tokens per sequence over the MXFP4
// paged cache (decode, speculative decode).
//
// For a query row q (one token of one query head) at position t of its
// sequence, over the keys k_j and values v_j of its key/value head, j <= t:
//   s_j = scale * <q, k_j>,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m).
//
// Work split.  A tile is R = 8 NT rows (query tokens x the heads that share a
// key/value head) of one sequence and head; its cost is the sequence's length
// in chunks.  All tiles' chunks stand in one line, which is cut into equal
// parts, one per CTA, whatever the lengths; a tile that is cut leaves partial
// results (unnormalised sum, maximum, sum of weights), which the CTA that
// arrives last at the tile's counter joins in a fixed order.  The plan is
// made on the device from the lengths, so nothing depends on a length that the
// host guessed, and a captured graph follows the lengths in memory.
//
// Arithmetic.  Keys and values stay in registers as the record holds them.
// E2M1 -> f16 is one exact conversion per two codes; a 16-token group is the
// 16-row side of m16n8k16 f16 matrix instructions, the rows the 8-column side:
//   S^T[token, row]  = sum over blocks b of 2^(e_k[token, b] - 127) * (K_b Q_b^T)
//   O^T[d, row]     += V_b^T (P 2^(e_v[token, b] - E_b))
// with fp32 accumulators.  Queries are f16 scaled by a power of two per row,
// so that their 8 significant bits are kept from the row's maximum down to
// 2^-27 of it.  A key block's exponent is applied to its fp32 accumulator.
// A value block's exponent joins the weights in fp32, relative to a reference
// E_b, and the product is rounded to f16 once: 11 bits down to 2^-26 of the
// reference, fewer down to 2^-36.  E_b follows the largest weight * 2^e that
// the tile's rows have met, as the softmax's maximum follows the largest
// score, so a token of no weight does not raise it, however large its values.
#pragma once

#include <climits>

#include "kv4.cuh"

namespace fp8mm {

struct KvAttnArgs {
  KvCache kv;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;  // [rows][q heads], or nullptr
  int64_t q_st, q_sh, o_st, o_sh, lse_st;  // elements
  const int32_t *cu, *lens;
  int64_t rows;
  int32_t batch, group;  // group: query heads per key/value head
  float scale_log2;      // scale * log2(e)
  float* partials;       // nullptr: tiles are not cut
  unsigned* counters;    // one per CTA, zero between calls
};

constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kChunkGroups = kAttnWarps;  // groups of a chunk: one per warp
constexpr float kLn2 = 0.69314718055994531f;

template <int D, int NT>
struct AttnCfg {
  static constexpr int R = 8 * NT;
  static constexpr int kRowFloats = D + 4;  // padded row of a warp's partial result
  static constexpr int kSmemBytes = kAttnWarps * R * (kRowFloats + 2) * 4;
  static constexpr int kPartFloats = R * (D + 2);
};

// m16n8k16, f16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held by a warp (lane: row
// lane / 4, columns 2 (lane % 4) and + 1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x * 2^n for |n| <= 250 (clamped; beyond that every finite x under- or
// overflows, but for |x| near the type's limits), by two exact factors.
__device__ __forceinline__ float scale2(float x, int n) {
  n = max(-250, min(250, n));
  const int h = n >> 1;
  return x * __uint_as_float(static_cast<uint32_t>(h + 127) << 23) *
         __uint_as_float(static_cast<uint32_t>(n - h + 127) << 23);
}

// ------------------------------------------------------------------ the plan

struct AttnSeq {
  int lo, n, len;
  int64_t tiles;   // row tiles x heads
  int64_t chunks;  // of one tile
};

template <int R>
__device__ __forceinline__ AttnSeq attn_seq(const KvAttnArgs& p, int s) {
  AttnSeq q;
  q.lo = p.cu != nullptr ? p.cu[s] : s;
  q.n = p.cu != nullptr ? p.cu[s + 1] - q.lo : 1;
  if (q.lo < 0 || q.n < 0 || static_cast<int64_t>(q.lo) + q.n > p.rows) {
    record_index_error(kSiteSequence);
    q.n = 0;
  }
  q.len = p.lens[s];
  const int64_t most = static_cast<int64_t>(p.kv.max_pages) * p.kv.page_groups * kGroup;
  if (q.len < 0 || q.len > most) {
    record_index_error(kSiteSequence);
    q.len = q.len < 0 ? 0 : static_cast<int>(most);
  }
  q.tiles = (static_cast<int64_t>(q.n) * p.group + R - 1) / R * p.kv.kv_heads;
  constexpr int kChunk = kChunkGroups * kGroup;
  q.chunks = p.partials == nullptr ? 1 : max(1, (q.len + kChunk - 1) / kChunk);
  return q;
}

// Units before each strip of sequences; strip i is [i * per, (i + 1) * per).
struct AttnPlan {
  int64_t before[kAttnThreads + 1];
  int64_t warp_sum[kAttnWarps];
  int last;
};

template <int R>
__device__ __forceinline__ int attn_plan(const KvAttnArgs& p, AttnPlan& pl) {
  const int per = (p.batch + kAttnThreads - 1) / kAttnThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t mine = 0;
  const int s1 = min(p.batch, static_cast<int>((threadIdx.x + 1) * per));
  for (int s = threadIdx.x * per; s < s1; ++s) {
    const AttnSeq q = attn_seq<R>(p, s);
    mine += q.tiles * q.chunks;
  }
  int64_t sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) pl.warp_sum[warp] = sum;
  __syncthreads();
  int64_t base = 0;
  for (int w = 0; w < warp; ++w) base += pl.warp_sum[w];
  pl.before[threadIdx.x + 1] = base + sum;
  if (threadIdx.x == 0) pl.before[0] = 0;
  __syncthreads();
  return per;
}

// ------------------------------------------------------------------ one warp's part of a tile

constexpr float kSlack = 2.f;  // how far (log2) a score may pass the running maximum before that moves
constexpr int kBias = 12;      // weights enter the second product times 2^kBias: 2^(kSlack + 1 + kBias) < 2^16

template <int D, int NT>
struct AttnWarp {
  static constexpr int NB = D / 32;
  static constexpr int NJ = D / 16;
  float o[NT][NJ][4];          // O^T: rows d = 16 j + g (+ 8), columns 2 c (+ 1)
  uint32_t qf[NT][NB][4];      // query fragments: column g, elements 32 b + 8 c + 0..7
  float sc[NT][2], m[NT][2], l[NT][2];  // columns 2 c, 2 c + 1
  int ref[NB];                 // E_b
  uint32_t ref_half;           // E_b / 2 in bytes, with the bytes' top bits set
  int vis[NT][2];              // tokens visible to columns 2 c, 2 c + 1; INT_MAX where the column is no row
  int vis_min, vis_max;        // over the tile's rows

  __device__ __forceinline__ void pack_refs() {
    ref_half = 0x80808080u;
#pragma unroll
    for (int b = 0; b < NB; ++b) ref_half |= static_cast<uint32_t>(min(ref[b] >> 1, 127)) << (8 * b);
  }

  // Rows rho = row0 + column of the tile; sequence rows from q.lo.
  __device__ __forceinline__ void begin(const KvAttnArgs& p, const AttnSeq& q, int64_t row0, int head) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int64_t rows = static_cast<int64_t>(q.n) * p.group;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t rho = row0 + 8 * t + g;
      uint4 v[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) v[b] = make_uint4(0, 0, 0, 0);
      if (rho < rows) {
        const int64_t i = rho / p.group;
        const int64_t h = head * static_cast<int64_t>(p.group) + (rho - i * p.group);
        const __nv_bfloat16* src = p.q + (q.lo + i) * p.q_st + h * p.q_sh + 8 * c;
#pragma unroll
        for (int b = 0; b < NB; ++b) v[b] = *reinterpret_cast<const uint4*>(src + 32 * b);
      }
      uint32_t mx = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[b].x & 0x7FFF7FFFu, v[b].y & 0x7FFF7FFFu),
                                   __vmaxu2(v[b].z & 0x7FFF7FFFu, v[b].w & 0x7FFF7FFFu)));
      mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      // the row's maximum to [2^13, 2^14): exponent shift in two exact factors
      const int ex = mx == 0 ? 0 : 13 + 127 - static_cast<int>(max(mx & 0xFFFFu, mx >> 16) >> 7);
      const float f0 = scale2(1.f, ex / 2), f1 = scale2(1.f, ex - ex / 2);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float f[8];
        bf16x8_to_f32(v[b], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[t][b][i] = pack_f16(f[2 * i] * f0 * f1, f[2 * i + 1] * f0 * f1);
      }
      // 2^(e + 1 - 127) is what scores are multiplied by: one factor 2 to take back
      const float inv = scale2(p.scale_log2, -ex - 1);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = 2 * c + k;
        sc[t][k] = __shfl_sync(0xFFFFFFFFu, inv, 4 * col);
        m[t][k] = -INFINITY;
        l[t][k] = 0.f;
        const int64_t r = row0 + 8 * t + col;
        vis[t][k] = r < rows ? q.len - q.n + static_cast<int>(r / p.group) + 1 : INT_MAX;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[t][j][k] = 0.f;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) ref[b] = 0;
    pack_refs();
    const int64_t last = min(row0 + 8 * NT, rows) - 1;
    vis_min = q.len - q.n + static_cast<int>(row0 / p.group) + 1;
    vis_max = q.len - q.n + static_cast<int>(last / p.group) + 1;
  }

  // One group: kw, vw its code words, ke / ve the exponent words of tokens g
  // and g + 8; base: position of its first token; len: the sequence's length.
  __device__ __forceinline__ void group(const uint32_t (&kw)[2][NB], const uint32_t (&ke)[2], const uint32_t (&vw)[NJ],
                                        uint32_t (&ve)[2], int base, int len) {
    float x[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[t][k] = 0.f;
    // exponents one up (their factor 2 is in sc), so that 0 is no zero
    const uint32_t k0 = ke[0] + 0x01010101u, k1 = ke[1] + 0x01010101u;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t a[4], a8[4];
      e2m1x8_to_f16(kw[0][b], a);
      e2m1x8_to_f16(kw[1][b], a8);
      const float f0 = __uint_as_float(((k0 >> (8 * b)) & 0xFFu) << 23);
      const float f1 = __uint_as_float(((k1 >> (8 * b)) & 0xFFu) << 23);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(d, a[0], a8[0], a[1], a8[1], qf[t][b][0], qf[t][b][1]);
        mma_f16(d, a[2], a8[2], a[3], a8[3], qf[t][b][2], qf[t][b][3]);
        x[t][0] = fmaf(d[0], f0, x[t][0]);
        x[t][1] = fmaf(d[1], f0, x[t][1]);
        x[t][2] = fmaf(d[2], f1, x[t][2]);
        x[t][3] = fmaf(d[3], f1, x[t][3]);
      }
    }
    bool slow = base + kGroup > vis_min;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[t][k] *= sc[t][k & 1];
      slow |= fmaxf(x[t][0], x[t][2]) > m[t][0] + kSlack || fmaxf(x[t][1], x[t][3]) > m[t][1] + kSlack;
    }
    // e <= E_b + 1 in every byte, compared by halves; and no E_b past what 2^(e - E_b) needs as a normal fp32
    const uint32_t fit = (ref_half - ((ve[0] >> 1) & 0x7F7F7F7Fu)) & (ref_half - ((ve[1] >> 1) & 0x7F7F7F7Fu));
    slow |= (fit & 0x80808080u) != 0x80808080u;
#pragma unroll
    for (int b = 0; b < NB; ++b) slow |= ref[b] > 126 + kBias;
    if (__any_sync(0xFFFFFFFFu, slow)) {
      group_slow(x, vw, ve, base, len);
      return;
    }
    float pr[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < 4; ++k) pr[t][k] = ex2(x[t][k] - m[t][k & 1]);
      l[t][0] += pr[t][0] + pr[t][2];
      l[t][1] += pr[t][1] + pr[t][3];
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t one = static_cast<uint32_t>(127 + kBias - ref[b]) << 23;
      const float f0 = __uint_as_float((((ve[0] >> (8 * b)) & 0xFFu) << 23) + one);
      const float f1 = __uint_as_float((((ve[1] >> (8 * b)) & 0xFFu) << 23) + one);
      value_product(pr, vw, b, f0, f1);
    }
  }

  // O^T += V_b^T (P f), f0 / f1 the factors of tokens g and g + 8.
  __device__ __forceinline__ void value_product(const float (&pr)[NT][4], const uint32_t (&vw)[NJ], int b, float f0,
                                                float f1) {
    uint32_t v0[4], v1[4];
    e2m1x8_to_f16(vw[2 * b], v0);
    e2m1x8_to_f16(vw[2 * b + 1], v1);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // P^T (token g, columns 2 c, 2 c + 1) to the product's B side (column g, tokens 2 c, 2 c + 1)
      const uint32_t b0 = movmatrix_trans(pack_f16(pr[t][0] * f0, pr[t][1] * f0));
      const uint32_t b1 = movmatrix_trans(pack_f16(pr[t][2] * f1, pr[t][3] * f1));
      mma_f16(o[t][2 * b], v0[0], v0[1], v0[2], v0[3], b0, b1);
      mma_f16(o[t][2 * b + 1], v1[0], v1[1], v1[2], v1[3], b0, b1);
    }
  }

  // The same with masks, a new maximum or new references.
  __device__ __forceinline__ void group_slow(float (&x)[NT][4], const uint32_t (&vw)[NJ], uint32_t (&ve)[2], int base,
                                             int len) {
    const int g = (threadIdx.x & 31) >> 2;
    // exponents of tokens behind the sequence may be anything: 0
    if (base + g >= len) ve[0] = 0;
    if (base + g + 8 >= len) ve[1] = 0;
    float pr[NT][4], r[NT][2];
    int top[2] = {-1000, -1000};  // exponents of the largest weights of tokens g and g + 8 (p < 2^top)
    int drop = 1000;              // how far the references may fall: the maxima's least rise
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool row = vis[t][k] != INT_MAX;
        if (base + g >= min(vis[t][k], len)) x[t][k] = -INFINITY;
        if (base + g + 8 >= min(vis[t][k], len)) x[t][k + 2] = -INFINITY;
        float mx = fmaxf(x[t][k], x[t][k + 2]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        const float mn = fmaxf(m[t][k], mx);
        const bool same = m[t][k] == mn;
        r[t][k] = same ? 1.f : ex2(m[t][k] - mn);
        // a column that is no row, or has met nothing yet, holds no sum that the references must keep
        if (row && m[t][k] != -INFINITY) drop = min(drop, same ? 0 : static_cast<int>(fminf(mn - m[t][k], 1000.f)));
        m[t][k] = mn;
        const float at = mn == -INFINITY ? 0.f : mn;
        pr[t][k] = ex2(x[t][k] - at);
        pr[t][k + 2] = ex2(x[t][k + 2] - at);
        l[t][k] = l[t][k] * r[t][k] + pr[t][k] + pr[t][k + 2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (row && pr[t][k + 2 * h] > 0.f)
            top[h] = max(top[h], static_cast<int>(__float_as_uint(pr[t][k + 2 * h]) >> 23) - 126);
      }
    drop = __reduce_min_sync(0xFFFFFFFFu, drop);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int e0 = static_cast<int>((ve[0] >> (8 * b)) & 0xFFu), e1 = static_cast<int>((ve[1] >> (8 * b)) & 0xFFu);
      const int old = ref[b];
      ref[b] = __reduce_max_sync(0xFFFFFFFFu, max(max(old - drop, 0), max(e0 + top[0], e1 + top[1])));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float s0 = scale2(r[t][0], old - ref[b]), s1 = scale2(r[t][1], old - ref[b]);
#pragma unroll
        for (int j = 2 * b; j < 2 * b + 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[t][j][k] *= (k & 1) ? s1 : s0;
      }
      float pb[NT][4];  // weight * 2^(e - E_b) first, in two steps that neither overflow nor lose bits, then kBias
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) pb[t][k] = fminf(scale2(pr[t][k], (k < 2 ? e0 : e1) - ref[b]), 1.f);
      value_product(pb, vw, b, static_cast<float>(1 << kBias), static_cast<float>(1 << kBias));
    }
    pack_refs();
  }

  // Results to shared memory: [R][kRowFloats] sums in real units, maxima and
  // sums of weights behind them.
  __device__ __forceinline__ void publish(float* so, float* sm, float* sl) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    constexpr int RF = AttnCfg<D, NT>::kRowFloats;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[t][k] += __shfl_xor_sync(0xFFFFFFFFu, l[t][k], off);
        if (g == 0) {
          sm[8 * t + 2 * c + k] = m[t][k];
          sl[8 * t + 2 * c + k] = l[t][k];
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int j = 2 * b; j < 2 * b + 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            so[(8 * t + 2 * c + (k & 1)) * RF + 16 * j + g + 8 * (k >> 1)] =
                scale2(o[t][j][k], ref[b] - 127 - kBias);
      }
    }
  }
};

// Output row `rho` of a tile's sequence and head.
template <int D>
__device__ __forceinline__ void attn_store(const KvAttnArgs& p, const AttnSeq& q, int64_t rho, int head, int d4,
                                           const float (&acc)[4], float mx, float sum) {
  const int64_t i = rho / p.group;
  const int64_t h = head * static_cast<int64_t>(p.group) + (rho - i * p.group);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
  const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
  *reinterpret_cast<uint2*>(p.out + (q.lo + i) * p.o_st + h * p.o_sh + 4 * d4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (p.lse != nullptr && d4 == 0)
    p.lse[(q.lo + i) * p.lse_st + h] = sum > 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// Weight of a partial result with maximum m under the joint maximum mx.
__device__ __forceinline__ float join_weight(float m, float mx) { return m == -INFINITY ? 0.f : ex2(m - mx); }

template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads) kv4_attn_kernel(const KvAttnArgs p) {
  using Cfg = AttnCfg<D, NT>;
  constexpr int R = Cfg::R, RF = Cfg::kRowFloats, NB = D / 32, NJ = D / 16;
  extern __shared__ __align__(16) float smem[];
  __shared__ AttnPlan plan;
  float* so = smem;                               // [warps][R][RF]
  float* sm = smem + kAttnWarps * R * RF;         // [warps][R]
  float* sl = sm + kAttnWarps * R;                // [warps][R]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  griddep_launch_dependents();
  griddep_wait();

  const int per = attn_plan<R>(p, plan);
  const int64_t total = plan.before[kAttnThreads];
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);  // each has at least one unit
  if (blockIdx.x >= ctas) return;
  int64_t u = blockIdx.x * total / ctas;
  const int64_t u_begin = u, u1 = (blockIdx.x + 1) * total / ctas;
  int s;
  int64_t base;  // units before sequence s
  {
    int lo = 0, hi = kAttnThreads;  // before[lo] <= u < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (plan.before[mid] <= u) lo = mid; else hi = mid;
    }
    s = lo * per;
    base = plan.before[lo];
  }
  AttnSeq q = attn_seq<R>(p, s);
  AttnWarp<D, NT> w;
  while (u < u1) {
    while (u >= base + q.tiles * q.chunks) {
      base += q.tiles * q.chunks;
      q = attn_seq<R>(p, ++s);
    }
    const int64_t tile = (u - base) / q.chunks;
    const int64_t i0 = base + tile * q.chunks, i1 = i0 + q.chunks;
    const int head = static_cast<int>(tile % p.kv.kv_heads);
    const int64_t row0 = tile / p.kv.kv_heads * R;
    const int64_t end = min(u1, i1);
    const int groups = (q.len + kGroup - 1) / kGroup;
    int g0 = 0, g1 = groups;
    if (p.partials != nullptr) {
      g0 = static_cast<int>(u - i0) * kChunkGroups;
      g1 = min(groups, static_cast<int>(end - i0) * kChunkGroups);
    }
    w.begin(p, q, row0, head);
    g1 = min(g1, (max(w.vis_max, 0) + kGroup - 1) / kGroup);
    for (int gi = g0 + warp; gi < g1; gi += kAttnWarps) {
      const uint8_t* rec = kv_record<D>(p.kv, s, gi, head);
      if (rec == nullptr) continue;
      uint32_t kw[2][NB], ke[2], vw[NJ], ve[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t* kp = reinterpret_cast<const uint32_t*>(rec + (g + 8 * h) * (D / 2) + c * (D / 8));
#pragma unroll
        for (int b = 0; b < NB; ++b) kw[h][b] = kp[b];
        ke[h] = load_exponents<NB>(rec + 16 * D + (g + 8 * h) * NB);
        ve[h] = load_exponents<NB>(rec + 16 * D + D / 2 + (g + 8 * h) * NB);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        vw[j] = *reinterpret_cast<const uint32_t*>(rec + 8 * D + (j / 4) * 512 + lane * 16 + (j % 4) * 4);
      w.group(kw, ke, vw, ve, gi * kGroup, q.len);
    }
    w.publish(so + warp * R * RF, sm + warp * R, sl + warp * R);
    __syncthreads();
    const bool whole = u == i0 && end == i1;
    const int64_t rows = static_cast<int64_t>(q.n) * p.group;
    float* part = nullptr;
    if (!whole) part = p.partials + (2 * blockIdx.x + (i0 >= u_begin ? 1 : 0)) * static_cast<int64_t>(Cfg::kPartFloats);
    for (int i = threadIdx.x; i < R * D / 4; i += kAttnThreads) {
      const int row = i / (D / 4), d4 = i % (D / 4);
      float mx = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kAttnWarps; ++k) mx = fmaxf(mx, sm[k * R + row]);
#pragma unroll
      for (int k = 0; k < kAttnWarps; ++k) {
        const float f = join_weight(sm[k * R + row], mx);
        const float4 v = *reinterpret_cast<const float4*>(so + (k * R + row) * RF + 4 * d4);
        sum = fmaf(f, sl[k * R + row], sum);
        acc[0] = fmaf(f, v.x, acc[0]);
        acc[1] = fmaf(f, v.y, acc[1]);
        acc[2] = fmaf(f, v.z, acc[2]);
        acc[3] = fmaf(f, v.w, acc[3]);
      }
      if (whole) {
        if (row0 + row < rows) attn_store<D>(p, q, row0 + row, head, d4, acc, mx, sum);
      } else {
        *reinterpret_cast<float4*>(part + row * D + 4 * d4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (d4 == 0) {
          part[R * D + row] = mx;
          part[R * D + R + row] = sum;
        }
      }
    }
    __syncthreads();
    if (!whole) {
      // CTA that holds unit x: the largest b with b * total / ctas <= x
      const int64_t first = ((i0 + 1) * ctas - 1) / total, last = (i1 * ctas - 1) / total;
      if (threadIdx.x == 0) {
        __threadfence();
        const unsigned before = atomicAdd(p.counters + first, 1u);
        plan.last = before == static_cast<unsigned>(last - first);
        if (plan.last) p.counters[first] = 0;  // as found, for the next call
        __threadfence();
      }
      __syncthreads();
      if (plan.last) {
        for (int i = threadIdx.x; i < R * D / 4; i += kAttnThreads) {
          const int row = i / (D / 4), d4 = i % (D / 4);
          if (row0 + row >= rows) continue;
          float mx = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
          for (int64_t b = first; b <= last; ++b) {  // slot 1: the tile begins in that CTA
            const float* pt = p.partials + (2 * b + (b == first ? 1 : 0)) * static_cast<int64_t>(Cfg::kPartFloats);
            mx = fmaxf(mx, __ldcg(pt + R * D + row));
          }
          for (int64_t b = first; b <= last; ++b) {
            const float* pt = p.partials + (2 * b + (b == first ? 1 : 0)) * static_cast<int64_t>(Cfg::kPartFloats);
            const float f = join_weight(__ldcg(pt + R * D + row), mx);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(pt + row * D + 4 * d4));
            sum = fmaf(f, __ldcg(pt + R * D + R + row), sum);
            acc[0] = fmaf(f, v.x, acc[0]);
            acc[1] = fmaf(f, v.y, acc[1]);
            acc[2] = fmaf(f, v.z, acc[2]);
            acc[3] = fmaf(f, v.w, acc[3]);
          }
          attn_store<D>(p, q, row0 + row, head, d4, acc, mx, sum);
        }
      }
      __syncthreads();
    }
    u = end;
  }
}

}  // namespace fp8mm
