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
  uint64_t timeout_ns;
  float* partials;       // nullptr: tiles are not cut
  unsigned* counters;    // one per CTA, zero between calls
};

constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kStep = 2;                        // groups that a warp takes at once
constexpr int kAttnStages = 2;                  // steps of a warp's ring
constexpr int kChunkGroups = kStep * kAttnWarps;  // groups of a chunk: one step per warp
constexpr float kLn2 = 0.69314718055994531f;

template <int D, int NT>
struct AttnCfg {
  static constexpr int R = 8 * NT;
  static constexpr int kRowFloats = D + 4;  // padded row of a warp's partial result
  static constexpr int kRecord = 17 * D;
  static constexpr int kRingBytes = kAttnWarps * kAttnStages * kStep * kRecord;
  static constexpr int kSmemBytes = kRingBytes + kAttnWarps * R * (kRowFloats + 2) * 4;
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
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
constexpr float kHead = 2.f;   // to so far above it
constexpr int kSpare = 8;      // how far E_b may be above what the weights need, to take in the step's exponents
constexpr int kMinRef = 13;    // so that 2^(127 + kBias - E_b) is finite
constexpr int kBias = 12;      // weights enter the second product times 2^kBias: 2^(kSlack + 1 + kBias) < 2^16

template <int D, int NT>
struct AttnWarp {
  static constexpr int NB = D / 32;
  static constexpr int NJ = D / 16;
  float o[NT][NJ][4];          // O^T: rows d = 16 j + g (+ 8), columns 2 c (+ 1)
  uint32_t qf[NT][NB][4];      // query fragments: column g, elements 32 b + 8 c + 0..7
  float sc[NT][2], m[NT][2], l[NT][2];  // columns 2 c, 2 c + 1
  float unit[NB];              // 2^(127 + kBias - E_b), which tells E_b (kMinRef and up)
  uint32_t ref_half;           // E_b / 2 in bytes, with the bytes' top bits set
  int vis[NT][2];              // tokens visible to columns 2 c, 2 c + 1; INT_MAX where the column is no row
  int vis_min, vis_max;        // over the tile's rows

  __device__ __forceinline__ int ref(int b) const {
    return 254 + kBias - static_cast<int>(__float_as_uint(unit[b]) >> 23);
  }
  __device__ __forceinline__ void set_ref(int b, int e) {
    unit[b] = __uint_as_float(static_cast<uint32_t>(254 + kBias - e) << 23);
    ref_half = (b == 0 ? 0x80808080u : ref_half) | static_cast<uint32_t>(min(e >> 1, 127)) << (8 * b);
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
    for (int b = 0; b < NB; ++b) set_ref(b, kMinRef);
    const int64_t last = min(row0 + 8 * NT, rows) - 1;
    vis_min = q.len - q.n + static_cast<int>(row0 / p.group) + 1;
    vis_max = q.len - q.n + static_cast<int>(last / p.group) + 1;
  }

  // Code words of this lane: keys of tokens g (h = 0) and g + 8; values.
  static __device__ __forceinline__ void load_keys(const uint8_t* rec, int h, uint32_t (&kw)[NB]) {
    const uint8_t* kp = rec + h * 4 * D + (threadIdx.x & 31) * (D / 8);
    if constexpr (NB == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(kp);
      kw[0] = v.x, kw[1] = v.y, kw[2] = v.z, kw[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(kp);
      kw[0] = v.x, kw[1] = v.y;
    }
  }
  static __device__ __forceinline__ void load_values(const uint8_t* rec, uint32_t (&vw)[NJ]) {
#pragma unroll
    for (int j = 0; j < NJ; j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(rec + 8 * D + (j / 4) * 512 + (threadIdx.x & 31) * 16);
      vw[j] = v.x, vw[j + 1] = v.y, vw[j + 2] = v.z, vw[j + 3] = v.w;
    }
  }
  // 2^(byte b of w - 127) as fp32 bits (0 for a byte of 0).
  static __device__ __forceinline__ float exp_byte(uint32_t w, int b) {
    return __uint_as_float((b == 3 ? w >> 1 : w << (23 - 8 * b)) & 0x7F800000u);
  }

  // S^T of one group into x (not yet scaled).
  __device__ __forceinline__ void scores(const uint8_t* rec, float (&x)[NT][4]) {
    const int g = (threadIdx.x & 31) >> 2;
    uint32_t k0w[NB], k1w[NB];
    load_keys(rec, 0, k0w);
    load_keys(rec, 1, k1w);
    // exponents one up (their factor 2 is in sc), so that 0 is no zero
    const uint32_t k0 = load_exponents<NB>(rec + 16 * D + g * NB) + 0x01010101u;
    const uint32_t k1 = load_exponents<NB>(rec + 16 * D + (g + 8) * NB) + 0x01010101u;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t a[4], a8[4];
      e2m1x8_to_f16(k0w[b], a);
      e2m1x8_to_f16(k1w[b], a8);
      const float f0 = exp_byte(k0, b), f1 = exp_byte(k1, b);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float d[4];
        mma_f16_zero(d, a[0], a8[0], a[1], a8[1], qf[t][b][0], qf[t][b][1]);
        mma_f16(d, a[2], a8[2], a[3], a8[3], qf[t][b][2], qf[t][b][3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[t][k] = b == 0 ? d[k] * (k < 2 ? f0 : f1) : fmaf(d[k], k < 2 ? f0 : f1, x[t][k]);
      }
    }
  }

  // O^T += V_b^T (P f) for one group, f0 / f1 the factors of tokens g and g + 8.
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

  // kStep groups at rec, rec + 17 D, from token position base on; good: bit u
  // where group u is there (else its tokens count as unseen); len: the
  // sequence's length.
  __device__ __forceinline__ void step(const uint8_t* rec, uint32_t good, int base, int len) {
    const int g = (threadIdx.x & 31) >> 2;
    float x[kStep][NT][4];
    uint32_t ve[kStep][2];
#pragma unroll
    for (int u = 0; u < kStep; ++u) scores(rec + u * 17 * D, x[u]);
    // e <= E_b + 1 in every byte, compared by halves
    uint32_t fit = 0x80808080u;
#pragma unroll
    for (int u = 0; u < kStep; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ve[u][h] = load_exponents<NB>(rec + u * 17 * D + 16 * D + D / 2 + (g + 8 * h) * NB);
        fit &= ref_half - ((ve[u][h] >> 1) & 0x7F7F7F7Fu);
      }
    bool slow = fit != 0x80808080u || base + kStep * kGroup > vis_min || good != (1u << kStep) - 1;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          x[u][t][k] *= sc[t][k];
          x[u][t][k + 2] *= sc[t][k];
          mx = fmaxf(mx, fmaxf(x[u][t][k], x[u][t][k + 2]));
        }
        slow |= mx > m[t][k] + kSlack;
      }
    if (__any_sync(0xFFFFFFFFu, slow)) {
      step_slow(x, rec, ve, good, base, len);
      return;
    }
#pragma unroll
    for (int u = 0; u < kStep; ++u) {
      uint32_t vw[NJ];
      load_values(rec + u * 17 * D, vw);
      float pr[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int k = 0; k < 4; ++k) pr[t][k] = ex2(x[u][t][k] - m[t][k & 1]);
        l[t][0] += pr[t][0] + pr[t][2];
        l[t][1] += pr[t][1] + pr[t][3];
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
        value_product(pr, vw, b, exp_byte(ve[u][0], b) * unit[b], exp_byte(ve[u][1], b) * unit[b]);
    }
  }

  // The same with masks, a new maximum or new references.
  __device__ __forceinline__ void step_slow(float (&x)[kStep][NT][4], const uint8_t* rec, uint32_t (&ve)[kStep][2],
                                            uint32_t good, int base, int len) {
    const int g = (threadIdx.x & 31) >> 2;
    float r[NT][2];
    int top[kStep][2];  // exponents of the largest weights of tokens g and g + 8 (p < 2^top)
    int drop = 1000;    // how far the references may fall: the maxima's least rise
#pragma unroll
    for (int u = 0; u < kStep; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[u][h] = -1000;
        // exponents of tokens behind the sequence may be anything: 0
        if (base + kGroup * u + g + 8 * h >= len || !((good >> u) & 1u)) ve[u][h] = 0;
      }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool row = vis[t][k] != INT_MAX;
        const int end = min(vis[t][k], len);
        float mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < kStep; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (base + kGroup * u + g + 8 * h >= end || !((good >> u) & 1u)) x[u][t][k + 2 * h] = -INFINITY;
            mx = fmaxf(mx, x[u][t][k + 2 * h]);
          }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        const bool same = !(mx > m[t][k] + kSlack);
        const float mn = same ? m[t][k] : mx + kHead;
        r[t][k] = same ? 1.f : ex2(m[t][k] - mn);
        // a column that is no row, or has met nothing yet, holds no sum that the references must keep
        if (row && m[t][k] != -INFINITY) drop = min(drop, same ? 0 : static_cast<int>(fminf(mn - m[t][k], 1000.f)));
        m[t][k] = mn;
        const float at = mn == -INFINITY ? 0.f : mn;
        l[t][k] *= r[t][k];
#pragma unroll
        for (int u = 0; u < kStep; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float pr = ex2(x[u][t][k + 2 * h] - at);
            x[u][t][k + 2 * h] = pr;
            l[t][k] += pr;
            if (row && pr > 0.f) top[u][h] = max(top[u][h], static_cast<int>(__float_as_uint(pr) >> 23) - 126);
          }
      }
    drop = __reduce_min_sync(0xFFFFFFFFu, drop);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int old = ref(b);
      int e = max(old - drop, kMinRef), all = 0;
#pragma unroll
      for (int u = 0; u < kStep; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int one = static_cast<int>((ve[u][h] >> (8 * b)) & 0xFFu);
          e = max(e, one + top[u][h]);
          all = max(all, one);
        }
      e = __reduce_max_sync(0xFFFFFFFFu, e);
      e = max(e, min(e + kSpare, __reduce_max_sync(0xFFFFFFFFu, all)));
      set_ref(b, e);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float s0 = scale2(r[t][0], old - e), s1 = scale2(r[t][1], old - e);
#pragma unroll
        for (int j = 2 * b; j < 2 * b + 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[t][j][k] *= (k & 1) ? s1 : s0;
      }
    }
#pragma unroll
    for (int u = 0; u < kStep; ++u) {
      uint32_t vw[NJ];
      load_values(rec + u * 17 * D, vw);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int e0 = static_cast<int>((ve[u][0] >> (8 * b)) & 0xFFu) - ref(b);
        const int e1 = static_cast<int>((ve[u][1] >> (8 * b)) & 0xFFu) - ref(b);
        float pb[NT][4];  // weight * 2^(e - E_b): at most 1 where the column is a row
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) pb[t][k] = fminf(scale2(x[u][t][k], k < 2 ? e0 : e1), 1.f);
        value_product(pb, vw, b, static_cast<float>(1 << kBias), static_cast<float>(1 << kBias));
      }
    }
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
                scale2(o[t][j][k], ref(b) - 127 - kBias);
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

// A CTA's part of a tile: groups [g0, g1) of sequence s and one head.
struct AttnPiece {
  AttnSeq q;
  int s, head, g0, g1;
  int64_t base;             // units before sequence s
  int64_t i0, i1, u, end;   // units of the tile; of the piece
  int64_t row0;             // the tile's first row among the sequence's rows of a head
};

// The piece that begins at unit u (which [.., u1) contains), going on from
// sequence pc.s.
template <int R>
__device__ __forceinline__ void attn_piece(const KvAttnArgs& p, AttnPiece& pc, int64_t u, int64_t u1) {
  while (u >= pc.base + pc.q.tiles * pc.q.chunks) {
    pc.base += pc.q.tiles * pc.q.chunks;
    pc.q = attn_seq<R>(p, ++pc.s);
  }
  const int64_t tile = (u - pc.base) / pc.q.chunks;
  pc.i0 = pc.base + tile * pc.q.chunks;
  pc.i1 = pc.i0 + pc.q.chunks;
  pc.u = u;
  pc.end = min(u1, pc.i1);
  pc.head = static_cast<int>(tile % p.kv.kv_heads);
  pc.row0 = tile / p.kv.kv_heads * R;
  // groups up to the last row's position
  const int64_t last = min(pc.row0 + R, static_cast<int64_t>(pc.q.n) * p.group) - 1;
  const int seen = pc.q.len - pc.q.n + static_cast<int>(last / p.group) + 1;
  pc.g0 = 0;
  pc.g1 = (max(seen, 0) + kGroup - 1) / kGroup;
  if (p.partials != nullptr) {
    pc.g0 = static_cast<int>(u - pc.i0) * kChunkGroups;
    pc.g1 = min(pc.g1, static_cast<int>(pc.end - pc.i0) * kChunkGroups);
  }
}

// Joins the warps' results of a piece (in shared memory) and writes the tile's
// rows, or the piece's partial result, and then the tile if this CTA is the
// last of its contributors.
template <int D, int NT>
__device__ __forceinline__ void attn_join(const KvAttnArgs& p, const AttnPiece& pc, const float* so, const float* sm,
                                          const float* sl, int& is_last, int64_t u_begin, int64_t ctas, int64_t total) {
  using Cfg = AttnCfg<D, NT>;
  constexpr int R = Cfg::R, RF = Cfg::kRowFloats;
  const bool whole = pc.u == pc.i0 && pc.end == pc.i1;
  const int64_t rows = static_cast<int64_t>(pc.q.n) * p.group;
  float* part = nullptr;
  if (!whole) part = p.partials + (2 * blockIdx.x + (pc.i0 >= u_begin ? 1 : 0)) * static_cast<int64_t>(Cfg::kPartFloats);
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
      if (pc.row0 + row < rows) attn_store<D>(p, pc.q, pc.row0 + row, pc.head, d4, acc, mx, sum);
    } else {
      *reinterpret_cast<float4*>(part + row * D + 4 * d4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (d4 == 0) {
        part[R * D + row] = mx;
        part[R * D + R + row] = sum;
      }
    }
  }
  __syncthreads();
  if (whole) return;
  // CTA that holds unit x: the largest b with b * total / ctas <= x
  const int64_t first = ((pc.i0 + 1) * ctas - 1) / total, last = (pc.i1 * ctas - 1) / total;
  if (threadIdx.x == 0) {
    __threadfence();
    const unsigned before = atomicAdd(p.counters + first, 1u);
    is_last = before == static_cast<unsigned>(last - first);
    if (is_last) p.counters[first] = 0;  // as found, for the next call
    __threadfence();
  }
  __syncthreads();
  if (is_last) {
    for (int i = threadIdx.x; i < R * D / 4; i += kAttnThreads) {
      const int row = i / (D / 4), d4 = i % (D / 4);
      if (pc.row0 + row >= rows) continue;
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
      attn_store<D>(p, pc.q, pc.row0 + row, pc.head, d4, acc, mx, sum);
    }
  }
  __syncthreads();
}

// A warp's ring of steps (kStep records each), filled by bulk copies that
// its first lanes issue, one per record.
template <int D>
struct AttnRing {
  static constexpr int S = kAttnStages, kRecord = 17 * D, kLook = 32 / kStep;
  uint8_t* buf;
  uint64_t* bar;        // [S]
  uint32_t phase;       // bit i: parity of stage i's next completion
  uint32_t good;        // bit kStep i + u: record u of stage i is there
  uint64_t addr;        // lane kStep i + u: record u of the window's step i, 0 where there is none
  int first, last;      // the piece's groups: this warp's steps begin at first, first + kChunkGroups, .. < last
  int issued, taken;    // steps

  __device__ __forceinline__ void issue(const KvCache& kv, int seq, int head) {
    if (first + issued * kChunkGroups >= last) return;
    const int lane = threadIdx.x & 31;
    if (issued % kLook == 0) {  // look up the records of the next kLook steps
      const int gi = first + (issued + lane / kStep) * kChunkGroups + lane % kStep;
      addr = gi < last ? reinterpret_cast<uint64_t>(kv_record<D>(kv, seq, gi, head)) : 0;
    }
    const uint64_t src = __shfl_sync(0xFFFFFFFFu, addr, issued % kLook * kStep + lane % kStep);
    const int st = issued % S;
    const uint32_t there = __ballot_sync(0xFFFFFFFFu, src != 0) & ((1u << kStep) - 1);
    good = (good & ~(((1u << kStep) - 1) << (kStep * st))) | (there << (kStep * st));
    if (lane == 0 && there != 0) mbar_arrive_expect_tx(bar + st, __popc(there) * kRecord);
    __syncwarp();
    if (lane < kStep && src != 0)
      bulk_load(buf + (st * kStep + lane) * kRecord, reinterpret_cast<const void*>(src), kRecord, bar + st);
    ++issued;
  }
  __device__ __forceinline__ uint32_t there(int st) const { return (good >> (kStep * st)) & ((1u << kStep) - 1); }
  __device__ __forceinline__ void begin(const KvCache& kv, const AttnPiece& pc) {
    first = pc.g0 + (threadIdx.x >> 5) * kStep;
    last = pc.g1;
    issued = taken = 0;
    for (int i = 0; i < S; ++i) issue(kv, pc.s, pc.head);
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, NT == 1 ? 2 : 1) kv4_attn_kernel(const KvAttnArgs p) {
  using Cfg = AttnCfg<D, NT>;
  constexpr int R = Cfg::R, RF = Cfg::kRowFloats, S = kAttnStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ AttnPlan plan;
  __shared__ uint64_t bars[kAttnWarps][S];
  float* so = reinterpret_cast<float*>(smem + Cfg::kRingBytes);  // [warps][R][RF]
  float* sm = so + kAttnWarps * R * RF;                          // [warps][R]
  float* sl = sm + kAttnWarps * R;                               // [warps][R]
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x < kAttnWarps * S) mbar_init(&bars[0][0] + threadIdx.x, 1);
  fence_mbar_init();
  griddep_launch_dependents();
  griddep_wait();

  const int per = attn_plan<R>(p, plan);  // and makes the barriers' set-up visible to the CTA
  const int64_t total = plan.before[kAttnThreads];
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);  // each has at least one unit
  if (blockIdx.x >= ctas) return;
  const int64_t u_begin = blockIdx.x * total / ctas, u1 = (blockIdx.x + 1) * total / ctas;
  AttnPiece pc;
  {
    int lo = 0, hi = kAttnThreads;  // before[lo] <= u_begin < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (plan.before[mid] <= u_begin) lo = mid; else hi = mid;
    }
    pc.s = lo * per;
    pc.base = plan.before[lo];
    pc.q = attn_seq<R>(p, pc.s);
  }
  AttnRing<D> ring;
  ring.buf = smem + warp * (S * kStep * Cfg::kRecord);
  ring.bar = bars[warp];
  ring.phase = ring.good = 0;
  bool dead = false;  // a wait expired: no further copies or waits
  AttnWarp<D, NT> w;
  attn_piece<R>(p, pc, u_begin, u1);
  ring.begin(p.kv, pc);
  while (true) {
    w.begin(p, pc.q, pc.row0, pc.head);
    for (int gi = ring.first; gi < ring.last && !dead; gi += kChunkGroups) {
      const int st = ring.taken % S;
      const uint32_t there = ring.there(st);
      if (there != 0) {
        if (!warp_wait(ring.bar + st, (ring.phase >> st) & 1u, p.timeout_ns, nullptr, kSiteKvRecord)) {
          dead = true;
          break;
        }
        ring.phase ^= 1u << st;
        w.step(ring.buf + st * kStep * Cfg::kRecord, there, gi * kGroup, pc.q.len);
        __syncwarp();  // the stage is free
      }
      ++ring.taken;
      ring.issue(p.kv, pc.s, pc.head);
    }
    // the next piece's first records are on their way while this one is joined
    const AttnPiece done = pc;
    const bool more = pc.end < u1;
    if (more) {
      attn_piece<R>(p, pc, done.end, u1);
      if (!dead) ring.begin(p.kv, pc);
    }
    w.publish(so + warp * R * RF, sm + warp * R, sl + warp * R);
    __syncthreads();
    attn_join<D, NT>(p, done, so, sm, sl, plan.last, u_begin, ctas, total);
    if (!more) break;
  }
  if (dead) {  // the copies in flight land before the CTA gives its shared memory back
    for (; ring.taken < ring.issued; ++ring.taken) {
      const int st = ring.taken % S;
      if (ring.there(st) != 0) warp_wait(ring.bar + st, (ring.phase >> st) & 1u, p.timeout_ns, nullptr, kSiteKvDrain);
    }
  }
}

}  // namespace fp8mm
