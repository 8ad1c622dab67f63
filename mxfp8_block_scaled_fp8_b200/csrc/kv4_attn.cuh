// kv4_attn.cuh -- attention of a few query tokens per sequence over the MXFP4
// paged cache (decode, speculative decode).
//
// For a query row q (one token of one query head) at position t of its
// sequence, over the keys k_j and values v_j of its key/value head, j <= t:
//   s_j = scale * <q, k_j>,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m).
//
// Work split.  A tile is R rows (4, 8 or 16; query tokens x the heads that
// share a key/value head) of one sequence and head; its cost is the sequence's
// length in steps of 32 tokens.  All tiles' steps stand in one line, which is
// cut into equal jobs, whatever the lengths, and every warp works on its own
// job: it lays out its tile, fills its own ring of records by bulk copies and
// keeps its own softmax, with no barrier in the CTA after the plan.  A job's
// part of one tile is a piece.  A tile that is cut leaves partial results
// (unnormalised sum, maximum, sum of weights) and a line in a list, by which a
// second kernel joins them in the order of the jobs.  The plan is made on the
// device from the lengths, so nothing depends on a length that the host
// guessed, and a captured graph follows the lengths in memory.
// Bound by reading the cache, 17 D bytes per 16 tokens and head, once, and close
// behind it by the conversions (two a clock and SM, 8 per record and lane of
// each operand: the ALU pipe is about 60 % busy, HBM about 55 %; neither is
// full).  Measured: 4 contexts of 100003 to 131072 tokens, 32 heads on 8, 100 to
// 109 us a call on different cards, 77 to 71 % of the rate of a copy; 64 of 1 to
// 8192 tokens 68 us, 64 %.  Measured on the way, the long contexts: eight warps of
// a CTA on one piece, joined through shared memory, 117 us; the same with a warp
// that brings the records and one that joins results, 122 us (a CTA waits for its
// slowest warp).
//
// Matrix instructions on registers, not tcgen05: with 4 to 16 rows the product
// is a hundredth of what the tensor cores give, and tcgen05 would want the codes
// as bf16 tiles in shared memory, four times the record's bytes written and read
// again; kv4_prefill.cuh does that where there are rows enough to pay for it.
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
// The rows of a tile share it.  A row whose sums come out small in its units
// (kLow), since another row has met values far above what this one has, is taken
// again by itself with its own: a token with huge values, seen by some of the
// rows, leaves the others their bits.  (That look at the sums takes 0.8 us of 64
// sequences of 1 to 8192 tokens, 66.0 us in a graph; references by row, which cost
// multiplications and registers in every step, took 4 to 8.)
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
  float* partials;       // two per job; nullptr: tiles are not cut
  struct AttnCut* cuts;  // of the tiles that are cut
  struct AttnCounters* counters;
  int32_t unit_steps;    // steps of a unit: 1, or more where the units would not fit 31 bits
  int32_t jobs;          // that the grid has: lines of the list
};

constexpr int kAttnCtas = 2;      // CTAs of an SM (NT = 1)
constexpr int kAttnWarps = 8;     // of a CTA
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kStep = 2;          // groups that a warp takes at once
constexpr int kAttnStages = 2;    // steps of a warp's ring

// Zero between calls.
struct AttnCounters {
  unsigned cut, done;
  unsigned zero[62];  // always: what a workspace that was not zeroed is known by
};
// A tile that is cut over jobs first..last: rows row0.. of a head, of the
// sequence whose rows begin at lo.
struct AttnCut {
  int32_t first, last, lo, head, row0, rows;
};
constexpr float kLn2 = 0.69314718055994531f;

// NT tiles of 8 columns.  FOLD = 2 where a tile has at most four rows: its
// rows stand twice in the eight columns, and columns 4..7 take the second of
// two groups, so that softmax and weights have no idle columns.
template <int D, int NT, int FOLD>
struct AttnCfg {
  static constexpr int R = 8 * NT / FOLD;  // rows of a tile
  static constexpr int kRecord = 17 * D;
  static constexpr int kRingBytes = kAttnStages * kStep * kRecord;  // of a warp
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

// What laying a tile out costs a warp, in steps (each short tile of a batch
// adds its latency: queries, page table, first records, results).  64 sequences
// of 1 to 8192 tokens, in a graph: 74.6 us with 4, 66.9 with 6 (66.0 since), 66.9 with 10.
constexpr int kTileSteps = 6;

struct AttnSeq {
  int lo, n, len;
  uint32_t tiles;  // row tiles x heads
  uint32_t units;  // of one tile; the first ones stand for its layout
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
  const int most = min(p.kv.max_pages * p.kv.page_groups * kGroup, kMostTokens);  // fits: checked on the host
  if (q.len < 0 || q.len > most) {
    record_index_error(kSiteSequence);
    q.n = q.len = 0;
  }
  // rows of a head below 2^31: checked on the host
  q.tiles = (static_cast<uint32_t>(q.n) * p.group + R - 1) / R * p.kv.kv_heads;
  const uint32_t steps = (static_cast<uint32_t>(q.len) + kStep * kGroup - 1) / (kStep * kGroup) + kTileSteps;
  q.units = p.unit_steps == 1 ? steps : (steps + p.unit_steps - 1) / p.unit_steps;
  if (p.partials == nullptr) q.units = 1;
  return q;
}

// Units before each strip of sequences; strip i is [i * per, (i + 1) * per).
// Rising bounds keep the total below 2^31 (the host chose unit_steps for it);
// others, whose rows may count twice, are recorded and nothing is done.
struct AttnPlan {
  uint32_t before[kAttnThreads + 1];
  uint64_t warp_sum[kAttnWarps];
};

template <int R>
__device__ __forceinline__ int attn_plan(const KvAttnArgs& p, AttnPlan& pl) {
  const int per = (p.batch + kAttnThreads - 1) / kAttnThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t sum = 0;
  const int s1 = static_cast<int>(min(static_cast<int64_t>(p.batch), static_cast<int64_t>(threadIdx.x + 1) * per));
  for (int64_t s = static_cast<int64_t>(threadIdx.x) * per; s < s1; ++s) {
    const AttnSeq q = attn_seq<R>(p, static_cast<int>(s));
    sum += min(static_cast<uint64_t>(q.tiles) * q.units, uint64_t{1} << 32);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) pl.warp_sum[warp] = sum;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAttnWarps; ++w) sum += w < warp ? pl.warp_sum[w] : 0u;
  if (threadIdx.x == kAttnThreads - 1 && sum > INT32_MAX) {
    record_index_error(kSiteSequence);
    sum = 0;
  }
  pl.before[threadIdx.x + 1] = static_cast<uint32_t>(sum);
  if (threadIdx.x == 0) pl.before[0] = 0;
  __syncthreads();
  return per;
}

// `total` units cut into `jobs` (<= total) jobs of `q` units, the first `r`
// of them of one more.
struct AttnCutting {
  uint32_t total, jobs, q, r;
  __device__ __forceinline__ uint32_t begin(uint32_t job) const { return job * q + min(job, r); }
  __device__ __forceinline__ uint32_t job_of(uint32_t unit) const {
    const uint32_t wide = r * (q + 1);
    return unit < wide ? unit / (q + 1) : r + (unit - wide) / q;
  }
};

// ------------------------------------------------------------------ one warp's part of a tile

constexpr float kSlack = 2.f;  // how far (log2) a score may pass the running maximum before that moves
constexpr float kHead = 2.f;   // to so far above it
// Scores (log2) from this size on are taken one by one (step_slow): a fused x sc - m has the exact product, m a rounded
// one, and the difference, half an ulp of the score, is below 2^-12 only under it.
constexpr float kExact = 4096.f;
constexpr int kSpare = 10;     // how far E_b may be above what the weights need, to take in the steps' exponents
constexpr int kMinRef = 13;    // so that 2^(127 + kBias - E_b) is finite
// A row's sums below this, in the units that its weights were rounded in, are not to be had from shared references: each
// token is off by 6 * 2^-25 at most where its weight is below f16's normal range (weights of the row's largest score alone
// give 2^(kBias - kHead) * |code| * 2^(e - E_b)).
constexpr float kLow = 1.f;
constexpr int kBias = 12;      // weights enter the second product times 2^kBias: 2^(kSlack + 1 + kBias) < 2^16

// A tile's queries in shared memory, the same for all warps: fragments of the
// columns (lane: column g, elements 32 b + 8 c + 0..7 of each block; FOLD = 2:
// columns 4..7 are zero, and lane ^ 16 has the rows in columns 4..7).
template <int D, int NT, int FOLD>
struct __align__(16) AttnQuery {
  uint4 frag[NT][D / 32][32];
  float factor[8 * NT / FOLD];  // of the rows' scores
};

template <int D, int NT, int FOLD>
struct AttnWarp {
  static constexpr int NB = D / 32, NJ = D / 16, R = 8 * NT / FOLD;
  static constexpr int U = kStep / FOLD;  // score tiles of a step
  using Query = AttnQuery<D, NT, FOLD>;
  float o[NT][NJ][4];          // O^T: rows d = 16 j + g (+ 8), columns 2 c (+ 1)
  float sc[NT][2], m[NT][2], l[NT][2];  // of columns 2 c, 2 c + 1
  float limit[NT][2];          // (m + kSlack) / sc: raw scores above it move the maximum; -inf: all go the slow way
  float unit[NB];              // 2^(127 + kBias - E_b), which tells E_b (kMinRef and up)
  uint32_t ref_half;           // E_b / 2 in bytes, with the bytes' top bits set
  uint32_t spare;              // how far E_b is above what the weights need, in bytes
  int vis[NT][2];              // tokens visible to columns 2 c, 2 c + 1; INT_MAX where the column is no row
  int vis_min;                 // least of them

  // Group, of the FOLD of a score tile, that this lane's columns belong to.
  static __device__ __forceinline__ int fold() { return FOLD == 2 ? (threadIdx.x & 3) >> 1 : 0; }

  __device__ __forceinline__ int ref(int b) const {
    return 254 + kBias - static_cast<int>(__float_as_uint(unit[b]) >> 23);
  }
  __device__ __forceinline__ void set_ref(int b, int e) {
    unit[b] = __uint_as_float(static_cast<uint32_t>(254 + kBias - e) << 23);
    ref_half = (b == 0 ? 0x80808080u : ref_half) | static_cast<uint32_t>(min(e >> 1, 126)) << (8 * b);  // 255: never below
  }

  // The tile's rows, row0 on: this lane's part of column g of each tile.
  static __device__ __forceinline__ void load_queries(const KvAttnArgs& p, const AttnSeq& q, int row0, int head,
                                                      uint4 (&v)[NT][NB]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int rows = q.n * p.group;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int rho = row0 + 8 * t + g;
#pragma unroll
      for (int b = 0; b < NB; ++b) v[t][b] = make_uint4(0, 0, 0, 0);
      if (8 * t + g < R && rho < rows) {
        const int i = rho / p.group;
        const int h = head * p.group + (rho - i * p.group);
        const __nv_bfloat16* src = p.q + static_cast<int64_t>(q.lo + i) * p.q_st + h * p.q_sh + 8 * c;
#pragma unroll
        for (int b = 0; b < NB; ++b) v[t][b] = *reinterpret_cast<const uint4*>(src + 32 * b);
      }
    }
  }
  // The same as query fragments and score factors.
  static __device__ __forceinline__ void put_queries(const KvAttnArgs& p, const uint4 (&v)[NT][NB], Query& to) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t mx = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[t][b].x & 0x7FFF7FFFu, v[t][b].y & 0x7FFF7FFFu),
                                   __vmaxu2(v[t][b].z & 0x7FFF7FFFu, v[t][b].w & 0x7FFF7FFFu)));
      mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      // the row's maximum to [2^13, 2^14): exponent shift in two exact
      // factors, with the scale's sign, so that a score's factor is not negative
      const int ex = mx == 0 ? 0 : 13 + 127 - static_cast<int>(max(mx & 0xFFFFu, mx >> 16) >> 7);
      const float f0 = scale2(p.scale_log2 < 0.f ? -1.f : 1.f, ex / 2), f1 = scale2(1.f, ex - ex / 2);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float f[8];
        bf16x8_to_f32(v[t][b], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * f0 * f1;  // one after the other: f0 f1 may be 2^140
        to.frag[t][b][lane] = make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
      }
      if (c == 0 && 8 * t + g < R) to.factor[8 * t + g] = scale2(fabsf(p.scale_log2), -ex);
    }
  }

  // active: bit i where row i of the tile is worked on.
  __device__ __forceinline__ void begin(const KvAttnArgs& p, const AttnSeq& q, int row0, const Query& from, uint32_t active) {
    const int c = threadIdx.x & 3;
    const int at = row0 / p.group, off = row0 - at * p.group;
    const int seen = q.len - q.n + at + 1;  // tokens visible to the tile's first row
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (8 * t + 2 * c + k) % R;
        sc[t][k] = from.factor[row];
        m[t][k] = limit[t][k] = -INFINITY;
        l[t][k] = 0.f;
        vis[t][k] = (active >> row) & 1u ? seen + (off + row) / p.group : INT_MAX;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[t][j][k] = 0.f;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) set_ref(b, kMinRef);
    spare = 0;
    vis_min = seen;
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
  // 2^(byte b of w - 127) as fp32; 0 for a byte of 0: such blocks, of magnitudes up to 6 * 2^-127, count as zeros in scores
  // and in the fast path's sums.
  static __device__ __forceinline__ float exp_byte(uint32_t w, int b) {
    return __uint_as_float((b == 3 ? w >> 1 : w << (23 - 8 * b)) & 0x7F800000u);
  }

  // S^T of one score tile (FOLD groups at rec) into x, not yet scaled; NaN for a key with a NaN (0 * 2^128).
  __device__ __forceinline__ void scores(const Query& q, const uint8_t* rec, float (&x)[NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    uint32_t kw[FOLD][2][NB];
#pragma unroll
    for (int f = 0; f < FOLD; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h) load_keys(rec + f * 17 * D, h, kw[f][h]);
    // exponents of the lane's tokens
    const uint8_t* er = rec + fold() * 17 * D + 16 * D + g * NB;
    const uint32_t k0 = load_exponents<NB>(er), k1 = load_exponents<NB>(er + 8 * NB);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float d[NT][4];
#pragma unroll
      for (int f = 0; f < FOLD; ++f) {
        uint32_t a[4], a8[4];
        e2m1x8_to_f16(kw[f][0][b], a);
        e2m1x8_to_f16(kw[f][1][b], a8);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint4 qf = q.frag[t][b][lane ^ (16 * f)];
          if (f == 0) mma_f16_zero(d[t], a[0], a8[0], a[1], a8[1], qf.x, qf.y);
          else mma_f16(d[t], a[0], a8[0], a[1], a8[1], qf.x, qf.y);
          mma_f16(d[t], a[2], a8[2], a[3], a8[3], qf.z, qf.w);
        }
      }
      const float f0 = exp_byte(k0, b), f1 = exp_byte(k1, b);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[t][k] = b == 0 ? d[t][k] * (k < 2 ? f0 : f1) : fmaf(d[t][k], k < 2 ? f0 : f1, x[t][k]);
    }
  }

  // O^T += V_b^T (P f) for one score tile, f0 / f1 the factors of the lane's
  // tokens g and g + 8; vw: value words of its groups.
  __device__ __forceinline__ void value_product(const float (&pr)[NT][4], const uint32_t (&vw)[FOLD][NJ], int b,
                                                float f0, float f1) {
    uint32_t b0[NT], b1[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // P^T (token g, columns 2 c, 2 c + 1) to the product's B side (column g, tokens 2 c, 2 c + 1)
      b0[t] = movmatrix_trans(pack_f16(pr[t][0] * f0, pr[t][1] * f0));
      b1[t] = movmatrix_trans(pack_f16(pr[t][2] * f1, pr[t][3] * f1));
    }
#pragma unroll
    for (int f = 0; f < FOLD; ++f) {
      uint32_t v0[4], v1[4];
      e2m1x8_to_f16(vw[f][2 * b], v0);
      e2m1x8_to_f16(vw[f][2 * b + 1], v1);
      // columns of the other group: no weight
      const uint32_t mine = FOLD == 1 || ((threadIdx.x >> 4) & 1) == f ? 0xFFFFFFFFu : 0u;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma_f16(o[t][2 * b], v0[0], v0[1], v0[2], v0[3], b0[t] & mine, b1[t] & mine);
        mma_f16(o[t][2 * b + 1], v1[0], v1[1], v1[2], v1[3], b0[t] & mine, b1[t] & mine);
      }
    }
  }

  // kStep groups at rec, rec + 17 D, .., from token position base on; good:
  // bit i where group i is there (else its tokens count as unseen); len: the
  // sequence's length; release(): called once the records are in registers.
  template <typename F>
  __device__ __forceinline__ void step(const Query& q, const uint8_t* rec, uint32_t good, int base, int len, F release) {
    const int g = (threadIdx.x & 31) >> 2;
    float x[U][NT][4];
    uint32_t ve[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) scores(q, rec + u * FOLD * 17 * D, x[u]);
    // e <= E_b + 1 in every byte, compared by halves
    uint32_t fit = 0x80808080u;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ve[u][h] = load_exponents<NB>(rec + (u * FOLD + fold()) * 17 * D + 16 * D + D / 2 + (g + 8 * h) * NB);
        fit &= ref_half - ((ve[u][h] >> 1) & 0x7F7F7F7Fu);
      }
    bool slow = fit != 0x80808080u || base + kStep * kGroup > vis_min || good != (1u << kStep) - 1;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float mx = fmaxf(x[0][t][k], x[0][t][k + 2]);
#pragma unroll
        for (int u = 1; u < U; ++u) mx = fmaxf(mx, fmaxf(x[u][t][k], x[u][t][k + 2]));
        slow |= mx > limit[t][k];
      }
    if (__any_sync(0xFFFFFFFFu, slow)) {
      step_slow(x, rec, ve, good, base, len, release);
      return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t vw[FOLD][NJ];
#pragma unroll
      for (int f = 0; f < FOLD; ++f) load_values(rec + (u * FOLD + f) * 17 * D, vw[f]);
      if (u == U - 1) release();
      float pr[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int k = 0; k < 4; ++k) pr[t][k] = ex2(fmaf(x[u][t][k], sc[t][k & 1], -m[t][k & 1]));
        l[t][0] += pr[t][0] + pr[t][2];
        l[t][1] += pr[t][1] + pr[t][3];
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
        value_product(pr, vw, b, exp_byte(ve[u][0], b) * unit[b], exp_byte(ve[u][1], b) * unit[b]);
    }
  }

  // Value blocks with a NaN: into the sums of the rows that see their tokens, and their exponents out of the way.  end:
  // positions of the lane's tokens.
  __device__ __forceinline__ void put_nan(uint32_t (&ve)[U][2], const int (&end)[U][2]) {
    const float nan = __int_as_float(0x7FC00000);
    uint32_t hit[NT][2] = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t values = bytes_255(ve[u][h]);
        ve[u][h] &= ~((values >> 7) * 0xFFu);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (end[u][h] < vis[t][k]) hit[t][k] |= values;
      }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) hit[t][k] |= __shfl_xor_sync(0xFFFFFFFFu, hit[t][k], off);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if ((hit[t][k] >> (8 * (j / 2) + 7)) & 1u) o[t][j][k] = o[t][j][k + 2] = nan;
      }
  }

  // The same with masks, a new maximum or new references.
  template <typename F>
  __device__ __forceinline__ void step_slow(float (&x)[U][NT][4], const uint8_t* rec, uint32_t (&ve)[U][2],
                                            uint32_t good, int base, int len, F release) {
    const int g = (threadIdx.x & 31) >> 2;
    float r[NT][2];
    int top[U][2];    // exponents of the largest weights of the lane's tokens (p < 2^top)
    int drop = 1000;  // how far the references may fall: the maxima's least rise
    int end[U][2];    // position of the lane's tokens, INT_MAX where there is no record
    uint32_t nan = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int gr = u * FOLD + fold();
        const int at = (good >> gr) & 1u ? base + kGroup * gr + g + 8 * h : INT_MAX;
        end[u][h] = at;
        top[u][h] = -1000;
        if (at >= len) ve[u][h] = 0;  // exponents of tokens behind the sequence may be anything
        nan |= bytes_255(ve[u][h]);
      }
    if (__builtin_expect(__any_sync(0xFFFFFFFFu, nan != 0), 0)) put_nan(ve, end);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool row = vis[t][k] != INT_MAX;
        const int seen = min(vis[t][k], len);
        float mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& y = x[u][t][k + 2 * h];
            y = end[u][h] >= seen ? -INFINITY : __fmul_rn(y, sc[t][k]);
            mx = fmaxf(mx, y);
          }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        if constexpr (FOLD == 2) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));  // one maximum for both halves of a row
        const bool same = !(mx > m[t][k] + kSlack);
        const float mn = same ? m[t][k] : mx + kHead;
        r[t][k] = same ? 1.f : ex2(m[t][k] - mn);
        // a column that is no row, or has met nothing yet, holds no sum that the references must keep
        if (row && m[t][k] != -INFINITY) drop = min(drop, same ? 0 : static_cast<int>(fminf(mn - m[t][k], 1000.f)));
        m[t][k] = mn;
        limit[t][k] = fabsf(mn) >= kExact ? -INFINITY : (sc[t][k] > 0.f ? (mn + kSlack) / sc[t][k] : INFINITY);
        const float at = mn == -INFINITY ? 0.f : mn;
        l[t][k] *= r[t][k];
#pragma unroll
        for (int u = 0; u < U; ++u)
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
      int need = max(old - static_cast<int>((spare >> (8 * b)) & 0xFFu) - drop, kMinRef), all = 0;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int one = static_cast<int>((ve[u][h] >> (8 * b)) & 0xFFu);
          need = max(need, one + top[u][h]);
          all = max(all, one);
        }
      need = __reduce_max_sync(0xFFFFFFFFu, need);
      const int e = max(need, min(need + kSpare, max(old, __reduce_max_sync(0xFFFFFFFFu, all))));
      spare = (spare & ~(0xFFu << (8 * b))) | static_cast<uint32_t>(e - need) << (8 * b);
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
    for (int u = 0; u < U; ++u) {
      uint32_t vw[FOLD][NJ];
#pragma unroll
      for (int f = 0; f < FOLD; ++f) load_values(rec + (u * FOLD + f) * 17 * D, vw[f]);
      if (u == U - 1) release();
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

  // Sums in real units, maxima and sums of weights of the columns; the two
  // folds joined (then columns 2 c, 2 c + 1 of the lanes with c < 2 count).
  // Returns the rows, of several active ones, whose sums in a block are below kLow.
  __device__ __forceinline__ uint32_t finish(uint32_t active) {
    uint32_t low = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      bool under[2] = {false, false};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[t][k] += __shfl_xor_sync(0xFFFFFFFFu, l[t][k], off);
        if constexpr (FOLD == 2) l[t][k] += __shfl_xor_sync(0xFFFFFFFFu, l[t][k], 2);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float top[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 2 * b; j < 2 * b + 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float& y = o[t][j][k];
            if constexpr (FOLD == 2) y += __shfl_xor_sync(0xFFFFFFFFu, y, 2);
            top[k & 1] = fmaxf(top[k & 1], fabsf(y));
            y = scale2(y, ref(b) - 127 - kBias);
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // (a block of zeros leaves E_b where it began)
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], off));
          under[k] |= top[k] < kLow && ref(b) > kMinRef;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, under[k] && l[t][k] > 0.f);  // lane c of a column 8 t + 2 c + k
#pragma unroll
        for (int c = 0; c < (FOLD == 2 ? 2 : 4); ++c) low |= ((who >> c) & 1u) << (8 * t + 2 * c + k);
      }
    }
    return (active & (active - 1)) != 0 ? low & active : 0;
  }
  // After finish(): f(row, d, value) for this lane's elements.
  template <typename F>
  __device__ __forceinline__ void elements(F f) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    if (FOLD == 2 && c >= 2) return;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < NJ; ++j) f(t, k & 1, 8 * t + 2 * c + (k & 1), 16 * j + g + 8 * (k >> 1), o[t][j][k]);
  }
};

// A job's part of a tile: groups [g0, g1) of sequence s and one head.
struct AttnPiece {
  AttnSeq q;
  int s, head, g0, g1;
  int row0;             // the tile's first row among the sequence's rows of a head
  uint32_t i0, i1;      // units of the tile
  uint32_t u, end;      // units of the piece
  uint32_t base;        // units before sequence s
  uint32_t job, job_u, job_end;  // the job and its units
};

// The piece that begins at unit pc.u of its job, going on from sequence pc.s.
template <int R>
__device__ __forceinline__ void attn_piece(const KvAttnArgs& p, AttnPiece& pc) {
  while (pc.u >= pc.base + pc.q.tiles * pc.q.units) {
    pc.base += pc.q.tiles * pc.q.units;
    pc.q = attn_seq<R>(p, ++pc.s);
  }
  const uint32_t tile = (pc.u - pc.base) / pc.q.units;
  pc.i0 = pc.base + tile * pc.q.units;
  pc.i1 = pc.i0 + pc.q.units;
  pc.end = min(pc.job_end, pc.i1);
  const uint32_t rt = tile / p.kv.kv_heads;
  pc.head = static_cast<int>(tile - rt * p.kv.kv_heads);
  pc.row0 = static_cast<int>(rt * R);
  // groups up to the last row's position
  const int last = min(pc.row0 + R, pc.q.n * p.group) - 1;
  const int seen = pc.q.len - pc.q.n + last / p.group + 1;
  pc.g0 = 0;
  pc.g1 = (max(seen, 0) + kGroup - 1) / kGroup;
  if (p.partials != nullptr) {
    const int from = static_cast<int>(pc.u - pc.i0) * p.unit_steps - kTileSteps;
    const int to = static_cast<int>(pc.end - pc.i0) * p.unit_steps - kTileSteps;
    pc.g0 = max(from, 0) * kStep;
    pc.g1 = min(pc.g1, max(to, 0) * kStep);
  }
}

// The first piece of a job.
template <int R>
__device__ __forceinline__ void attn_job(const KvAttnArgs& p, const AttnPlan& pl, int per, const AttnCutting& cut,
                                         uint32_t job, AttnPiece& pc) {
  pc.job = job;
  pc.job_u = pc.u = cut.begin(job);
  pc.job_end = cut.begin(job + 1);
  int lo = 0, hi = min(kAttnThreads, (p.batch + per - 1) / per);  // before[lo] <= u < before[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pl.before[mid] <= pc.u) lo = mid; else hi = mid;
  }
  pc.s = lo * per;
  pc.base = pl.before[lo];
  pc.q = attn_seq<R>(p, pc.s);
  attn_piece<R>(p, pc);
}

// The rows of the piece's tile, a bit each.
template <int R>
__device__ __forceinline__ uint32_t attn_rows(const KvAttnArgs& p, const AttnPiece& pc) {
  return (1u << min(pc.q.n * p.group - pc.row0, R)) - 1;
}

// Output row `rho` of a tile's sequence and head.
template <int D>
__device__ __forceinline__ void attn_store(const KvAttnArgs& p, int lo, int rho, int head, int d4,
                                           const float (&acc)[4], float mx, float sum) {
  const int64_t i = rho / p.group;
  const int64_t h = head * static_cast<int64_t>(p.group) + (rho - i * p.group);
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
  const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
  *reinterpret_cast<uint2*>(p.out + (lo + i) * p.o_st + h * p.o_sh + 4 * d4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (p.lse != nullptr && d4 == 0)
    p.lse[(lo + i) * p.lse_st + h] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// The rows `done` of a tile that one warp has done alone.
template <int D, int NT, int FOLD>
__device__ __forceinline__ void attn_store_warp(const KvAttnArgs& p, const AttnPiece& pc, const AttnWarp<D, NT, FOLD>& w,
                                                uint32_t done) {
  float inv[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int k = 0; k < 2; ++k) inv[t][k] = w.l[t][k] != 0.f ? 1.f / w.l[t][k] : 0.f;
  w.elements([&](int t, int k, int row, int d, float v) {
    const int rho = pc.row0 + row;
    if (((done >> row) & 1u) == 0) return;
    const int i = rho / p.group;
    const int h = pc.head * p.group + (rho - i * p.group);
    p.out[static_cast<int64_t>(pc.q.lo + i) * p.o_st + h * p.o_sh + d] = __float2bfloat16_rn(v * inv[t][k]);
    if (p.lse != nullptr && d == 0)
      p.lse[static_cast<int64_t>(pc.q.lo + i) * p.lse_st + h] = w.l[t][k] != 0.f ? (w.m[t][k] + log2f(w.l[t][k])) * kLn2 : -INFINITY;
  });
}

// Weight of a partial result with maximum m under the joint maximum mx.
__device__ __forceinline__ float join_weight(float m, float mx) { return m == -INFINITY ? 0.f : ex2(m - mx); }

// A line of the list of cut tiles.  (The join sees to counters that were not zero: nothing is written past the list.)
__device__ __forceinline__ void attn_list_cut(const KvAttnArgs& p, const AttnCut& cut) {
  const unsigned at = atomicAdd(&p.counters->cut, 1u);
  if (at < static_cast<unsigned>(p.jobs)) p.cuts[at] = cut;
}
// The look at a line before it is followed, since in a workspace that was not zeroed it may be anything.
template <int R>
__device__ __forceinline__ bool attn_cut_fits(const KvAttnArgs& p, const AttnCut& cut) {
  if (cut.first >= 0 && cut.first <= cut.last && cut.last < p.jobs && cut.head >= 0 && cut.head < p.kv.kv_heads &&
      cut.lo >= 0 && cut.row0 >= 0 && cut.rows >= 1 && cut.rows <= R &&
      cut.lo + static_cast<int64_t>((static_cast<uint32_t>(cut.row0) + cut.rows - 1) / p.group) < p.rows)
    return true;
  record_error(kDevErrWorkspace, kSiteKvCuts);
  return false;
}

constexpr int kJoinThreads = 256;
constexpr int kJoinAlone = 32;  // pieces that one warp joins alone

// What a warp has of a row: the joint maximum, sum of weights, and elements
// 4 lane .. + 3 of the sum.
struct JoinSum {
  float mx, sum, acc[4];
};

// Pieces from, from + step, .. < n of a cut tile's row, several loads in flight.
template <int D, int R>
__device__ __forceinline__ JoinSum attn_join_pieces(const KvAttnArgs& p, const AttnCut& cut, int row, int from, int step) {
  constexpr int L = D / 4, kAhead = 8, kPart = R * (D + 2);
  const int lane = threadIdx.x & 31, n = cut.last - cut.first + 1;
  // slot 1 of its job where the tile begins there, else slot 0
  const float* part0 = p.partials + 2 * cut.first * static_cast<int64_t>(kPart);
  JoinSum s{-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
  for (int b0 = from; b0 < n; b0 += step * kAhead) {
    float4 v[kAhead];
    float m[kAhead], l[kAhead], top = s.mx;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int b = min(b0 + k * step, n - 1);
      const float* pt = part0 + (2 * b + (b == 0 ? 1 : 0)) * static_cast<int64_t>(kPart);
      m[k] = b0 + k * step < n ? pt[R * D + row] : -INFINITY;
      l[k] = pt[R * D + R + row];
      v[k] = reinterpret_cast<const float4*>(pt + row * D)[lane % L];
      top = fmaxf(top, m[k]);
    }
    const float r = join_weight(s.mx, top);
    s.mx = top;
    s.sum *= r;
#pragma unroll
    for (int k = 0; k < 4; ++k) s.acc[k] *= r;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float f = join_weight(m[k], top);
      s.sum = fmaf(f, l[k], s.sum);
      s.acc[0] = fmaf(f, v[k].x, s.acc[0]);
      s.acc[1] = fmaf(f, v[k].y, s.acc[1]);
      s.acc[2] = fmaf(f, v[k].z, s.acc[2]);
      s.acc[3] = fmaf(f, v[k].w, s.acc[3]);
    }
  }
  return s;
}

// Rows of the cut tiles from their pieces' results, in a fixed order: a warp
// per row, or where a tile has many pieces a CTA per row, its warps taking
// every eighth piece.
template <int D, int R>
__global__ void __launch_bounds__(kJoinThreads) kv4_attn_join_kernel(const KvAttnArgs p) {
  constexpr int W = kJoinThreads / 32, L = D / 4;
  __shared__ float s_mx[W], s_sum[W];
  __shared__ float4 s_acc[W][L];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const unsigned lines = p.counters->cut, items = lines <= static_cast<unsigned>(p.jobs) ? lines * R : 0;
  if (blockIdx.x == 0 && threadIdx.x < 62 && (p.counters->zero[threadIdx.x] != 0 || lines > static_cast<unsigned>(p.jobs)))
    record_error(kDevErrWorkspace, kSiteKvCounters);
  for (unsigned it = blockIdx.x * W + warp; it < items; it += gridDim.x * W) {
    const AttnCut cut = p.cuts[it / R];
    const int row = it % R;
    if (row >= cut.rows || cut.last - cut.first >= kJoinAlone || !attn_cut_fits<R>(p, cut)) continue;
    const JoinSum s = attn_join_pieces<D, R>(p, cut, row, 0, 1);
    if (lane < L) attn_store<D>(p, cut.lo, cut.row0 + row, cut.head, lane, s.acc, s.mx, s.sum);
  }
  for (unsigned it = blockIdx.x; it < items; it += gridDim.x) {
    const AttnCut cut = p.cuts[it / R];
    const int row = it % R;
    if (row >= cut.rows || cut.last - cut.first < kJoinAlone || !attn_cut_fits<R>(p, cut)) continue;
    const JoinSum s = attn_join_pieces<D, R>(p, cut, row, warp, W);
    if (lane < L) s_acc[warp][lane] = make_float4(s.acc[0], s.acc[1], s.acc[2], s.acc[3]);
    if (lane == 0) {
      s_mx[warp] = s.mx;
      s_sum[warp] = s.sum;
    }
    __syncthreads();
    if (threadIdx.x < L) {
      float top = -INFINITY, all = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, s_mx[w]);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = join_weight(s_mx[w], top);
        const float4 v = s_acc[w][threadIdx.x];
        all = fmaf(f, s_sum[w], all);
        o[0] = fmaf(f, v.x, o[0]);
        o[1] = fmaf(f, v.y, o[1]);
        o[2] = fmaf(f, v.z, o[2]);
        o[3] = fmaf(f, v.w, o[3]);
      }
      attn_store<D>(p, cut.lo, cut.row0 + row, cut.head, threadIdx.x, o, top, all);
    }
    __syncthreads();
  }
  __syncthreads();
  // the last CTA that has read the list leaves the counters as they were found
  if (threadIdx.x == 0 && atomicAdd(&p.counters->done, 1u) + 1 == gridDim.x) p.counters->cut = p.counters->done = 0;
}

// A warp's part of the CTA's shared memory.
template <int D, int NT, int FOLD>
struct __align__(128) AttnShared {
  uint8_t ring[AttnCfg<D, NT, FOLD>::kRingBytes];
  AttnQuery<D, NT, FOLD> query;
  AttnPiece piece;
  uint32_t active, low;  // rows of the piece that are worked on; that are to be taken again
  uint64_t full[kAttnStages];
};

// A warp's ring of steps (kStep records each), filled by bulk copies that its
// lane 0 issues: one for a step whose records stand together in a page.
template <int D>
struct AttnRing {
  static constexpr int S = kAttnStages, kRecord = 17 * D;
  uint8_t* buf;
  uint64_t* bar;        // [S]
  uint32_t phase;       // bit i: parity of stage i's next completion
  uint32_t good;        // bits 2 i, 2 i + 1: records of stage i that are there
  uint64_t addr;        // lane i: the first record of the window's step i; bits 0, 1: its records that are there, bit 2: together
  int g0, steps;        // the piece's first group, and its steps
  int last;             // behind its last group
  int issued, taken;    // steps

  // The records of the 32 steps from `issued` on.
  __device__ __forceinline__ void look(const KvCache& kv, int seq, int head) {
    const int gi = g0 + (issued + (threadIdx.x & 31)) * kStep;
    uint64_t a = 0, b = 0;
    if (gi < last) a = reinterpret_cast<uint64_t>(kv_record<D>(kv, seq, gi, head));
    if (gi + 1 < last) b = reinterpret_cast<uint64_t>(kv_record<D>(kv, seq, gi + 1, head));
    addr = a | (a != 0 ? 1u : 0u) | (b != 0 ? 2u : 0u) | (a != 0 && b == a + kRecord ? 4u : 0u);
  }
  __device__ __forceinline__ void issue(const KvCache& kv, int seq, int head) {
    if (issued >= steps) return;
    if (issued % 32 == 0) look(kv, seq, head);
    const uint64_t src = __shfl_sync(0xFFFFFFFFu, addr, issued % 32);
    const int st = issued % S;
    const uint32_t there = static_cast<uint32_t>(src) & 3u;
    good = (good & ~(3u << (2 * st))) | (there << (2 * st));
    if ((threadIdx.x & 31) == 0 && there != 0) {
      uint8_t* dst = buf + st * kStep * kRecord;
      const uint8_t* from = reinterpret_cast<const uint8_t*>(src & ~7ull);
      const bool together = (src & 4u) != 0;
      mbar_arrive_expect_tx(bar + st, there == 3u ? 2 * kRecord : kRecord);
      if (there & 1u) bulk_load(dst, from, together ? 2 * kRecord : kRecord, bar + st);
      if ((there & 2u) && !together)
        bulk_load(dst + kRecord, kv_record<D>(kv, seq, g0 + issued * kStep + 1, head), kRecord, bar + st);
    }
    ++issued;
  }
  __device__ __forceinline__ uint32_t there(int st) const { return (good >> (2 * st)) & 3u; }
  __device__ __forceinline__ void begin(const KvCache& kv, const AttnPiece& pc) {
    g0 = pc.g0;
    last = pc.g1;
    steps = max(0, (pc.g1 - pc.g0 + kStep - 1) / kStep);
    issued = taken = 0;
    for (int i = 0; i < S; ++i) issue(kv, pc.s, pc.head);
  }
};

template <int D, int NT, int FOLD>
__global__ void __launch_bounds__(kAttnThreads, NT == 1 ? kAttnCtas : 1) kv4_attn_kernel(const KvAttnArgs p) {
  using Cfg = AttnCfg<D, NT, FOLD>;
  constexpr int R = Cfg::R, S = kAttnStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ AttnPlan plan;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  AttnShared<D, NT, FOLD>& sh = reinterpret_cast<AttnShared<D, NT, FOLD>*>(smem)[warp];
  if (lane < S) mbar_init(&sh.full[lane], 1);
  fence_mbar_init();
  __syncwarp();
  griddep_launch_dependents();
  griddep_wait();

  const int per = attn_plan<R>(p, plan);
  AttnCutting cut;
  cut.total = plan.before[kAttnThreads];
  cut.jobs = min(gridDim.x * kAttnWarps, cut.total);
  // a job per warp, neighbouring ones on different SMs
  const uint32_t job = warp * gridDim.x + blockIdx.x;
  if (job >= cut.jobs) return;
  cut.q = cut.total / cut.jobs;
  cut.r = cut.total - cut.q * cut.jobs;
  AttnRing<D> ring;
  ring.buf = sh.ring;
  ring.bar = sh.full;
  ring.phase = ring.good = 0;
  AttnWarp<D, NT, FOLD> w;
  AttnPiece& pc = sh.piece;
  bool dead = false;  // a wait expired
  if (lane == 0) attn_job<R>(p, plan, per, cut, job, pc);
  if (lane == 0) sh.active = attn_rows<R>(p, pc), sh.low = 0;
  __syncwarp();
  while (true) {
    {
      uint4 raw[NT][D / 32];
      w.load_queries(p, pc.q, pc.row0, pc.head, raw);
      ring.begin(p.kv, pc);
      w.put_queries(p, raw, sh.query);
    }
    __syncwarp();
    w.begin(p, pc.q, pc.row0, sh.query, sh.active);
    const int len = pc.q.len, seq = pc.s, head = pc.head;
    while (ring.taken < ring.steps) {
      const int st = ring.taken % S;
      const uint32_t there = ring.there(st);
      auto release = [&] {  // the stage is free
        __syncwarp();
        ++ring.taken;
        ring.issue(p.kv, seq, head);
      };
      if (there == 0) {
        release();
        continue;
      }
      if (!warp_wait(ring.bar + st, (ring.phase >> st) & 1u, p.timeout_ns, nullptr, kSiteKvRecord)) {
        dead = true;
        break;
      }
      ring.phase ^= 1u << st;
      w.step(sh.query, ring.buf + st * kStep * Cfg::kRecord, there, (ring.g0 + ring.taken * kStep) * kGroup, len, release);
    }
    if (dead) break;
    // the tile's rows, or the piece's partial result
    const uint32_t active = sh.active, low = w.finish(active), done = active & ~low;
    const bool whole = pc.u == pc.i0 && pc.end == pc.i1, begins = pc.i0 >= pc.job_u;
    if (whole) {
      attn_store_warp<D, NT, FOLD>(p, pc, w, done);
    } else {
      float* part = p.partials + (2 * pc.job + (begins ? 1 : 0)) * static_cast<int64_t>(Cfg::kPartFloats);
      w.elements([&](int t, int k, int row, int d, float v) {
        if (((done >> row) & 1u) == 0) return;
        part[row * D + d] = v;
        if (d == 0) {
          part[R * D + row] = w.m[t][k];
          part[R * D + R + row] = w.l[t][k];
        }
      });
    }
    const uint32_t more = sh.low | low;  // rows to take again, one by one
    __syncwarp();
    if (more != 0) {
      if (lane == 0) sh.active = more & (0u - more), sh.low = more & (more - 1);
      __syncwarp();
      continue;
    }
    if (!whole && begins && lane == 0)  // to the list of cut tiles
      attn_list_cut(p, AttnCut{static_cast<int>(pc.job), static_cast<int>(cut.job_of(pc.i1 - 1)), pc.q.lo, pc.head, pc.row0,
                               min(pc.q.n * p.group - pc.row0, R)});
    if (pc.end >= pc.job_end) break;
    __syncwarp();
    if (lane == 0) {
      pc.u = pc.end;
      attn_piece<R>(p, pc);
      sh.active = attn_rows<R>(p, pc);
    }
    __syncwarp();
  }
  if (dead) {  // copies in flight land before the CTA gives its shared memory back
    for (; ring.taken < ring.issued; ++ring.taken) {
      const int st = ring.taken % S;
      if (ring.there(st) != 0) warp_wait(ring.bar + st, (ring.phase >> st) & 1u, p.timeout_ns, nullptr, kSiteKvDrain);
    }
  }
}

}  // namespace fp8mm
