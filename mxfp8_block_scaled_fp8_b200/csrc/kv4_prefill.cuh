// kv4_prefill.cuh -- attention of many query tokens per sequence over the
// MXFP4 paged cache (chunked prefill), on tcgen05.
//
// The arithmetic of kv4_attn.cuh for tiles of 256 rows (query tokens x the
// heads that share a key/value head), two halves of 128, the TMEM lanes:
//   S = Q K^T       Q, K bf16 in shared memory, fp32 in TMEM
//   P = 2^(S scale log2 e - m), bf16, written over S
//   O += P V        P from TMEM, V^T bf16 in shared memory, fp32 in TMEM
// Codes become bf16 exactly (a code has two significant bits, the exponent is
// bf16's), so keys and values enter without error; weights are rounded to 8
// bits, and the row's sum is of the fp32 weights.
//
// Warps: 0-3 and 4-7 the softmax of the two halves (a thread per row), 8-10
// bring keys and 11-13 values and write them as bf16 tiles, 14 and 15 issue the
// matrix instructions of a half each.  A step is 64 tokens; its scores have two
// places in TMEM per half, so that the products fill one while the softmax is at
// the other.  Keys and values have a ring of four steps each, freed apart: a key
// tile after its QKs, a value tile after its PVs.  Every warp goes from piece to
// piece on its own, ordered by the barriers of what it reads and writes.
//
// Bounds of a step (256 rows, D = 128), in SM clocks: tensor 1290 (PV 8 x 64;
// QK 16 x 48.6, because its operands' 6 KB pass shared memory at 128 bytes a
// clock), exponentials 1024, writing tiles 400 of shared memory's clocks.
// At D = 64 a step has half the products and the same exponentials, 1024 clocks,
// which bound it: two chunks of 2048 tokens at 16384 take 937 us, 432 of them
// exponentials.
// Measured on two prompts' chunks of 1025 to 2048 tokens in contexts of up to
// 16384, 32 heads on 8 (541 GFLOP): 621 us in a graph, 871 TFLOP/s, 53 % of the
// rate that a plain bf16 GEMM reaches here (626 to 632 a call); when it took 618,
// it was 546 without the conversion to bf16, 598 without the exponentials, 500
// without both: what is left is the tensor pipe beside the softmax's reads and
// writes of TMEM.  What was tried on the way, same work: steps of 128 tokens with
// one place for scores 871 us (the softmax waits for its own products); scores in
// two places but tiles of 128 tokens freed whole 918 us (conversion in the chain);
// steps of 128 tokens whose products are issued as they are ready 713 us; one
// issuing warp 627 us (its waits are the tensor pipe's); four warps for values and
// two for keys 677 us.
//
// Work split: as in kv4_attn.cuh, a job per CTA in a line of costs, which here
// follow the causal mask; cut tiles are joined by the same second kernel.
#pragma once

#include "kv4_attn.cuh"

namespace fp8mm {

constexpr int kPreRows = 256;        // rows of a tile
constexpr int kPreFrom = 96;         // rows of a head and sequence from which this kernel is the faster one (kv4.cu)
constexpr int kPreTokens = 64;       // tokens of a step
constexpr int kPreGroups = kPreTokens / kGroup;
constexpr int kPreStages = 4;        // steps whose keys, and whose values, have a place in shared memory
constexpr int kPreThreads = 512;
constexpr int kPreKeyWarps = 3, kPreValueWarps = 3;  // that write key and value tiles
constexpr float kPreSlack = 8.f;
// A fused s sc - m has the exact product, m a rounded one: from this size of m (log2) on they may be 1 and more apart, up or
// down.  Such a row's weights are 2^((s - base) sc), base its largest raw score, and its m stands at -inf, so that every
// step is searched (pre_search).
constexpr float kPreExact = 16777216.f;
// What a tile costs beside its tokens, in units of 64 tokens (queries to shared
// memory, the chain's fill and drain, the rows' store): 665 us with 6, 630 with
// 8, 621 with 9, 624 with 11.
constexpr int kPreTileCost = 9;
constexpr uint32_t kIdescBf16 = (1u << 4) | (1u << 7) | (1u << 10) | (128u >> 4 << 24);

template <int D>
struct PreCfg {
  static constexpr int kQBlock = 128 * 128;              // 128 rows of 64 bf16
  static constexpr int kKBlock = kPreTokens * 128;
  static constexpr int kQBytes = kPreRows * D * 2;
  static constexpr int kTileBytes = kPreTokens * D * 2;  // of keys: D / 64 blocks; of values: one block of D rows
  static constexpr int kSmemBytes = kQBytes + 2 * kPreStages * kTileBytes + 1024;  // tiles stand on 1024-byte boundaries
};

// kind::f16 products, A from shared memory or from TMEM.
__device__ __forceinline__ void mma_bf16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
#define FP8MM_RIN32(r)                                                                                     \
  "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),       \
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),       \
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),      \
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
// Columns of this thread's lane, loaded and waited for in one statement, so
// that no register is touched before it holds its value.
__device__ __forceinline__ void tmem_load_32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : FP8MM_R32(r)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load_64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Stores of this thread's lane.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::FP8MM_RIN32(r),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------ the plan

struct PreSeq {
  int lo, n, len;
  int rows;        // of a head
  int tiles;       // of a head
};

__device__ __forceinline__ PreSeq pre_seq(const KvAttnArgs& p, int s) {
  const AttnSeq q = attn_seq<kPreRows>(p, s);
  PreSeq r;
  r.lo = q.lo;
  r.n = q.n;
  r.len = q.len;
  r.rows = q.n * p.group;
  r.tiles = (r.rows + kPreRows - 1) / kPreRows;
  return r;
}
// Cost, in units of 64 tokens, of the first `tile` row tiles of one head: a
// tile costs its prefix and the new tokens up to its last row.
__device__ __forceinline__ int64_t pre_cost(const KvAttnArgs& p, const PreSeq& q, int tile) {
  const int64_t t = tile;
  return t * (max(q.len - q.n, 0) / 64 + kPreTileCost) + t * (t + 1) / 2 * kPreRows / p.group / 64;
}

struct PrePiece {
  PreSeq q;
  int s, head, tile;       // sequence, head, row tile
  int row0, k0, k1;        // first row; steps
  int64_t i0, i1, u, end;  // units of the tile; of the piece
  int64_t job_u, job_end;
};

// Above what a call can ask for: the host lets rows * group * heads be 4e9 at
// most, so there are 4e9 / 256 + 4e9 / 128 tiles, of 2^25 units.
constexpr int64_t kPreMostUnits = int64_t{1} << 52;
struct PrePlan {
  int64_t before[kAttnThreads + 1];
  int64_t warp_sum[kAttnThreads / 32];
};

__device__ __forceinline__ int pre_plan(const KvAttnArgs& p, PrePlan& pl) {
  const int per = (p.batch + kAttnThreads - 1) / kAttnThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t sum = 0;
  if (threadIdx.x < kAttnThreads) {
    const int s1 = static_cast<int>(min(static_cast<int64_t>(p.batch), static_cast<int64_t>(threadIdx.x + 1) * per));
    for (int64_t s = static_cast<int64_t>(threadIdx.x) * per; s < s1; ++s) {
      const PreSeq q = pre_seq(p, static_cast<int>(s));
      sum = min(sum + min(pre_cost(p, q, q.tiles), kPreMostUnits / p.kv.kv_heads) * p.kv.kv_heads, kPreMostUnits);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) pl.warp_sum[warp] = sum;
  }
  __syncthreads();
  if (threadIdx.x < kAttnThreads) {
    for (int w = 0; w < warp; ++w) sum += pl.warp_sum[w];
    if (threadIdx.x == kAttnThreads - 1 && sum >= kPreMostUnits) {  // bounds that do not rise, whose rows count twice
      record_index_error(kSiteSequence);
      sum = 0;
    }
    pl.before[threadIdx.x + 1] = sum;
    if (threadIdx.x == 0) pl.before[0] = 0;
  }
  __syncthreads();
  return per;
}

// The piece's rows and its share of the tile's steps.
__device__ __forceinline__ void pre_share(const KvAttnArgs& p, PrePiece& pc) {
  pc.end = min(pc.job_end, pc.i1);
  pc.row0 = pc.tile * kPreRows;
  const int last = min(pc.row0 + kPreRows, pc.q.rows) - 1;
  const int seen = max(pc.q.len - pc.q.n + last / p.group + 1, 0);
  const int64_t steps = (seen + kPreTokens - 1) / kPreTokens, c = pc.i1 - pc.i0;
  pc.k0 = pc.u == pc.i0 ? 0 : static_cast<int>((pc.u - pc.i0) * steps / c);
  pc.k1 = static_cast<int>(pc.end == pc.i1 ? steps : (pc.end - pc.i0) * steps / c);
}
// A job's first piece.  Within a sequence the heads of a row tile stand side
// by side.
__device__ __forceinline__ void pre_first(const KvAttnArgs& p, const PrePlan& pl, int per, int64_t job, int64_t jobs,
                                          int64_t total, PrePiece& pc) {
  const int heads = p.kv.kv_heads;
  pc.job_u = pc.u = job * total / jobs;
  pc.job_end = (job + 1) * total / jobs;
  int lo = 0, hi = min(kAttnThreads, (p.batch + per - 1) / per);
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pl.before[mid] <= pc.u) lo = mid; else hi = mid;
  }
  pc.s = lo * per;
  int64_t base = pl.before[lo];
  pc.q = pre_seq(p, pc.s);
  for (int64_t c; pc.u >= base + (c = pre_cost(p, pc.q, pc.q.tiles) * heads);) {
    base += c;
    pc.q = pre_seq(p, ++pc.s);
  }
  const int64_t x = pc.u - base;
  lo = 0, hi = pc.q.tiles;  // cost(lo) heads <= x < cost(hi) heads
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pre_cost(p, pc.q, mid) * heads <= x) lo = mid; else hi = mid;
  }
  const int64_t c0 = pre_cost(p, pc.q, lo), c = pre_cost(p, pc.q, lo + 1) - c0;
  pc.tile = lo;
  pc.head = static_cast<int>((x - c0 * heads) / c);
  pc.i0 = base + c0 * heads + pc.head * c;
  pc.i1 = pc.i0 + c;
  pre_share(p, pc);
}
// The next one: the next tile's beginning.
__device__ __forceinline__ void pre_next(const KvAttnArgs& p, PrePiece& pc) {
  int64_t c = pc.i1 - pc.i0;
  if (++pc.head == p.kv.kv_heads) {
    pc.head = 0;
    ++pc.tile;
    while (pc.tile >= pc.q.tiles) {
      pc.q = pre_seq(p, ++pc.s);
      pc.tile = 0;
    }
    c = pre_cost(p, pc.q, pc.tile + 1) - pre_cost(p, pc.q, pc.tile);
  }
  pc.u = pc.i0 = pc.i1;
  pc.i1 = pc.i0 + c;
  pre_share(p, pc);
}

// ------------------------------------------------------------------ the kernel

template <int D>
struct PreShared {
  PrePlan plan;
  PrePiece piece[kPreThreads / 32];  // of each warp: they go from piece to piece on their own
  uint64_t full[2][kPreStages], empty[2][kPreStages];  // of keys, of values
  uint64_t q_full[2], s_full[2][2], p_full[2][2], pv_done[2][2], drain;
  float base[kPreRows];  // PreRow::base
  uint32_t tmem;
  int abort;
};

// One group's keys or values in registers, as the lanes of a warp hold them
// (zeros without a record); base: position of its first token.
template <int D>
struct PreKeys {
  static constexpr int NB = D / 32;
  uint32_t w[2][NB], e[2];

  // (a score is written over where a row does not see its token)
  static __device__ __forceinline__ void make_finite(uint8_t*, int) {}
  __device__ __forceinline__ void load(const uint8_t* rec, int, int) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      e[h] = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) w[h][b] = 0;
      if (rec == nullptr) continue;
      const uint8_t* kp = rec + h * 4 * D + lane * (D / 8);
      if constexpr (NB == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(kp);
        w[h][0] = v.x, w[h][1] = v.y, w[h][2] = v.z, w[h][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(kp);
        w[h][0] = v.x, w[h][1] = v.y;
      }
      e[h] = load_exponents<NB>(rec + 16 * D + (g + 8 * h) * NB);
    }
  }
  // Into the tile [token][d]: blocks of 64 d, rows of 128 bytes whose 16-byte
  // chunks are permuted by the row (128-byte swizzle).  at: the group's place.
  __device__ __forceinline__ void store(uint8_t* tile, int at) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        // rows of odd g take the other half of their 128 bytes: the 8 lanes
        // of a phase meet all banks
        const int odd = (b ^ g) & 1, row = at * kGroup + g + 8 * h, chunk = odd * 4 + c;
        *reinterpret_cast<uint4*>(tile + (b >> 1) * PreCfg<D>::kKBlock + row * 128 + ((chunk ^ g) << 4)) =
            e2m1x8_to_bf16(odd ? w[h][b | 1] : w[h][b & ~1], ue8m0_to_f32((e[h] >> (8 * ((b & ~1) + odd))) & 0xFFu));
      }
  }
};

template <int D>
struct PreValues {
  static constexpr int NB = D / 32, NJ = D / 16;
  uint32_t w[NJ], e[4];  // e: of tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9

  __device__ __forceinline__ void load(const uint8_t* rec, int base, int len) {
    const int lane = threadIdx.x & 31, c = lane & 3;
#pragma unroll
    for (int j = 0; j < NJ; ++j) w[j] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = 0;
    if (rec == nullptr) return;
#pragma unroll
    for (int j = 0; j < NJ; j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(rec + 8 * D + (j / 4) * 512 + lane * 16);
      w[j] = v.x, w[j + 1] = v.y, w[j + 2] = v.z, w[j + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 2 * c + (i & 1) + 8 * (i >> 1);
      // tokens behind the sequence may hold anything: exponent 0, finite, for weights of 0
      if (base + t < len) e[i] = load_exponents<NB>(rec + 16 * D + D / 2 + t * NB);
    }
  }
  // Into the tile [d][token], swizzled rows as the keys'.
  __device__ __forceinline__ void store(uint8_t* tile, int at) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = ue8m0_to_f32((e[i] >> (8 * b)) & 0xFFu);
#pragma unroll
      for (int j = 2 * b; j < 2 * b + 2; ++j) {
        uint32_t h[4];  // (d, pair c), (d + 8, pair c), (d, pair c + 4), (d + 8, pair c + 4)
        e2m1x8_to_f16(w[j], h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
          const __nv_bfloat162 r = __floats2bfloat162_rn(v.x * f[2 * (i >> 1)], v.y * f[2 * (i >> 1) + 1]);
          const int d = 16 * j + g + 8 * (i & 1), chunk = 2 * at + (i >> 1);
          *reinterpret_cast<uint32_t*>(tile + d * 128 + ((chunk ^ g) << 4) + 4 * c) =
              *reinterpret_cast<const uint32_t*>(&r);
        }
      }
    }
  }
  // What this lane stored: infinities and NaN become the type's largest, so that the weights of 0 of rows that do not see
  // their tokens leave them out.
  static __device__ __forceinline__ void make_finite(uint8_t* tile, int at) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll 1
    for (int i = 0; i < 4 * NJ; ++i) {
      const int d = 16 * (i >> 2) + g + 8 * (i & 1), chunk = 2 * at + ((i >> 1) & 1);
      uint32_t* at32 = reinterpret_cast<uint32_t*>(tile + d * 128 + ((chunk ^ g) << 4) + 4 * c);
      uint32_t v = *at32;
      if ((v & 0x7F80u) == 0x7F80u) v = (v & 0xFFFF8000u) | 0x7F7Fu;
      if ((v & 0x7F800000u) == 0x7F800000u) v = (v & 0x8000FFFFu) | 0x7F7F0000u;
      *at32 = v;
    }
  }
};

// What a softmax thread keeps of its row.
struct PreRow {
  float m, l;  // the maximum that the weights are taken under, the sum of weights
  float base;  // the largest raw score, of a row past kPreExact; else -inf
  bool ok;     // no wait has expired
};
// A step's scores at buf searched for the row's maximum, `left` of them to be seen; where it moves, the sums at o_addr are
// scaled, after the products of the step before have landed (`done`; nullptr: there are none).  Not inlined: in the loop it
// takes registers from the steps that are not searched (641 us instead of 618, by the place of its branch).
template <int D>
__device__ __noinline__ PreRow pre_search(PreRow r, uint32_t buf, uint32_t o_addr, int left, float sc, uint64_t* done,
                                          uint32_t parity, uint64_t timeout, volatile int* abort) {
  float raw = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < 64; i += 32) {
    uint32_t s[32];
    tmem_load_32(buf + i, s);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (i + e < left) raw = fmaxf(raw, __uint_as_float(s[e]));
  }
  const float mx = raw * sc;
  float f = 1.f;
  if (r.base != -INFINITY) {
    if (raw > r.base) {
      f = ex2((r.base - raw) * sc);
      r.base = raw;
    }
  } else if (mx > r.m + kPreSlack || (r.m == -INFINITY && mx != -INFINITY)) {
    f = ex2(r.m - mx);
    r.m = mx;
    if (fabsf(r.m) >= kPreExact) r.base = raw, r.m = -INFINITY;
  }
  r.l *= f;
  if (__any_sync(0xFFFFFFFFu, f != 1.f) && done != nullptr) {
    r.ok = warp_wait(done, parity, timeout, abort, kSiteEpiSync);
    if (!r.ok) return r;
    tc_fence_after();
#pragma unroll 1
    for (int i = 0; i < D / 16; ++i) {
      uint32_t o[16];
      tmem_load_16(o_addr + 16 * i, o);
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
      tmem_st_32x32b_x16(o_addr + 16 * i, o);
    }
    tmem_st_wait();
  }
  if (__any_sync(0xFFFFFFFFu, r.base != -INFINITY)) {  // the differences take the scores' place
#pragma unroll 1
    for (int i = 0; i < 64; i += 16) {
      uint32_t s[16];
      tmem_load_16(buf + i, s);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (r.base != -INFINITY) s[e] = __float_as_uint(__uint_as_float(s[e]) - r.base);
      tmem_st_32x32b_x16(buf + i, s);
    }
    tmem_st_wait();
  }
  return r;
}

template <int D>
__global__ void __launch_bounds__(kPreThreads, 1) kv4_prefill_kernel(const KvAttnArgs p) {
  using Cfg = PreCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ PreShared<D> sh;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* qs = smem;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  volatile int* abort = &sh.abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPreStages; ++i) {
      for (int v = 0; v < 2; ++v) {
        mbar_init(&sh.full[v][i], kPreGroups);
        mbar_init(&sh.empty[v][i], 2);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sh.s_full[i][b], 1);
        mbar_init(&sh.p_full[i][b], 4);
        mbar_init(&sh.pv_done[i][b], 1);
      }
    }
    mbar_init(&sh.drain, 2);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 15) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  griddep_launch_dependents();
  griddep_wait();
  const int per = pre_plan(p, sh.plan);
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int64_t total = sh.plan.before[kAttnThreads];
  const int64_t jobs = min(static_cast<int64_t>(gridDim.x), total);
  const uint64_t timeout = p.timeout_ns;
  uint32_t tile0 = 0;    // steps of earlier pieces
  uint32_t filled = 0;   // earlier pieces that have steps

  if (blockIdx.x < jobs) {
    PrePiece& pc = sh.piece[warp];
    if (lane == 0) pre_first(p, sh.plan, per, blockIdx.x, jobs, total, pc);
    __syncwarp();
    // A half's queries, with the scale's sign, to shared memory, by its softmax warps.
    auto queries = [&](int t) {
      constexpr int N = 128 * D / 8 / 128;
      const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
      uint8_t* half = qs + t * (128 * D * 2);
#pragma unroll
      for (int j0 = 0; j0 < N; j0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = (threadIdx.x & 127) + (j0 + j) * 128, rho = pc.row0 + 128 * t + i / (D / 8), ch = i % (D / 8);
          v[j] = make_uint4(0, 0, 0, 0);
          if (rho < pc.q.rows) {
            const int tok = rho / p.group, h = pc.head * p.group + (rho - tok * p.group);
            v[j] = ld_stream_16(p.q + static_cast<int64_t>(pc.q.lo + tok) * p.q_st + h * p.q_sh + 8 * ch);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = (threadIdx.x & 127) + (j0 + j) * 128, r = i / (D / 8), ch = i % (D / 8);
          *reinterpret_cast<uint4*>(half + (ch >> 3) * Cfg::kQBlock + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
              make_uint4(v[j].x ^ sign, v[j].y ^ sign, v[j].z ^ sign, v[j].w ^ sign);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[t]);
    };
    if (warp < 8 && pc.k0 < pc.k1) queries(warp >> 2);
    while (true) {
      const int row0 = pc.row0, rows = pc.q.rows, head = pc.head, len = pc.q.len, n = pc.q.n, k0 = pc.k0, k1 = pc.k1;
      const bool more = pc.end < pc.job_end;
      if (warp >= 8 && warp < 14) {
        // ---- records to bf16 tiles
        const int groups = (len + kGroup - 1) / kGroup, seq = pc.s, units = (k1 - k0) * kPreGroups;
        const int first_sees = len - n + row0 / p.group + 1;
        // this warp's groups of the piece: first, first + warps, ..; one is
        // written while the next is on its way
        auto bring = [&](auto rec, int which, int first, int warps) {
          uint64_t addr = 0;  // lane i: the record of the warp's group 32 n + i
          auto load = [&](int n) {
            const int unit = first + n * warps;
            if ((n & 31) == 0) {
              const int u = unit + lane * warps, group = k0 * kPreGroups + u;
              addr = u < units && group < groups ? reinterpret_cast<uint64_t>(kv_record<D>(p.kv, seq, group, head)) : 0;
            }
            const uint64_t a = __shfl_sync(0xFFFFFFFFu, addr, n & 31);
            rec.load(reinterpret_cast<const uint8_t*>(a), (k0 * kPreGroups + unit) * kGroup, len);
          };
          if (first < units) load(0);
#pragma unroll 1
          for (int unit = first, n = 0; unit < units; unit += warps, ++n) {
            const uint32_t it = tile0 + unit / kPreGroups;
            const int st = it % kPreStages;
            auto cur = rec;
            if (unit + warps < units) load(n + 1);
            if (!warp_wait(&sh.empty[which][st], ((it / kPreStages) & 1) ^ 1, timeout, abort, kSiteKvRecord)) break;
            uint8_t* tile = smem + Cfg::kQBytes + (which * kPreStages + st) * Cfg::kTileBytes;
            cur.store(tile, unit % kPreGroups);
            if ((k0 * kPreGroups + unit + 1) * kGroup > first_sees) cur.make_finite(tile, unit % kPreGroups);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.full[which][st]);
          }
        };
        if (warp < 8 + kPreKeyWarps)
          bring(PreKeys<D>(), 0, warp - 8, kPreKeyWarps);
        else
          bring(PreValues<D>(), 1, warp - 8 - kPreKeyWarps, kPreValueWarps);
      } else if (warp >= 14) {
        // ---- products of a half
        const int t = warp - 14;
        const uint32_t idesc_s = kIdescBf16 | (static_cast<uint32_t>(kPreTokens >> 3) << 17);
        const uint32_t idesc_o = kIdescBf16 | (static_cast<uint32_t>(D >> 3) << 17);
        // an address takes 16-byte steps in a descriptor's low bits
        const uint64_t q_desc = sw128_kmajor_desc(smem_u32(qs)), k_desc = q_desc + Cfg::kQBytes / 16;
        const uint64_t v_desc = k_desc + kPreStages * Cfg::kTileBytes / 16;
        auto there = [&](int which, uint32_t it) {
          return warp_wait(&sh.full[which][it % kPreStages], (it / kPreStages) & 1, timeout, abort, kSiteMmaFull);
        };
        auto qk = [&](uint32_t it) {
          if (!there(0, it)) return false;
          tc_fence_after();
          if (elect_one_sync()) {
            const uint64_t qd = q_desc + t * (128 * D * 2 / 16), kd = k_desc + it % kPreStages * (Cfg::kTileBytes / 16);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              mma_bf16_ss(tmem + 128 * t + 64 * (it & 1), qd + (i >> 2) * (Cfg::kQBlock / 16) + (i & 3) * 2,
                          kd + (i >> 2) * (Cfg::kKBlock / 16) + (i & 3) * 2, idesc_s, i != 0);
            tc_commit(&sh.s_full[t][it & 1]);
            tc_commit(&sh.empty[0][it % kPreStages]);
          }
          __syncwarp();
          return true;
        };
        const uint32_t it0 = tile0, it1 = tile0 + (k1 - k0);
        bool ok = k0 >= k1 || warp_wait(&sh.q_full[t], filled & 1, timeout, abort, kSiteMmaFull);
        for (uint32_t it = it0; it < min(it0 + 2, it1) && ok; ++it) ok = qk(it);
        for (uint32_t it = it0; it < it1 && ok; ++it) {
          ok = there(1, it) && warp_wait(&sh.p_full[t][it & 1], (it >> 1) & 1, timeout, abort, kSiteMmaAccEmpty);
          if (!ok) break;
          tc_fence_after();
          if (elect_one_sync()) {
            const uint64_t vd = v_desc + it % kPreStages * (Cfg::kTileBytes / 16);
            const uint32_t more = it != it0;
#pragma unroll
            for (int i = 0; i < kPreTokens / 16; ++i)
              mma_bf16_ts(tmem + 256 + 128 * t, tmem + 128 * t + 64 * (it & 1) + 8 * i, vd + 2 * i, idesc_o, i != 0 ? 1u : more);
            tc_commit(&sh.pv_done[t][it & 1]);
            tc_commit(&sh.empty[1][it % kPreStages]);
          }
          __syncwarp();
          if (it + 2 < it1) ok = qk(it + 2);
        }
      } else {
        // ---- softmax: a thread per row
        const int t = warp >> 2, r = threadIdx.x & 127;
        const int rho = row0 + 128 * t + r;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + 128 * t + lane_base, o_addr = tmem + 256 + 128 * t + lane_base;
        const int vis = rho < rows ? min(len, max(len - n + rho / p.group + 1, 0)) : 0;
        const float sc = fabsf(p.scale_log2);
        float m = -INFINITY, l = 0.f;
        sh.base[threadIdx.x] = -INFINITY;
        bool ok = true;
        const uint32_t it0 = tile0, it1 = tile0 + (k1 - k0);
        for (uint32_t it = it0; it < it1; ++it) {
          ok = warp_wait(&sh.s_full[t][it & 1], (it >> 1) & 1, timeout, abort, kSiteEpiAccFull);
          if (!ok) break;
          tc_fence_after();
          const uint32_t buf = s_addr + 64 * (it & 1);
          const int left = vis - (k0 + static_cast<int>(it - it0)) * kPreTokens;  // tokens of the step that the row sees
          const bool masked = __any_sync(0xFFFFFFFFu, left < kPreTokens);
          // The maximum only keeps weights and sums in fp32's range (a bf16
          // weight has 8 bits at any size), so a step is not searched for it: the
          // rows' first sets it, and one whose weights sum to more than 2^16 is
          // taken again with a new one (values up to 2^100 stay in range).
          bool search = __any_sync(0xFFFFFFFFu, it == it0 || (m == -INFINITY && left > 0));
          uint32_t w[32];
          for (bool searched = false;;) {
            if (search) {
              const PreRow row = pre_search<D>({m, l, sh.base[threadIdx.x], true}, buf, o_addr, left, sc,
                                               it != it0 ? &sh.pv_done[t][(it - 1) & 1] : nullptr, ((it - 1) >> 1) & 1,
                                               timeout, abort);
              m = row.m, l = row.l, sh.base[threadIdx.x] = row.base, ok = row.ok;
              if (!ok) break;
              searched = true;
            }
            uint32_t s[64];
            tmem_load_64(buf, s);
            if (masked) {
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (e >= left) s[e] = 0xFF800000u;
            }
            const float at = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float x = ex2(fmaf(__uint_as_float(s[2 * e]), sc, -at));
              const float y = ex2(fmaf(__uint_as_float(s[2 * e + 1]), sc, -at));
              sum[2 * (e & 1)] += x;
              sum[2 * (e & 1) + 1] += y;
              const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
              w[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            const float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            search = !searched && __any_sync(0xFFFFFFFFu, !(all <= 0x1p16f));
            if (search) continue;
            l += all;
            break;
          }
          if (!ok) break;
          tmem_st_32x32b_x32(buf, w);  // over the scores, which have been read
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_full[t][it & 1]);
        }
        const bool whole = pc.u == pc.i0 && pc.end == pc.i1, begins = pc.i0 >= pc.job_u;
        const int lo = pc.q.lo;
        if (!whole && begins && threadIdx.x == 0) {  // to the list of cut tiles
          const int64_t last = (pc.i1 * jobs - 1) / total;  // the job that holds unit i1 - 1
          attn_list_cut(p, AttnCut{static_cast<int>(blockIdx.x), static_cast<int>(last), lo, head, row0,
                                   min(rows - row0, kPreRows)});
        }
        // ---- the next piece's queries: every QK of this one is done, since its scores have been read
        if (more && ok) {
          __syncwarp();
          if (lane == 0) pre_next(p, pc);
          __syncwarp();
          if (pc.k0 < pc.k1) queries(t);
        }
        if (sh.base[threadIdx.x] != -INFINITY) m = sh.base[threadIdx.x] * sc;
        // ---- the rows, or the piece's partial result
        if (ok && k0 < k1) ok = warp_wait(&sh.pv_done[t][(it1 - 1) & 1], ((it1 - 1) >> 1) & 1, timeout, abort, kSiteEpiSync);
        if (ok) {
          tc_fence_after();
          const bool row = rho < rows;
          float* part = nullptr;
          __nv_bfloat16* out = nullptr;
          const int tok = rho / p.group, h = head * p.group + (rho - tok * p.group);
          if (!whole) part = p.partials + (2 * static_cast<int64_t>(blockIdx.x) + (begins ? 1 : 0)) * (kPreRows * (D + 2));
          else out = p.out + static_cast<int64_t>(lo + tok) * p.o_st + h * p.o_sh;
          const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            if (k0 < k1) {
              tmem_load_32(o_addr + 32 * i, o);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0;
            }
            if (!whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<uint4*>(part + (128 * t + r) * D + 32 * i + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            } else if (row) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[e + 2 * j]) * inv, __uint_as_float(o[e + 2 * j + 1]) * inv);
                  w[j] = *reinterpret_cast<const uint32_t*>(&v);
                }
                *reinterpret_cast<uint4*>(out + 32 * i + e) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          if (!whole) {
            part[kPreRows * D + 128 * t + r] = m;
            part[kPreRows * D + kPreRows + 128 * t + r] = l;
          } else if (row && p.lse != nullptr) {
            p.lse[static_cast<int64_t>(lo + tok) * p.lse_st + h] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
          }
          tc_fence_before();
        }
      }
      tile0 += k1 - k0;
      filled += k0 < k1;
      // (the whole warp, should its lanes read the flag apart: those that go on wait for all)
      if (!more || __any_sync(0xFFFFFFFFu, *abort != 0)) break;
      if (warp >= 8) {
        __syncwarp();
        if (lane == 0) pre_next(p, pc);
        __syncwarp();
      }
    }
  }
  // the matrix instructions in flight land before the tensor memory is given back
  if (warp >= 14) {
    if (elect_one_sync()) tc_commit(&sh.drain);
    __syncwarp();
    warp_wait(&sh.drain, 0, timeout, nullptr, kSiteDrain);
  }
  __syncthreads();
  if (warp == 15) tmem_dealloc(tmem, 512);
}

}  // namespace fp8mm
