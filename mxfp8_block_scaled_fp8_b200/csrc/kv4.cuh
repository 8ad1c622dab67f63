// kv4.cuh -- the MXFP4 paged key/value cache: its format, the kernels that
// write and read it (append, gather), the moving of pages, and the norm and
// rotation of queries and keys that stand before it.
//
// Format.  E2M1 codes with one UE8M0 exponent e per 32 elements along the
// head dimension (value = code * 2^(e - 127)); e is the smallest power of two
// with 6 * 2^(e - 127) >= the block's largest magnitude, so no element
// saturates, 0 for a block of zeros: the library's MX rule (the maximum's
// scale rounded up to a power of two) with E2M1's largest value 6.  255 marks a
// block with a NaN, as in MX, with codes of zero (0 * inf is NaN); an infinity is
// the code 6 under 253, the largest exponent of a number.
//
// Record.  The unit is one head's 16 consecutive tokens ("group"), 17 * D
// bytes, in the order in which the attention kernel's matrix instructions
// take them, so that a warp loads a group with 16-byte reads and no shuffle:
//   key codes     [16 tokens][4 quarters][D/32 blocks] 32-bit words; the word
//                 of (token, quarter c, block b) holds the elements
//                 32 b + 8 c .. + 7, element 0 in the lowest nibble
//   value codes   [D/64][8 g][4 c][4] 32-bit words; word (d64, g, c, w) is of
//                 dimensions d = 64 d64 + 16 w + g (bytes 0, 2) and d + 8
//                 (bytes 1, 3), tokens 2c, 2c+1 (bytes 0, 1) and 2c+8, 2c+9
//                 (bytes 2, 3), the even token in the low nibble
//   key exponents, value exponents  [16 tokens][D/32] bytes each
// A page holds page_size tokens (a multiple of 16) as [head][group][record].
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <cstdint>

#include "ptx.cuh"
#include "vec.cuh"

namespace fp8mm {

constexpr int kGroup = 16;  // tokens of a record
// Tokens of a sequence at most: below it no position of a last step passes an int.
constexpr int kMostTokens = 0x7FFFFFFF - 64;

struct KvCache {
  uint8_t* base;
  int64_t page_stride;     // bytes
  const int32_t* table;    // [batch][table_stride] page ids
  int64_t table_stride;    // elements
  int32_t num_pages, max_pages;
  int32_t kv_heads;
  int32_t page_groups;     // groups per page
};

// Records the first data error; `site` tells which index was out of range.
__device__ __forceinline__ void record_index_error(unsigned site) { record_error(kDevErrIndex, site); }

// Record of (sequence, group, head), or nullptr where the page table has no
// such page (recorded): nothing is read or written through a bad page id.
template <int D>
__device__ __forceinline__ uint8_t* kv_record(const KvCache& kv, int seq, int group, int head) {
  const int slot = group / kv.page_groups;
  int page = -1;
  if (slot < kv.max_pages) page = kv.table[seq * kv.table_stride + slot];
  if (page < 0 || page >= kv.num_pages) {
    record_index_error(kSitePage);
    return nullptr;
  }
  return kv.base + page * kv.page_stride +
         (static_cast<int64_t>(head) * kv.page_groups + (group - slot * kv.page_groups)) * (17 * D);
}

// Sequence of row r in the ragged batch cu[0..batch] (r < cu[batch]), found
// by the whole warp: each step probes 32 bounds at once.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int r) {
  int lo = 0, hi = batch;  // cu[lo] <= r < cu[hi]
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const bool below = at < hi && cu[at] <= r;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, below));
    lo += n * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// 8 E2M1 codes of a word as 4 f16x2 (exact).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 8 fp32 -> 8 E2M1 codes (round to nearest even, saturating), element 0 in
// the lowest nibble.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&y)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= static_cast<uint32_t>(
             __nv_cvt_float2_to_fp4x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_E2M1, cudaRoundNearest))
         << (8 * i);
  return w;
}

// 2^(e - 127) as fp32 for every exponent byte (255 gives infinity).
__device__ __forceinline__ float ue8m0_to_f32(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e << 23);
}
// The top bits of those bytes of w that are 255.
__device__ __forceinline__ uint32_t bytes_255(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u; }

// Exponent byte of a block whose largest bf16 magnitude has the bits m (sign
// cleared): amax = (1 + f / 128) 2^(E - 127) <= 6 * 2^(e - 127) = 1.5 *
// 2^(e - 125) for e = E - 2 where f <= 64, else E - 1; at least 0.
__device__ __forceinline__ uint32_t mxfp4_exponent(uint32_t m) {
  const int e = static_cast<int>(m >> 7) - 2 + ((m & 0x7Fu) > 64u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));
}

// Transpose of an 8 x 8 matrix of nibbles, row i in w[i], column j at bits
// 4 j: three rounds of swaps between rows 4, 2 and 1 apart.
__device__ __forceinline__ void transpose_nibbles_8x8(uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 16-bit halves of rows i and i + 4
    const uint32_t a = w[i], b = w[i + 4];
    w[i] = __byte_perm(a, b, 0x5410);
    w[i + 4] = __byte_perm(a, b, 0x7632);
  }
#pragma unroll
  for (int q = 0; q < 8; q += 4)
#pragma unroll
    for (int i = q; i < q + 2; ++i) {  // bytes of rows i and i + 2
      const uint32_t a = w[i], b = w[i + 2];
      w[i] = __byte_perm(a, b, 0x6240);
      w[i + 2] = __byte_perm(a, b, 0x7351);
    }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {  // nibbles of rows i and i + 1
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0F0F0F0Fu) | ((b & 0x0F0F0F0Fu) << 4);
    w[i + 1] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
  }
}

// ------------------------------------------------------------------ append

struct KvAppendArgs {
  KvCache kv;
  const __nv_bfloat16 *k, *v;
  int64_t k_st, k_sh, v_st, v_sh;  // elements
  const int32_t* cu;               // nullptr: one row per sequence
  const int32_t* lens;
  int32_t batch;
  int64_t rows;
};

constexpr int kKvThreads = 128;

// The rows of one 16-token group that a call touches.  A row leads the group
// if it is its sequence's first row or starts a group; the warp that has the
// leading row handles the whole group, so that no two warps of a call write
// into one record.
struct KvSpan {
  int seq, group;
  int first, end;  // token slots of the group that the call touches: [first, end)
  int row0;        // row of token slot `first`
};

// Rows r0 .. r0 + count - 1 (count <= 32, one per lane): true in the lanes
// whose row leads a span.  lens: lengths with the rows; else starts (may be
// nullptr: 0): positions of the sequences' first rows.
__device__ __forceinline__ bool kv_span(const int32_t* cu, int batch, int rows, int r0, int count, const int32_t* lens,
                                        const int32_t* starts, KvSpan* sp) {
  const int r = r0 + (threadIdx.x & 31);
  int seq = r, lo = r, n = 1;
  if (cu != nullptr) {
    const int end = min(cu[batch], rows);  // rows behind the last sequence are padding
    if (r0 >= end) return false;
    int a = find_sequence(cu, batch, r0);
    int z = count == 1 ? a + 1 : find_sequence(cu, batch, min(r0 + count, end) - 1) + 1;
    if (r >= end || r >= r0 + count) return false;
    while (z - a > 1) {
      const int mid = (a + z) / 2;
      if (cu[mid] <= r) a = mid; else z = mid;
    }
    seq = a;
    lo = cu[seq];
    const int64_t next = cu[seq + 1];
    if (seq == 0 && r < lo) return false;  // rows before the first sequence are padding too
    if (lo < 0 || r < lo || r >= next || next > rows) {
      record_index_error(kSiteSequence);
      return false;
    }
    n = static_cast<int>(next) - lo;
  } else if (r >= rows || r >= r0 + count) {
    return false;
  }
  int64_t start = starts != nullptr ? starts[seq] : 0;
  if (lens != nullptr) {
    if (lens[seq] == 0) return false;  // a padding sequence: nothing of it is kept
    start = static_cast<int64_t>(lens[seq]) - n;
  }
  if (start < 0 || start + n > kMostTokens) {
    record_index_error(kSiteSequence);
    return false;
  }
  const int pos = static_cast<int>(start) + (r - lo);
  if (r != lo && pos % kGroup != 0) return false;
  sp->seq = seq;
  sp->group = pos / kGroup;
  sp->first = pos % kGroup;
  sp->end = min(kGroup, static_cast<int>(start) + n - pos / kGroup * kGroup);
  sp->row0 = r;
  return true;
}
// The span of lane `from`.
__device__ __forceinline__ KvSpan span_of(const KvSpan& sp, int from) {
  KvSpan o;
  o.seq = __shfl_sync(0xFFFFFFFFu, sp.seq, from);
  o.group = __shfl_sync(0xFFFFFFFFu, sp.group, from);
  o.first = __shfl_sync(0xFFFFFFFFu, sp.first, from);
  o.end = __shfl_sync(0xFFFFFFFFu, sp.end, from);
  o.row0 = __shfl_sync(0xFFFFFFFFu, sp.row0, from);
  return o;
}

// A warp's group of keys or values.  Lane (g, c) = (lane / 4, lane % 4) has the
// eighth c of every block of token slots g and g + 8: a block's maximum is over
// four neighbouring lanes.
template <int D>
__device__ __forceinline__ void load_group(const __nv_bfloat16* x, int64_t st, const KvSpan& sp, int lane,
                                           uint4 (&v)[2][D / 32]) {
  constexpr int NB = D / 32;
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int slot = g + 8 * h;
    const bool ok = slot >= sp.first && slot < sp.end;
    const __nv_bfloat16* row = x + (sp.row0 + static_cast<int64_t>(slot - sp.first)) * st + 8 * c;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      v[h][b] = ok ? ld_stream_16(row + 32 * b) : make_uint4(0, 0, 0, 0);
  }
}
template <int D>
__device__ __forceinline__ void quantize_group(const uint4 (&v)[2][D / 32], uint32_t (&code)[2][D / 32],
                                               uint32_t (&e)[2][D / 32]) {
  constexpr int NB = D / 32;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint4 q = v[h][b];
      uint32_t m = __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu),
                            __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
      m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      m = max(m & 0xFFFFu, m >> 16);
      const uint32_t ex = mxfp4_exponent(m);
      e[h][b] = ex;
      const float s = __uint_as_float((254u - min(ex, 253u)) << 23);  // 2^(127 - e), a normal power of two
      float f[8];
      bf16x8_to_f32(q, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= s;
      code[h][b] = f32x8_to_e2m1(f);
      if (m > 0x7F80u) e[h][b] = 255u, code[h][b] = 0u;  // a NaN
    }
}

// A token's exponents as one word.
template <int NB>
__device__ __forceinline__ void store_exponents(uint8_t* dst, const uint32_t (&e)[NB]) {
  if constexpr (NB == 4)
    *reinterpret_cast<uint32_t*>(dst) = e[0] | (e[1] << 8) | (e[2] << 16) | (e[3] << 24);
  else
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(e[0] | (e[1] << 8));
}
template <int NB>
__device__ __forceinline__ uint32_t load_exponents(const uint8_t* src) {
  return NB == 4 ? *reinterpret_cast<const uint32_t*>(src) : *reinterpret_cast<const uint16_t*>(src);
}

// One warp per (kRows rows, head): 1 where most rows lead a group (decode),
// 16 for prompts.  Bound by HBM for long prompts (4 D bytes
// in, 17 D / 16 bytes out per token and head; 8 prompts of 1 to 2047 tokens, 8
// heads, written and read back: 23.4 us, 27.6 with the values' loads behind the
// keys' conversion; 131072 tokens 124 us, 5.5 TB/s) and by the latency of the
// index loads for a decode step (64 tokens 4.4 us).  A group that is written only in part keeps the
// codes of its other tokens: values share bytes between neighbouring tokens,
// so those words are merged with what the record held.
template <int D, int kRows>
__global__ void __launch_bounds__(kKvThreads) kv4_append_kernel(const KvAppendArgs p) {
  constexpr int NB = D / 32;
  __shared__ uint32_t s_code[kKvThreads / 32][kGroup][D / 8 + 4];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = static_cast<int>((p.rows + kRows - 1) / kRows);
  const int64_t tasks = static_cast<int64_t>(blocks) * p.kv.kv_heads;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kKvThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kKvThreads / 32) + warp; t < tasks; t += stride) {
    const int block = static_cast<int>(t / p.kv.kv_heads);
    const int head = static_cast<int>(t - static_cast<int64_t>(block) * p.kv.kv_heads);
    KvSpan mine;
    const bool leads = kv_span(p.cu, p.batch, static_cast<int>(p.rows), block * kRows, kRows, p.lens, nullptr, &mine);
    for (unsigned todo = __ballot_sync(0xFFFFFFFFu, leads); todo != 0; todo &= todo - 1) {
      const KvSpan sp = span_of(mine, __ffs(todo) - 1);
      uint4 kx[2][NB], vx[2][NB];
      load_group<D>(p.k + head * p.k_sh, p.k_st, sp, lane, kx);
      load_group<D>(p.v + head * p.v_sh, p.v_st, sp, lane, vx);
      uint8_t* rec = kv_record<D>(p.kv, sp.seq, sp.group, head);
      if (rec == nullptr) continue;
      const int g = lane >> 2, c = lane & 3;
      uint32_t code[2][NB], e[2][NB];
      // keys: every token's codes and exponents are its own bytes
      quantize_group<D>(kx, code, e);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int slot = g + 8 * h;
        if (slot < sp.first || slot >= sp.end) continue;
        uint32_t* dst = reinterpret_cast<uint32_t*>(rec + slot * (D / 2) + c * (D / 8));
        if constexpr (NB == 4)
          *reinterpret_cast<uint4*>(dst) = make_uint4(code[h][0], code[h][1], code[h][2], code[h][3]);
        else
          *reinterpret_cast<uint2*>(dst) = make_uint2(code[h][0], code[h][1]);
        if (c == 0) store_exponents<NB>(rec + 16 * D + slot * NB, e[h]);
      }
      // values: exponents by token, codes through shared memory and an 8 x 8 transpose
      quantize_group<D>(vx, code, e);
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int slot = g + 8 * h;
#pragma unroll
        for (int b = 0; b < NB; ++b) s_code[warp][slot][4 * b + c] = code[h][b];
        if (slot >= sp.first && slot < sp.end && c == 0) store_exponents<NB>(rec + 16 * D + D / 2 + slot * NB, e[h]);
      }
      __syncwarp();
      if (lane < D / 4) {  // lane = (16-dimension slice j, pair cc)
        const int j = lane & (D / 16 - 1), cc = lane / (D / 16);
        uint32_t w[8];
        uint32_t mask = 0;  // bits that the call writes
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // byte i / 2 = (half, d + 8), nibble i % 2: token 2 cc + i % 2 + 8 half
          const int slot = 2 * cc + (i & 1) + 8 * (i >> 2);
          w[i] = s_code[warp][slot][2 * j + ((i >> 1) & 1)];
          if (slot >= sp.first && slot < sp.end) mask |= 0xFu << (4 * i);
        }
        transpose_nibbles_8x8(w);
        uint32_t* dst = reinterpret_cast<uint32_t*>(rec + 8 * D + (j / 4) * 512 + cc * 16 + (j % 4) * 4);
        if (mask == 0xFFFFFFFFu) {
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[16 * i] = w[i];
        } else if (mask != 0) {
          uint32_t old[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) old[i] = dst[16 * i];
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[16 * i] = (old[i] & ~mask) | (w[i] & mask);
        }
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ gather

struct KvGatherArgs {
  KvCache kv;
  __nv_bfloat16 *k, *v;
  int64_t k_st, k_sh, v_st, v_sh;
  const int32_t* cu;
  const int32_t* starts;  // nullptr: from position 0
  int32_t batch;
  int64_t rows;
};

// 8 codes times 2^(e - 127) as 8 bf16: exact, as a code has two significant
// bits (down to 2^-128, which bf16 holds as a subnormal).
__device__ __forceinline__ uint4 e2m1x8_to_bf16(uint32_t w, float s) {
  uint32_t h[4], o[4];
  e2m1x8_to_f16(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);
    o[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// 16 consecutive bf16 (32-byte store where the rows allow it).
template <bool kWide>
__device__ __forceinline__ void store_bf16x16(__nv_bfloat16* dst, const uint4& a, const uint4& b) {
  if constexpr (kWide) {
    st_global_v8(dst, a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w);
  } else {
    reinterpret_cast<uint4*>(dst)[0] = a;
    reinterpret_cast<uint4*>(dst)[1] = b;
  }
}

// One warp per (16 rows, head), 17 D bytes in, 4 D bytes per token out.
// Bound by HBM (79 % of the bytes are the writes): 131072 tokens of 8 heads of
// 128 in 110 us, 6.2 TB/s, 94 % of a copy.  kWide: v's rows are 32-byte aligned.
template <int D, bool kWide>
__global__ void __launch_bounds__(kKvThreads) kv4_gather_kernel(const KvGatherArgs p) {
  constexpr int NB = D / 32;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int j = lane & (D / 16 - 1), cc = (lane / (D / 16)) & 3;
  const int blocks = static_cast<int>((p.rows + kGroup - 1) / kGroup);
  const int64_t tasks = static_cast<int64_t>(blocks) * p.kv.kv_heads;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kKvThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kKvThreads / 32) + warp; t < tasks; t += stride) {
    const int block = static_cast<int>(t / p.kv.kv_heads);
    const int head = static_cast<int>(t - static_cast<int64_t>(block) * p.kv.kv_heads);
    KvSpan mine;
    const bool leads = kv_span(p.cu, p.batch, static_cast<int>(p.rows), block * kGroup, kGroup, nullptr, p.starts, &mine);
    for (unsigned todo = __ballot_sync(0xFFFFFFFFu, leads); todo != 0; todo &= todo - 1) {
      const KvSpan sp = span_of(mine, __ffs(todo) - 1);
      const uint8_t* rec = kv_record<D>(p.kv, sp.seq, sp.group, head);
      if (rec == nullptr) continue;
      uint32_t kw[2][NB], ke[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* src = rec + (g + 8 * h) * (D / 2) + c * (D / 8);
        if constexpr (NB == 4) {
          const uint4 q = *reinterpret_cast<const uint4*>(src);
          kw[h][0] = q.x, kw[h][1] = q.y, kw[h][2] = q.z, kw[h][3] = q.w;
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(src);
          kw[h][0] = q.x, kw[h][1] = q.y;
        }
        ke[h] = load_exponents<NB>(rec + 16 * D + (g + 8 * h) * NB);
      }
      uint32_t w[8], ve[4];  // ve: of tokens 2 cc, 2 cc + 1, 2 cc + 8, 2 cc + 9
      const uint32_t* vsrc = reinterpret_cast<const uint32_t*>(rec + 8 * D + (j / 4) * 512 + cc * 16 + (j % 4) * 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = vsrc[16 * i];
#pragma unroll
      for (int i = 0; i < 4; ++i) ve[i] = rec[16 * D + D / 2 + (2 * cc + (i & 1) + 8 * (i >> 1)) * NB + j / 2];
      __nv_bfloat16* kd = p.k + head * p.k_sh + 8 * c;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int slot = g + 8 * h;
        if (slot < sp.first || slot >= sp.end) continue;
        __nv_bfloat16* dst = kd + (sp.row0 + static_cast<int64_t>(slot - sp.first)) * p.k_st;
#pragma unroll
        for (int b = 0; b < NB; ++b)
          *reinterpret_cast<uint4*>(dst + 32 * b) = e2m1x8_to_bf16(kw[h][b], ue8m0_to_f32((ke[h] >> (8 * b)) & 0xFFu));
      }
      if (lane < D / 4) {
        transpose_nibbles_8x8(w);  // w[i]: dimensions 16 j + 8 ((i / 2) % 2) + 0..7 of token 2 cc + i % 2 + 8 (i / 4)
        __nv_bfloat16* vd = p.v + head * p.v_sh + 16 * j;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int slot = 2 * cc + (i & 1) + 8 * (i >> 1);
          if (slot < sp.first || slot >= sp.end) continue;
          const float f = ue8m0_to_f32(ve[i]);
          const int at = 4 * (i >> 1) + (i & 1);
          store_bf16x16<kWide>(vd + (sp.row0 + static_cast<int64_t>(slot - sp.first)) * p.v_st, e2m1x8_to_bf16(w[at], f),
                               e2m1x8_to_bf16(w[at + 2], f));
        }
      }
    }
  }
}

// ------------------------------------------------------------------ pages

constexpr int kPageMoves = 480;  // moves of one launch: 3840 bytes of kernel parameters

struct KvCopyArgs {
  uint8_t* base;
  int64_t page_stride, layer_stride;  // bytes
  int32_t layers, moves;
  uint32_t page_vecs;                 // 16-byte vectors of a page
  int32_t src[kPageMoves], dst[kPageMoves];
};
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

// One block per slice of kCopyThreads * kCopyUnroll vectors of one move's
// page in one layer.  The moves come by value as kernel parameters, so that a
// captured graph holds them; no destination is another move's source, so the
// order does not matter.  Bound by HBM: 400 pages of 68 KB in 16 layers in 138
// us, 6.5 TB/s, 99 % of a copy.
__global__ void __launch_bounds__(kCopyThreads) kv_copy_pages_kernel(const __grid_constant__ KvCopyArgs p,
                                                                     uint32_t slices) {
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t page = blockIdx.x / slices;  // (layer, move)
  const uint32_t slice = blockIdx.x - page * slices;
  const uint32_t layer = page / p.moves, m = page - layer * p.moves;
  const uint8_t* src = p.base + layer * p.layer_stride + p.src[m] * p.page_stride;
  uint8_t* dst = p.base + layer * p.layer_stride + p.dst[m] * p.page_stride;
  const uint32_t v0 = slice * (kCopyThreads * kCopyUnroll) + threadIdx.x;
  uint4 v[kCopyUnroll];
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i)
    if (v0 + i * kCopyThreads < p.page_vecs) v[i] = ld_stream_16(src + static_cast<int64_t>(v0 + i * kCopyThreads) * 16);
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i)
    if (v0 + i * kCopyThreads < p.page_vecs)
      *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(v0 + i * kCopyThreads) * 16) = v[i];
}

// ------------------------------------------------------------------ norm and rotation

struct QkNormArgs {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *qo, *ko;
  int64_t q_st, q_sh, k_st, k_sh, qo_st, qo_sh, ko_st, ko_sh;  // elements
  const __nv_bfloat16 *qw, *kw;  // both nullptr: no norm
  const float* cos_sin;          // [max_pos][rot]: rot / 2 cosines, rot / 2 sines
  int64_t cs_stride;
  const int32_t* pos;
  int64_t tokens;
  int32_t q_heads, k_heads, rot, max_pos;
  float eps;
  int32_t slices;  // warps per token
};
constexpr int kNormThreads = 128;
constexpr int kNormUnroll = 4;

// One warp per (token, slice of the heads); D / 8 lanes per head, so a warp
// takes 256 / D heads side by side and kNormUnroll of these in a step, while the
// next step's loads are in flight.  y = r (x_i w_i cos +- x_j w_j sin), r =
// rsqrt(mean x^2 + eps): the weights join the token's angles once for all its
// query heads and once for its key heads, and partners exchange bf16 pairs.
// fp32 throughout, rounded once.  Bound by HBM for long prompts (each element
// read and written once), by latency for a decode step (64 tokens 2.5 us).
// 8192 tokens of 40 heads of 128: 33.4 us in a graph, 5.1 TB/s; steps of 2 heads 41.8, of 4
// 37.0, of 16 42.0; weights and angles apart, fp32 partners 39.6.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_kernel(const QkNormArgs p) {
  constexpr int L = D / 8;         // lanes of a head
  constexpr int HW = 32 / L;       // heads that a warp takes side by side
  constexpr int U = kNormUnroll;   // and of these, one after the other, in a step
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int l = lane % L, sub = lane / L, e0 = 8 * l;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * (kNormThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = wid / p.slices;
  if (t >= p.tokens) return;
  // steps of queries, then of keys
  const int q_steps = (p.q_heads + HW * U - 1) / (HW * U), steps = q_steps + (p.k_heads + HW * U - 1) / (HW * U);
  uint4 v[U];
  auto load = [&](int s) {
    const bool keys = s >= q_steps;
    const __nv_bfloat16* x = (keys ? p.k + t * p.k_st : p.q + t * p.q_st) + e0;
    const int64_t sh = keys ? p.k_sh : p.q_sh;
    const int h0 = (keys ? s - q_steps : s) * (HW * U) + sub, heads = keys ? p.k_heads : p.q_heads;
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = h0 + u * HW < heads ? ld_stream_16(x + (h0 + u * HW) * sh) : make_uint4(0, 0, 0, 0);
  };
  int s = static_cast<int>(wid - t * p.slices);
  const int pos = p.pos[t];
  load(s);              // beside the position and the angles
  if (pos < 0) return;  // a padding row
  if (pos >= p.max_pos) {
    if (lane == 0) record_index_error(kSitePosition);
    return;
  }
  const int half = p.rot / 2;
  const bool turned = e0 < p.rot, second = !kInterleaved && e0 >= half;
  // element e0 + i turns with element pe + i (interleaved: with its neighbour)
  const int pe = kInterleaved || !turned ? e0 : (second ? e0 - half : e0 + half), partner = lane + (pe - e0) / 8;
  // y_i = r (x_i a_i + x_partner b_i): the weights joined with the angles
  float a[8], b[8];
  auto factors = [&](const __nv_bfloat16* w) {
    float c[8], d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, d[i] = 0.f;
    if (turned) {
      const float* row = p.cos_sin + pos * p.cs_stride + (kInterleaved ? e0 / 2 : (second ? pe : e0));
#pragma unroll
      for (int i = 0; i < (kInterleaved ? 4 : 8); i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(row + i), y = *reinterpret_cast<const float4*>(row + half + i);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (kInterleaved) {
            c[2 * k] = c[2 * k + 1] = xs[k];
            d[2 * k] = -ys[k], d[2 * k + 1] = ys[k];
          } else {
            c[i + k] = xs[k], d[i + k] = second ? ys[k] : -ys[k];
          }
        }
      }
    }
    float wa[8], wb[8];
    const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    bf16x8_to_f32(w != nullptr ? *reinterpret_cast<const uint4*>(w + e0) : ones, wa);
    bf16x8_to_f32(w != nullptr ? *reinterpret_cast<const uint4*>(w + pe) : ones, wb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = wa[i] * c[i];
      b[i] = wb[kInterleaved ? i ^ 1 : i] * d[i];
    }
  };
  for (int have = -1; s < steps; s += p.slices) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = v[u];
    if (s + p.slices < steps) load(s + p.slices);
    const int keys = s >= q_steps;
    if (keys != have) {
      factors(keys ? p.kw : p.qw);
      have = keys;
    }
    __nv_bfloat16* out = (keys ? p.ko + t * p.ko_st : p.qo + t * p.qo_st) + e0;
    const int64_t sh = keys ? p.ko_sh : p.qo_sh;
    const int h0 = (keys ? s - q_steps : s) * (HW * U) + sub, heads = keys ? p.k_heads : p.q_heads;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8], o[8];
      bf16x8_to_f32(x[u], f);
      float r = 1.f;
      if (p.qw != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
        for (int k = 1; k < L; k <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, k);
        r = rsqrtf(ss * (1.f / D) + p.eps);
      }
      if constexpr (kInterleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = f[i ^ 1];
      } else {
        const uint4 y = make_uint4(__shfl_sync(0xFFFFFFFFu, x[u].x, partner), __shfl_sync(0xFFFFFFFFu, x[u].y, partner),
                                   __shfl_sync(0xFFFFFFFFu, x[u].z, partner), __shfl_sync(0xFFFFFFFFu, x[u].w, partner));
        bf16x8_to_f32(y, o);
      }
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(fmaf(f[2 * i], a[2 * i], o[2 * i] * b[2 * i]) * r,
                                                       fmaf(f[2 * i + 1], a[2 * i + 1], o[2 * i + 1] * b[2 * i + 1]) * r);
        y[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if (h0 + u * HW < heads) *reinterpret_cast<uint4*>(out + (h0 + u * HW) * sh) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

}  // namespace fp8mm
