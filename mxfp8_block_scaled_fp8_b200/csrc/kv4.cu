// kv4.cu -- the C ABI of the MXFP4 key/value cache operators: argument checks
// and launches (kernels in kv4.cuh and kv4_attn.cuh).
#include "kv4.cuh"

#include <algorithm>
#include <climits>
#include <cmath>
#include <limits>
#include <memory>
#include <new>

#include "host.cuh"
#include "kv4_attn.cuh"
#include "kv4_prefill.cuh"

namespace fp8mm {

unsigned int kv_take_device_error() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  const unsigned int zero = 0;
  cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero));
  return v;
}

constexpr int64_t kMaxRows = INT32_MAX / 2;

static int64_t page_bytes(int64_t page_size, int64_t kv_heads, int64_t d) { return page_size / 16 * kv_heads * 17 * d; }

// The cache's description, checked; no CUDA call.
static fp8mm_status check_cache(const fp8mm_kv_cache* c, KvCache* out) {
  if (c == nullptr) return FP8MM_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128) return FP8MM_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size % 16 != 0 || c->page_size > 4096) return FP8MM_ERR_SHAPE;
  if (c->kv_heads < 1 || c->kv_heads > 65535 || c->num_pages < 0 || c->num_pages > INT32_MAX || c->batch < 0 ||
      c->batch > kMaxRows || c->max_pages < 0 || c->max_pages > INT32_MAX / c->page_size ||
      c->table_stride < c->max_pages)
    return FP8MM_ERR_SHAPE;
  if (c->page_stride < page_bytes(c->page_size, c->kv_heads, c->head_dim)) return FP8MM_ERR_SHAPE;
  if (c->batch > 0 && c->max_pages > 0 && (c->pages == nullptr || c->page_table == nullptr)) return FP8MM_ERR_NULL;
  if (!aligned(c->pages, 16) || c->page_stride % 16 != 0 || !aligned(c->page_table, 4)) return FP8MM_ERR_ALIGN;
  out->base = static_cast<uint8_t*>(c->pages);
  out->page_stride = c->page_stride;
  out->table = c->page_table;
  out->table_stride = c->table_stride;
  out->num_pages = static_cast<int32_t>(c->num_pages);
  out->max_pages = static_cast<int32_t>(c->max_pages);
  out->kv_heads = static_cast<int32_t>(c->kv_heads);
  out->page_groups = static_cast<int32_t>(c->page_size / 16);
  return FP8MM_OK;
}

// Rows of [rows][heads][dim] bf16 with these strides in elements: 16-byte
// vectors along dim.
static fp8mm_status check_rows(const void* x, int64_t stride_t, int64_t stride_h, int64_t heads, int64_t d, bool out) {
  if (x == nullptr) return FP8MM_ERR_NULL;
  if (stride_t < 0 || stride_h < 0 || (heads > 1 && stride_h < d) || (out && stride_t < d)) return FP8MM_ERR_SHAPE;
  if (!aligned(x, 16) || stride_t % 8 != 0 || stride_h % 8 != 0) return FP8MM_ERR_ALIGN;
  return FP8MM_OK;
}

static int kv_grid(int64_t tasks, int threads, const DeviceInfo& dev) {
  return static_cast<int>(std::min<int64_t>(cdiv(tasks, threads / 32), static_cast<int64_t>(dev.sms) * 64));
}

// Every page in range, a destination written once and never a source.
static bool valid_moves(const int32_t* src, const int32_t* dst, int64_t moves, int64_t num_pages) {
  for (int64_t i = 0; i < moves; ++i)
    if (src[i] < 0 || src[i] >= num_pages || dst[i] < 0 || dst[i] >= num_pages) return false;
  std::unique_ptr<int32_t[]> sorted(new (std::nothrow) int32_t[moves]);
  if (!sorted) return false;
  std::copy(dst, dst + moves, sorted.get());
  std::sort(sorted.get(), sorted.get() + moves);
  if (std::adjacent_find(sorted.get(), sorted.get() + moves) != sorted.get() + moves) return false;
  for (int64_t i = 0; i < moves; ++i)
    if (std::binary_search(sorted.get(), sorted.get() + moves, src[i])) return false;
  return true;
}

// Jobs of an attention call with a workspace, and that workspace: counters,
// the list of cut tiles (one may begin in each job), two partial tiles per job.
static int attn_jobs(int sms) { return kAttnCtas * kAttnWarps * sms; }
static size_t attn_list_bytes(int sms) { return (256 + attn_jobs(sms) * sizeof(AttnCut) + 255) / 256 * 256; }
// Rows of the partial tiles: 8 per job of a warp (16 of half as many jobs), or
// kPreRows per job of a CTA.
static size_t attn_part_rows(int sms) {
  return std::max(static_cast<size_t>(attn_jobs(sms)) * 2 * 8, static_cast<size_t>(sms) * 2 * kPreRows);
}
static size_t attn_workspace(int sms, int64_t d) {
  return attn_list_bytes(sms) + attn_part_rows(sms) * static_cast<size_t>(d + 2) * sizeof(float);
}

template <int D, int NT, int FOLD>
static fp8mm_status launch_attn(KvAttnArgs& p, cudaStream_t s, const DeviceInfo& dev) {
  using Cfg = AttnCfg<D, NT, FOLD>;
  auto kern = kv4_attn_kernel<D, NT, FOLD>;
  const int grid = (NT == 1 ? kAttnCtas : 1) * dev.sms;
  p.jobs = grid * kAttnWarps;
  const int smem = kAttnWarps * static_cast<int>(sizeof(AttnShared<D, NT, FOLD>));
  fp8mm_status st = ensure_smem(reinterpret_cast<const void*>(kern), smem, dev.device);
  if (st != FP8MM_OK) return st;
  st = launch_pdl(kern, dim3(grid), dim3(kAttnThreads), smem, s, p);
  if (st != FP8MM_OK || p.partials == nullptr) return st;
  return launch_pdl(kv4_attn_join_kernel<D, Cfg::R>, dim3(2 * dev.sms), dim3(kJoinThreads), 0, s, p);
}

template <int D>
static fp8mm_status launch_prefill(KvAttnArgs& p, cudaStream_t s, const DeviceInfo& dev) {
  auto kern = kv4_prefill_kernel<D>;
  p.jobs = dev.sms;
  fp8mm_status st = ensure_smem(reinterpret_cast<const void*>(kern), PreCfg<D>::kSmemBytes, dev.device);
  if (st != FP8MM_OK) return st;
  st = launch_pdl(kern, dim3(dev.sms), dim3(kPreThreads), PreCfg<D>::kSmemBytes, s, p);
  if (st != FP8MM_OK || p.partials == nullptr) return st;
  return launch_pdl(kv4_attn_join_kernel<D, kPreRows>, dim3(2 * dev.sms), dim3(kJoinThreads), 0, s, p);
}

}  // namespace fp8mm

using namespace fp8mm;

extern "C" {

size_t mxfp4_kv_page_bytes(int64_t page_size, int64_t kv_heads, int64_t head_dim) {
  if (page_size < 16 || page_size % 16 != 0 || page_size > 4096 || kv_heads < 1 || kv_heads > 65535 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return static_cast<size_t>(page_bytes(page_size, kv_heads, head_dim));
}

fp8mm_status mxfp4_kv_append(const void* k_bf16, int64_t k_stride_t, int64_t k_stride_h, const void* v_bf16,
                             int64_t v_stride_t, int64_t v_stride_h, int64_t rows, const int32_t* cu_seqlens,
                             const int32_t* seq_lens, const fp8mm_kv_cache* cache, void* stream) {
  KvAppendArgs p{};
  fp8mm_status st = check_cache(cache, &p.kv);
  if (st != FP8MM_OK) return st;
  if (rows < 0 || rows > kMaxRows || (cu_seqlens == nullptr && rows != cache->batch)) return FP8MM_ERR_SHAPE;
  if (rows == 0 || cache->batch == 0) return FP8MM_OK;
  if (seq_lens == nullptr) return FP8MM_ERR_NULL;
  if ((st = check_rows(k_bf16, k_stride_t, k_stride_h, cache->kv_heads, cache->head_dim, false)) != FP8MM_OK) return st;
  if ((st = check_rows(v_bf16, v_stride_t, v_stride_h, cache->kv_heads, cache->head_dim, false)) != FP8MM_OK) return st;
  if (!aligned(cu_seqlens, 4) || !aligned(seq_lens, 4)) return FP8MM_ERR_ALIGN;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FP8MM_OK) return st;
  p.k = static_cast<const __nv_bfloat16*>(k_bf16);
  p.v = static_cast<const __nv_bfloat16*>(v_bf16);
  p.k_st = k_stride_t;
  p.k_sh = k_stride_h;
  p.v_st = v_stride_t;
  p.v_sh = v_stride_h;
  p.cu = cu_seqlens;
  p.lens = seq_lens;
  p.batch = static_cast<int32_t>(cache->batch);
  p.rows = rows;
  // A warp per row while few rows share a group, else per 16 rows (64 sequences, 8 heads: 4 new tokens
  // each 5.5 us against 9.5, 8 tokens 6.3 against 6.1, 16 tokens 7.9 against 4.6).
  const bool prompts = rows >= 8 * cache->batch;
  const int grid = kv_grid((prompts ? cdiv(rows, kGroup) : rows) * cache->kv_heads, kKvThreads, dev);
  auto kern = prompts ? (cache->head_dim == 128 ? kv4_append_kernel<128, kGroup> : kv4_append_kernel<64, kGroup>)
                      : (cache->head_dim == 128 ? kv4_append_kernel<128, 1> : kv4_append_kernel<64, 1>);
  st = launch_pdl(kern, dim3(grid), dim3(kKvThreads), 0, static_cast<cudaStream_t>(stream), p);
  return st != FP8MM_OK ? st : launched();
}

fp8mm_status mxfp4_kv_gather(const fp8mm_kv_cache* cache, const int32_t* starts, const int32_t* cu_seqlens,
                             int64_t rows, void* k_bf16, int64_t k_stride_t, int64_t k_stride_h, void* v_bf16,
                             int64_t v_stride_t, int64_t v_stride_h, void* stream) {
  KvGatherArgs p{};
  fp8mm_status st = check_cache(cache, &p.kv);
  if (st != FP8MM_OK) return st;
  if (rows < 0 || rows > kMaxRows) return FP8MM_ERR_SHAPE;
  if (rows == 0 || cache->batch == 0) return FP8MM_OK;
  if (cu_seqlens == nullptr) return FP8MM_ERR_NULL;
  if ((st = check_rows(k_bf16, k_stride_t, k_stride_h, cache->kv_heads, cache->head_dim, true)) != FP8MM_OK) return st;
  if ((st = check_rows(v_bf16, v_stride_t, v_stride_h, cache->kv_heads, cache->head_dim, true)) != FP8MM_OK) return st;
  if (!aligned(cu_seqlens, 4) || !aligned(starts, 4)) return FP8MM_ERR_ALIGN;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FP8MM_OK) return st;
  p.k = static_cast<__nv_bfloat16*>(k_bf16);
  p.v = static_cast<__nv_bfloat16*>(v_bf16);
  p.k_st = k_stride_t;
  p.k_sh = k_stride_h;
  p.v_st = v_stride_t;
  p.v_sh = v_stride_h;
  p.cu = cu_seqlens;
  p.starts = starts;
  p.batch = static_cast<int32_t>(cache->batch);
  p.rows = rows;
  const int grid = kv_grid(cdiv(rows, kGroup) * cache->kv_heads, kKvThreads, dev);
  // 32-byte stores of values where rows allow them (131072 tokens of 8 heads: 110 us, 114 with 16-byte ones)
  const bool wide = aligned(v_bf16, 32) && v_stride_t % 16 == 0 && v_stride_h % 16 == 0;
  auto kern = cache->head_dim == 128 ? (wide ? kv4_gather_kernel<128, true> : kv4_gather_kernel<128, false>)
                                     : (wide ? kv4_gather_kernel<64, true> : kv4_gather_kernel<64, false>);
  st = launch_pdl(kern, dim3(grid), dim3(kKvThreads), 0, static_cast<cudaStream_t>(stream), p);
  return st != FP8MM_OK ? st : launched();
}

size_t mxfp4_kv_attention_workspace_bytes(int64_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  DeviceInfo dev;
  const int sms = current_device(&dev) == FP8MM_OK ? dev.sms : 148;
  return attn_workspace(sms, head_dim);
}

fp8mm_status mxfp4_kv_attention(const void* q_bf16, int64_t q_stride_t, int64_t q_stride_h, int64_t rows,
                                int64_t q_heads, const int32_t* cu_seqlens, const int32_t* seq_lens,
                                const fp8mm_kv_cache* cache, float scale, void* out_bf16, int64_t out_stride_t,
                                int64_t out_stride_h, float* lse, int64_t lse_stride, void* workspace,
                                size_t workspace_bytes, void* stream) {
  KvAttnArgs p{};
  fp8mm_status st = check_cache(cache, &p.kv);
  if (st != FP8MM_OK) return st;
  if (rows < 0 || rows > kMaxRows || q_heads < 1 || q_heads > 65535 || q_heads % cache->kv_heads != 0 ||
      (cu_seqlens == nullptr && rows != cache->batch))
    return FP8MM_ERR_SHAPE;
  p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  if (!std::isfinite(p.scale_log2)) return FP8MM_ERR_SHAPE;
  if (rows == 0 || cache->batch == 0) return FP8MM_OK;
  if (seq_lens == nullptr) return FP8MM_ERR_NULL;
  const int64_t d = cache->head_dim;
  if ((st = check_rows(q_bf16, q_stride_t, q_stride_h, q_heads, d, false)) != FP8MM_OK) return st;
  if ((st = check_rows(out_bf16, out_stride_t, out_stride_h, q_heads, d, true)) != FP8MM_OK) return st;
  if (lse != nullptr && lse_stride < q_heads) return FP8MM_ERR_SHAPE;
  if (!aligned(cu_seqlens, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4)) return FP8MM_ERR_ALIGN;
  if (workspace != nullptr && !aligned(workspace, 256)) return FP8MM_ERR_ALIGN;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FP8MM_OK) return st;
  if (workspace != nullptr && workspace_bytes < attn_workspace(dev.sms, d)) return FP8MM_ERR_WORKSPACE;
  p.q = static_cast<const __nv_bfloat16*>(q_bf16);
  p.out = static_cast<__nv_bfloat16*>(out_bf16);
  p.lse = lse;
  p.q_st = q_stride_t;
  p.q_sh = q_stride_h;
  p.o_st = out_stride_t;
  p.o_sh = out_stride_h;
  p.lse_st = lse_stride;
  p.cu = cu_seqlens;
  p.lens = seq_lens;
  p.rows = rows;
  p.batch = static_cast<int32_t>(cache->batch);
  p.group = static_cast<int32_t>(q_heads / cache->kv_heads);
  // a masked score stays -inf after scaling, any other one becomes next to nothing
  if (p.scale_log2 == 0.f) p.scale_log2 = std::numeric_limits<float>::denorm_min();
  p.timeout_ns = wait_timeout_ns();
  if (workspace != nullptr) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.counters = reinterpret_cast<AttnCounters*>(ws);
    p.cuts = reinterpret_cast<AttnCut*>(ws + 256);
    p.partials = reinterpret_cast<float*>(ws + attn_list_bytes(dev.sms));
  }
  if (rows * p.group > INT32_MAX) return FP8MM_ERR_SHAPE;
  // units: every tile's steps and layout, at most; more steps a unit where they would not fit 31 bits
  const double steps = static_cast<double>(p.kv.max_pages) * p.kv.page_groups / kStep + 1 + kTileSteps;
  const double tiles = (static_cast<double>(rows) * p.group / 4 + p.batch) * p.kv.kv_heads;
  if (tiles > 1e9) return FP8MM_ERR_SHAPE;
  p.unit_steps = static_cast<int32_t>(std::min(1e9, 1 + steps * tiles / 2e9));
  // Rows that a sequence has on average decide the tile: 4, 8 or 16 of them, or 256 (which needs the workspace).
  // 32 sequences of 4096 tokens, 8 heads: 4 rows 39.1 us in tiles of 4, 41.4 of 8, 58.5 of 16; 8 rows 42.4 in
  // tiles of 8, 60.5 of 16.  Tiles of 16 and of 256, head size 128 | 64, us in a graph:
  //   16 sequences of 4096: 64 rows 111, 133 | 81, 120;  96 rows 158, 139 | 115, 125;  128 rows 206, 138 | 150, 118
  //   64 of 512:            64 rows 183, 134 | 99, 104;  96 rows 268, 148 | 136, 115;  128 rows 327, 153 | 165, 111
  //   1 of 32768:           64 rows 56, 70 | 42, 58;     96 rows 79, 70 | 57, 57;      128 rows 97, 67 | 70, 54
  //   2 of 1024:            96 rows 23, 39 | 19, 28;     128 rows 24, 40 | 20, 28;     256 rows 34, 42 | 26, 29
  // Little work in short contexts would be better off in tiles of 16 throughout, at most 16 us; one size serves a
  // whole call, whatever its sequences' own rows.
  const int64_t tile = cdiv(rows, cache->batch) * p.group;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.partials != nullptr && tile >= kPreFrom)
    st = d == 128 ? launch_prefill<128>(p, s, dev) : launch_prefill<64>(p, s, dev);
  else if (d == 128)
    st = tile <= 4   ? launch_attn<128, 1, 2>(p, s, dev)
         : tile <= 8 ? launch_attn<128, 1, 1>(p, s, dev)
                     : launch_attn<128, 2, 1>(p, s, dev);
  else
    st = tile <= 4   ? launch_attn<64, 1, 2>(p, s, dev)
         : tile <= 8 ? launch_attn<64, 1, 1>(p, s, dev)
                     : launch_attn<64, 2, 1>(p, s, dev);
  return st != FP8MM_OK ? st : launched();
}

fp8mm_status kv_copy_pages(void* pages, int64_t num_pages, int64_t page_bytes, int64_t page_stride, int64_t layers,
                           int64_t layer_stride, const int32_t* src, const int32_t* dst, int64_t moves, void* stream) {
  if (num_pages < 0 || num_pages > INT32_MAX || page_bytes < 0 || page_bytes > INT32_MAX || layers < 0 ||
      layers > INT32_MAX || moves < 0 || moves > num_pages)
    return FP8MM_ERR_SHAPE;
  if (moves == 0 || layers == 0 || page_bytes == 0) return FP8MM_OK;
  // pages apart in each layer, and layers apart or, with a page's layers side by side, pages apart
  if (page_stride < page_bytes ||
      (layers > 1 && (layer_stride < page_bytes || ((layer_stride - page_bytes) / page_stride < num_pages - 1 &&
                                                    (page_stride - page_bytes) / layer_stride < layers - 1))))
    return FP8MM_ERR_SHAPE;
  if (pages == nullptr || src == nullptr || dst == nullptr) return FP8MM_ERR_NULL;
  if (!aligned(pages, 16) || page_bytes % 16 != 0 || page_stride % 16 != 0 || layer_stride % 16 != 0)
    return FP8MM_ERR_ALIGN;
  if (!valid_moves(src, dst, moves, num_pages)) return FP8MM_ERR_SHAPE;
  DeviceInfo dev;
  fp8mm_status st = current_device(&dev);
  if (st != FP8MM_OK) return st;
  KvCopyArgs p{};
  p.page_stride = page_stride;
  p.layer_stride = layer_stride;
  p.page_vecs = static_cast<uint32_t>(page_bytes / 16);
  const int64_t slices = cdiv(p.page_vecs, kCopyThreads * kCopyUnroll);
  for (int64_t m0 = 0; m0 < moves; m0 += kPageMoves) {
    p.moves = static_cast<int32_t>(std::min<int64_t>(kPageMoves, moves - m0));
    std::copy(src + m0, src + m0 + p.moves, p.src);
    std::copy(dst + m0, dst + m0 + p.moves, p.dst);
    const int64_t per_launch = std::max<int64_t>(1, INT32_MAX / (p.moves * slices));  // layers within the grid's limit
    for (int64_t l0 = 0; l0 < layers; l0 += per_launch) {
      p.base = static_cast<uint8_t*>(pages) + l0 * layer_stride;
      p.layers = static_cast<int32_t>(std::min<int64_t>(per_launch, layers - l0));
      st = launch_pdl(kv_copy_pages_kernel, dim3(static_cast<unsigned>(p.layers * p.moves * slices)), dim3(kCopyThreads),
                      0, static_cast<cudaStream_t>(stream), p, static_cast<uint32_t>(slices));
      if (st != FP8MM_OK) return st;
    }
  }
  return launched();
}

fp8mm_status qk_norm_rope(const void* q_bf16, int64_t q_stride_t, int64_t q_stride_h, const void* k_bf16,
                          int64_t k_stride_t, int64_t k_stride_h, int64_t tokens, int64_t q_heads, int64_t k_heads,
                          int64_t head_dim, const void* q_weight, const void* k_weight, float eps,
                          const float* cos_sin, int64_t max_pos, int64_t rot_dim, int64_t cos_sin_stride,
                          int32_t interleaved, const int32_t* positions, void* q_out, int64_t q_out_stride_t,
                          int64_t q_out_stride_h, void* k_out, int64_t k_out_stride_t, int64_t k_out_stride_h,
                          void* stream) {
  if (tokens < 0 || tokens > kMaxRows || q_heads < 0 || k_heads < 0 || q_heads + k_heads > 65535) return FP8MM_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return FP8MM_ERR_SHAPE;
  if (rot_dim < 16 || rot_dim > head_dim || rot_dim % 16 != 0 || max_pos < 1 || max_pos > INT32_MAX ||
      cos_sin_stride < rot_dim || !(eps >= 0.f) || !std::isfinite(eps) || (interleaved != 0 && interleaved != 1))
    return FP8MM_ERR_SHAPE;
  if (tokens == 0 || q_heads + k_heads == 0) return FP8MM_OK;
  if (cos_sin == nullptr || positions == nullptr || ((q_weight == nullptr) != (k_weight == nullptr)))
    return FP8MM_ERR_NULL;
  fp8mm_status st = FP8MM_OK;
  if (q_heads > 0 && ((st = check_rows(q_bf16, q_stride_t, q_stride_h, q_heads, head_dim, false)) != FP8MM_OK ||
                      (st = check_rows(q_out, q_out_stride_t, q_out_stride_h, q_heads, head_dim, true)) != FP8MM_OK))
    return st;
  if (k_heads > 0 && ((st = check_rows(k_bf16, k_stride_t, k_stride_h, k_heads, head_dim, false)) != FP8MM_OK ||
                      (st = check_rows(k_out, k_out_stride_t, k_out_stride_h, k_heads, head_dim, true)) != FP8MM_OK))
    return st;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(cos_sin, 16) || cos_sin_stride % 4 != 0 ||
      !aligned(positions, 4))
    return FP8MM_ERR_ALIGN;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != FP8MM_OK) return st;
  QkNormArgs p{};
  p.q = static_cast<const __nv_bfloat16*>(q_bf16);
  p.k = static_cast<const __nv_bfloat16*>(k_bf16);
  p.qo = static_cast<__nv_bfloat16*>(q_out);
  p.ko = static_cast<__nv_bfloat16*>(k_out);
  p.q_st = q_stride_t;
  p.q_sh = q_stride_h;
  p.k_st = k_stride_t;
  p.k_sh = k_stride_h;
  p.qo_st = q_out_stride_t;
  p.qo_sh = q_out_stride_h;
  p.ko_st = k_out_stride_t;
  p.ko_sh = k_out_stride_h;
  p.qw = static_cast<const __nv_bfloat16*>(q_weight);
  p.kw = static_cast<const __nv_bfloat16*>(k_weight);
  p.cos_sin = cos_sin;
  p.cs_stride = cos_sin_stride;
  p.pos = positions;
  p.tokens = tokens;
  p.q_heads = static_cast<int32_t>(q_heads);
  p.k_heads = static_cast<int32_t>(k_heads);
  p.rot = static_cast<int32_t>(rot_dim);
  p.max_pos = static_cast<int32_t>(max_pos);
  p.eps = eps;
  // warps of a token: one that walks all its heads, keeping the angles, and more, down to one step each, while the
  // tokens alone would not fill the SMs (40 heads of 128, one warp and one per step: 8192 tokens 33.7 and 45.9 us, 2048
  // tokens 11.3 and 10.9, 1024 tokens 8.8 and 6.2, 7.9 by this rule, 64 tokens 6.2 and 2.5)
  const int64_t step = kNormUnroll * (256 / head_dim), steps = cdiv(q_heads, step) + cdiv(k_heads, step);
  const int64_t fill = std::max<int64_t>(1, static_cast<int64_t>(dev.sms) * 32 / tokens);
  p.slices = static_cast<int32_t>(std::min(steps, fill));
  const int64_t blocks = cdiv(tokens * p.slices, kNormThreads / 32);
  if (blocks > INT32_MAX) return FP8MM_ERR_SHAPE;
  auto pick = [&](auto half, auto inter) { return interleaved ? inter : half; };
  auto kern = head_dim == 64    ? pick(qk_norm_rope_kernel<64, false>, qk_norm_rope_kernel<64, true>)
              : head_dim == 128 ? pick(qk_norm_rope_kernel<128, false>, qk_norm_rope_kernel<128, true>)
                                : pick(qk_norm_rope_kernel<256, false>, qk_norm_rope_kernel<256, true>);
  st = launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kNormThreads), 0, static_cast<cudaStream_t>(stream), p);
  return st != FP8MM_OK ? st : launched();
}

}  // extern "C"
