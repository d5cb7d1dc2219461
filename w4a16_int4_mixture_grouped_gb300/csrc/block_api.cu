// Host side of the paged cache, its attention and the block norms (declared in
// include/moe_w4a16.h): argument checks and launches. No device memory is allocated here.
#include <cmath>

#include <cuda_runtime.h>

#include "block.h"
#include "internal.h"
#include "moe_w4a16.h"

using namespace moe;

#define MOE_CUDA_TRY(expr)                            \
  do {                                                \
    if ((expr) != cudaSuccess) return MOE_W4A16_ERR_CUDA; \
  } while (0)

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool ws_fits(const void* ws, size_t bytes, size_t need) {
  return ws != nullptr && aligned16(ws) && bytes >= need && bytes >= MOE_W4A16_WS_HEADER_BYTES;
}

// A layer's pages for rows of `heads` heads of `dim` channels.
moe_w4a16_status check_pages(const moe_w4a16_pages* c, int heads, int dim, bool latent) {
  if (c == nullptr || c->k == nullptr || (c->v == nullptr) != latent) return MOE_W4A16_ERR_INVALID_ARG;
  if (c->dtype != MOE_W4A16_CACHE_BF16 && c->dtype != MOE_W4A16_CACHE_E4M3) return MOE_W4A16_ERR_INVALID_ARG;
  if (latent && c->dtype != MOE_W4A16_CACHE_BF16) return MOE_W4A16_ERR_UNSUPPORTED;
  if (c->num_pages < 1 || c->page_size < 1 || c->page_size > MOE_W4A16_MAX_PAGE_SIZE || c->reserved != 0)
    return MOE_W4A16_ERR_INVALID_ARG;
  const int vec = c->dtype == MOE_W4A16_CACHE_E4M3 ? 16 : 8;   // elements of 16 bytes
  if (dim % vec != 0) return MOE_W4A16_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v)) return MOE_W4A16_ERR_INVALID_ARG;
  if (c->page_stride % vec != 0 || c->token_stride % vec != 0 || c->head_stride % vec != 0)
    return MOE_W4A16_ERR_INVALID_ARG;
  if (c->page_stride < 0 || c->token_stride < dim || (heads > 1 && c->head_stride < dim))
    return MOE_W4A16_ERR_INVALID_ARG;
  if (c->dtype == MOE_W4A16_CACHE_E4M3) {
    if (!std::isfinite(c->k_scale) || !std::isfinite(c->v_scale) || c->k_scale <= 0.f || c->v_scale <= 0.f)
      return MOE_W4A16_ERR_INVALID_ARG;
  } else if (c->k_scale != 1.f || c->v_scale != 1.f) {
    return MOE_W4A16_ERR_INVALID_ARG;
  }
  return MOE_W4A16_OK;
}

// Tokens of a full table row stay below 2^31.
bool table_ok(const void* tables, int64_t stride, int max_pages, int page_size, int num_seqs) {
  return tables != nullptr && max_pages >= 1 && stride >= max_pages && num_seqs >= 1 &&
         static_cast<int64_t>(max_pages) * page_size < (int64_t(1) << 31);
}

TableView table_view(const int32_t* tables, int64_t stride, int max_pages, int page_size, int num_pages, int num_seqs) {
  return TableView{tables, stride, max_pages, page_size, num_pages, num_seqs};
}

moe_w4a16_status pool_view(const moe_w4a16_pool* pool, PoolView* out) {
  if (pool == nullptr || pool->base == nullptr || pool->num_planes < 1 || pool->num_pages < 1 || pool->page_bytes < 16)
    return MOE_W4A16_ERR_INVALID_ARG;
  if (!aligned16(pool->base) || (pool->plane_stride | pool->page_stride | pool->page_bytes) % 16 != 0)
    return MOE_W4A16_ERR_INVALID_ARG;
  if (pool->page_stride < pool->page_bytes || pool->plane_stride < 0) return MOE_W4A16_ERR_INVALID_ARG;
  if (pool->page_bytes >= (int64_t(1) << 34)) return MOE_W4A16_ERR_UNSUPPORTED;
  *out = PoolView{static_cast<uint8_t*>(pool->base), pool->num_planes, pool->num_pages, pool->plane_stride,
                  pool->page_stride, pool->page_bytes};
  return MOE_W4A16_OK;
}

moe_w4a16_status page_ops(int32_t* refs, int num_pages, int32_t* tables, int64_t table_stride, int max_pages,
                          int32_t* lens, int num_seqs, int count, int page_size, void* ws, size_t ws_bytes,
                          PageOps* o) {
  if (refs == nullptr || lens == nullptr || num_pages < 1 || count < 0 || page_size < 1 ||
      page_size > MOE_W4A16_MAX_PAGE_SIZE || !table_ok(tables, table_stride, max_pages, page_size, num_seqs))
    return MOE_W4A16_ERR_INVALID_ARG;
  // a call's page needs are summed in 32 bits
  if (static_cast<int64_t>(count) * max_pages >= (int64_t(1) << 31)) return MOE_W4A16_ERR_UNSUPPORTED;
  size_t need = 0;
  const moe_w4a16_status st = moe_w4a16_cache_workspace_size(num_pages, count, &need);
  if (st != MOE_W4A16_OK) return st;
  if (!ws_fits(ws, ws_bytes, need)) return MOE_W4A16_ERR_WORKSPACE;
  o->t = table_view(tables, table_stride, max_pages, page_size, num_pages, num_seqs);
  o->tables = tables;
  o->lens = lens;
  o->refs = refs;
  o->count = count;
  o->scratch = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kBlockWsOffset);
  o->entries = count > num_pages ? count : num_pages;
  o->err = static_cast<int*>(ws);
  return MOE_W4A16_OK;
}

moe_w4a16_status attention_call(AttnParams& p, const moe_w4a16_pages* cache, const int32_t* tables,
                                int64_t table_stride, int max_pages, int num_seqs, float scale, void* ws,
                                size_t ws_bytes, bool latent, cudaStream_t stream) {
  if (p.batch < 0 || p.heads < 1 || p.kv_heads < 1 || p.heads % p.kv_heads != 0 || p.window < 0 || !std::isfinite(scale))
    return MOE_W4A16_ERR_INVALID_ARG;
  if (p.dim < 16 || p.dim % 16 != 0 || (!latent && p.dim > MOE_W4A16_MAX_HEAD_DIM)) return MOE_W4A16_ERR_UNSUPPORTED;
  moe_w4a16_status st = check_pages(cache, p.kv_heads, p.dim, latent);
  if (st != MOE_W4A16_OK) return st;
  if (static_cast<int64_t>(p.batch) * p.heads >= (int64_t(1) << 31)) return MOE_W4A16_ERR_UNSUPPORTED;
  size_t need = 0;
  st = moe_w4a16_attention_workspace_size(p.heads, p.kv_heads, p.dim, &need);
  if (st != MOE_W4A16_OK) return st;
  if (!ws_fits(ws, ws_bytes, need)) return MOE_W4A16_ERR_WORKSPACE;
  if (p.batch == 0) return MOE_W4A16_OK;
  if (p.q == nullptr || p.out == nullptr || p.lens == nullptr || !aligned16(p.q) || !aligned16(p.out) ||
      p.q_stride % 8 != 0 || p.q_stride < static_cast<int64_t>(p.heads) * p.dim)
    return MOE_W4A16_ERR_INVALID_ARG;
  if (p.seq_ids == nullptr && num_seqs < p.batch) return MOE_W4A16_ERR_INVALID_ARG;
  if (!table_ok(tables, table_stride, max_pages, cache->page_size, num_seqs)) return MOE_W4A16_ERR_INVALID_ARG;
  p.group = p.heads / p.kv_heads;
  p.k = cache->k;
  p.v = cache->v;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  p.t = table_view(tables, table_stride, max_pages, cache->page_size, cache->num_pages, num_seqs);
  p.score_scale = static_cast<float>(static_cast<double>(scale) * cache->k_scale * 1.4426950408889634);
  p.v_scale = cache->v_scale;
  p.err = static_cast<int*>(ws);
  p.counters = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + MOE_W4A16_WS_HEADER_BYTES);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kBlockWsOffset);
  int device = 0;
  MOE_CUDA_TRY(cudaGetDevice(&device));
  p.wait_ns = wait_limit_ns(device);
  MOE_CUDA_TRY(latent ? launch_latent_attention(p, device, stream) : launch_attention(p, cache->dtype, device, stream));
  return MOE_W4A16_OK;
}

}  // namespace

extern "C" {

moe_w4a16_status moe_w4a16_attention_workspace_size(int num_heads, int num_kv_heads, int head_dim, size_t* bytes) {
  if (bytes == nullptr || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0)
    return MOE_W4A16_ERR_INVALID_ARG;
  const bool latent = num_kv_heads == 1 && head_dim == MOE_W4A16_LATENT_DIM;
  if (head_dim < 16 || head_dim % 16 != 0 || (!latent && head_dim > MOE_W4A16_MAX_HEAD_DIM))
    return MOE_W4A16_ERR_UNSUPPORTED;
  // header | arrival counters | parts of split rows
  *bytes = kBlockWsOffset + (latent ? latent_part_bytes(num_heads) : attention_part_bytes(num_heads, num_kv_heads, head_dim));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_paged_attention(const uint16_t* q, int64_t q_stride, int batch, int num_heads,
                                           int num_kv_heads, int head_dim, const moe_w4a16_pages* cache,
                                           const int32_t* tables, int64_t table_stride, int max_pages,
                                           const int32_t* lens, const int32_t* seq_ids, int num_seqs, float scale,
                                           int window, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                                           moe_w4a16_stream_t stream) {
  AttnParams p{};
  p.q = q;
  p.q_stride = q_stride;
  p.batch = batch;
  p.heads = num_heads;
  p.kv_heads = num_kv_heads;
  p.dim = head_dim;
  p.lens = lens;
  p.seq_ids = seq_ids;
  p.window = window;
  p.out = out;
  p.lse = lse;
  return attention_call(p, cache, tables, table_stride, max_pages, num_seqs, scale, ws, ws_bytes, false,
                        reinterpret_cast<cudaStream_t>(stream));
}

moe_w4a16_status moe_w4a16_latent_attention(const uint16_t* q, int64_t q_stride, int batch, int num_heads,
                                            const moe_w4a16_pages* cache, const int32_t* tables, int64_t table_stride,
                                            int max_pages, const int32_t* lens, const int32_t* seq_ids, int num_seqs,
                                            float scale, int window, uint16_t* out, float* lse, void* ws,
                                            size_t ws_bytes, moe_w4a16_stream_t stream) {
  AttnParams p{};
  p.q = q;
  p.q_stride = q_stride;
  p.batch = batch;
  p.heads = num_heads;
  p.kv_heads = 1;
  p.dim = MOE_W4A16_LATENT_DIM;
  p.lens = lens;
  p.seq_ids = seq_ids;
  p.window = window;
  p.out = out;
  p.lse = lse;
  return attention_call(p, cache, tables, table_stride, max_pages, num_seqs, scale, ws, ws_bytes, true,
                        reinterpret_cast<cudaStream_t>(stream));
}

moe_w4a16_status moe_w4a16_cache_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                        int num_tokens, int num_heads, int head_dim, const moe_w4a16_pages* cache,
                                        const int32_t* tables, int64_t table_stride, int max_pages, int num_seqs,
                                        const int32_t* seq_ids, const int32_t* positions, void* ws, size_t ws_bytes,
                                        moe_w4a16_stream_t stream) {
  if (num_tokens < 0 || num_heads < 1 || head_dim < 8 || head_dim > (1 << 16) || num_heads > (1 << 12))
    return MOE_W4A16_ERR_INVALID_ARG;
  if (cache == nullptr) return MOE_W4A16_ERR_INVALID_ARG;
  const bool latent = cache->v == nullptr;
  moe_w4a16_status st = check_pages(cache, num_heads, head_dim, latent);
  if (st != MOE_W4A16_OK) return st;
  if (!table_ok(tables, table_stride, max_pages, cache->page_size, num_seqs)) return MOE_W4A16_ERR_INVALID_ARG;
  if (!ws_fits(ws, ws_bytes, MOE_W4A16_WS_HEADER_BYTES)) return MOE_W4A16_ERR_WORKSPACE;
  const int64_t width = static_cast<int64_t>(num_heads) * head_dim;
  if ((v == nullptr) != latent && num_tokens > 0) return MOE_W4A16_ERR_INVALID_ARG;
  if (k_stride < width || k_stride % 8 != 0 || (!latent && (v_stride < width || v_stride % 8 != 0)))
    return MOE_W4A16_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_W4A16_OK;
  if (k == nullptr || seq_ids == nullptr || positions == nullptr || !aligned16(k) || !aligned16(v))
    return MOE_W4A16_ERR_INVALID_ARG;
  AppendParams p{};
  p.src[0] = k;
  p.src[1] = v;
  p.src_stride[0] = k_stride;
  p.src_stride[1] = v_stride;
  p.pages[0] = cache->k;
  p.pages[1] = cache->v;
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.tokens = num_tokens;
  p.heads = num_heads;
  p.dim = head_dim;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  p.t = table_view(tables, table_stride, max_pages, cache->page_size, cache->num_pages, num_seqs);
  p.seq_ids = seq_ids;
  p.positions = positions;
  p.err = static_cast<int*>(ws);
  MOE_CUDA_TRY(launch_cache_append(p, cache->dtype, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_cache_workspace_size(int num_pages, int count, size_t* bytes) {
  if (bytes == nullptr || num_pages < 0 || count < 0 || count > (1 << 28) || num_pages > (1 << 28))
    return MOE_W4A16_ERR_INVALID_ARG;
  // header | the attention calls' counters, left alone | scratch
  *bytes = kBlockWsOffset + cache_ws_words(num_pages, count) * sizeof(int32_t);
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_cache_extend(int32_t* refs, int num_pages, int32_t* tables, int64_t table_stride,
                                        int max_pages, int32_t* lens, int num_seqs, const int32_t* seq_ids,
                                        const int32_t* counts, int count, int page_size, int32_t* positions, void* ws,
                                        size_t ws_bytes, moe_w4a16_stream_t stream) {
  PageOps o{};
  moe_w4a16_status st = page_ops(refs, num_pages, tables, table_stride, max_pages, lens, num_seqs, count, page_size, ws,
                                 ws_bytes, &o);
  if (st != MOE_W4A16_OK) return st;
  if (count == 0) return MOE_W4A16_OK;
  if (seq_ids == nullptr || positions == nullptr) return MOE_W4A16_ERR_INVALID_ARG;
  MOE_CUDA_TRY(launch_cache_extend(o, seq_ids, counts, positions, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_cache_fork(const moe_w4a16_pool* pool, int32_t* refs, int32_t* tables, int64_t table_stride,
                                      int max_pages, int32_t* lens, int num_seqs, const int32_t* parents,
                                      const int32_t* children, int count, int page_size, void* ws, size_t ws_bytes,
                                      moe_w4a16_stream_t stream) {
  PoolView view;
  moe_w4a16_status st = pool_view(pool, &view);
  if (st != MOE_W4A16_OK) return st;
  PageOps o{};
  st = page_ops(refs, view.num_pages, tables, table_stride, max_pages, lens, num_seqs, count, page_size, ws, ws_bytes,
                &o);
  if (st != MOE_W4A16_OK) return st;
  if (count == 0) return MOE_W4A16_OK;
  if (parents == nullptr || children == nullptr) return MOE_W4A16_ERR_INVALID_ARG;
  int device = 0;
  MOE_CUDA_TRY(cudaGetDevice(&device));
  MOE_CUDA_TRY(launch_cache_fork(o, view, parents, children, device, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_cache_free(int32_t* refs, int num_pages, int32_t* tables, int64_t table_stride,
                                      int max_pages, int32_t* lens, int num_seqs, const int32_t* seq_ids,
                                      const int32_t* keep, int count, int page_size, void* ws, size_t ws_bytes,
                                      moe_w4a16_stream_t stream) {
  PageOps o{};
  moe_w4a16_status st = page_ops(refs, num_pages, tables, table_stride, max_pages, lens, num_seqs, count, page_size, ws,
                                 ws_bytes, &o);
  if (st != MOE_W4A16_OK) return st;
  if (count == 0) return MOE_W4A16_OK;
  if (seq_ids == nullptr) return MOE_W4A16_ERR_INVALID_ARG;
  MOE_CUDA_TRY(launch_cache_free(o, seq_ids, keep, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_cache_copy(const moe_w4a16_pool* pool, const int32_t* src, const int32_t* dst, int count,
                                      void* ws, size_t ws_bytes, moe_w4a16_stream_t stream) {
  PoolView view;
  moe_w4a16_status st = pool_view(pool, &view);
  if (st != MOE_W4A16_OK) return st;
  if (count < 0) return MOE_W4A16_ERR_INVALID_ARG;
  if (!ws_fits(ws, ws_bytes, MOE_W4A16_WS_HEADER_BYTES)) return MOE_W4A16_ERR_WORKSPACE;
  if (count == 0) return MOE_W4A16_OK;
  if (src == nullptr || dst == nullptr) return MOE_W4A16_ERR_INVALID_ARG;
  int device = 0;
  MOE_CUDA_TRY(cudaGetDevice(&device));
  MOE_CUDA_TRY(launch_cache_copy(view, src, dst, count, static_cast<int*>(ws), device,
                                 reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_cache_compact(const moe_w4a16_pool* pool, const int32_t* refs, const int32_t* tables,
                                         int64_t table_stride, int max_pages, int num_seqs, int32_t* refs_out,
                                         int32_t* tables_out, int32_t* page_map, int32_t* num_live, void* ws,
                                         size_t ws_bytes, moe_w4a16_stream_t stream) {
  PoolView view;
  moe_w4a16_status st = pool_view(pool, &view);
  if (st != MOE_W4A16_OK) return st;
  if (tables_out == nullptr || refs_out == nullptr || page_map == nullptr || num_live == nullptr || refs == nullptr)
    return MOE_W4A16_ERR_INVALID_ARG;
  PageOps o{};
  // the lengths play no part; the tables are read, never written through this view
  st = page_ops(refs_out, view.num_pages, const_cast<int32_t*>(tables), table_stride, max_pages, refs_out, num_seqs, 0,
                1, ws, ws_bytes, &o);
  if (st != MOE_W4A16_OK) return st;
  int device = 0;
  MOE_CUDA_TRY(cudaGetDevice(&device));
  MOE_CUDA_TRY(launch_cache_compact(o, view, refs, refs_out, tables_out, page_map, num_live, device,
                                    reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_block_norm(const uint16_t* x, int64_t x_stride, const void* h, int64_t h_stride,
                                      int residual_dtype, const uint16_t* gate, int gate_rows, const uint16_t* w_post,
                                      const uint16_t* w_pre, int rows, int n, float eps, float residual_scale,
                                      float block_scale, void* h_out, int64_t h_out_stride, uint16_t* y,
                                      int64_t y_stride, moe_w4a16_stream_t stream) {
  if (residual_dtype != MOE_W4A16_RESIDUAL_BF16 && residual_dtype != MOE_W4A16_RESIDUAL_F32)
    return MOE_W4A16_ERR_INVALID_ARG;
  if (rows < 0 || n < 1 || !(eps >= 0.f) || !std::isfinite(eps)) return MOE_W4A16_ERR_INVALID_ARG;
  if (n > MOE_W4A16_MAX_NORM_WIDTH) return MOE_W4A16_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_W4A16_OK;
  if (h == nullptr || (h_out == nullptr && y == nullptr) || (y == nullptr) != (w_pre == nullptr))
    return MOE_W4A16_ERR_INVALID_ARG;
  if (x == nullptr && (gate != nullptr || w_post != nullptr)) return MOE_W4A16_ERR_INVALID_ARG;
  if (gate != nullptr && (gate_rows < 1 || rows % gate_rows != 0)) return MOE_W4A16_ERR_INVALID_ARG;
  if (h_stride < n || (x != nullptr && x_stride < n) || (h_out != nullptr && h_out_stride < n) ||
      (y != nullptr && y_stride < n))
    return MOE_W4A16_ERR_INVALID_ARG;
  const bool res32 = residual_dtype == MOE_W4A16_RESIDUAL_F32;
  const auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  // element alignment of every tensor, then the widest access that all rows of all of them allow: 2 bytes a column
  // for BF16, 4 (up to 16 in all) for an FP32 residual
  const uintptr_t res = bits(h) | bits(h_out), rest = bits(x) | bits(gate) | bits(w_post) | bits(w_pre) | bits(y);
  if ((res & (res32 ? 3u : 1u)) != 0 || (rest & 1u) != 0) return MOE_W4A16_ERR_INVALID_ARG;
  int64_t columns = n;
  if (rows > 1) {
    columns |= h_stride;
    if (x != nullptr) columns |= x_stride;
    if (h_out != nullptr) columns |= h_out_stride;
    if (y != nullptr) columns |= y_stride;
  }
  int width = 8;
  while (width > 1 && (columns % width != 0 || (rest & (2u * width - 1u)) != 0 ||
                       (res & (res32 ? (width > 4 ? 15u : 4u * width - 1u) : 2u * width - 1u)) != 0))
    width /= 2;
  // rows that start at any column, but all tensors' alike
  const auto alike = [&](const void* t, int64_t stride) { return t == nullptr || rows == 1 || (stride - h_stride) % 8 == 0; };
  const bool shift = width < 8 && ((res | bits(x) | bits(y)) & 15u) == 0 && alike(x, x_stride) &&
                     alike(h_out, h_out_stride) && alike(y, y_stride);
  NormParams p{};
  p.x = x;
  p.x_stride = x_stride;
  p.h = h;
  p.h_stride = h_stride;
  p.gate = gate;
  p.rows_per_gate = gate != nullptr ? rows / gate_rows : 1;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.rows = rows;
  p.n = n;
  p.eps = eps;
  p.res_scale = residual_scale;
  p.blk_scale = block_scale;
  p.h_out = h_out;
  p.h_out_stride = h_out_stride;
  p.y = y;
  p.y_stride = y_stride;
  int device = 0;
  MOE_CUDA_TRY(cudaGetDevice(&device));
  MOE_CUDA_TRY(launch_block_norm(p, res32, width, shift, device, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

}  // extern "C"
