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

// Places in memory: `tokens` x `heads` rows of `width` bytes.
struct Rows {
  int64_t at, tokens, token_stride, heads, head_stride, width;
  Rows(const void* p, int64_t t, int64_t ts, int64_t h, int64_t hs, int64_t w)
      : at(static_cast<int64_t>(reinterpret_cast<uintptr_t>(p))), tokens(t), token_stride(ts), heads(h), head_stride(hs), width(w) {
    if (token_stride == 0) tokens = 1;                     // (a broadcast row is one)
    if (head_stride == 0) heads = 1;
    if (heads > 1 && head_stride == width) width *= heads, heads = 1;
    if (tokens > 1 && token_stride == width) width *= tokens, tokens = 1;
  }
  int64_t end() const { return at + (tokens - 1) * token_stride + (heads - 1) * head_stride + width; }
};
int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && (a < 0) != (b < 0) ? 1 : 0); }
// Whether x + k * stride lies between low and high (neither included) for a k of from .. to.
bool between(int64_t x, int64_t stride, int64_t from, int64_t to, int64_t low, int64_t high) {
  if (from > to) return false;
  if (stride <= 0) return low < x && x < high;
  const int64_t first = floor_div(low - x, stride) + 1, k = first > from ? first : from;
  return k <= to && x + k * stride < high;
}
// Whether a byte is in both, exactly; the rows of b lie apart from each other. Rows that lie between each other's (queries and keys
// of one buffer) are no overlap.
bool overlap(const Rows& a, const Rows& b) {
  if (a.end() <= b.at || b.end() <= a.at) return false;
  if ((a.tokens == 1 || b.tokens == 1 || a.token_stride == b.token_stride) &&
      (a.heads == 1 || b.heads == 1 || a.head_stride == b.head_stride)) {
    // all distances between rows are x + token steps + head steps
    const int64_t ts = a.tokens > 1 ? a.token_stride : b.token_stride, hs = a.heads > 1 ? a.head_stride : b.head_stride;
    for (int64_t h = 1 - a.heads; h < b.heads; ++h)
      if (between(b.at - a.at + h * hs, b.tokens > 1 || a.tokens > 1 ? ts : 0, 1 - a.tokens, b.tokens - 1, -b.width, a.width)) return true;
    return false;
  }
  // row by row of a (rare): b's outer steps near it, then the inner ones
  const bool by_token = b.heads == 1 || (b.tokens > 1 && b.token_stride >= b.head_stride);
  const int64_t outer = by_token ? b.tokens : b.heads, outer_step = by_token ? b.token_stride : b.head_stride;
  const int64_t inner = by_token ? b.heads : b.tokens, inner_step = by_token ? b.head_stride : b.token_stride;
  const int64_t span = (inner - 1) * inner_step + b.width;
  for (int64_t t = 0; t < a.tokens; ++t)
    for (int64_t h = 0; h < a.heads; ++h) {
      const int64_t x = a.at + t * a.token_stride + h * a.head_stride - b.at;
      int64_t o = outer > 1 ? floor_div(x - span, outer_step) + 1 : 0;
      for (o = o < 0 ? 0 : o; o < outer && o * outer_step < x + a.width; ++o)
        if (between(o * outer_step - x, inner > 1 ? inner_step : 0, 0, inner - 1, -b.width, a.width)) return true;
    }
  return false;
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

// The arguments that both append calls take; p.tokens of 0: nothing to do.
moe_w4a16_status append_params(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, int num_tokens,
                               int num_heads, int head_dim, const moe_w4a16_pages* cache, const int32_t* tables,
                               int64_t table_stride, int max_pages, int num_seqs, const int32_t* seq_ids,
                               const int32_t* positions, void* ws, size_t ws_bytes, AppendParams* out) {
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
  AppendParams& p = *out;
  p.tokens = num_tokens;
  if (num_tokens == 0) return MOE_W4A16_OK;
  if (k == nullptr || seq_ids == nullptr || positions == nullptr || !aligned16(k) || !aligned16(v))
    return MOE_W4A16_ERR_INVALID_ARG;
  p.src[0] = k;
  p.src[1] = v;
  p.src_stride[0] = k_stride;
  p.src_stride[1] = v_stride;
  p.pages[0] = cache->k;
  p.pages[1] = cache->v;
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.heads = num_heads;
  p.dim = head_dim;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  p.t = table_view(tables, table_stride, max_pages, cache->page_size, cache->num_pages, num_seqs);
  p.seq_ids = seq_ids;
  p.positions = positions;
  p.err = static_cast<int*>(ws);
  return MOE_W4A16_OK;
}

bool rotary_ok(const moe_w4a16_rotary_desc* r, int head_dim) {
  return r != nullptr && r->turns != nullptr && (reinterpret_cast<uintptr_t>(r->turns) & 7u) == 0 && r->dim >= 2 &&
         r->dim % 2 == 0 && r->dim <= MOE_W4A16_MAX_ROTARY_DIM && r->offset >= 0 && r->offset <= head_dim - r->dim &&
         (r->interleaved == 0 || r->interleaved == 1) && std::isfinite(r->magnitude);
}
RotaryView rotary_view(const moe_w4a16_rotary_desc* r) {
  return RotaryView{r->turns, r->dim, r->offset, r->interleaved, r->magnitude};
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
  AppendParams p{};
  const moe_w4a16_status st = append_params(k, k_stride, v, v_stride, num_tokens, num_heads, head_dim, cache, tables,
                                            table_stride, max_pages, num_seqs, seq_ids, positions, ws, ws_bytes, &p);
  if (st != MOE_W4A16_OK || p.tokens == 0) return st;
  MOE_CUDA_TRY(launch_cache_append(p, cache->dtype, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_cache_append_rotary(
    const uint16_t* q, int64_t q_stride, int num_q_heads, uint16_t* q_out, int64_t q_out_stride, const uint16_t* k,
    int64_t k_stride, const uint16_t* v, int64_t v_stride, int num_tokens, int num_heads, int head_dim,
    const moe_w4a16_rotary_desc* rotary, const moe_w4a16_pages* cache, const int32_t* tables, int64_t table_stride,
    int max_pages, int num_seqs, const int32_t* seq_ids, const int32_t* positions, void* ws, size_t ws_bytes,
    moe_w4a16_stream_t stream) {
  AppendRotaryParams p{};
  const moe_w4a16_status st =
      append_params(k, k_stride, v, v_stride, num_tokens, num_heads, head_dim, cache, tables, table_stride, max_pages,
                    num_seqs, seq_ids, positions, ws, ws_bytes, &p.a);
  if (st != MOE_W4A16_OK) return st;
  if (!rotary_ok(rotary, head_dim)) return MOE_W4A16_ERR_INVALID_ARG;
  if (rotary->offset % 8 != 0 || rotary->dim % (rotary->interleaved ? 8 : 16) != 0) return MOE_W4A16_ERR_UNSUPPORTED;
  if (q != nullptr || q_out != nullptr) {
    const int64_t width = static_cast<int64_t>(num_q_heads) * head_dim;
    if (num_q_heads < 1 || num_q_heads > (1 << 16) || q_stride < width || q_out_stride < width || q_stride % 8 != 0 ||
        q_out_stride % 8 != 0 || (num_tokens > 0 && (q == nullptr || q_out == nullptr)) || !aligned16(q) || !aligned16(q_out))
      return MOE_W4A16_ERR_INVALID_ARG;
    if (num_tokens > 0) {
      // in place, row by row, or apart; and apart from the keys and values, which other threads read meanwhile
      const Rows turned(q_out, num_tokens, 2 * q_out_stride, 1, 0, 2 * width);
      const int64_t key_width = int64_t(2) * num_heads * head_dim;
      if (!(q == q_out && (num_tokens == 1 || q_stride == q_out_stride)) &&
          overlap(Rows(q, num_tokens, 2 * q_stride, 1, 0, 2 * width), turned))
        return MOE_W4A16_ERR_INVALID_ARG;
      if (overlap(Rows(k, num_tokens, 2 * k_stride, 1, 0, key_width), turned) ||
          (v != nullptr && overlap(Rows(v, num_tokens, 2 * v_stride, 1, 0, key_width), turned)))
        return MOE_W4A16_ERR_INVALID_ARG;
    }
    p.q = q;
    p.q_stride = q_stride;
    p.q_out = q_out;
    p.q_out_stride = q_out_stride;
    p.q_heads = num_q_heads;
  }
  if (num_tokens == 0) return MOE_W4A16_OK;
  p.r = rotary_view(rotary);
  int device = 0;
  MOE_CUDA_TRY(cudaGetDevice(&device));
  MOE_CUDA_TRY(launch_cache_append_rotary(p, cache->dtype, device, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_rotary_frequencies(int dim, double theta, int scaling, double factor, int trained_length,
                                              double low, double high, const double* given, uint64_t* turns) {
  if (turns == nullptr || dim < 2 || dim % 2 != 0 || dim > MOE_W4A16_MAX_ROTARY_DIM) return MOE_W4A16_ERR_INVALID_ARG;
  if (scaling < MOE_W4A16_ROTARY_NONE || scaling > MOE_W4A16_ROTARY_GIVEN) return MOE_W4A16_ERR_INVALID_ARG;
  const bool bands = scaling == MOE_W4A16_ROTARY_TURNS || scaling == MOE_W4A16_ROTARY_INDEX;
  const bool scaled = bands || scaling == MOE_W4A16_ROTARY_LINEAR || scaling == MOE_W4A16_ROTARY_BASE;
  if (scaling == MOE_W4A16_ROTARY_GIVEN ? given == nullptr : !(theta > 0) || !std::isfinite(theta))
    return MOE_W4A16_ERR_INVALID_ARG;
  if (scaled && (!(factor >= 1) || !std::isfinite(factor))) return MOE_W4A16_ERR_INVALID_ARG;
  if (bands && (trained_length < 1 || !(low > 0) || !(high > low) || !std::isfinite(high))) return MOE_W4A16_ERR_INVALID_ARG;
  if (scaling == MOE_W4A16_ROTARY_INDEX && theta == 1) return MOE_W4A16_ERR_INVALID_ARG;
  if (scaling == MOE_W4A16_ROTARY_BASE && dim == 2 && factor != 1) return MOE_W4A16_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  if (scaling == MOE_W4A16_ROTARY_BASE && factor != 1) theta *= std::pow(factor, dim / (dim - 2.0));
  double edge[2] = {0, 0};                                    // INDEX: the pairs that turn `high` and `low` times
  if (scaling == MOE_W4A16_ROTARY_INDEX) {
    const double most = dim - 1;
    edge[0] = std::floor(dim * std::log(trained_length / (two_pi * high)) / (2 * std::log(theta)));
    edge[1] = std::ceil(dim * std::log(trained_length / (two_pi * low)) / (2 * std::log(theta)));
    for (double& e : edge) e = e < 0 ? 0 : e > most ? most : e;
  }
  for (int i = 0; i < dim / 2; ++i) {
    double f = scaling == MOE_W4A16_ROTARY_GIVEN ? given[i] : std::pow(theta, -2.0 * i / dim);
    if (scaling == MOE_W4A16_ROTARY_LINEAR) f /= factor;
    if (bands) {
      double keep = scaling == MOE_W4A16_ROTARY_TURNS
                        ? (trained_length * f / two_pi - low) / (high - low)
                        : 1 - (i - edge[0]) / (edge[1] - edge[0] > 0.001 ? edge[1] - edge[0] : 0.001);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      f = keep * f + (1 - keep) * f / factor;
    }
    if (!std::isfinite(f)) return MOE_W4A16_ERR_INVALID_ARG;
    const double t = std::fabs(f) / two_pi;                   // within 2^-52 of itself, as 2 pi is rounded too
    const double part = t - std::floor(t);                    // modulo one turn: exact, as t is not negative
    // 32 bits at a time; what lies below 2^-64 is cut off
    const double top = std::floor(part * 4294967296.0);
    const double rest = std::floor((part * 4294967296.0 - top) * 4294967296.0);
    const uint64_t bits = (static_cast<uint64_t>(top) << 32) + static_cast<uint64_t>(rest);
    turns[i] = f < 0 ? 0 - bits : bits;
  }
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_rotary(const uint16_t* x, int64_t x_stride, int64_t x_head_stride, const int32_t* positions,
                                  int num_tokens, int num_heads, int head_dim, const moe_w4a16_rotary_desc* rotary,
                                  uint16_t* out, int64_t out_stride, int64_t out_head_stride,
                                  moe_w4a16_stream_t stream) {
  if (num_tokens < 0 || num_heads < 1 || num_heads > (1 << 16) || head_dim < 2 || head_dim > (1 << 16) ||
      !rotary_ok(rotary, head_dim))
    return MOE_W4A16_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_W4A16_OK;
  const auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if (x == nullptr || out == nullptr || positions == nullptr || ((bits(x) | bits(out)) & 1u) != 0)
    return MOE_W4A16_ERR_INVALID_ARG;
  if (x_stride < 0 || x_head_stride < 0) return MOE_W4A16_ERR_INVALID_ARG;
  // rows of out lie apart: heads within tokens, or tokens within heads
  const int64_t heads_span = num_heads > 1 ? (num_heads - 1) * out_head_stride : 0;
  const int64_t tokens_span = num_tokens > 1 ? (num_tokens - 1) * out_stride : 0;
  const bool by_token = (num_heads == 1 || out_head_stride >= head_dim) &&
                        (num_tokens == 1 || out_stride >= heads_span + head_dim);
  const bool by_head = (num_tokens == 1 || out_stride >= head_dim) &&
                       (num_heads == 1 || out_head_stride >= tokens_span + head_dim);
  if (!by_token && !by_head) return MOE_W4A16_ERR_INVALID_ARG;
  if (x == out && ((num_tokens > 1 && x_stride != out_stride) || (num_heads > 1 && x_head_stride != out_head_stride)))
    return MOE_W4A16_ERR_INVALID_ARG;
  if (x != out && overlap(Rows(x, num_tokens, 2 * x_stride, num_heads, 2 * x_head_stride, int64_t(2) * head_dim),
                          Rows(out, num_tokens, 2 * out_stride, num_heads, 2 * out_head_stride, int64_t(2) * head_dim)))
    return MOE_W4A16_ERR_INVALID_ARG;
  int64_t units = head_dim | rotary->offset | (rotary->interleaved ? rotary->dim : rotary->dim / 2);
  if (num_tokens > 1) units |= x_stride | out_stride;
  if (num_heads > 1) units |= x_head_stride | out_head_stride;
  int width = 8;
  while (width > 1 && (units % width != 0 || ((bits(x) | bits(out)) & (2u * width - 1u)) != 0)) width /= 2;
  RotaryParams p{};
  p.x = x;
  p.x_stride = x_stride;
  p.x_head_stride = x_head_stride;
  p.positions = positions;
  p.tokens = num_tokens;
  p.heads = num_heads;
  p.dim = head_dim;
  p.r = rotary_view(rotary);
  p.out = out;
  p.out_stride = out_stride;
  p.out_head_stride = out_head_stride;
  int device = 0;
  MOE_CUDA_TRY(cudaGetDevice(&device));
  MOE_CUDA_TRY(launch_rotary(p, width, device, reinterpret_cast<cudaStream_t>(stream)));
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_paged_chunk_workspace_size(int num_heads, int num_kv_heads, int head_dim, size_t* bytes) {
  if (bytes == nullptr || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0)
    return MOE_W4A16_ERR_INVALID_ARG;
  if (head_dim < 16 || head_dim % 16 != 0 || head_dim > MOE_W4A16_MAX_HEAD_DIM) return MOE_W4A16_ERR_UNSUPPORTED;
  // header | the one-token calls' counters, left alone | scratch
  *bytes = kBlockWsOffset + chunk_scratch_bytes(num_heads, num_kv_heads, head_dim);
  return MOE_W4A16_OK;
}

moe_w4a16_status moe_w4a16_paged_chunk_attention(const uint16_t* q, int64_t q_stride, int num_tokens,
                                                 const int32_t* starts, int batch, int num_heads, int num_kv_heads,
                                                 int head_dim, const moe_w4a16_pages* cache, const int32_t* tables,
                                                 int64_t table_stride, int max_pages, const int32_t* lens,
                                                 const int32_t* seq_ids, int num_seqs, float scale, int window,
                                                 uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                                                 moe_w4a16_stream_t stream) {
  return moe_w4a16_paged_chunk_attention_at(q, q_stride, num_tokens, starts, nullptr, batch, num_heads, num_kv_heads,
                                            head_dim, cache, tables, table_stride, max_pages, lens, seq_ids, num_seqs,
                                            scale, window, out, lse, ws, ws_bytes, stream);
}

moe_w4a16_status moe_w4a16_paged_chunk_attention_at(const uint16_t* q, int64_t q_stride, int num_tokens,
                                                    const int32_t* starts, const int32_t* positions, int batch,
                                                    int num_heads, int num_kv_heads, int head_dim,
                                                    const moe_w4a16_pages* cache, const int32_t* tables,
                                                    int64_t table_stride, int max_pages, const int32_t* lens,
                                                    const int32_t* seq_ids, int num_seqs, float scale, int window,
                                                    uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                                                    moe_w4a16_stream_t stream) {
  if (num_tokens < 0 || batch < 0 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0 || window < 0 ||
      !std::isfinite(scale))
    return MOE_W4A16_ERR_INVALID_ARG;
  if (head_dim < 16 || head_dim % 16 != 0 || head_dim > MOE_W4A16_MAX_HEAD_DIM) return MOE_W4A16_ERR_UNSUPPORTED;
  moe_w4a16_status st = check_pages(cache, num_kv_heads, head_dim, false);
  if (st != MOE_W4A16_OK) return st;
  if (static_cast<int64_t>(num_tokens) * num_heads >= (int64_t(1) << 31)) return MOE_W4A16_ERR_UNSUPPORTED;
  size_t need = 0;
  st = moe_w4a16_paged_chunk_workspace_size(num_heads, num_kv_heads, head_dim, &need);
  if (st != MOE_W4A16_OK) return st;
  if (!ws_fits(ws, ws_bytes, need)) return MOE_W4A16_ERR_WORKSPACE;
  if (num_tokens == 0 || batch == 0) return MOE_W4A16_OK;
  const int64_t width = static_cast<int64_t>(num_heads) * head_dim;
  if (q == nullptr || out == nullptr || lens == nullptr || starts == nullptr || !aligned16(q) || !aligned16(out) ||
      q_stride % 8 != 0 || q_stride < width)
    return MOE_W4A16_ERR_INVALID_ARG;
  // outputs are stored while other rows' queries are still to be read
  const Rows queries(q, num_tokens, 2 * q_stride, 1, 0, 2 * width), outs(out, num_tokens, 2 * width, 1, 0, 2 * width);
  if (overlap(queries, outs)) return MOE_W4A16_ERR_INVALID_ARG;
  if (lse != nullptr) {
    const Rows sums(lse, num_tokens, int64_t(4) * num_heads, 1, 0, int64_t(4) * num_heads);
    if (overlap(queries, sums) || overlap(outs, sums)) return MOE_W4A16_ERR_INVALID_ARG;
  }
  if (seq_ids == nullptr && num_seqs < batch) return MOE_W4A16_ERR_INVALID_ARG;
  if (!table_ok(tables, table_stride, max_pages, cache->page_size, num_seqs)) return MOE_W4A16_ERR_INVALID_ARG;
  ChunkParams p{};
  p.q = q;
  p.q_stride = q_stride;
  p.tokens = num_tokens;
  p.starts = starts;
  p.positions = positions;
  p.batch = batch;
  p.heads = num_heads;
  p.kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.dim = head_dim;
  p.k = cache->k;
  p.v = cache->v;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  p.t = table_view(tables, table_stride, max_pages, cache->page_size, cache->num_pages, num_seqs);
  p.lens = lens;
  p.seq_ids = seq_ids;
  p.score_scale = static_cast<float>(static_cast<double>(scale) * cache->k_scale * 1.4426950408889634);
  p.v_scale = cache->v_scale;
  p.window = window;
  p.out = out;
  p.lse = lse;
  p.err = static_cast<int*>(ws);
  p.scratch = static_cast<uint8_t*>(ws) + kBlockWsOffset;
  int device = 0;
  MOE_CUDA_TRY(cudaGetDevice(&device));
  p.wait_ns = wait_limit_ns(device);
  MOE_CUDA_TRY(launch_chunk_attention(p, cache->dtype, device, reinterpret_cast<cudaStream_t>(stream)));
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
