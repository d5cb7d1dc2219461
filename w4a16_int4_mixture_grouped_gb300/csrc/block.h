// Internal host/device declarations of the paged cache, its attention and the block norms
// (not part of the ABI).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "moe_w4a16.h"

namespace moe {

constexpr int kLatentDim = MOE_W4A16_LATENT_DIM;
constexpr int kLatentValue = MOE_W4A16_LATENT_VALUE_DIM;

// Pages of sequences as every cache kernel reads them.
struct TableView {
  const int32_t* tables;
  int64_t table_stride;
  int max_pages;
  int page_size;
  int num_pages;
  int num_seqs;
};

struct AttnParams {
  const uint16_t* q;
  int64_t q_stride;
  int batch, heads, kv_heads, group;   // group = heads / kv_heads
  int dim;                             // channels of a key (= of a value; latent: 576 and 512)
  const void* k;
  const void* v;
  int64_t page_stride, token_stride, head_stride;   // elements
  TableView t;
  const int32_t* lens;
  const int32_t* seq_ids;
  float score_scale;                   // scale * k_scale * log2(e): scores in units of log 2
  float v_scale;
  int window;
  int lanes;                           // grouped form: work rows of a sequence that go side by side
  uint16_t* out;
  float* lse;
  int* err;
  uint64_t wait_ns;                    // latent form: limit of a pipeline wait
  int* counters;                       // [kAttnMaxCtas] arrivals of split rows' parts, zero between calls
  float* parts;                        // FP32 parts of split rows, two to a CTA
};
// CTAs of an attention launch: two on each of the GPU's 152 SMs.
constexpr int kAttnMaxCtas = 304;
// Arrival counters of grouped attention, behind the 256-byte header of the workspace. They have to be zero between calls,
// so no other call on cache or attention puts anything there: all of them may share a workspace.
constexpr size_t kAttnCounterBytes = (kAttnMaxCtas * sizeof(int) + 255) / 256 * 256;
constexpr size_t kBlockWsOffset = MOE_W4A16_WS_HEADER_BYTES + kAttnCounterBytes;   // what a call need not leave at zero
constexpr int kLatentMaxCtas = 152;    // the latent kernel: one
constexpr int kLatentMinTiles = 2;     // tiles a CTA of the latent kernel takes at least: a part costs as much as a tile
size_t attention_part_bytes(int heads, int kv_heads, int dim);
size_t latent_part_bytes(int heads);

// First and past-the-last seen token of query b; a length out of range is cut and recorded.
__device__ __forceinline__ void seen_range(const AttnParams& p, int b, int& row, int& lo, int& hi) {
  row = p.seq_ids != nullptr ? p.seq_ids[b] : b;
  lo = hi = 0;
  if (row < 0 || row >= p.t.num_seqs) {
    atomicCAS(p.err, 0, MOE_W4A16_ERR_BAD_INDEX);
    row = -1;
    return;
  }
  const int cap = p.t.max_pages * p.t.page_size;
  hi = p.lens[row];
  if (hi < 0 || hi > cap) {
    atomicCAS(p.err, 0, MOE_W4A16_ERR_BAD_INDEX);
    hi = hi < 0 ? 0 : cap;
  }
  lo = p.window > 0 && hi > p.window ? hi - p.window : 0;
}

cudaError_t launch_attention(const AttnParams& p, int dtype, int device, cudaStream_t stream);
cudaError_t launch_latent_attention(const AttnParams& p, int device, cudaStream_t stream);

struct AppendParams {
  const uint16_t* src[2];
  int64_t src_stride[2];
  void* pages[2];                      // keys, values; values null for a latent cache
  float scale[2];
  int tokens, heads, dim;
  int64_t page_stride, token_stride, head_stride;
  TableView t;
  const int32_t* seq_ids;
  const int32_t* positions;
  int* err;
};
cudaError_t launch_cache_append(const AppendParams& p, int dtype, cudaStream_t stream);

struct PoolView {
  uint8_t* base;
  int planes, num_pages;
  int64_t plane_stride, page_stride, page_bytes;
};
// Workspace of the page calls from kBlockWsOffset on, in int32 words: [0] number of copies, then
// per entry {source, destination} of a copy, {pages of its table row, granted}, then one word per page.
constexpr size_t kCacheWsPairs = 16;
inline size_t cache_ws_words(int num_pages, int count) {
  const size_t entries = count > num_pages ? count : num_pages;
  return kCacheWsPairs + 4 * entries + static_cast<size_t>(num_pages);
}
struct PageOps {
  TableView t;
  int32_t* tables;
  int32_t* lens;
  int32_t* refs;
  int count;
  int32_t* scratch;                    // cache_ws_words
  int entries;                         // capacity of the entry arrays in scratch
  int* err;
};
cudaError_t launch_cache_extend(const PageOps& o, const int32_t* seq_ids, const int32_t* counts, int32_t* positions,
                                cudaStream_t stream);
cudaError_t launch_cache_fork(const PageOps& o, const PoolView& pool, const int32_t* parents, const int32_t* children,
                              int device, cudaStream_t stream);
cudaError_t launch_cache_free(const PageOps& o, const int32_t* seq_ids, const int32_t* keep, cudaStream_t stream);
cudaError_t launch_cache_copy(const PoolView& pool, const int32_t* src, const int32_t* dst, int count, int* err,
                              int device, cudaStream_t stream);
cudaError_t launch_cache_compact(const PageOps& o, const PoolView& pool, const int32_t* refs_in, int32_t* refs_out,
                                 int32_t* tables_out, int32_t* page_map, int32_t* num_live, int device,
                                 cudaStream_t stream);

struct NormParams {
  const uint16_t* x;
  int64_t x_stride;
  const void* h;
  int64_t h_stride;
  const uint16_t* gate;
  int rows_per_gate;
  const uint16_t* w_post;
  const uint16_t* w_pre;
  int rows, n;
  float eps, res_scale, blk_scale;
  void* h_out;
  int64_t h_out_stride;
  uint16_t* y;
  int64_t y_stride;
};
// width: columns of one access (8, 4, 2 or 1) that every row of every tensor allows; shift: rows that start anywhere, but
// all tensors' alike, from 16-byte aligned first rows.
cudaError_t launch_block_norm(const NormParams& p, bool res32, int width, bool shift, int device, cudaStream_t stream);

}  // namespace moe
