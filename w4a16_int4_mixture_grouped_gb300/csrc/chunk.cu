// Attention of a chunk of new tokens per sequence over a paged cache, grouped heads.
//
// One warp a query row (token and head): lanes take 32 tokens' scores at a time, the softmax runs with a maximum and
// a sum of its own, and lanes take channels for the value product.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace chunk {

constexpr int kWarps = 8;
constexpr int kMaxDim = MOE_W4A16_MAX_HEAD_DIM;

template <bool E4M3>
__device__ __forceinline__ float element(const void* p, int64_t at) {
  if (E4M3) {
    __nv_fp8_e4m3 x;
    x.__x = static_cast<const uint8_t*>(p)[at];
    return static_cast<float>(x);
  }
  return bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
}

template <bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) chunk_kernel(const ChunkParams p) {
  __shared__ float q_s[kWarps][kMaxDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
  const ChunkRange c = chunk_range(p, b);
  const int64_t rows = int64_t(c.n) * p.heads;
  for (int64_t r = int64_t(blockIdx.x) * kWarps + warp; r < rows; r += int64_t(gridDim.x) * kWarps) {
    const int i = static_cast<int>(r / p.heads), h = static_cast<int>(r % p.heads), tok = c.first + i;
    const int pos = c.base + i, hi = c.row < 0 ? 0 : pos + 1, lo = p.window > 0 && hi > p.window ? hi - p.window : 0;
    const int64_t head = int64_t(h / p.group) * p.head_stride;
    __syncwarp();
    for (int d = lane; d < p.dim; d += 32) q_s[warp][d] = bf16_to_f32(p.q[tok * p.q_stride + int64_t(h) * p.dim + d]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[kMaxDim / 32];
#pragma unroll
    for (int k = 0; k < kMaxDim / 32; ++k) o[k] = 0.f;
    const int32_t* table = p.t.tables + int64_t(c.row < 0 ? 0 : c.row) * p.t.table_stride;
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      int64_t at = -1;
      if (j < hi) {
        const int page = table[j / p.t.page_size];
        if (page >= p.t.num_pages) set_error(p.err, MOE_W4A16_ERR_BAD_INDEX);
        else if (page >= 0) at = int64_t(page) * p.page_stride + int64_t(j % p.t.page_size) * p.token_stride + head;
      }
      float s = -INFINITY;
      if (at >= 0) {
        s = 0.f;
        for (int d = 0; d < p.dim; ++d) s = fmaf(q_s[warp][d], element<E4M3>(p.k, at + d), s);
        s *= p.score_scale;
      }
      float top = s;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
      top = fmaxf(top, m);
      const float base = top == -INFINITY ? 0.f : top, keep = exp2f(m - base);
      const float e = at >= 0 ? exp2f(s - base) : 0.f;
      float sum = e;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(~0u, sum, x);
      l = l * keep + sum;
      m = top;
#pragma unroll
      for (int k = 0; k < kMaxDim / 32; ++k) o[k] *= keep;
      for (int t = 0; t < 32; ++t) {
        const int64_t v = __shfl_sync(~0u, at, t);
        const float w = __shfl_sync(~0u, e, t);
        if (v < 0) continue;
#pragma unroll
        for (int k = 0; k < kMaxDim / 32; ++k)
          if (k * 32 + lane < p.dim) o[k] = fmaf(w, element<E4M3>(p.v, v + k * 32 + lane), o[k]);
      }
    }
    const float inv = l == 0.f ? 0.f : p.v_scale / l;
    uint16_t* out = p.out + (int64_t(tok) * p.heads + h) * p.dim;
#pragma unroll
    for (int k = 0; k < kMaxDim / 32; ++k)
      if (k * 32 + lane < p.dim) out[k * 32 + lane] = f32_to_bf16_rn(o[k] * inv);
    if (lane == 0 && p.lse != nullptr)
      p.lse[int64_t(tok) * p.heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
  }
}

}  // namespace chunk

size_t chunk_scratch_bytes(int, int, int) { return 0; }

cudaError_t launch_chunk_attention(const ChunkParams& p, int dtype, int, cudaStream_t stream) {
  const int64_t rows = int64_t(p.tokens) * p.heads;
  const int64_t want = (rows + chunk::kWarps - 1) / chunk::kWarps;
  const dim3 grid(static_cast<unsigned>(want < 4096 ? want : 4096), p.batch < 65535 ? p.batch : 65535);
  if (dtype == MOE_W4A16_CACHE_E4M3) chunk::chunk_kernel<true><<<grid, chunk::kWarps * 32, 0, stream>>>(p);
  else chunk::chunk_kernel<false><<<grid, chunk::kWarps * 32, 0, stream>>>(p);
  note_launch();
  return cudaGetLastError();
}

}  // namespace moe
