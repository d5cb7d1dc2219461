// Attention of one new token per sequence over a latent cache.
//
// Simple form: one CTA per (sequence, query head), tokens in strides of the CTA, a running
// maximum and sum per thread joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace latent {

constexpr int kThreads = 128;

template <bool E4M3>
__device__ __forceinline__ float element(const void* base, int64_t i) {
  if (E4M3) return static_cast<float>(static_cast<const __nv_fp8_e4m3*>(base)[i]);
  return bf16_to_f32(static_cast<const uint16_t*>(base)[i]);
}

// DV channels of values per row (the latent form: 512 of 576); values at the key's own base when V is null.
template <bool E4M3>
__global__ void __launch_bounds__(kThreads) attention_kernel(const AttnParams p, int dv) {
  __shared__ float qs[kLatentDim], prob[kThreads], red[kThreads / 32];
  __shared__ int64_t rows[kThreads];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  int seq, lo, hi;
  seen_range(p, b, seq, lo, hi);
  for (int c = tid; c < p.dim; c += kThreads) qs[c] = bf16_to_f32(p.q[b * p.q_stride + int64_t(h) * p.dim + c]);
  __syncthreads();
  const void* values = p.v != nullptr ? p.v : p.k;
  const int64_t head = int64_t(h / p.group) * p.head_stride;
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = lo; j0 < hi; j0 += kThreads) {
    const int j = j0 + tid;
    float s = -INFINITY;
    int64_t row = -1;
    if (j < hi) {
      const int page = p.t.tables[int64_t(seq) * p.t.table_stride + j / p.t.page_size];
      if (page >= p.t.num_pages) set_error(p.err, MOE_W4A16_ERR_BAD_INDEX);
      if (page >= 0 && page < p.t.num_pages) {
        row = int64_t(page) * p.page_stride + int64_t(j % p.t.page_size) * p.token_stride + head;
        float d = 0.f;
        for (int c = 0; c < p.dim; ++c) d = fmaf(qs[c], element<E4M3>(p.k, row + c), d);
        s = d * p.score_scale;
      }
    }
    rows[tid] = row;
    float top = s;
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, red[w]);
    const float mn = fmaxf(m, top);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float keep = exp2f(m - base);
    prob[tid] = row >= 0 ? exp2f(s - base) : 0.f;
    m = mn;
    l *= keep;
    for (int i = 0; i < 4; ++i) acc[i] *= keep;
    __syncthreads();
    const int n = min(kThreads, hi - j0);
    for (int t = 0; t < n; ++t) {
      if (rows[t] < 0) continue;
      l += prob[t];
      for (int i = 0; i < 4; ++i) {
        const int c = tid + i * kThreads;
        if (c < dv) acc[i] = fmaf(prob[t], element<E4M3>(values, rows[t] + c), acc[i]);
      }
    }
    __syncthreads();
  }
  const float inv = l > 0.f ? p.v_scale / l : 0.f;
  for (int i = 0; i < 4; ++i) {
    const int c = tid + i * kThreads;
    if (c < dv) p.out[(int64_t(b) * p.heads + h) * dv + c] = f32_to_bf16_rn(l > 0.f ? acc[i] * inv : 0.f);
  }
  if (tid == 0 && p.lse != nullptr) p.lse[int64_t(b) * p.heads + h] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace latent

size_t latent_part_bytes(int) { return 0; }

cudaError_t launch_latent_attention(const AttnParams& p, int, cudaStream_t stream) {
  latent::attention_kernel<false><<<dim3(p.heads, p.batch), latent::kThreads, 0, stream>>>(p, kLatentValue);
  note_launch();
  return cudaGetLastError();
}

}  // namespace moe
