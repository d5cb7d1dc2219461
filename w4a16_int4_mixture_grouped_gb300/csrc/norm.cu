// Norms before and after a block on the residual stream (moe_w4a16_block_norm).
//
// Simple form: one CTA per row, the unrounded residual row kept in shared memory between the
// two norms.
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace norm {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

template <bool RES32>
__global__ void __launch_bounds__(kThreads) block_norm_kernel(const NormParams p) {
  extern __shared__ float row[];
  __shared__ float red[kThreads / 32];
  const int64_t t = blockIdx.x;
  const uint16_t* x = p.x != nullptr ? p.x + t * p.x_stride : nullptr;
  float post = 1.f;
  if (p.w_post != nullptr) {
    float s = 0.f;
    for (int c = threadIdx.x; c < p.n; c += kThreads) {
      const float v = bf16_to_f32(x[c]);
      s = fmaf(v, v, s);
    }
    post = rsqrtf(block_sum(s, red) / p.n + p.eps);
  }
  const uint16_t* gate = p.gate != nullptr ? p.gate + t / p.rows_per_gate * p.n : nullptr;
  float s = 0.f;
  for (int c = threadIdx.x; c < p.n; c += kThreads) {
    float h = p.res_scale * (RES32 ? static_cast<const float*>(p.h)[t * p.h_stride + c]
                                   : bf16_to_f32(static_cast<const uint16_t*>(p.h)[t * p.h_stride + c]));
    if (x != nullptr) {
      float u = bf16_to_f32(x[c]);
      if (p.w_post != nullptr) u = u * post * bf16_to_f32(p.w_post[c]);
      if (gate != nullptr) u *= bf16_to_f32(gate[c]);
      h = fmaf(p.blk_scale, u, h);
    }
    row[c] = h;
    s = fmaf(h, h, s);
    if (p.h_out != nullptr) {
      if (RES32) static_cast<float*>(p.h_out)[t * p.h_out_stride + c] = h;
      else static_cast<uint16_t*>(p.h_out)[t * p.h_out_stride + c] = f32_to_bf16_rn(h);
    }
  }
  if (p.y == nullptr) return;
  const float pre = rsqrtf(block_sum(s, red) / p.n + p.eps);
  for (int c = threadIdx.x; c < p.n; c += kThreads)
    p.y[t * p.y_stride + c] = f32_to_bf16_rn(row[c] * pre * bf16_to_f32(p.w_pre[c]));
}

}  // namespace norm

cudaError_t launch_block_norm(const NormParams& p, bool res32, bool, int device, cudaStream_t stream) {
  static bool attr_set[2][64] = {{false}};
  const size_t smem = static_cast<size_t>(p.n) * sizeof(float);
  if (device >= 0 && device < 64 && !attr_set[res32][device]) {
    const void* fn = res32 ? reinterpret_cast<const void*>(norm::block_norm_kernel<true>)
                           : reinterpret_cast<const void*>(norm::block_norm_kernel<false>);
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               MOE_W4A16_MAX_NORM_WIDTH * sizeof(float));
    if (e != cudaSuccess) return e;
    attr_set[res32][device] = true;
  }
  if (res32) norm::block_norm_kernel<true><<<p.rows, norm::kThreads, smem, stream>>>(p);
  else norm::block_norm_kernel<false><<<p.rows, norm::kThreads, smem, stream>>>(p);
  note_launch();
  return cudaGetLastError();
}

}  // namespace moe
