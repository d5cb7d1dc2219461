// Norms before and after a block on the residual stream (moe_w4a16_block_norm):
//
//   u = x * rsqrt(mean(x^2) + eps) * w_post,  h' = rs * h + bs * gate * u,  y = h' * rsqrt(mean(h'^2) + eps) * w_pre
//
// Bound by HBM: x and h are read once, h' and y written once, nothing else moves. A row stays in the
// registers of its threads between the two norms (FP32, never rounded in between); everything that a
// row needs, weights and gate included, is requested before the first sum, so a single row costs one
// memory latency and two sums.
//
//   * Rows of up to 1024 elements: a warp a row, sums by shuffles alone, eight rows a CTA.
//   * Longer rows: a CTA a row, one barrier a sum (every warp adds up the warps' sums itself).
//   * Many long rows: as many CTAs as fit, each walking through rows. A thread keeps the same columns, so it
//     holds their weights, and copies its own 16-byte pieces of the rows to come into shared memory
//     (cp.async, no barrier): the bytes in flight no longer hang on registers and on the two sums.
//   * 16-byte accesses where n, strides and pointers allow; else element by element, coalesced.
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace norm {

constexpr int kRowWarps = 8;             // rows of a CTA in the warp-a-row form

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the row's threads: a warp, or a CTA (one barrier; `red` is not reused).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (WARP) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

// E consecutive elements: 8 by 16-byte accesses, or a single one.
template <int E>
struct Pack {
  float v[E];
};
template <int E>
__device__ __forceinline__ Pack<E> load_bf16(const uint16_t* p) {
  Pack<E> r;
  if (E == 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < E; ++i) r.v[i] = __uint_as_float(i & 1 ? a[i / 2] & 0xffff0000u : a[i / 2] << 16);
  } else {
    r.v[0] = bf16_to_f32(*p);
  }
  return r;
}
template <int E>
__device__ __forceinline__ Pack<E> load_f32(const float* p) {
  Pack<E> r;
  if (E == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    const float c[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < E; ++i) r.v[i] = c[i];
  } else {
    r.v[0] = *p;
  }
  return r;
}
template <int E>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Pack<E>& x) {
  if (E == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2_rn(x.v[(2 * i) % E], x.v[(2 * i + 1) % E]);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *p = f32_to_bf16_rn(x.v[0]);
  }
}
template <int E>
__device__ __forceinline__ void store_f32(float* p, const Pack<E>& x) {
  if (E == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x.v[0], x.v[1 % E], x.v[2 % E], x.v[3 % E]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x.v[4 % E], x.v[5 % E], x.v[6 % E], x.v[7 % E]);
  } else {
    *p = x.v[0];
  }
}

// A thread holds K packs of E elements, pack k at (thread + k * threads of the row).
template <bool RES32, int E, int K, bool WARP, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_kernel(const NormParams p) {
  __shared__ float red[2][32];
  const int64_t t = WARP ? int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= p.rows) return;               // (a whole warp, and only in the form without barriers)
  const int first = (WARP ? threadIdx.x & 31 : threadIdx.x) * E, step = (WARP ? 32 : blockDim.x) * E;
  const uint16_t* gate_row = p.gate != nullptr ? p.gate + t / p.rows_per_gate * p.n : nullptr;

  Pack<E> h[K], x[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = first + k * step;
#pragma unroll
    for (int i = 0; i < E; ++i) h[k].v[i] = x[k].v[i] = 0.f;
    if (c < p.n) {
      if (p.x != nullptr) x[k] = load_bf16<E>(p.x + t * p.x_stride + c);
      h[k] = RES32 ? load_f32<E>(static_cast<const float*>(p.h) + t * p.h_stride + c)
                   : load_bf16<E>(static_cast<const uint16_t*>(p.h) + t * p.h_stride + c);
    }
  }
  if (p.x != nullptr) {
    // the block's own factors, before the sum that they wait for
    Pack<E> f[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = first + k * step;
#pragma unroll
      for (int i = 0; i < E; ++i) f[k].v[i] = p.blk_scale;
      if (c < p.n) {
        if (p.w_post != nullptr) {
          const Pack<E> w = load_bf16<E>(p.w_post + c);
#pragma unroll
          for (int i = 0; i < E; ++i) f[k].v[i] *= w.v[i];
        }
        if (gate_row != nullptr) {
          const Pack<E> w = load_bf16<E>(gate_row + c);
#pragma unroll
          for (int i = 0; i < E; ++i) f[k].v[i] *= w.v[i];
        }
      }
    }
    float post = 1.f;
    if (p.w_post != nullptr) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(x[k].v[i], x[k].v[i], s);
      post = rsqrtf(row_sum<WARP>(s, red[0]) / p.n + p.eps);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) h[k].v[i] = fmaf(x[k].v[i] * post, f[k].v[i], p.res_scale * h[k].v[i]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) h[k].v[i] *= p.res_scale;
  }
  if (p.h_out != nullptr) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = first + k * step;
      if (c >= p.n) continue;
      if (RES32) store_f32<E>(static_cast<float*>(p.h_out) + t * p.h_out_stride + c, h[k]);
      else store_bf16<E>(static_cast<uint16_t*>(p.h_out) + t * p.h_out_stride + c, h[k]);
    }
  }
  if (p.y == nullptr) return;
  Pack<E> w[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (first + k * step < p.n) w[k] = load_bf16<E>(p.w_pre + first + k * step);
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(h[k].v[i], h[k].v[i], s);
  const float pre = rsqrtf(row_sum<WARP>(s, red[1]) / p.n + p.eps);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = first + k * step;
    if (c >= p.n) continue;
#pragma unroll
    for (int i = 0; i < E; ++i) h[k].v[i] *= pre * w[k].v[i];
    store_bf16<E>(p.y + t * p.y_stride + c, h[k]);
  }
}

// ---------------------------------------------------------------------------
// many long rows
// ---------------------------------------------------------------------------
// Shared memory: [stage][piece][thread] of 16 bytes; pieces of a pack: x, h (two with an FP32 residual), gate.
template <bool RES32, bool GATE>
constexpr int kPieces = 1 + (RES32 ? 2 : 1) + (GATE ? 1 : 0);

__device__ __forceinline__ Pack<8> unpack_bf16(uint32_t slot) {
  const uint4 w = lds128(slot);
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
  Pack<8> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = __uint_as_float(i & 1 ? a[i / 2] & 0xffff0000u : a[i / 2] << 16);
  return r;
}

// K packs of 8 columns a thread, STAGES rows in flight; GATE: a gate that changes with the row (else part of
// the thread's own factors).
template <bool RES32, int K, bool GATE, int STAGES, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 512 ? 2 : 1) block_norm_rows_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[4][32];
  constexpr int kPc = kPieces<RES32, GATE>;
  const int threads = blockDim.x, first = threadIdx.x * 8, step = threads * 8;
  const uint32_t own = smem_u32(ring) + threadIdx.x * 16;
  const uint32_t piece = threads * 16, stage_bytes = piece * kPc * K;
  const bool norm_x = p.w_post != nullptr;

  Pack<8> f[K];                          // block_scale * w_post * (a gate for all rows)
  uint4 wpre[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = first + k * step;
    wpre[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[k].v[i] = p.blk_scale;
    if (c >= p.n) continue;
    if (norm_x) {
      const Pack<8> w = load_bf16<8>(p.w_post + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[k].v[i] *= w.v[i];
    }
    if (!GATE && p.gate != nullptr) {
      const Pack<8> w = load_bf16<8>(p.gate + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[k].v[i] *= w.v[i];
    }
    if (p.y != nullptr) wpre[k] = *reinterpret_cast<const uint4*>(p.w_pre + c);
  }

  auto issue = [&](int64_t t, int stage) {
    if (t < p.rows) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = first + k * step;
        if (c >= p.n) continue;
        const uint32_t to = own + stage * stage_bytes + k * kPc * piece;
        cp_async16(to, p.x + t * p.x_stride + c, 16);
        if (RES32) {
          const float* h = static_cast<const float*>(p.h) + t * p.h_stride + c;
          cp_async16(to + piece, h, 16);
          cp_async16(to + 2 * piece, h + 4, 16);
        } else {
          cp_async16(to + piece, static_cast<const uint16_t*>(p.h) + t * p.h_stride + c, 16);
        }
        if (GATE) cp_async16(to + (kPc - 1) * piece, p.gate + t / p.rows_per_gate * p.n + c, 16);
      }
    }
    cp_async_commit();
  };
  const int64_t grid = gridDim.x;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) issue(blockIdx.x + i * grid, i);

  int stage = 0, parity = 0;
  for (int64_t t = blockIdx.x; t < p.rows; t += grid) {
    issue(t + (STAGES - 1) * grid, stage == 0 ? STAGES - 1 : stage - 1);
    cp_async_wait<STAGES - 1>();
    Pack<8> h[K], x[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k].v[i] = x[k].v[i] = 0.f;
      if (first + k * step >= p.n) continue;
      const uint32_t at = own + stage * stage_bytes + k * kPc * piece;
      x[k] = unpack_bf16(at);
      if (RES32) {
        const uint4 a = lds128(at + piece), b = lds128(at + 2 * piece);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k].v[i] = __uint_as_float(w[i]);
      } else {
        h[k] = unpack_bf16(at + piece);
      }
    }
    float post = 1.f;
    if (norm_x) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[k].v[i], x[k].v[i], s);
      post = rsqrtf(row_sum<false>(s, red[2 * parity]) / p.n + p.eps);
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = first + k * step;
      if (c >= p.n) continue;
      if (GATE) {
        const Pack<8> w = unpack_bf16(own + stage * stage_bytes + (k * kPc + kPc - 1) * piece);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k].v[i] *= w.v[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[k].v[i] = fmaf(x[k].v[i] * post, f[k].v[i], p.res_scale * h[k].v[i]);
        s = fmaf(h[k].v[i], h[k].v[i], s);
      }
      if (p.h_out != nullptr) {
        if (RES32) store_f32<8>(static_cast<float*>(p.h_out) + t * p.h_out_stride + c, h[k]);
        else store_bf16<8>(static_cast<uint16_t*>(p.h_out) + t * p.h_out_stride + c, h[k]);
      }
    }
    if (p.y != nullptr) {
      const float pre = rsqrtf(row_sum<false>(s, red[2 * parity + 1]) / p.n + p.eps);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = first + k * step;
        if (c >= p.n) continue;
        const uint32_t a[4] = {wpre[k].x, wpre[k].y, wpre[k].z, wpre[k].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          h[k].v[i] *= pre * __uint_as_float(i & 1 ? a[i / 2] & 0xffff0000u : a[i / 2] << 16);
        store_bf16<8>(p.y + t * p.y_stride + c, h[k]);
      }
    }
    parity ^= 1;                         // a sum's buffer is used again two rows (two barriers) later
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

// Shared memory that a CTA of the walking form may take, and its CTAs on an SM.
constexpr int kRowsSmem = 224 * 1024;
int rows_ctas(int threads, int smem) {
  const int by_smem = kRowsSmem / (smem + 1536), by_threads = threads <= 512 ? 1024 / threads : 1;
  const int n = by_smem < by_threads ? by_smem : by_threads;
  return n < 1 ? 1 : n;
}

template <bool RES32, int K, bool GATE, int STAGES, int THREADS>
cudaError_t launch_rows(const NormParams& p, int threads, int device, cudaStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(block_norm_rows_kernel<RES32, K, GATE, STAGES, THREADS>);
  static bool attr_set[64] = {false};
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  constexpr int kPackBytes = kPieces<RES32, GATE> * 16;
  if (!attr_set[device]) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kRowsSmem);
    if (e != cudaSuccess) return e;
    attr_set[device] = true;
  }
  const int smem = threads * K * kPackBytes * STAGES;
  if (smem > kRowsSmem) return cudaErrorInvalidValue;    // (rows_fit)
  const int ctas = device_info(device).sm_count * rows_ctas(threads, smem);
  block_norm_rows_kernel<RES32, K, GATE, STAGES, THREADS>
      <<<p.rows < ctas ? p.rows : ctas, threads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <bool RES32, int E, int K>
void launch_warp(const NormParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.rows + kRowWarps - 1) / kRowWarps);
  block_norm_kernel<RES32, E, K, true, kRowWarps * 32><<<grid, kRowWarps * 32, 0, stream>>>(p);
}
template <bool RES32, int E, int K, int THREADS>
void launch_cta(const NormParams& p, cudaStream_t stream) {
  const int threads = ((p.n + E * K - 1) / (E * K) + 31) / 32 * 32;
  block_norm_kernel<RES32, E, K, false, THREADS><<<p.rows, threads, 0, stream>>>(p);
}

// Many long rows: 16-byte pieces, more than a warp a row, at least four rows for each CTA that fits, and two rows
// in flight in shared memory.
bool rows_fit(const NormParams& p, bool res32, bool vec, bool gate, int device) {
  if (!vec || p.x == nullptr || p.n <= 1024 || p.n > 16384 || p.rows < 8 * device_info(device).sm_count) return false;
  const int pieces = 1 + (res32 ? 2 : 1) + (gate ? 1 : 0), threads = (p.n / 8 + 63) / 64 * 32;
  return p.n <= 2048 || threads * 2 * pieces * 16 * 2 <= kRowsSmem;
}

template <bool RES32, bool GATE>
cudaError_t rows_form(const NormParams& p, int device, cudaStream_t stream) {
  const int vecs = p.n / 8;
  const auto threads = [&](int k) { return ((vecs + k - 1) / k + 31) / 32 * 32; };
  if (vecs <= 256) return launch_rows<RES32, 1, GATE, 4, 256>(p, threads(1), device, stream);
  if (vecs <= 1024) return launch_rows<RES32, 2, GATE, 2, 512>(p, threads(2), device, stream);
  return launch_rows<RES32, 2, GATE, 2, 1024>(p, threads(2), device, stream);
}

template <bool RES32>
void launch(const NormParams& p, bool vec, cudaStream_t stream) {
  if (vec) {
    if (p.n <= 256) return launch_warp<RES32, 8, 1>(p, stream);
    if (p.n <= 512) return launch_warp<RES32, 8, 2>(p, stream);
    if (p.n <= 1024) return launch_warp<RES32, 8, 4>(p, stream);
    if (p.n <= 8192) return launch_cta<RES32, 8, 1, 1024>(p, stream);
    if (p.n <= 16384) return launch_cta<RES32, 8, 2, 1024>(p, stream);
    return launch_cta<RES32, 8, 4, 1024>(p, stream);
  }
  if (p.n <= 256) return launch_warp<RES32, 1, 8>(p, stream);
  if (p.n <= 1024) return launch_warp<RES32, 1, 32>(p, stream);
  if (p.n <= 8192) return launch_cta<RES32, 1, 8, 1024>(p, stream);
  return launch_cta<RES32, 1, 32, 1024>(p, stream);
}

}  // namespace norm

cudaError_t launch_block_norm(const NormParams& p, bool res32, bool vec, int device, cudaStream_t stream) {
  const bool gate = p.gate != nullptr && p.rows_per_gate != p.rows;
  if (norm::rows_fit(p, res32, vec, gate, device)) {
    const cudaError_t e = res32 ? (gate ? norm::rows_form<true, true>(p, device, stream)
                                        : norm::rows_form<true, false>(p, device, stream))
                                : (gate ? norm::rows_form<false, true>(p, device, stream)
                                        : norm::rows_form<false, false>(p, device, stream));
    note_launch();
    return e;
  }
  if (res32) norm::launch<true>(p, vec, stream);
  else norm::launch<false>(p, vec, stream);
  note_launch();
  return cudaGetLastError();
}

}  // namespace moe
