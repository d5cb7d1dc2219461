// Norms before and after a block on the residual stream (moe_w4a16_block_norm):
//
//   u = x * rsqrt(mean(x^2) + eps) * w_post,  h' = rs * h + bs * gate * u,  y = h' * rsqrt(mean(h'^2) + eps) * w_pre
//
// Bound by HBM: x and h are read once, h' and y written once, nothing else moves. A row stays in the
// registers of its threads between the two norms (FP32, never rounded in between).
//
//   * Short rows (up to 64 packs): 8, 16 or 32 lanes a row, sums by shuffles alone.
//   * Longer rows: a CTA a row, one barrier a sum (every warp adds up the warps' sums itself). Few rows: all that a
//     row needs, weights and gate included, is requested before the first sum.
//   * Many long rows: two packs of 8 columns a thread in 40 registers (FP32 residual: 40 bytes spilled), weights read
//     (from L1) where they are used, so that three CTAs share an SM and one's loads run beside the others' sums.
//     8192 x 7168 with an FP32 residual: 109 us, 6.46 TB/s (a plain copy of as many bytes: 108.7 us). At 64 registers
//     and two CTAs it takes 133 us; one CTA an SM that walks through rows with four of them in flight in shared
//     memory, by cp.async or by bulk copies, 125 us.
//   * Packs of 8 columns, 16 bytes of BF16. Rows of any width do with them too where all tensors' rows start alike
//     (contiguous tensors): only the packs at a row's two ends go column by column. Otherwise packs of 2 or 1.
//
// Slower forms, by the bytes that they need: odd widths, whose weights are read a column at a time (8192 x 7167: 2.7 TB/s BF16
// residual, 4.2 FP32; 8192 x 1021: 2.5); rows wider than 16384 columns, whose packs spill (728 to 2856 bytes of stores a
// thread; 4096 x 20000: 2.1 and 2.6 TB/s, 2048 x 32768: 2.0 and 2.4); rows that start at different alignments (8192 x 7167:
// 1.2, 2048 x 20001: 0.8).
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace norm {

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the row's threads: LANES lanes of a warp, or the CTA (0; one barrier, `red` is not reused).
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* red) {
  if (LANES != 0) return lanes_sum<LANES == 0 ? 32 : LANES>(v);
  v = lanes_sum<32>(v);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return lanes_sum<32>(lane < warps ? red[lane] : 0.f);
}

// E (1, 2 or 8) consecutive elements by one access (FP32: of at most 16 bytes), from an address aligned to it.
template <int E>
struct Pack {
  float v[E];
};
// Element i of a pack, i known at run time only.
template <int E>
__device__ __forceinline__ float element(const Pack<E>& x, int i) {
  float v = x.v[0];
#pragma unroll
  for (int k = 1; k < E; ++k)
    if (k == i) v = x.v[k];
  return v;
}
template <int E>
__device__ __forceinline__ Pack<E> load_bf16(const uint16_t* p) {
  Pack<E> r;
  uint32_t a[4] = {0, 0, 0, 0};
  if (E == 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    a[0] = w.x, a[1] = w.y, a[2] = w.z, a[3] = w.w;
  } else if (E == 2) {
    a[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    a[0] = *p;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) r.v[i] = __uint_as_float(i & 1 ? a[i / 2] & 0xffff0000u : a[i / 2] << 16);
  return r;
}
template <int E>
__device__ __forceinline__ Pack<E> load_f32(const float* p) {
  Pack<E> r;
  if (E == 8) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const float4 a = reinterpret_cast<const float4*>(p)[i];
      r.v[(4 * i) % E] = a.x, r.v[(4 * i + 1) % E] = a.y, r.v[(4 * i + 2) % E] = a.z, r.v[(4 * i + 3) % E] = a.w;
    }
  } else if (E == 2) {
    const float2 a = *reinterpret_cast<const float2*>(p);
    r.v[0] = a.x, r.v[1 % E] = a.y;
  } else {
    r.v[0] = *p;
  }
  return r;
}
template <int E>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Pack<E>& x) {
  if (E == 1) {
    *p = f32_to_bf16_rn(x.v[0]);
    return;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < E / 2; ++i) w[i] = pack_bf16x2_rn(x.v[(2 * i) % E], x.v[(2 * i + 1) % E]);
  if (E == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint32_t*>(p) = w[0];
}
template <int E>
__device__ __forceinline__ void store_f32(float* p, const Pack<E>& x) {
  if (E == 8 && (reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    // 32 bytes at once: two 16-byte stores of a warp would each write half of every 32-byte sector
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x.v[0]), "f"(x.v[1 % E]),
                 "f"(x.v[2 % E]), "f"(x.v[3 % E]), "f"(x.v[4 % E]), "f"(x.v[5 % E]), "f"(x.v[6 % E]), "f"(x.v[7 % E])
                 : "memory");
  } else if (E == 8) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
      reinterpret_cast<float4*>(p)[i] =
          make_float4(x.v[(4 * i) % E], x.v[(4 * i + 1) % E], x.v[(4 * i + 2) % E], x.v[(4 * i + 3) % E]);
  } else if (E == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(x.v[0], x.v[1 % E]);
  } else {
    *p = x.v[0];
  }
}

// Eight columns [c, c + 8) of a row whose pack is 16-byte aligned there but may stick out of the row at its ends.
__device__ __forceinline__ Pack<8> load_edge(const uint16_t* row, int c, int n) {
  if (c >= 0 && c + 8 <= n) return load_bf16<8>(row + c);
  Pack<8> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = c + i >= 0 && c + i < n ? bf16_to_f32(row[c + i]) : 0.f;
  return r;
}
__device__ __forceinline__ Pack<8> load_edge(const float* row, int c, int n) {
  if (c >= 0 && c + 8 <= n) return load_f32<8>(row + c);
  Pack<8> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = c + i >= 0 && c + i < n ? row[c + i] : 0.f;
  return r;
}
// Eight columns of a weight row at any alignment; zero outside the row (an edge column's factor, infinite perhaps, must
// not reach the zeros beside it: their product enters the row's sum).
__device__ __forceinline__ Pack<8> load_any(const uint16_t* row, int c, int n) {
  Pack<8> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = c + i >= 0 && c + i < n ? bf16_to_f32(__ldg(row + c + i)) : 0.f;
  return r;
}

// A thread holds K packs of E elements, pack k at (thread + k * threads of the row). SHIFT (E = 8): rows that
// start anywhere, all tensors' alike (odd widths): the packs lie at the 16-byte boundaries of the row, the
// first from up to seven columns before it, and only the weights are read a column at a time (from L1).
template <bool RES32, int E, int K, int LANES, int THREADS, int CTAS, bool SHIFT>
__global__ void __launch_bounds__(THREADS, CTAS) block_norm_kernel(const NormParams p) {
  __shared__ float red[2][32];
  constexpr bool kPart = LANES != 0;
  constexpr int kDiv = kPart ? LANES : 1;
  int64_t t = kPart ? int64_t(blockIdx.x) * (THREADS / kDiv) + threadIdx.x / kDiv : blockIdx.x;
  const bool live = t < p.rows;          // (lanes past the last row take part in the sums of their warp)
  if (!live) t = p.rows - 1;
  int first = (kPart ? threadIdx.x % kDiv : threadIdx.x) * E;
  const int step = (kPart ? LANES : blockDim.x) * E;
  if (SHIFT) first -= static_cast<int>(t * p.h_stride & 7);
  const uint16_t* gate_row = p.gate != nullptr ? p.gate + t / p.rows_per_gate * p.n : nullptr;

  Pack<E> h[K], x[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = first + k * step;
#pragma unroll
    for (int i = 0; i < E; ++i) h[k].v[i] = x[k].v[i] = 0.f;
    if (c < p.n) {
      if constexpr (SHIFT) {
        if (p.x != nullptr) x[k] = load_edge(p.x + t * p.x_stride, c, p.n);
        if (RES32) h[k] = load_edge(static_cast<const float*>(p.h) + t * p.h_stride, c, p.n);
        else h[k] = load_edge(static_cast<const uint16_t*>(p.h) + t * p.h_stride, c, p.n);
      } else {
        if (p.x != nullptr) x[k] = load_bf16<E>(p.x + t * p.x_stride + c);
        h[k] = RES32 ? load_f32<E>(static_cast<const float*>(p.h) + t * p.h_stride + c)
                     : load_bf16<E>(static_cast<const uint16_t*>(p.h) + t * p.h_stride + c);
      }
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
          Pack<E> w;
          if constexpr (SHIFT) w = load_any(p.w_post, c, p.n);
          else w = load_bf16<E>(p.w_post + c);
#pragma unroll
          for (int i = 0; i < E; ++i) f[k].v[i] *= w.v[i];
        }
        if (gate_row != nullptr) {
          Pack<E> w;
          if constexpr (SHIFT) w = load_any(gate_row, c, p.n);
          else w = load_bf16<E>(gate_row + c);
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
      post = rsqrtf(row_sum<LANES>(s, red[0]) / p.n + p.eps);
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
  if (p.h_out != nullptr && live) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = first + k * step;
      if (c >= p.n) continue;
      if (SHIFT && (c < 0 || c + E > p.n)) {
        for (int i = max(0, -c); i < E && c + i < p.n; ++i) {
          const float v = element(h[k], i);
          if (RES32) static_cast<float*>(p.h_out)[t * p.h_out_stride + c + i] = v;
          else static_cast<uint16_t*>(p.h_out)[t * p.h_out_stride + c + i] = f32_to_bf16_rn(v);
        }
      } else if (RES32) {
        store_f32<E>(static_cast<float*>(p.h_out) + t * p.h_out_stride + c, h[k]);
      } else {
        store_bf16<E>(static_cast<uint16_t*>(p.h_out) + t * p.h_out_stride + c, h[k]);
      }
    }
  }
  if (p.y == nullptr) return;
  Pack<E> w[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (first + k * step < p.n) {
      if constexpr (SHIFT) w[k] = load_any(p.w_pre, first + k * step, p.n);
      else w[k] = load_bf16<E>(p.w_pre + first + k * step);
    }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(h[k].v[i], h[k].v[i], s);
  const float pre = rsqrtf(row_sum<LANES>(s, red[1]) / p.n + p.eps);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = first + k * step;
    if (c >= p.n || !live) continue;
#pragma unroll
    for (int i = 0; i < E; ++i) h[k].v[i] *= pre * w[k].v[i];
    if (SHIFT && (c < 0 || c + E > p.n)) {
      for (int i = max(0, -c); i < E && c + i < p.n; ++i) p.y[t * p.y_stride + c + i] = f32_to_bf16_rn(element(h[k], i));
    } else {
      store_bf16<E>(p.y + t * p.y_stride + c, h[k]);
    }
  }
}

// ---------------------------------------------------------------------------
// many long rows
// ---------------------------------------------------------------------------
// Two FP32 lanes in a 64-bit register: the packed multiply-add halves the arithmetic, which at two bytes an
// element is a third of this kernel's instructions.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_get(F2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// The two BF16 of a word.
__device__ __forceinline__ F2 f2_bf16(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }

// K packs of 8 columns a thread, one row a CTA.
template <bool RES32, int K, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) block_norm_many_kernel(const NormParams p) {
  __shared__ float red[2][32];
  const int64_t t = blockIdx.x;
  const int first = threadIdx.x * 8, step = blockDim.x * 8;
  const float inv_n = 1.f / p.n;
  const uint16_t* gate_row = p.gate != nullptr ? p.gate + t / p.rows_per_gate * p.n : nullptr;
  uint4 x[K];
  F2 h[K][4];
  bool in[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = first + k * step;
    in[k] = c < p.n;
    x[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[k][i].v = 0;
    if (!in[k]) continue;
    // (x is there: launch(). With a BF16 residual the compiler keeps the loads within 40 registers only behind a test;
    // without it the spills cost 13%, 87 -> 99 us at 9362 x 7168. With an FP32 residual the test costs 8%.)
    if (RES32 || p.x != nullptr) x[k] = *reinterpret_cast<const uint4*>(p.x + t * p.x_stride + c);
    if (RES32) {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.h) + t * p.h_stride + c);
      const float4 a = src[0], b2 = src[1];
      h[k][0] = f2(a.x, a.y);
      h[k][1] = f2(a.z, a.w);
      h[k][2] = f2(b2.x, b2.y);
      h[k][3] = f2(b2.z, b2.w);
    } else {
      const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.h) + t * p.h_stride + c);
      h[k][0].v = r.x;
      h[k][1].v = r.y;
      h[k][2].v = r.z;
      h[k][3].v = r.w;
    }
  }
  float post = 1.f;
  if (p.w_post != nullptr) {
    F2 s = f2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(f2_bf16(w[i]), f2_bf16(w[i]), s);
    }
    float a, b2;
    f2_get(s, a, b2);
    post = rsqrtf(row_sum<0>(a + b2, red[0]) * inv_n + p.eps);
  }
  const float scale = post * p.blk_scale;
  const F2 scale2 = f2(scale, scale), rs = f2(p.res_scale, p.res_scale);
  F2 s = f2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = first + k * step;
    if (!in[k]) continue;
    uint4 wr = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), gr = wr;
    if (p.w_post != nullptr) wr = __ldg(reinterpret_cast<const uint4*>(p.w_post + c));
    if (gate_row != nullptr) gr = *reinterpret_cast<const uint4*>(gate_row + c);
    const uint32_t xw[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, ww[4] = {wr.x, wr.y, wr.z, wr.w}, gw[4] = {gr.x, gr.y, gr.z, gr.w};
    Pack<8> out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 factor = mul2(mul2(f2_bf16(ww[i]), scale2), f2_bf16(gw[i]));
      const F2 hv = RES32 ? h[k][i] : f2_bf16(static_cast<uint32_t>(h[k][i].v));
      h[k][i] = fma2(f2_bf16(xw[i]), factor, mul2(rs, hv));
      s = fma2(h[k][i], h[k][i], s);
      f2_get(h[k][i], out.v[2 * i], out.v[2 * i + 1]);
    }
    if (p.h_out != nullptr) {
      if (RES32) store_f32<8>(static_cast<float*>(p.h_out) + t * p.h_out_stride + c, out);
      else store_bf16<8>(static_cast<uint16_t*>(p.h_out) + t * p.h_out_stride + c, out);
    }
  }
  if (p.y == nullptr) return;
  float a, b2;
  f2_get(s, a, b2);
  const float pre = rsqrtf(row_sum<0>(a + b2, red[1]) * inv_n + p.eps);
  const F2 pre2 = f2(pre, pre);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = first + k * step;
    if (!in[k]) continue;
    const uint4 wr = __ldg(reinterpret_cast<const uint4*>(p.w_pre + c));
    const uint32_t w[4] = {wr.x, wr.y, wr.z, wr.w};
    Pack<8> out;
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_get(mul2(mul2(h[k][i], pre2), f2_bf16(w[i])), out.v[2 * i], out.v[2 * i + 1]);
    store_bf16<8>(p.y + t * p.y_stride + c, out);
  }
}

template <bool RES32, int E, int K, int LANES, bool SHIFT>
void launch_part(const NormParams& p, cudaStream_t stream) {
  constexpr int kThreads = 256, kRows = kThreads / LANES;
  const unsigned grid = static_cast<unsigned>((p.rows + kRows - 1) / kRows);
  block_norm_kernel<RES32, E, K, LANES, kThreads, 1, SHIFT><<<grid, kThreads, 0, stream>>>(p);
}
template <bool RES32, int E, int K, bool SHIFT, int THREADS = 1024, int CTAS = 1>
void launch_cta(const NormParams& p, int packs, cudaStream_t stream) {
  const int threads = ((packs + K - 1) / K + 31) / 32 * 32;
  block_norm_kernel<RES32, E, K, 0, THREADS, CTAS, SHIFT><<<p.rows, threads, 0, stream>>>(p);
}

// E: columns of a pack.
template <bool RES32, int E, bool SHIFT>
void launch(const NormParams& p, int sm_count, cudaStream_t stream) {
  const int packs = (p.n + (SHIFT ? 7 : 0) + E - 1) / E;
  if (packs <= 8) return launch_part<RES32, E, 1, 8, SHIFT>(p, stream);
  if (packs <= 16) return launch_part<RES32, E, 1, 16, SHIFT>(p, stream);
  if (packs <= 32) return launch_part<RES32, E, 1, 32, SHIFT>(p, stream);
  if (packs <= 64) return launch_part<RES32, E, 2, 32, SHIFT>(p, stream);
  if constexpr (E == 8) {
    if (!SHIFT && packs <= 2048 && p.x != nullptr && p.rows > 2 * sm_count) {
      const int threads = (packs + 63) / 64 * 32;        // two packs each
      if (packs <= 1024) block_norm_many_kernel<RES32, 2, 512, 3><<<p.rows, threads, 0, stream>>>(p);
      else if (packs <= 1536) block_norm_many_kernel<RES32, 2, 768, 2><<<p.rows, threads, 0, stream>>>(p);
      else block_norm_many_kernel<RES32, 2, 1024, 1><<<p.rows, threads, 0, stream>>>(p);
      return;
    }
    if (SHIFT && packs <= 1024 && p.rows > 2 * sm_count) return launch_cta<RES32, E, 2, SHIFT, 512, 2>(p, packs, stream);
    if (packs <= 1024) return launch_cta<RES32, E, 1, SHIFT>(p, packs, stream);
    if (packs <= 2048) return launch_cta<RES32, E, 2, SHIFT>(p, packs, stream);
    return launch_cta<RES32, E, 5, SHIFT>(p, packs, stream);       // (up to 4097 packs)
  } else {
    if (packs <= 8192) return launch_cta<RES32, E, 8, SHIFT>(p, packs, stream);
    return launch_cta<RES32, E, 32, SHIFT>(p, packs, stream);
  }
}

template <bool RES32>
void launch_width(const NormParams& p, int width, bool shift, int sm_count, cudaStream_t stream) {
  if (shift) launch<RES32, 8, true>(p, sm_count, stream);
  else if (width == 8) launch<RES32, 8, false>(p, sm_count, stream);
  else if (width >= 2) launch<RES32, 2, false>(p, sm_count, stream);
  else launch<RES32, 1, false>(p, sm_count, stream);
}

}  // namespace norm

cudaError_t launch_block_norm(const NormParams& p, bool res32, int width, bool shift, int device, cudaStream_t stream) {
  const int sm_count = device_info(device).sm_count;
  if (res32) norm::launch_width<true>(p, width, shift, sm_count, stream);
  else norm::launch_width<false>(p, width, shift, sm_count, stream);
  note_launch();
  return cudaGetLastError();
}

}  // namespace moe
