// Rotation of positions: of queries or keys by themselves, and of a step's queries and keys on the way into the cache.
//
// A pair (a, b) at position p turns by the angle p f_i. The frequency is kept as f_i / 2 pi modulo one, in units of
// 2^-64 turns: p times that, modulo 2^64, is the angle modulo a turn with no rounding however far p is (an FP32 product
// is off by 0.008 radians at position 131072). Its upper half, as a signed number of turns in [-0.5, 0.5), goes to the
// sine and cosine.
//
// Bound by HBM: every element is read once and written once. A CTA takes the heads of one token, so that its sines and
// cosines are computed once, by as many threads as there are pairs, and kept in shared memory.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace rotary {

constexpr int kThreads = 256;

// (cos, sin) of the pairs at position pos, times the magnitude.
__device__ __forceinline__ void fill_table(const RotaryView& r, int pos, float2* table) {
  for (int i = threadIdx.x; i < r.dim / 2; i += kThreads) {
    const uint64_t turn = r.turns[i] * static_cast<uint64_t>(static_cast<int64_t>(pos));
    const int part = static_cast<int>(static_cast<uint32_t>((turn + 0x80000000ull) >> 32));   // 2^-32 turns
    float s, c;
    sincospif(static_cast<float>(part) * 4.656612873077393e-10f, &s, &c);                    // 2^-31: half turns
    table[i] = make_float2(c * r.magnitude, s * r.magnitude);
  }
}

// N BF16 elements from W-element accesses, as floats, and back.
template <int W> struct Access;
template <> struct Access<8> { using type = uint4; };
template <> struct Access<4> { using type = uint2; };
template <> struct Access<2> { using type = uint32_t; };
template <> struct Access<1> { using type = uint16_t; };
template <int N, int W>
__device__ __forceinline__ void load(const uint16_t* src, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += W) {
    const auto v = *reinterpret_cast<const typename Access<W>::type*>(src + i);
    const uint16_t* e = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
    for (int j = 0; j < W; ++j) x[i + j] = bf16_to_f32(e[j]);
  }
}
template <int N, int W>
__device__ __forceinline__ void store(uint16_t* dst, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += W) {
    typename Access<W>::type v;
    if constexpr (W == 1) {
      v = f32_to_bf16_rn(x[i]);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int j = 0; j < W / 2; ++j) w[j] = pack_bf16x2_rn(x[i + 2 * j], x[i + 2 * j + 1]);
    }
    *reinterpret_cast<typename Access<W>::type*>(dst + i) = v;
  }
}

// A head's units: first those of the rotated part (half layout: N channels of each half; interleaved: N channels that
// are pairs), then the rest by accesses.
template <int N>
__device__ __forceinline__ int turned_units(const RotaryView& r) { return r.interleaved ? r.dim / N : r.dim / (2 * N); }
template <int N>
__device__ __forceinline__ int plain_channel(const RotaryView& r, int i) {
  const int c = i * N;
  return c < r.offset ? c : c + r.dim;
}
// Turns a unit in place: lo of pairs i .. (and hi, half a rotation on).
template <int N>
__device__ __forceinline__ void turn_half(const float2* table, int i, float (&lo)[N], float (&hi)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float2 t = table[i + j];
    const float a = lo[j], b = hi[j];
    lo[j] = a * t.x - b * t.y;
    hi[j] = a * t.y + b * t.x;
  }
}
template <int N>
__device__ __forceinline__ void turn_pairs(const float2* table, int i, float (&x)[N]) {
#pragma unroll
  for (int j = 0; j + 1 < N; j += 2) {
    const float2 t = table[i + j / 2];
    const float a = x[j], b = x[j + 1];
    x[j] = a * t.x - b * t.y;
    x[j + 1] = a * t.y + b * t.x;
  }
}

// One unit of a head's row from src to dst.
template <int N, int W>
__device__ __forceinline__ void turn_unit(const RotaryView& r, const float2* table, int unit, const uint16_t* src,
                                          uint16_t* dst) {
  const int turned = turned_units<N>(r);
  if (unit >= turned) {
    float x[W];
    const int c = plain_channel<W>(r, unit - turned);
    load<W, W>(src + c, x);
    store<W, W>(dst + c, x);
  } else if (r.interleaved) {
    float x[N];
    const int c = r.offset + unit * N;
    load<N, W>(src + c, x);
    turn_pairs<N>(table, unit * N / 2, x);
    store<N, W>(dst + c, x);
  } else {
    float lo[N], hi[N];
    const int c = r.offset + unit * N;
    load<N, W>(src + c, lo);
    load<N, W>(src + c + r.dim / 2, hi);
    turn_half<N>(table, unit * N, lo, hi);
    store<N, W>(dst + c, lo);
    store<N, W>(dst + c + r.dim / 2, hi);
  }
}

// Block (token, part of the heads). W: elements of an access.
template <int W, bool PAIRS>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p, int parts) {
  constexpr int N = PAIRS && W == 1 ? 2 : W;
  extern __shared__ float2 table[];
  const bool in_place = p.x == p.out;
  const int units = turned_units<N>(p.r) + (in_place ? 0 : (p.dim - p.r.dim) / W);
  const int64_t blocks = int64_t(p.tokens) * parts;
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const int tok = static_cast<int>(blk / parts), part = static_cast<int>(blk % parts);
    __syncthreads();
    fill_table(p.r, p.positions[tok], table);
    __syncthreads();
    const int h0 = static_cast<int>(int64_t(p.heads) * part / parts), h1 = static_cast<int>(int64_t(p.heads) * (part + 1) / parts);
    const uint16_t* src = p.x + tok * p.x_stride;
    uint16_t* dst = p.out + tok * p.out_stride;
    for (int i = threadIdx.x; i < (h1 - h0) * units; i += kThreads) {
      const int h = h0 + i / units;
      turn_unit<N, W>(p.r, table, i % units, src + h * p.x_head_stride, dst + h * p.out_head_stride);
    }
  }
}

// ---------------------------------------------------------------------------
// rotation on the way into the cache
// ---------------------------------------------------------------------------
// Eight channels to a page: BF16, or E4M3 as in cache_append (a true division).
template <bool E4M3>
__device__ __forceinline__ void to_page(void* pages, int64_t at, const float (&x)[8], float scale) {
  if (!E4M3) {
    store<8, 8>(static_cast<uint16_t*>(pages) + at, x);
  } else {
    uint32_t out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[4 * j], scale), __fdiv_rn(x[4 * j + 1], scale)), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[4 * j + 2], scale), __fdiv_rn(x[4 * j + 3], scale)), __NV_SATFINITE, __NV_E4M3);
      out[j] = lo | hi << 16;
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + at) = make_uint2(out[0], out[1]);
  }
}

// Block (token, part): the token's query heads and key heads unit by unit, then its values.
template <bool E4M3>
__global__ void __launch_bounds__(kThreads) append_rotary_kernel(const AppendRotaryParams p, int parts) {
  extern __shared__ float2 table[];
  const AppendParams& a = p.a;
  const RotaryView& r = p.r;
  const int turned = turned_units<8>(r), units = turned + (a.dim - r.dim) / 8;
  const bool q_in_place = p.q == p.q_out;
  const int q_units = p.q == nullptr ? 0 : q_in_place ? turned : units;
  const int nq = p.q_heads * q_units, nk = a.heads * units, nv = a.src[1] != nullptr ? a.heads * (a.dim / 8) : 0;
  const int64_t blocks = int64_t(a.tokens) * parts;
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const int tok = static_cast<int>(blk / parts), part = static_cast<int>(blk % parts);
    const int seq = a.seq_ids[tok], pos = a.positions[tok];
    // the row's place in the pages, -1: none
    int64_t row = -1;
    if (pos >= 0) {
      const int col = pos / a.t.page_size;
      int page = -1;
      if (seq >= 0 && seq < a.t.num_seqs && col < a.t.max_pages) page = a.t.tables[seq * a.t.table_stride + col];
      if (page >= 0 && page < a.t.num_pages) row = page * a.page_stride + (pos - col * a.t.page_size) * a.token_stride;
      else if (threadIdx.x == 0) set_error(a.err, MOE_W4A16_ERR_BAD_INDEX);
    }
    __syncthreads();
    fill_table(r, pos, table);
    __syncthreads();
    const int all = nq + (row >= 0 ? nk + nv : 0);
    for (int i = threadIdx.x + part * kThreads; i < all; i += kThreads * parts) {
      if (i < nq) {
        const int h = i / q_units;
        const int64_t off = int64_t(h) * a.dim;
        turn_unit<8, 8>(r, table, i - h * q_units, p.q + tok * p.q_stride + off, p.q_out + tok * p.q_out_stride + off);
      } else if (i < nq + nk) {
        const int h = (i - nq) / units, unit = i - nq - h * units;
        const uint16_t* src = a.src[0] + tok * a.src_stride[0] + int64_t(h) * a.dim;
        const int64_t at = row + h * a.head_stride;
        float x[8];
        if (unit >= turned) {
          const int c = plain_channel<8>(r, unit - turned);
          load<8, 8>(src + c, x);
          to_page<E4M3>(a.pages[0], at + c, x, a.scale[0]);
        } else if (r.interleaved) {
          const int c = r.offset + unit * 8;
          load<8, 8>(src + c, x);
          turn_pairs<8>(table, unit * 4, x);
          to_page<E4M3>(a.pages[0], at + c, x, a.scale[0]);
        } else {
          const int c = r.offset + unit * 8;
          float y[8];
          load<8, 8>(src + c, x);
          load<8, 8>(src + c + r.dim / 2, y);
          turn_half<8>(table, unit * 8, x, y);
          to_page<E4M3>(a.pages[0], at + c, x, a.scale[0]);
          to_page<E4M3>(a.pages[0], at + c + r.dim / 2, y, a.scale[0]);
        }
      } else {
        const int j = i - nq - nk, h = j / (a.dim / 8), c = (j - h * (a.dim / 8)) * 8;
        const uint16_t* src = a.src[1] + tok * a.src_stride[1] + int64_t(h) * a.dim + c;
        const int64_t at = row + h * a.head_stride + c;
        if (!E4M3) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.pages[1]) + at) = *reinterpret_cast<const uint4*>(src);
        } else {
          float x[8];
          load<8, 8>(src, x);
          to_page<E4M3>(a.pages[1], at, x, a.scale[1]);
        }
      }
    }
  }
}

// CTAs a token: enough that few tokens still reach every SM, each with at least `least` units of work.
static int parts_of(int64_t tokens, int64_t units, int least, int device) {
  const int64_t want = (2 * int64_t(device_info(device).sm_count) + tokens - 1) / tokens;
  const int64_t most = (units + least - 1) / least;
  return static_cast<int>(want < 1 ? 1 : want < most ? want : most < 1 ? 1 : most);
}
static unsigned grid_of(int64_t blocks) { return static_cast<unsigned>(blocks < (1 << 20) ? blocks : 1 << 20); }

template <int W>
static void run_rotary(const RotaryParams& p, int device, cudaStream_t stream) {
  const int n = W == 1 && p.r.interleaved ? 2 : W;
  const int64_t units = int64_t(p.heads) * (p.r.dim / (p.r.interleaved ? n : 2 * n) + (p.x == p.out ? 0 : (p.dim - p.r.dim) / W));
  int parts = parts_of(p.tokens, units, kThreads, device);
  if (parts > p.heads) parts = p.heads;
  const unsigned grid = grid_of(int64_t(p.tokens) * parts);
  const size_t smem = sizeof(float2) * (p.r.dim / 2);
  if (p.r.interleaved) rotary_kernel<W, true><<<grid, kThreads, smem, stream>>>(p, parts);
  else rotary_kernel<W, false><<<grid, kThreads, smem, stream>>>(p, parts);
}

}  // namespace rotary

using namespace rotary;

cudaError_t launch_rotary(const RotaryParams& p, int width, int device, cudaStream_t stream) {
  if (width == 8) run_rotary<8>(p, device, stream);
  else if (width == 4) run_rotary<4>(p, device, stream);
  else if (width == 2) run_rotary<2>(p, device, stream);
  else run_rotary<1>(p, device, stream);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_cache_append_rotary(const AppendRotaryParams& p, int dtype, int device, cudaStream_t stream) {
  const int units = p.r.dim / (p.r.interleaved ? 8 : 16) + (p.a.dim - p.r.dim) / 8;
  const int64_t all = int64_t(p.q_heads + p.a.heads) * units + (p.a.src[1] != nullptr ? p.a.heads * (p.a.dim / 8) : 0);
  const int parts = parts_of(p.a.tokens, all, kThreads, device);
  const unsigned grid = grid_of(int64_t(p.a.tokens) * parts);
  const size_t smem = sizeof(float2) * (p.r.dim / 2);
  if (dtype == MOE_W4A16_CACHE_E4M3) append_rotary_kernel<true><<<grid, kThreads, smem, stream>>>(p, parts);
  else append_rotary_kernel<false><<<grid, kThreads, smem, stream>>>(p, parts);
  note_launch();
  return cudaGetLastError();
}

}  // namespace moe
