// Rotation of positions: of queries or keys by themselves, and of a step's queries and keys on the way into the cache.
//
// A pair (a, b) at position p turns by the angle p f_i. The frequency is kept as f_i / 2 pi modulo one, in units of
// 2^-64 turns: p times that, modulo 2^64, is its angle modulo a turn with no further rounding however far p is (an FP32 product
// is off by 0.008 radians at position 131072). Its upper half, as a signed number of turns in [-0.5, 0.5), goes to the
// sine and cosine.
//
// Bound by HBM: every element is read once and written once. A CTA takes all heads of one to four tokens, so that the sines
// and cosines of a token are computed once, by all threads, and kept in shared memory; a thread's first loads are in flight
// before. Measured (GB300, copy of the same bytes at 6.78 TB/s in brackets): 8191 tokens of 64 query and 8 key and value
// heads of 128 channels into BF16 pages 57.8 us (49.5), 2048 of 64 query rows and a cached row of 576 channels 55.9 us
// (45.3), 8192 tokens of 64 heads of 192 channels by themselves 73.7 us (59.4). Few tokens (a decode step) are bound by the
// launch.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace rotary {

constexpr int kThreads = 256;
constexpr int kMostTokens = 4;                          // of a CTA at a time

// A token's table holds (cos, sin) of its pairs, times the magnitude: the j-th two of each unit's EACH pairs side by side, so
// that threads on neighbouring units read neighbouring 16 bytes (pair after pair: 8-way bank conflicts, 66 us for 54, see
// append_rotary_kernel).
template <int EACH>
__device__ __forceinline__ int table_at(int units, int unit, int j) {
  constexpr int kTwo = EACH > 1 ? 2 : 1;
  return ((j / kTwo) * units + unit) * kTwo + j % kTwo;
}
template <int EACH>
__device__ __forceinline__ void fill_tables(const RotaryView& r, const int32_t* positions, int tok, int tokens, float2* table) {
  const int pairs = r.dim / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs, pair = i - t * pairs;
    const uint64_t turn = r.turns[pair] * static_cast<uint64_t>(static_cast<int64_t>(positions[tok + t]));
    const int part = static_cast<int>(static_cast<uint32_t>((turn + 0x80000000ull) >> 32));   // 2^-32 turns
    float s, c;
    sincospif(static_cast<float>(part) * 4.656612873077393e-10f, &s, &c);                    // 2^-31: half turns
    table[t * pairs + table_at<EACH>(pairs / EACH, pair / EACH, pair % EACH)] = make_float2(c * r.magnitude, s * r.magnitude);
  }
}

// N BF16 elements as they are loaded and stored: accesses of W.
template <int W> struct Access;
template <> struct Access<8> { using type = uint4; };
template <> struct Access<4> { using type = uint2; };
template <> struct Access<2> { using type = uint32_t; };
template <> struct Access<1> { using type = uint16_t; };
template <int N, int W>
struct Vec {
  typename Access<W>::type v[N / W];
  // (the first `count` accesses)
  __device__ __forceinline__ void load(const uint16_t* src, int count = N / W) {
#pragma unroll
    for (int i = 0; i < N / W; ++i)
      if (i < count) v[i] = reinterpret_cast<const typename Access<W>::type*>(src)[i];
  }
  __device__ __forceinline__ void store(uint16_t* dst, int count = N / W) const {
#pragma unroll
    for (int i = 0; i < N / W; ++i)
      if (i < count) reinterpret_cast<typename Access<W>::type*>(dst)[i] = v[i];
  }
  __device__ __forceinline__ void get(float (&x)[N]) const {
    const uint16_t* e = reinterpret_cast<const uint16_t*>(v);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = bf16_to_f32(e[j]);
  }
  __device__ __forceinline__ void set(const float (&x)[N]) {
    if constexpr (W == 1) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = f32_to_bf16_rn(x[j]);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) w[j] = pack_bf16x2_rn(x[2 * j], x[2 * j + 1]);
    }
  }
};

// A head's units: first those of the rotated part (half layout: N channels of each half; interleaved: N channels that
// are pairs), then the rest by accesses of W.
template <int N, bool PAIRS>
__host__ __device__ __forceinline__ int turned_units(const RotaryView& r) { return PAIRS ? r.dim / N : r.dim / (2 * N); }

// A CTA's part: `count` heads from h0 on of each of `tokens` tokens from tok0 on, `units` units each, the `turned` first of
// them pairs. `place` says where a head lies, whether it turns, and stores. A thread has LOADS loads in flight, the first of
// them before place.open(), which every thread calls, makes the sines and cosines.
struct Part {
  int tok0, tokens, h0, count;
};
template <int N, int W, bool PAIRS, int LOADS, typename Place>
__device__ __forceinline__ void turn_heads(const RotaryView& r, const float2* table, const Part& part, int units, Place& place) {
  constexpr int kAhead = PAIRS ? LOADS : LOADS / 2;
  const int turned = turned_units<N, PAIRS>(r), half = r.dim / 2;
  // kThreads units on are dt tokens, dh heads and du units on
  const int d = kThreads / units, du = kThreads - d * units, dt = d / part.count, dh = d - dt * part.count;
  int h = threadIdx.x / units, unit = threadIdx.x - h * units, t = h / part.count;
  h -= t * part.count;
  bool opened = false;
  do {
    Vec<N, W> lo[kAhead], hi[kAhead];
    int ts[kAhead], hs[kAhead], us[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      ts[k] = t;
      hs[k] = part.h0 + h;
      us[k] = unit;
      if (t < part.tokens && place.moved(hs[k], unit < turned)) {
        const uint16_t* src = place.source(part.tok0 + t, hs[k]);
        if (unit < turned) {
          const int c = r.offset + unit * N;
          lo[k].load(src + c);
          if (!PAIRS) hi[k].load(src + c + half);
        } else {
          const int c = (unit - turned) * W;
          lo[k].load(src + (c < r.offset ? c : c + r.dim), 1);
        }
      }
      unit += du;
      h += dh;
      t += dt;
      if (unit >= units) unit -= units, ++h;
      if (h >= part.count) h -= part.count, ++t;
    }
    if (!opened) {
      place.open(part);
      opened = true;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (ts[k] >= part.tokens || !place.moved(hs[k], us[k] < turned)) continue;
      if (us[k] >= turned) {
        const int c = (us[k] - turned) * W;
        place.copy(part, ts[k], hs[k], c < r.offset ? c : c + r.dim, lo[k], 1);
        continue;
      }
      const int c = r.offset + us[k] * N;
      if (!place.turns(hs[k])) {
        place.copy(part, ts[k], hs[k], c, lo[k], N / W);
        if (!PAIRS) place.copy(part, ts[k], hs[k], c + half, hi[k], N / W);
        continue;
      }
      float x[N];
      lo[k].get(x);
      constexpr int kEach = PAIRS ? N / 2 : N;
      float2 cs[kEach];
#pragma unroll
      for (int j = 0; j < kEach; j += kEach > 1 ? 2 : 1) {
        const float2* at = table + ts[k] * half + table_at<kEach>(turned, us[k], j);
        if constexpr (kEach > 1) {
          const float4 two = *reinterpret_cast<const float4*>(at);
          cs[j] = make_float2(two.x, two.y);
          cs[j + 1] = make_float2(two.z, two.w);
        } else {
          cs[j] = *at;
        }
      }
      if constexpr (PAIRS) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const float a = x[2 * j], b = x[2 * j + 1];
          x[2 * j] = a * cs[j].x - b * cs[j].y;
          x[2 * j + 1] = a * cs[j].y + b * cs[j].x;
        }
        place.store(part, ts[k], hs[k], c, x);
      } else {
        float y[N];
        hi[k].get(y);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float a = x[j], b = y[j];
          x[j] = a * cs[j].x - b * cs[j].y;
          y[j] = a * cs[j].y + b * cs[j].x;
        }
        place.store(part, ts[k], hs[k], c, x);
        place.store(part, ts[k], hs[k], c + half, y);
      }
    }
  } while (t < part.tokens);
}
// The CTAs' parts: groups of `tokens` tokens, or one token's heads in `parts`.
struct Split {
  int tokens, parts;
};
__device__ __forceinline__ bool part_of(int64_t blk, int tokens, int heads, const Split& s, Part& o) {
  const int64_t groups = (int64_t(tokens) + s.tokens - 1) / s.tokens;
  if (blk >= groups * s.parts) return false;
  const int group = static_cast<int>(blk / s.parts), part = static_cast<int>(blk - int64_t(group) * s.parts);
  o.tok0 = group * s.tokens;
  o.tokens = min(s.tokens, tokens - o.tok0);
  o.h0 = static_cast<int>(int64_t(heads) * part / s.parts);
  o.count = static_cast<int>(int64_t(heads) * (part + 1) / s.parts) - o.h0;
  return true;
}

// Heads of rows in BF16.
template <int N, int W, bool PAIRS>
struct RowPlace {
  const RotaryParams& p;
  float2* table;
  __device__ __forceinline__ const uint16_t* source(int tok, int h) const { return p.x + tok * p.x_stride + h * p.x_head_stride; }
  __device__ __forceinline__ void open(const Part& part) {
    fill_tables<PAIRS ? N / 2 : N>(p.r, p.positions, part.tok0, part.tokens, table);
    __syncthreads();
  }
  __device__ __forceinline__ bool moved(int, bool) const { return true; }
  __device__ __forceinline__ bool turns(int) const { return true; }
  __device__ __forceinline__ uint16_t* at(const Part& part, int t, int h, int c) const {
    return p.out + (part.tok0 + t) * p.out_stride + h * p.out_head_stride + c;
  }
  __device__ __forceinline__ void copy(const Part& part, int t, int h, int c, const Vec<N, W>& x, int count) const {
    x.store(at(part, t, h, c), count);
  }
  __device__ __forceinline__ void store(const Part& part, int t, int h, int c, const float (&x)[N]) const {
    Vec<N, W> v;
    v.set(x);
    v.store(at(part, t, h, c));
  }
};

// W: elements of an access. (Two loads a thread and 8 CTAs an SM: 73.7 us for the 8192 tokens; four and 5 CTAs 80.2, four and 4
// CTAs 83.9.)
template <int W, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 8) rotary_kernel(const __grid_constant__ RotaryParams p, const Split split) {
  constexpr int N = PAIRS && W == 1 ? 2 : W;
  extern __shared__ __align__(16) float2 table[];
  const int units = turned_units<N, PAIRS>(p.r) + (p.x == p.out ? 0 : (p.dim - p.r.dim) / W);
  RowPlace<N, W, PAIRS> place{p, table};
  Part part;
  for (int64_t blk = blockIdx.x; part_of(blk, p.tokens, p.heads, split, part); blk += gridDim.x) {
    turn_heads<N, W, PAIRS, 2>(p.r, table, part, units, place);
    __syncthreads();                                    // (the tables are read)
  }
}

// ---------------------------------------------------------------------------
// rotation on the way into the cache
// ---------------------------------------------------------------------------

// A token's query heads in BF16, then its key heads and its value heads to their places in the pages: BF16, or E4M3 as in
// cache_append (a true division).
template <bool E4M3, bool PAIRS>
struct TokenPlace {
  const AppendRotaryParams& p;
  float2* table;
  int64_t* rows;                 // [tokens of the group] first element in the pages, -1: none
  __device__ __forceinline__ const uint16_t* source(int tok, int h) const {
    if (h < p.q_heads) return p.q + tok * p.q_stride + int64_t(h) * p.a.dim;
    h -= p.q_heads;
    const bool value = h >= p.a.heads;
    return p.a.src[value] + tok * p.a.src_stride[value] + int64_t(value ? h - p.a.heads : h) * p.a.dim;
  }
  __device__ __forceinline__ void open(const Part& part) {
    const AppendParams& a = p.a;
    if (threadIdx.x < part.tokens) {
      const int tok = part.tok0 + threadIdx.x;
      const int seq = a.seq_ids[tok], pos = a.positions[tok];
      int64_t row = -1;
      if (pos >= 0) {
        const int col = pos / a.t.page_size;
        int page = -1;
        if (seq >= 0 && seq < a.t.num_seqs && col < a.t.max_pages) page = a.t.tables[seq * a.t.table_stride + col];
        if (page >= 0 && page < a.t.num_pages) row = page * a.page_stride + (pos - col * a.t.page_size) * a.token_stride;
        else set_error(a.err, MOE_W4A16_ERR_BAD_INDEX);
      }
      rows[threadIdx.x] = row;
    }
    fill_tables<PAIRS ? 4 : 8>(p.r, a.positions, part.tok0, part.tokens, table);
    __syncthreads();
  }
  // (queries in place: only what turns)
  __device__ __forceinline__ bool moved(int h, bool turned) const { return turned || h >= p.q_heads || p.q != p.q_out; }
  __device__ __forceinline__ bool turns(int h) const { return h < p.q_heads + p.a.heads; }
  __device__ __forceinline__ uint16_t* query(const Part& part, int t, int h, int c) const {
    return p.q_out + (part.tok0 + t) * p.q_out_stride + int64_t(h) * p.a.dim + c;
  }
  __device__ __forceinline__ void copy(const Part& part, int t, int h, int c, const Vec<8, 8>& x, int) const {
    if (h < p.q_heads) return x.store(query(part, t, h, c));
    h -= p.q_heads;
    const bool value = h >= p.a.heads;
    if (rows[t] < 0) return;
    const int64_t at = rows[t] + (value ? h - p.a.heads : h) * p.a.head_stride + c;
    if constexpr (E4M3) {
      float f[8];
      x.get(f);
      to_e4m3(at, value, f);
    } else {
      x.store(static_cast<uint16_t*>(p.a.pages[value]) + at);
    }
  }
  __device__ __forceinline__ void store(const Part& part, int t, int h, int c, const float (&x)[8]) const {
    Vec<8, 8> w;
    if (h < p.q_heads) {
      w.set(x);
      return w.store(query(part, t, h, c));
    }
    if (rows[t] < 0) return;
    const int64_t at = rows[t] + (h - p.q_heads) * p.a.head_stride + c;
    if constexpr (E4M3) {
      to_e4m3(at, false, x);
    } else {
      w.set(x);
      w.store(static_cast<uint16_t*>(p.a.pages[0]) + at);
    }
  }
  __device__ __forceinline__ void to_e4m3(int64_t at, bool value, const float (&x)[8]) const {
    const float scale = p.a.scale[value];
    uint32_t out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[4 * j], scale), __fdiv_rn(x[4 * j + 1], scale)), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[4 * j + 2], scale), __fdiv_rn(x[4 * j + 3], scale)), __NV_SATFINITE, __NV_E4M3);
      out[j] = lo | hi << 16;
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.a.pages[value]) + at) = make_uint2(out[0], out[1]);
  }
};

// (Four loads a thread and 5 CTAs an SM: 57.8 us for the 8191 tokens; 4 CTAs 59.3, two loads and 6 CTAs 61.7, 8 CTAs 69.2.)
template <bool E4M3, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 5) append_rotary_kernel(const __grid_constant__ AppendRotaryParams p, const Split split) {
  extern __shared__ __align__(16) float2 table[];
  __shared__ int64_t rows[kMostTokens];
  const int units = turned_units<8, PAIRS>(p.r) + (p.a.dim - p.r.dim) / 8;
  const int heads = p.q_heads + p.a.heads * (p.a.src[1] != nullptr ? 2 : 1);
  TokenPlace<E4M3, PAIRS> place{p, table, rows};
  Part part;
  for (int64_t blk = blockIdx.x; part_of(blk, p.a.tokens, heads, split, part); blk += gridDim.x) {
    turn_heads<8, 8, PAIRS, 4>(p.r, table, part, units, place);
    __syncthreads();                                    // (the tables are read)
  }
}

// Few tokens: their heads in parts, so that every SM has work, each of at least kThreads units. Many: groups, so that the
// latency of positions, sines and page numbers is paid once for several rows (8191 tokens one by one: 84.5 us, two by two
// 68.4, four by four 66.0, eight by eight 65.6, with the tables in the pairs' order).
static Split split_of(int64_t tokens, int heads, int64_t units, int device) {
  const int64_t sms = device_info(device).sm_count;
  Split s{1, 1};
  while (s.tokens < kMostTokens && tokens >= 16 * s.tokens * sms) s.tokens *= 2;
  const int64_t want = (2 * sms + tokens - 1) / tokens, most = (heads * units + kThreads - 1) / kThreads;
  s.parts = static_cast<int>(want < most ? want : most);
  if (s.parts > heads) s.parts = heads;
  if (s.parts < 1) s.parts = 1;
  return s;
}
static unsigned grid_of(int64_t tokens, const Split& s) {
  const int64_t blocks = (tokens + s.tokens - 1) / s.tokens * s.parts;
  return static_cast<unsigned>(blocks < (1 << 20) ? blocks : 1 << 20);
}

template <int W>
static void run_rotary(const RotaryParams& p, int device, cudaStream_t stream) {
  const int n = W == 1 && p.r.interleaved ? 2 : W;
  const int units = p.r.dim / (p.r.interleaved ? n : 2 * n) + (p.x == p.out ? 0 : (p.dim - p.r.dim) / W);
  const Split split = split_of(p.tokens, p.heads, units, device);
  const unsigned grid = grid_of(p.tokens, split);
  const size_t smem = sizeof(float2) * (p.r.dim / 2) * split.tokens;
  if (p.r.interleaved) rotary_kernel<W, true><<<grid, kThreads, smem, stream>>>(p, split);
  else rotary_kernel<W, false><<<grid, kThreads, smem, stream>>>(p, split);
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
  const int heads = p.q_heads + p.a.heads * (p.a.src[1] != nullptr ? 2 : 1);
  const Split split = split_of(p.a.tokens, heads, units, device);
  const unsigned grid = grid_of(p.a.tokens, split);
  const size_t smem = sizeof(float2) * (p.r.dim / 2) * split.tokens;
  const bool e4m3 = dtype == MOE_W4A16_CACHE_E4M3;
  if (p.r.interleaved) {
    if (e4m3) append_rotary_kernel<true, true><<<grid, kThreads, smem, stream>>>(p, split);
    else append_rotary_kernel<false, true><<<grid, kThreads, smem, stream>>>(p, split);
  } else {
    if (e4m3) append_rotary_kernel<true, false><<<grid, kThreads, smem, stream>>>(p, split);
    else append_rotary_kernel<false, false><<<grid, kThreads, smem, stream>>>(p, split);
  }
  note_launch();
  return cudaGetLastError();
}

}  // namespace moe
