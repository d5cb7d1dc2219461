// How the attention kernels share out their work: every CTA takes an equal range of one line of
// tiles (all sequences' seen tokens, row by row) and finds its rows by itself, from the lengths on
// the device. Used by the grouped and the latent kernel.
#pragma once

#include <cuda_runtime.h>

#include "block.h"

namespace moe {

__device__ __forceinline__ int tiles_of(int lo, int hi, int tile) {
  return hi > lo ? (hi - 1) / tile + 1 - lo / tile : 0;     // (hi + tile - 1 may pass 2^31)
}

// First tile of CTA c, and the CTA of tile x.
__device__ __forceinline__ int64_t cta_begin(int64_t total, int ctas, int c) { return total * c / ctas; }
__device__ __forceinline__ int cta_of(int64_t total, int ctas, int64_t x) {
  return static_cast<int>(((x + 1) * ctas - 1) / total);
}

// A CTA's share. A row of work is one (sequence, head block); a sequence has `rows` of them, each of
// tiles_b tiles of `tile` tokens, the first tile starting at the multiple of `tile` at or below the first
// seen token. `first` is the line position of sequence b's first tile.
struct Share {
  int64_t total, x, x_end, first;
  int ctas, b;
  int sums[16];
  int longest;
};

// Fills *sh for CTA `cta` of `grid` (every thread calls it). ctas_of(tiles, longest) says into how many shares that many
// tiles go, of which the longest row has `longest`, where there are fewer than CTAs or than a split is worth.
// False: no work for it.
template <int THREADS, typename F>
__device__ __forceinline__ bool find_share(const AttnParams& p, int cta, int grid, int rows, int tile, F ctas_of, Share* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) sh->longest = 0;
  int64_t line = 0;                                   // tiles of the sequences before the chunk
  for (int pass = 0; pass < 2; ++pass) {
    line = 0;
    for (int b0 = 0; b0 < p.batch; b0 += THREADS) {
      const int b = b0 + threadIdx.x;
      int n = 0;
      if (b < p.batch) {
        int row, lo, hi;
        seen_range(p, b, row, lo, hi);
        n = tiles_of(lo, hi, tile);
      }
      int pre = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += y;
      }
      const int most = __reduce_max_sync(0xffffffffu, n);
      __syncthreads();
      if (lane == 31) sh->sums[warp] = pre;
      if (lane == 0) atomicMax(&sh->longest, most);
      __syncthreads();
      int64_t before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sh->sums[w];
        all += sh->sums[w];
      }
      const int64_t at = line + (before + pre - n) * rows;
      line += all * rows;
      if (pass == 0 && b0 + THREADS >= p.batch) {
        if (threadIdx.x == 0) {
          int64_t ctas = ctas_of(line, sh->longest);
          ctas = ctas < 1 ? 1 : ctas > grid ? grid : ctas;
          const bool work = line > 0 && cta < ctas;
          sh->total = line;
          sh->ctas = static_cast<int>(ctas);
          sh->x = work ? cta_begin(line, static_cast<int>(ctas), cta) : 0;
          sh->x_end = work ? cta_begin(line, static_cast<int>(ctas), cta + 1) : 0;
        }
        __syncthreads();
        if (sh->x >= sh->x_end) return false;
      }
      // the sequence at which the share begins (a batch of one chunk: without a second pass)
      if ((pass == 1 || p.batch <= THREADS) && n > 0 && sh->x >= at && sh->x < at + int64_t(n) * rows) {
        sh->b = b;
        sh->first = at;
      }
      if (pass == 1 && sh->x < line) break;
    }
    if (p.batch <= THREADS) break;
  }
  __syncthreads();
  return true;
}

// The tiles [tile0, tile1) of row r of sequence b, of the row's ntiles.
struct Piece {
  int b, r, seq, lo, hi, ntiles, tile0, tile1;
  int64_t row0;                                       // line position of the row's first tile
};

// A warp's walk through its CTA's share (every lane calls next; each lane holds one sequence's range).
struct PieceWalk {
  int64_t x, x_end, first;
  int b, held;
  int row, lo, hi;

  __device__ __forceinline__ void hold(const AttnParams& p, int b0) {
    held = b0;
    row = -1;
    lo = hi = 0;
    const int mine = b0 + (threadIdx.x & 31);
    if (mine < p.batch) seen_range(p, mine, row, lo, hi);
  }
  __device__ __forceinline__ void start(const AttnParams& p, const Share* sh) {
    x = sh->x;
    x_end = sh->x_end;
    first = sh->first;
    b = sh->b;
    hold(p, b);
  }
  __device__ __forceinline__ bool next(const AttnParams& p, int rows, int tile, Piece& out) {
    while (x < x_end) {
      if (b >= held + 32) hold(p, b);
      out.seq = __shfl_sync(0xffffffffu, row, b - held);
      out.lo = __shfl_sync(0xffffffffu, lo, b - held);
      out.hi = __shfl_sync(0xffffffffu, hi, b - held);
      out.ntiles = tiles_of(out.lo, out.hi, tile);
      const int64_t n = int64_t(out.ntiles) * rows;
      if (x < first + n) {
        out.b = b;
        out.r = rows == 1 ? 0 : static_cast<int>((x - first) / out.ntiles);
        out.row0 = first + int64_t(out.r) * out.ntiles;
        out.tile0 = static_cast<int>(x - out.row0);
        out.tile1 = static_cast<int>(min(int64_t(out.ntiles), x_end - out.row0));
        x = out.row0 + out.tile1;
        return true;
      }
      first += n;
      ++b;
    }
    return false;
  }
};

// Sequences that see nothing: zero outputs of `width` channels a head and a log-sum of -infinity, spread
// over the CTAs.
template <int THREADS>
__device__ __forceinline__ void zero_empty(const AttnParams& p, int width) {
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    int row, lo, hi;
    seen_range(p, b, row, lo, hi);
    if (hi > lo) continue;
    uint4* out = reinterpret_cast<uint4*>(p.out + int64_t(b) * p.heads * width);
    for (int64_t e = threadIdx.x; e < int64_t(p.heads) * width / 8; e += THREADS) out[e] = make_uint4(0, 0, 0, 0);
    if (p.lse != nullptr)
      for (int h = threadIdx.x; h < p.heads; h += THREADS) p.lse[int64_t(b) * p.heads + h] = -INFINITY;
  }
}

}  // namespace moe
