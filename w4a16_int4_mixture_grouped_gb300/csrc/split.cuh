// How the attention kernels share out their work: every CTA takes an equal range of one line of
// tiles (all sequences' seen tokens, row by row), finds its rows by itself and joins the rows that
// its range shares with other CTAs. Used by the grouped and the latent kernel.
#pragma once

#include <cuda_runtime.h>

#include "block.h"

namespace moe {

// A row of work is one (sequence, head block); a sequence has `rows` of them. Row r of sequence b holds
// tiles_b tiles of `tile` tokens, the first of them starting at the multiple of `tile` at or below the
// first seen token. Tile x of the line belongs to CTA (x + 1) * ctas - 1) / total.
constexpr int kSeqCache = 128;           // sequences whose ranges a CTA holds in shared memory
struct SeqRange {
  int row, lo, hi;                       // row of the table; seen tokens [lo, hi)
};
struct SeqCache {
  SeqRange s[kSeqCache];
  int sums[32];
};

__device__ __forceinline__ int tiles_of(int lo, int hi, int tile) {
  return hi > lo ? (hi + tile - 1) / tile - lo / tile : 0;
}

// First tile of CTA c and the CTA of tile x.
__device__ __forceinline__ int64_t cta_begin(int64_t total, int ctas, int c) { return total * c / ctas; }
__device__ __forceinline__ int cta_of(int64_t total, int ctas, int64_t x) {
  return static_cast<int>(((x + 1) * ctas - 1) / total);
}

// Ranges of the sequences [b0, b0 + kSeqCache) into the cache (a CTA-wide call; ends in a barrier).
__device__ __forceinline__ void load_ranges(const AttnParams& p, int b0, SeqCache* cache, int threads) {
  __syncthreads();
  for (int i = threadIdx.x; i < kSeqCache; i += threads) {
    SeqRange r{-1, 0, 0};
    if (b0 + i < p.batch) seen_range(p, b0 + i, r.row, r.lo, r.hi);
    cache->s[i] = r;
  }
  __syncthreads();
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Tiles of the cached sequences (per row of work); every thread gets the sum.
__device__ __forceinline__ int cached_tiles(const SeqCache* cache, int tile) {
  int n = 0;
  for (int i = threadIdx.x & 31; i < kSeqCache; i += 32) n += tiles_of(cache->s[i].lo, cache->s[i].hi, tile);
  return warp_sum(n);
}

}  // namespace moe
