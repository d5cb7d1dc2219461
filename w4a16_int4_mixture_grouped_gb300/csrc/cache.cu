// Pages of a cache: appending rows, growing, forking, freeing and compacting sequences.
//
// Which page goes where is decided by one CTA (the plan kernels: prefix sums over the call's
// entries and over the pool's reference counts, so that the lowest free ids go to the first
// entries whatever the launch's timing); the bytes are then moved by a grid over (page, plane,
// 16 KB piece).
//
// The page calls on tables are bound by their chain of dependent reads (ids, lengths, table, counts; one CTA because
// the entries' order decides): extend by a token a sequence 5 us, a fork's plan 6 us, free 4 us. A sequence's new
// pages are granted by one thread, 0.05 to 0.07 us each: room for a prompt of 8192 tokens in pages of 16 takes 38 us,
// for 131072 391. The copies are bound by HBM: 2048 pages of 128 KB in 16 planes, half of them live, compacted: 337 us,
// 6.4 TB/s of reads and writes. Four 16-byte loads a thread in flight with every SM full of threads are enough; table
// updates ride in the copying launch.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace cache {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kPieceBytes = 16384;       // bytes a CTA copies at a time: four 16-byte loads per thread

// Scratch after the workspace header (cache_ws_words).
struct Scratch {
  int32_t* copies;    // [1] entries of src / dst
  int32_t* src;       // [entries] page to copy, -1: none
  int32_t* dst;
  int32_t* cols;      // [entries] pages of the entry's table row
  int32_t* start;     // [entries] first free page of the entry
  int32_t* free;      // [num_pages] free page ids, ascending
};
__device__ __forceinline__ Scratch scratch_of(const PageOps& o) {
  Scratch s;
  s.copies = o.scratch;
  s.src = o.scratch + kCacheWsPairs;
  s.dst = s.src + o.entries;
  s.cols = s.dst + o.entries;
  s.start = s.cols + o.entries;
  s.free = s.start + o.entries;
  return s;
}

// Exclusive prefix of v over the CTA; `total` is the CTA's sum. Every thread calls it.
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[31];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// Lists the lowest `need` free pages, ascending; returns how many there are (at most `need`). Eight pages a thread and
// step (a read and a prefix sum, about 1.5 us): behind 16384 pages in use, growing and freeing 256 sequences takes 7.1 us, behind
// 131072 19.7 (a page a thread: 13.5 and 73).
__device__ __forceinline__ int list_free(const int32_t* refs, int num_pages, int need, int32_t* out, int* warp_sums) {
  constexpr int kEach = 8;
  const bool wide = (reinterpret_cast<uintptr_t>(refs) & 15u) == 0;
  int found = 0;
  for (int p0 = 0; p0 < num_pages && found < need; p0 += kPlanThreads * kEach) {
    const int p = p0 + threadIdx.x * kEach;
    int r[kEach];
    if (wide && p + kEach <= num_pages) {
      const int4 a = reinterpret_cast<const int4*>(refs + p)[0], b = reinterpret_cast<const int4*>(refs + p)[1];
      r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w, r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
    } else {
#pragma unroll
      for (int k = 0; k < kEach; ++k) r[k] = p + k < num_pages ? refs[p + k] : 1;
    }
    uint32_t is_free = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) is_free |= (r[k] <= 0 ? 1u : 0u) << k;
    int total;
    int at = found + block_prefix(__popc(is_free), warp_sums, total);
    for (; is_free != 0 && at < need; is_free &= is_free - 1) out[at++] = p + __ffs(is_free) - 1;
    found += total;
  }
  __syncthreads();
  return min(found, need);
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
  return tokens / page_size + (tokens % page_size != 0);
}

// ---------------------------------------------------------------------------
// extend
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) extend_kernel(const PageOps o, const int32_t* seq_ids,
                                                              const int32_t* counts, int32_t* positions) {
  __shared__ int warp_sums[32];
  const Scratch s = scratch_of(o);
  const int64_t cap = int64_t(o.t.max_pages) * o.t.page_size;
  int total = 0;
  for (int i0 = 0; i0 < o.count; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int need = 0;
    if (i < o.count) {
      const int seq = seq_ids[i];
      int cols = -1;                                   // not granted
      if (seq < 0 || seq >= o.t.num_seqs) {
        set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
      } else {
        const int len = o.lens[seq];
        const int add = counts != nullptr ? counts[i] : 1;
        if (len < 0 || len > cap || add < 0) {
          set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
        } else if (len + int64_t(add) > cap) {
          set_error(o.err, MOE_W4A16_ERR_CAPACITY);
        } else {
          cols = pages_of(len + add, o.t.page_size);
          need = cols - pages_of(len, o.t.page_size);
        }
      }
      s.cols[i] = cols;
    }
    int sum;
    const int at = total + block_prefix(need, warp_sums, sum);
    if (i < o.count) s.start[i] = at;
    total += sum;                                      // at most num_seqs * max_pages: checked on the host
  }
  const int have = list_free(o.refs, o.t.num_pages, min(total, o.t.num_pages), s.free, warp_sums);
  for (int i = threadIdx.x; i < o.count; i += kPlanThreads) {
    int pos = -1;
    const int cols = s.cols[i];
    if (cols >= 0) {
      const int seq = seq_ids[i], len = o.lens[seq];
      const int first = pages_of(len, o.t.page_size), need = cols - first;
      if (need == 0 || s.start[i] + need <= have) {
        for (int k = 0; k < need; ++k) {
          const int page = s.free[s.start[i] + k];
          o.tables[seq * o.t.table_stride + first + k] = page;
          o.refs[page] = 1;
        }
        o.lens[seq] = len + (counts != nullptr ? counts[i] : 1);
        pos = len;
      } else {
        set_error(o.err, MOE_W4A16_ERR_CAPACITY);
      }
    }
    positions[i] = pos;
  }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PageOps o, const int32_t* parents,
                                                                 const int32_t* children) {
  __shared__ int warp_sums[32];
  const Scratch s = scratch_of(o);
  int total = 0;
  for (int i0 = 0; i0 < o.count; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int need = 0;
    if (i < o.count) {
      const int from = parents[i], to = children[i];
      int cols = -1, src = -1;
      if (from < 0 || from >= o.t.num_seqs || to < 0 || to >= o.t.num_seqs || o.lens[to] != 0) {
        set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
      } else {
        const int len = o.lens[from];
        if (len < 0 || len > int64_t(o.t.max_pages) * o.t.page_size) {
          set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
        } else {
          cols = pages_of(len, o.t.page_size);
          if (len % o.t.page_size != 0) {
            src = o.tables[from * o.t.table_stride + cols - 1];
            if (src >= o.t.num_pages) {
              set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
              src = -1;
            }
            need = src >= 0;
          }
        }
      }
      s.cols[i] = cols;
      s.src[i] = src;
    }
    int sum;
    const int at = total + block_prefix(need, warp_sums, sum);
    if (i < o.count) s.start[i] = at;
    total += sum;
  }
  const int have = list_free(o.refs, o.t.num_pages, min(total, o.t.num_pages), s.free, warp_sums);
  for (int i = threadIdx.x; i < o.count; i += kPlanThreads) {
    int dst = -1;
    if (s.cols[i] >= 0) {
      if (s.src[i] < 0 || s.start[i] < have) {
        if (s.src[i] >= 0) {
          dst = s.free[s.start[i]];
          o.refs[dst] = 1;
        }
        o.lens[children[i]] = o.lens[parents[i]];
      } else {
        set_error(o.err, MOE_W4A16_ERR_CAPACITY);
        s.cols[i] = -1;
        s.src[i] = -1;
      }
    }
    s.dst[i] = dst;
  }
  if (threadIdx.x == 0) *s.copies = o.count;
}

// ---------------------------------------------------------------------------
// page copies
// ---------------------------------------------------------------------------
// Pieces of the copies src[i] -> dst[i], i < n, in every plane, over the CTAs of the grid.
__device__ __forceinline__ void copy_pages(const PoolView& pool, const int32_t* src, const int32_t* dst, int n,
                                           int* err) {
  const int pieces = static_cast<int>((pool.page_bytes + kPieceBytes - 1) / kPieceBytes);
  const int64_t units = int64_t(n) * pool.planes * pieces;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = static_cast<int>(u % pieces);
    const int64_t r = u / pieces;
    const int plane = static_cast<int>(r % pool.planes), i = static_cast<int>(r / pool.planes);
    const int a = src[i], b = dst[i];
    if (a < 0 && b < 0) continue;
    if (a < 0 || a >= pool.num_pages || b < 0 || b >= pool.num_pages) {
      set_error(err, MOE_W4A16_ERR_BAD_INDEX);
      continue;
    }
    const int64_t off = plane * pool.plane_stride + int64_t(piece) * kPieceBytes;
    const uint4* from = reinterpret_cast<const uint4*>(pool.base + off + a * pool.page_stride);
    uint4* to = reinterpret_cast<uint4*>(pool.base + off + b * pool.page_stride);
    const int vecs = static_cast<int>(min(int64_t(kPieceBytes), pool.page_bytes - int64_t(piece) * kPieceBytes) / 16);
    uint4 v[kPieceBytes / 16 / kCopyThreads];
#pragma unroll
    for (int k = 0; k < kPieceBytes / 16 / kCopyThreads; ++k)
      if (k * kCopyThreads + threadIdx.x < vecs) v[k] = from[k * kCopyThreads + threadIdx.x];
#pragma unroll
    for (int k = 0; k < kPieceBytes / 16 / kCopyThreads; ++k)
      if (k * kCopyThreads + threadIdx.x < vecs) to[k * kCopyThreads + threadIdx.x] = v[k];
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const PoolView pool, const int32_t* src, const int32_t* dst,
                                                            int n, int* err) {
  copy_pages(pool, src, dst, n, err);
}

__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const PageOps o, const PoolView pool,
                                                            const int32_t* parents, const int32_t* children) {
  const Scratch s = scratch_of(o);
  for (int i = blockIdx.x; i < o.count; i += gridDim.x) {
    const int cols = s.cols[i];
    if (cols <= 0) continue;
    const int32_t* from = o.tables + parents[i] * o.t.table_stride;
    int32_t* to = o.tables + children[i] * o.t.table_stride;
    const int own = s.dst[i];                       // the copied last page, or -1: shared like the others
    for (int c = threadIdx.x; c < cols; c += kCopyThreads) {
      int page = from[c];
      if (c == cols - 1 && own >= 0) {
        page = own;
      } else if (page >= o.t.num_pages) {
        set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
      } else if (page >= 0) {
        atomicAdd(o.refs + page, 1);
      }
      to[c] = page;
    }
  }
  copy_pages(pool, s.src, s.dst, o.count, o.err);
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kCopyThreads) free_kernel(const PageOps o, const int32_t* seq_ids,
                                                            const int32_t* keep) {
  const int seq = seq_ids[blockIdx.x];
  if (seq < 0 || seq >= o.t.num_seqs) {
    if (threadIdx.x == 0) set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
    return;
  }
  int cols = o.t.max_pages;
  const int kept = keep != nullptr ? keep[blockIdx.x] : 0;
  if (kept > 0) cols = min(cols, max(0, o.lens[seq] - kept) / o.t.page_size);
  int32_t* row = o.tables + seq * o.t.table_stride;
  for (int c = threadIdx.x; c < cols; c += kCopyThreads) {
    // a sequence named twice: the exchange gives each entry to one of the two
    const int page = row[c] >= 0 ? atomicExch(row + c, -1) : -1;
    if (page < 0) continue;
    if (page >= o.t.num_pages) {
      set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
    } else if (atomicSub(o.refs + page, 1) <= 0) {
      atomicAdd(o.refs + page, 1);
      set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
    }
  }
  if (kept <= 0 && threadIdx.x == 0) o.lens[seq] = 0;
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PageOps o, const int32_t* refs_in,
                                                                    int32_t* refs_out, int32_t* page_map,
                                                                    int32_t* num_live) {
  __shared__ int warp_sums[32];
  const Scratch s = scratch_of(o);
  const int n = o.t.num_pages;
  int live = 0;
  for (int p = threadIdx.x; p < n; p += kPlanThreads) live += refs_in[p] > 0;
  int count;
  block_prefix(live, warp_sums, count);
  int movers = 0, holes = 0;
  for (int p0 = 0; p0 < n; p0 += kPlanThreads) {
    const int p = p0 + threadIdx.x;
    const int ref = p < n ? refs_in[p] : 0;
    const bool mover = ref > 0 && p >= count, hole = p < count && ref <= 0;
    int sum;
    // a page is never both: one prefix over each part of the id range
    const int a = block_prefix(mover, warp_sums, sum);
    if (mover) s.src[movers + a] = p;
    movers += sum;
    const int b = block_prefix(hole, warp_sums, sum);
    if (hole) s.dst[holes + b] = p;
    holes += sum;
    if (p < n && !mover) {
      page_map[p] = ref > 0 ? p : -1;
      if (!hole) refs_out[p] = ref > 0 ? ref : 0;   // a hole's count is its mover's, written below
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += kPlanThreads) {   // as many holes as movers
    const int from = s.src[i], to = s.dst[i];
    page_map[from] = to;
    const int ref = refs_in[from];
    refs_out[to] = ref;
    refs_out[from] = 0;
  }
  if (threadIdx.x == 0) {
    *s.copies = movers;
    *num_live = count;
  }
}

__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const PageOps o, const PoolView pool,
                                                               int32_t* tables_out, const int32_t* page_map) {
  const Scratch s = scratch_of(o);
  const int64_t entries = int64_t(o.t.num_seqs) * o.t.max_pages;
  for (int64_t i = int64_t(blockIdx.x) * kCopyThreads + threadIdx.x; i < entries;
       i += int64_t(gridDim.x) * kCopyThreads) {
    const int64_t at = i / o.t.max_pages * o.t.table_stride + i % o.t.max_pages;
    int page = o.tables[at];
    if (page >= o.t.num_pages) set_error(o.err, MOE_W4A16_ERR_BAD_INDEX);
    else if (page >= 0) page = page_map[page];
    tables_out[at] = page;
  }
  copy_pages(pool, s.src, s.dst, *s.copies, o.err);
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// One thread per 16 bytes of pages: 8 BF16 channels copied, or 16 quantised to E4M3 (a true
// division, so that the element is the one nearest to k / scale). Bound by HBM for a prefill's rows, by its
// dependent reads for a step's: 256 tokens of 8 heads x 128 channels in E4M3 2.9 us, 8192 latent rows 6.4 us.
template <bool E4M3>
__global__ void __launch_bounds__(kCopyThreads) append_kernel(const AppendParams p) {
  constexpr int kVec = E4M3 ? 16 : 8;
  const int chunks = p.dim / kVec, per_row = p.heads * chunks;
  const int which = blockIdx.y;
  for (int64_t i = int64_t(blockIdx.x) * kCopyThreads + threadIdx.x; i < int64_t(p.tokens) * per_row;
       i += int64_t(gridDim.x) * kCopyThreads) {
    const int tok = static_cast<int>(i / per_row), rest = static_cast<int>(i % per_row);
    const int head = rest / chunks, c = rest % chunks * kVec;
    const int seq = p.seq_ids[tok], pos = p.positions[tok];
    if (pos < 0) continue;
    const int col = pos / p.t.page_size;
    int page = -1;
    if (seq >= 0 && seq < p.t.num_seqs && col < p.t.max_pages) page = p.t.tables[seq * p.t.table_stride + col];
    if (page < 0 || page >= p.t.num_pages) {
      set_error(p.err, MOE_W4A16_ERR_BAD_INDEX);
      continue;
    }
    const uint4* src = reinterpret_cast<const uint4*>(p.src[which] + tok * p.src_stride[which] + int64_t(head) * p.dim + c);
    const int64_t at = page * p.page_stride + (pos - col * p.t.page_size) * p.token_stride + head * p.head_stride + c;
    if (!E4M3) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.pages[which]) + at) = *src;
    } else {
      const uint4 v[2] = {src[0], src[1]};
      const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
      uint32_t out[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t pair[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t x = w[2 * j + q];
          const float lo = __fdiv_rn(bf16_to_f32(static_cast<uint16_t>(x)), p.scale[which]);
          const float hi = __fdiv_rn(bf16_to_f32(static_cast<uint16_t>(x >> 16)), p.scale[which]);
          pair[q] = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
        }
        out[j] = pair[0] | pair[1] << 16;
      }
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.pages[which]) + at) = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

static unsigned copy_grid(int64_t units, int device) {
  const int64_t most = int64_t(device_info(device).sm_count) * 8;   // every SM full of 256-thread CTAs
  return static_cast<unsigned>(units < 1 ? 1 : units < most ? units : most);
}
static int64_t copy_units(const PoolView& pool, int64_t pages) {
  return pages * pool.planes * ((pool.page_bytes + kPieceBytes - 1) / kPieceBytes);
}

}  // namespace cache

using namespace cache;

cudaError_t launch_cache_append(const AppendParams& p, int dtype, cudaStream_t stream) {
  const bool e4m3 = dtype == MOE_W4A16_CACHE_E4M3;
  const int64_t threads = int64_t(p.tokens) * p.heads * (p.dim / (e4m3 ? 16 : 8));
  int64_t blocks = (threads + kCopyThreads - 1) / kCopyThreads;
  if (blocks > (1 << 20)) blocks = 1 << 20;
  const dim3 grid(static_cast<unsigned>(blocks), p.src[1] != nullptr ? 2 : 1);
  if (e4m3) append_kernel<true><<<grid, kCopyThreads, 0, stream>>>(p);
  else append_kernel<false><<<grid, kCopyThreads, 0, stream>>>(p);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_cache_extend(const PageOps& o, const int32_t* seq_ids, const int32_t* counts, int32_t* positions,
                                cudaStream_t stream) {
  extend_kernel<<<1, kPlanThreads, 0, stream>>>(o, seq_ids, counts, positions);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_cache_fork(const PageOps& o, const PoolView& pool, const int32_t* parents, const int32_t* children,
                              int device, cudaStream_t stream) {
  fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(o, parents, children);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  fork_kernel<<<copy_grid(copy_units(pool, o.count), device), kCopyThreads, 0, stream>>>(o, pool, parents, children);
  note_launch(2);
  return cudaGetLastError();
}

cudaError_t launch_cache_free(const PageOps& o, const int32_t* seq_ids, const int32_t* keep, cudaStream_t stream) {
  free_kernel<<<o.count, kCopyThreads, 0, stream>>>(o, seq_ids, keep);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_cache_copy(const PoolView& pool, const int32_t* src, const int32_t* dst, int count, int* err,
                              int device, cudaStream_t stream) {
  copy_kernel<<<copy_grid(copy_units(pool, count), device), kCopyThreads, 0, stream>>>(pool, src, dst, count, err);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const PageOps& o, const PoolView& pool, const int32_t* refs_in, int32_t* refs_out,
                                 int32_t* tables_out, int32_t* page_map, int32_t* num_live, int device,
                                 cudaStream_t stream) {
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(o, refs_in, refs_out, page_map, num_live);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // at most half the pool moves
  compact_kernel<<<copy_grid(copy_units(pool, (pool.num_pages + 1) / 2), device), kCopyThreads, 0, stream>>>(
      o, pool, tables_out, page_map);
  note_launch(2);
  return cudaGetLastError();
}

}  // namespace moe
