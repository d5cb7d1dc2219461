// Attention of one new token per sequence over a latent cache: one row of 576 channels per token is
// every head's key, its first 512 channels every head's value.
//
// With up to 64 heads on one row of 1152 bytes a token costs 2 * 64 * (576 + 512) flops for those
// bytes, 121 a byte: at full HBM speed 0.8 PFLOP/s, beyond warp-level MMA. So both products run on
// tcgen05, and both read the one copy of the tile in shared memory:
//
//   S^T [keys x heads]  = K [keys x 576] . Q^T       A = the tile, K-major
//   O^T [512 x heads]  += V^T [512 x keys] . P^T      A = the same tile, M-major (no transposed copy)
//
// Sequences with more than 64 heads are read once for each block of 64, one block after the other: over 128 sequences of
// 2048 to 8192 tokens 128 heads take 265 us where 64 take 154.
//
//   * Tiles of 64 tokens, two in shared memory (2 x 72 KB) beside the 64 queries (72 KB), filled with cp.async
//     (rows gathered by page; unseen slots zero-filled); the tile two ahead is prefetched into L2, so that HBM does
//     not wait for a free buffer.
//   * S^T (M = 64: 16 lanes of each TMEM quarter) is double-buffered, O^T takes 256 columns (four 128-channel
//     tiles). The next tile's scores run beside this tile's softmax and values. A thread issues an MMA every 60
//     to 75 cycles whatever its size, 52 of them a tile, so each product has two issuing warps: S^T in two
//     accumulators (even and odd chunks of the reduction) that the softmax adds up, O^T two channel tiles each.
//     Both products' operands come from shared memory: 4 KB a 64x64x16 MMA and 6 KB a 128x64x16 one make
//     240 KB a tile, 1900 of the about 3250 cycles that a tile takes at HBM speed.
//   * Softmax: the heads are columns, the lanes keys; two groups of four warps take 32 heads each, read in the
//     MMA fragment layout (16 scores a thread). The base of the exponents only moves when a score passes it by
//     2^8 (BF16 probabilities keep their relative precision, FP32 sums their range), so a tile costs no
//     maximum over its keys, only a vote, and the accumulator in TMEM is seldom rescaled.
//   * Work is shared out as in split.cuh; a row that crosses CTAs is written as FP32 parts, which a second
//     kernel joins in order, 13 us of the 142 below (64 heads x 512 channels are 128 KB a part, too much for one last
//     CTA: 148 us; joined inside a cooperative launch: 151 to 159 us).
//
// 128 sequences of up to 8192 tokens, 64 heads, pages of 64: 142 us, 5.14 TB/s; the kernel itself 130 us at 5.6 TB/s,
// its tensor pipe 46% busy. Not better: tiles of 128 tokens in a single buffer 172 us, one issuing thread a product 157 us.
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"
#include "split.cuh"

namespace moe {
namespace latent {

constexpr int kHeads = 64;                    // heads of a work row (MMA N)
constexpr int kTile = 64;                     // tokens of a tile
constexpr int kChunks = kLatentDim / 64;      // 128-byte column chunks of a row: 9
constexpr int kChunkBytes64 = 64 * 128;       // 64 rows of one chunk, 128-byte swizzled
constexpr int kTileBytes = kChunks * kChunkBytes64;      // 73,728
constexpr int kValueTiles = kLatentValue / 128;          // M tiles of O^T: 4

// warps: 0-7 softmax / rescale / epilogue, 8-11 tile loaders, 12-13 queries and S^T, 14-15 O^T
constexpr int kThreads = 512;
constexpr int kGroups = 3;                    // chunk groups of a tile that the S issuer waits for

constexpr int kKOff = 0;
constexpr int kQOff = 2 * kTileBytes;
constexpr int kPOff = kQOff + kTileBytes;
constexpr int kBarOff = kPOff + kTile * 128;
enum {
  kBarFull = 0,                               // [2][kGroups] tile chunks loaded
  kBarScore = kBarFull + 2 * kGroups,         // [2] S^T of a tile computed
  kBarScoreFree = kBarScore + 2,              // [2] S^T read
  kBarProb = kBarScoreFree + 2,               // P of a tile written, O^T rescaled if need be
  kBarDone = kBarProb + 1,                    // [2] a tile's O^T product done: tile, P free, O^T stable
  kBarQ = kBarDone + 2,                       // queries of a piece loaded
  kBarQFree = kBarQ + 1,
  kBarDrain = kBarQFree + 1,
  kNumBars = kBarDrain + 2
};
constexpr int kMiscOff = kBarOff + kNumBars * 8;         // TMEM address, abort flag
constexpr int kMaskOff = kMiscOff + 8;                   // [2][4] masks of 16 tokens seen
constexpr int kMaxOff = kMaskOff + 32;                   // float [4][64] maxima or sums by key quarter
constexpr int kKeepOff = kMaxOff + 4 * kHeads * 4;       // float [64] factors of a rescale
constexpr int kBaseOff = kKeepOff + kHeads * 4;          // float [64] bases at a row's end
constexpr int kShareOff = (kBaseOff + kHeads * 4 + 15) / 16 * 16;
constexpr int kSmemBytes = kShareOff + static_cast<int>(sizeof(Share));
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
static_assert(kPOff % 1024 == 0 && kQOff % 1024 == 0 && kChunkBytes64 % 1024 == 0, "swizzled tiles");

constexpr int kTmemCols = 512;
constexpr int kScoreCol = 0;                  // S^T buffer b, accumulator a at 128 b + 64 a
constexpr int kAccCol = 256;                  // O^T tile i at 256 + 64 i

// A part of a row: base and sum of its 64 heads, then O^T unnormalised as [64][512].
constexpr int kPartFloats = 2 * kHeads + kHeads * kLatentValue;
// What a CTA left for the join: a row that starts in it and goes on in the next np - 1.
struct Record {
  int32_t np, b, head0, heads;
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Operand tiles are rows of 128 bytes in 128-byte swizzle, 8-row atoms of 1024 bytes. K-major (rows along
// M or N, 64 channels of the reduction a row): atoms follow each other along the rows at 1024 bytes. M-major
// (rows along the reduction, 64 channels of M or N a row): 8-row groups of the reduction at 1024 bytes, the next
// 64 channels one chunk further.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead_bytes) {
  return (static_cast<uint64_t>((addr & 0x3FFFFu) >> 4)) | (static_cast<uint64_t>(lead_bytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// kind::f16, FP32 accumulator, BF16 operands, N = 64; bits 15 / 16: A / B M-major.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kHeads >> 3) << 17);
constexpr uint32_t kIdescScore = kIdesc | (uint32_t(kTile >> 4) << 24);
constexpr uint32_t kIdescValue = kIdesc | (uint32_t(128 >> 4) << 24) | (1u << 15) | (1u << 16);

// 16 lanes x 32 columns in the MMA fragment layout: registers 4j, 4j+1 hold lane t/4, columns 8j + 2(t%4), +1
// (thread t), registers 4j+2, 4j+3 the same of lane t/4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
// Both accumulators of a score buffer.
__device__ __forceinline__ void tmem_ld_frag(uint32_t addr, uint32_t (&r)[16], uint32_t (&r2)[16]) {
  tmem_ld_frag(addr, r);
  tmem_ld_frag(addr + 64, r2);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Bytes (a multiple of 16, from a 16-byte boundary) on their way from HBM to L2.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Work rows of a sequence: blocks of up to 64 heads.
__device__ __forceinline__ int head_blocks(int heads) { return (heads + kHeads - 1) / kHeads; }

// DIAG: the diagnostic instantiation, whose waits take the launch's own limit (moe_w4a16_set_wait_limit_ns).
template <bool DIAG>
__global__ void __launch_bounds__(kThreads, 1) latent_kernel(const AttnParams p, Record* records) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);
  const uint32_t bars = base + kBarOff;
  auto bar = [&](int i) { return bars + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMiscOff + 4);
  Share* share = reinterpret_cast<Share*>(smem + kShareOff);
  const int rows = head_blocks(p.heads);

  asm volatile("griddepcontrol.launch_dependents;");
  zero_empty<kThreads>(p, kLatentValue);
  if (threadIdx.x == 0) records[blockIdx.x].np = 0;
  const auto min_tiles = [](int64_t tiles, int) { return tiles / kLatentMinTiles; };
  if (!find_share<kThreads>(p, blockIdx.x, gridDim.x, rows, kTile, min_tiles, share)) return;
  if ((base & 1023u) != 0) {                 // the swizzle is a function of address bits
    if (threadIdx.x == 0) set_error(p.err, MOE_W4A16_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * kGroups; ++i) mbar_init(bar(kBarFull + i), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarScore + i), 2);
      mbar_init(bar(kBarScoreFree + i), 8);
      mbar_init(bar(kBarDone + i), 2);
      mbar_init(bar(kBarDrain + i), 2);
    }
    mbar_init(bar(kBarProb), 8);
    mbar_init(bar(kBarQ), 64);
    mbar_init(bar(kBarQFree), 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + kMiscOff), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kMiscOff);
  const int64_t total = share->total;
  const int ctas = share->ctas;
  PieceWalk walk;
  walk.start(p, share);
  Piece pc;
  auto wait = [&](int i, uint32_t parity) { return warp_wait(bar(i), parity, abort_flag, p.err, DIAG ? p.wait_ns : kWaitLimitNs); };

  if (warp < 8) {
    // ------------------------------------------------------------- softmax, rescale, epilogue
    const int q = warp & 3, group = warp >> 2;           // TMEM lane quarter, heads 32 group ..
    const int r0 = lane >> 2, cc = lane & 3;             // this thread's keys 16 q + r0, + 8; heads 8 j + 2 cc, + 1
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    float* maxima = reinterpret_cast<float*>(smem + kMaxOff) + 32 * group;      // [4][64]
    float* keeps = reinterpret_cast<float*>(smem + kKeepOff) + 32 * group;
    float* bases = reinterpret_cast<float*>(smem + kBaseOff) + 32 * group;
    const volatile uint32_t* masks = reinterpret_cast<const volatile uint32_t*>(smem + kMaskOff);
    uint32_t it = 0;                                     // tiles of this CTA so far
    bool dead = false;                                   // a wait gave up
    auto wait_or_die = [&](int i, uint32_t parity) {
      if (!dead) dead = !wait(i, parity);
    };
    // The four warps of a column group meet at a hardware barrier, which also ORs their votes. After a wait that gave
    // up they go on (with nothing to show for it) rather than leave, so that all of them reach every barrier.
    auto any_of_group = [&](bool vote) {
      int r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\t"
          "selp.b32 %0, 1, 0, q;\n\t}"
          : "=r"(r)
          : "r"(static_cast<int>(vote)), "r"(1 + group)
          : "memory");
      return r != 0;
    };
    auto group_sync = [&]() { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory"); };
    while (walk.next(p, rows, kTile, pc)) {
      const int head0 = pc.r * kHeads, heads = min(kHeads, p.heads - head0);
      const int mine = min(32, heads - 32 * group);      // heads of this column group (may be <= 0)
      float at[8], l[8];                                 // bases and sums of heads 8 j + 2 cc + e at 2 j + e
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        at[h] = -INFINITY;
        l[h] = 0.f;
      }
      const int n = pc.tile1 - pc.tile0;
      for (int i = 0; i < n; ++i, ++it) {
        const int buf = it & 1;
        const uint32_t par = (it >> 1) & 1u;
        uint32_t s[16];
        wait_or_die(kBarFull + buf * kGroups, par);
        wait_or_die(kBarScore + buf, par);
        tc_fence_after();
        const uint32_t seen = masks[buf * 4 + q];             // 16 bits
        {
          uint32_t s2[16];
          tmem_ld_frag(tmem + kScoreCol + buf * 128 + 32 * group + lanes, s, s2);
#pragma unroll
          for (int k = 0; k < 16; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) + __uint_as_float(s2[k]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarScoreFree + buf));
        bool over = false;
        if (seen != 0xffffu) {
          const bool a = seen >> r0 & 1u, b = seen >> (r0 + 8) & 1u;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const bool in = (k & 2) ? b : a;
            const float v = in ? __uint_as_float(s[k]) * p.score_scale : -INFINITY;
            s[k] = __float_as_uint(v);
            over |= v > at[(k >> 2) * 2 + (k & 1)] + 8.f;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float v = __uint_as_float(s[k]) * p.score_scale;
            s[k] = __float_as_uint(v);
            over |= v > at[(k >> 2) * 2 + (k & 1)] + 8.f;   // at = -inf at first: any seen score
          }
        }
        over = any_of_group(over);
        if (over) {
          // new bases: the maximum over the tile's keys where it passes the old one
          float best[8];
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            best[h] = fmaxf(__uint_as_float(s[(h >> 1) * 4 + (h & 1)]), __uint_as_float(s[(h >> 1) * 4 + 2 + (h & 1)]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) best[h] = fmaxf(best[h], __shfl_xor_sync(0xffffffffu, best[h], o));
            if (r0 == 0) maxima[q * kHeads + (h >> 1) * 8 + 2 * cc + (h & 1)] = best[h];
          }
          group_sync();
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const int head = (h >> 1) * 8 + 2 * cc + (h & 1);
            float top = at[h];
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, maxima[k * kHeads + head]);
            const float keep = top == at[h] ? 1.f : exp2_fast(at[h] - top);
            at[h] = top;
            l[h] *= keep;
            if (q == 0 && r0 == 0) keeps[head] = keep;
          }
          group_sync();
          if (i > 0) {
            // O^T is stable once the previous tile's product is done
            wait_or_die(kBarDone + (buf ^ 1), ((it - 1) >> 1) & 1u);
            tc_fence_after();
            if (mine > 0) {
#pragma unroll 1
              for (int mt = 0; mt < kValueTiles; ++mt) {
                uint32_t o[32];
                const uint32_t acc = tmem + kAccCol + mt * 64 + 32 * group + lanes;
                tmem_ld32(acc, o);
#pragma unroll
                for (int h = 0; h < 32; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * keeps[h]);
                tmem_st32(acc, o);
              }
            }
          }
        }
        uint32_t packed[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float b0 = at[2 * j] == -INFINITY ? 0.f : at[2 * j], b1 = at[2 * j + 1] == -INFINITY ? 0.f : at[2 * j + 1];
          const float e0 = exp2_fast(__uint_as_float(s[4 * j]) - b0), e1 = exp2_fast(__uint_as_float(s[4 * j + 1]) - b1);
          const float e2 = exp2_fast(__uint_as_float(s[4 * j + 2]) - b0),
                      e3 = exp2_fast(__uint_as_float(s[4 * j + 3]) - b1);
          l[2 * j] += e0 + e2;
          l[2 * j + 1] += e1 + e3;
          packed[2 * j] = pack_bf16x2_rn(e0, e1);
          packed[2 * j + 1] = pack_bf16x2_rn(e2, e3);
        }
        // the previous tile's product is done: P is free
        if (it != 0) wait_or_die(kBarDone + (buf ^ 1), ((it - 1) >> 1) & 1u);
        {
          uint8_t* row = smem + kPOff + (16 * q + r0) * 128 + cc * 4;    // rows r0 and r0 + 8: the same swizzle
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int chunk = ((group * 4 + j) ^ r0) << 4;
            *reinterpret_cast<uint32_t*>(row + chunk) = packed[2 * j];
            *reinterpret_cast<uint32_t*>(row + 8 * 128 + chunk) = packed[2 * j + 1];
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarProb));
      }

      // ---- epilogue: the sums over keys, then this quarter's channels of O^T
#pragma unroll
      for (int h = 0; h < 8; ++h) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
        if (r0 == 0) {
          const int head = (h >> 1) * 8 + 2 * cc + (h & 1);
          maxima[q * kHeads + head] = l[h];
          if (q == 0) bases[head] = at[h];
        }
      }
      group_sync();
      const float top = bases[lane];                     // lane h: head 32 group + h
      const float sum = maxima[lane] + maxima[kHeads + lane] + maxima[2 * kHeads + lane] + maxima[3 * kHeads + lane];
      wait_or_die(kBarDone + ((it - 1) & 1), ((it - 1) >> 1) & 1u);
      tc_fence_after();
      const int c0 = cta_of(total, ctas, pc.row0), c1 = cta_of(total, ctas, pc.row0 + pc.ntiles - 1);
      const int64_t out0 = (int64_t(pc.b) * p.heads + head0 + 32 * group);
      const bool whole = c0 == c1;
      float* part = p.parts + (int64_t(blockIdx.x) * 2 + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0)) * kPartFloats;
      if (q == 0 && lane < mine) {
        if (whole) {
          if (p.lse != nullptr) p.lse[out0 + lane] = (top + log2f(sum)) * 0.69314718055994531f;
        } else {
          part[32 * group + lane] = top;
          part[kHeads + 32 * group + lane] = sum;
        }
      }
      if (!whole && static_cast<int>(blockIdx.x) == c0 && threadIdx.x == 0)
        records[blockIdx.x] = Record{c1 - c0 + 1, pc.b, head0, heads};
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      if (mine > 0) {
#pragma unroll 1
        for (int mt = 0; mt < kValueTiles; ++mt) {
          uint32_t o[32];
          tmem_ld32(tmem + kAccCol + mt * 64 + 32 * group + lanes, o);
          const int d = mt * 128 + 32 * q + lane;
          if (whole) {
            // lane pairs trade values so that each stores two channels of one head: the even lane of the first,
            // the odd lane of the second of two heads
#pragma unroll
            for (int h = 0; h < 32; h += 2) {
              const float v0 = __uint_as_float(o[h]) * __shfl_sync(0xffffffffu, inv, h);
              const float v1 = __uint_as_float(o[h + 1]) * __shfl_sync(0xffffffffu, inv, h + 1);
              const bool odd = lane & 1;
              const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
              const int head = h + (odd ? 1 : 0);
              if (head < mine)
                *reinterpret_cast<uint32_t*>(p.out + (out0 + head) * kLatentValue + (d & ~1)) =
                    odd ? pack_bf16x2_rn(got, v1) : pack_bf16x2_rn(v0, got);
            }
          } else {
            float* dst = part + 2 * kHeads + 32 * group * kLatentValue + d;
#pragma unroll
            for (int h = 0; h < 32; ++h)
              if (h < mine) __stcg(dst + h * kLatentValue, __uint_as_float(o[h]));
          }
        }
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------- tile loaders
    // A warp owns 16 of a tile's tokens: lane & 15 = token for the page look-up; copies of 8 lanes a row, 4 rows at
    // a time.
    const int quarter = warp - 8;
    uint32_t it = 0;
    bool ok = true;
    const uint8_t* src = static_cast<const uint8_t*>(p.k);
    volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + kMaskOff);
    uint32_t to[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = k * 4 + (lane >> 3);
      to[k] = base + kKOff + (quarter * 16 + r) * 128 + (((lane & 7) ^ (r & 7)) << 4);
    }
    while (ok && walk.next(p, rows, kTile, pc)) {
      const int32_t* table = p.t.tables + int64_t(pc.seq) * p.t.table_stride;
      const int n = pc.tile1 - pc.tile0;
      const int tok0 = (pc.lo / kTile + pc.tile0) * kTile + 16 * quarter + (lane & 15);
      auto entry_of = [&](int i) -> int {
        if (i >= n) return -1;
        const int tok = tok0 + i * kTile;
        if (tok < pc.lo || tok >= pc.hi) return -1;
        return table[tok / p.t.page_size];
      };
      // byte offset of this lane's token in tile i, -1 where it is not seen
      auto offset_of = [&](int entry, int i) -> int64_t {
        if (entry < 0) return -1;
        if (entry >= p.t.num_pages) {
          set_error(p.err, MOE_W4A16_ERR_BAD_INDEX);
          return -1;
        }
        return (int64_t(entry) * p.page_stride + int64_t((tok0 + i * kTile) % p.t.page_size) * p.token_stride) * 2;
      };
      // a tile two ahead on its way to L2: one request where its rows lie behind each other, else one a row (60
      // cycles each, so behind the arrivals)
      auto prefetch = [&](int64_t off) {
        const int64_t first = __shfl_sync(0xffffffffu, off, 0);
        if (__all_sync(0xffffffffu, first >= 0 && off == first + (lane & 15) * (kLatentDim * 2))) {
          if (lane == 0) prefetch_l2(src + first, 16 * kLatentDim * 2);
        } else if (off >= 0 && lane < 16) {
          prefetch_l2(src + off, kLatentDim * 2);
        }
      };
      int64_t off = offset_of(entry_of(0), 0), off1 = offset_of(entry_of(1), 1);
      for (int i = 0; i < n; ++i, ++it) {
        const int buf = it & 1;
        const uint32_t seen = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
        const uint8_t* from[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t o = __shfl_sync(0xffffffffu, off, k * 4 + (lane >> 3));
          from[k] = src + (o >= 0 ? o + (lane & 7) * 16 : 0);
        }
        if (it >= 2 && !(ok = wait(kBarDone + buf, ((it >> 1) - 1) & 1u))) break;
        if (lane == 0) masks[buf * 4 + quarter] = seen;
        const uint32_t shift = buf * kTileBytes;
        if (seen == 0xffffu) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to[k] + shift + c * kChunkBytes64),
                           "l"(from[k] + c * 128)
                           : "memory");
            if (c % (kChunks / kGroups) == kChunks / kGroups - 1) cp_async_commit();
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < kChunks; ++c) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const bool have = seen >> (k * 4 + (lane >> 3)) & 1u;
              cp_async16(to[k] + shift + c * kChunkBytes64, have ? from[k] + c * 128 : src, have ? 16 : 0);
            }
            if (c % (kChunks / kGroups) == kChunks / kGroups - 1) cp_async_commit();
          }
        }
        const int entry = entry_of(i + 2);
        auto landed = [&](int grp) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarFull + buf * kGroups + grp));
        };
        static_assert(kGroups == 3, "waits below");
        cp_async_wait<2>();
        landed(0);
        cp_async_wait<1>();
        landed(1);
        cp_async_wait<0>();
        landed(2);
        off = off1;
        off1 = offset_of(entry, i + 2);
        prefetch(off1);
      }
    }
    cp_async_wait<0>();
  } else if (warp < 14) {
    // ------------------------------------------------------------- queries of a piece, S^T = K Q^T
    // Query rows past the last head are zeros. Issuer 0 takes the even chunks, issuer 1 the odd ones.
    const int half = warp - 12;
    uint32_t it = 0, piece = 0;
    bool ok = true;
    while (ok && walk.next(p, rows, kTile, pc)) {
      if (!(ok = wait(kBarQFree, (piece & 1u) ^ 1u))) break;
      const int head0 = pc.r * kHeads, heads = min(kHeads, p.heads - head0);
      const uint16_t* src = p.q + int64_t(pc.b) * p.q_stride + int64_t(head0) * kLatentDim;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = half * 32 + k * 4 + (lane >> 3);
        const uint32_t to = base + kQOff + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
        const uint16_t* from = src + (r < heads ? r * kLatentDim + (lane & 7) * 8 : 0);
        const uint32_t bytes = r < heads ? 16 : 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) cp_async16(to + c * kChunkBytes64, from + (bytes ? c * 64 : 0), bytes);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      mbar_arrive(bar(kBarQ));
      if (!(ok = wait(kBarQ, piece & 1u))) break;
      const int n = pc.tile1 - pc.tile0;
      for (int i = 0; i < n; ++i, ++it) {
        const int buf = it & 1;
        const uint32_t par = (it >> 1) & 1u;
        if (!(ok = wait(kBarScoreFree + buf, par ^ 1u))) break;
        const uint32_t d = tmem + kScoreCol + buf * 128 + half * 64;
#pragma unroll
        for (int grp = 0; grp < kGroups; ++grp) {
          if (ok) ok = wait(kBarFull + buf * kGroups + grp, par);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int cc = 0; cc < kChunks / kGroups; ++cc) {
              const int c = grp * (kChunks / kGroups) + cc;
              if ((c & 1) != half) continue;
              const uint64_t a = smem_desc(base + kKOff + buf * kTileBytes + c * kChunkBytes64, 16);
              const uint64_t b = smem_desc(base + kQOff + c * kChunkBytes64, 16);
#pragma unroll
              for (int k = 0; k < 4; ++k)                // 16 channels = 32 bytes a step
                tc_mma(d, a + 2 * k, b + 2 * k, kIdescScore, c < 2 && k == 0 ? 0u : 1u);
            }
            if (grp == kGroups - 1) tc_commit(bar(kBarScore + buf));
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (lane == 0) tc_commit(bar(kBarQFree));
      __syncwarp();
      ++piece;
    }
    cp_async_wait<0>();
    if (lane == 0) {
      tc_commit(bar(kBarDrain));
      mbar_drain(bar(kBarDrain), 0);
    }
  } else {
    // ------------------------------------------------------------- O^T += V^T P^T, two channel tiles an issuer
    const int half = warp - 14;
    uint32_t it = 0;
    bool ok = true;
    while (ok && walk.next(p, rows, kTile, pc)) {
      const int n = pc.tile1 - pc.tile0;
      for (int i = 0; i < n; ++i, ++it) {
        const int buf = it & 1;
        if (!(ok = wait(kBarProb, it & 1u))) break;
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int m = 0; m < kValueTiles / 2; ++m) {
            const int mt = half * (kValueTiles / 2) + m;
            const uint64_t a = smem_desc(base + kKOff + buf * kTileBytes + mt * 2 * kChunkBytes64, kChunkBytes64);
            const uint64_t b = smem_desc(base + kPOff, kChunkBytes64);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)         // 16 tokens = two 1024-byte groups a step
              tc_mma(tmem + kAccCol + mt * 64, a + k * 128, b + k * 128, kIdescValue, i == 0 && k == 0 ? 0u : 1u);
          }
          tc_commit(bar(kBarDone + buf));
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      tc_commit(bar(kBarDrain + 1));
      mbar_drain(bar(kBarDrain + 1), 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the rows that cross CTAs. Every block lists the split rows (records with more than one part); an item
// is (row, head), 512 channels. Many items: a warp each; few: a block each, its warps taking every eighth part.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kLaneVecs = kLatentValue / 4 / 32;          // float4 of a lane: 4
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const AttnParams p, const Record* records, int ctas) {
  __shared__ int list[kLatentMaxCtas];
  __shared__ float4 acc_s[kJoinWarps][kLatentValue / 4];
  __shared__ int count_s;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    constexpr int kLoads = (kLatentMaxCtas + 31) / 32;     // all in flight together
    int np[kLoads], count = 0;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) np[k] = 32 * k + lane < ctas ? __ldcg(&records[32 * k + lane].np) : 0;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const uint32_t m = __ballot_sync(0xffffffffu, np[k] > 1);
      if (np[k] > 1) list[count + __popc(m & ((1u << lane) - 1u))] = 32 * k + lane + (np[k] << 16);
      count += __popc(m);
    }
    if (lane == 0) count_s = count;
  }
  __syncthreads();
  const int heads = min(kHeads, p.heads);
  const int64_t items = int64_t(count_s) * heads;
  const bool by_warp = items > int64_t(gridDim.x) * 2;
  const int64_t first = by_warp ? int64_t(blockIdx.x) * kJoinWarps + warp : blockIdx.x;
  const int64_t step = by_warp ? int64_t(gridDim.x) * kJoinWarps : gridDim.x;
  const int part0 = by_warp ? 0 : warp, parts_step = by_warp ? 1 : kJoinWarps;
  for (int64_t item = first; item < items; item += step) {
    const int entry = list[item / heads], c = entry & 0xffff, np = entry >> 16, h = static_cast<int>(item % heads);
    const Record r = records[c];                          // (needed last; the parts' loads do not wait for it)
    auto part_at = [&](int i) { return p.parts + (int64_t(c + i) * 2 + (i == 0 ? 1 : 0)) * kPartFloats; };
    // lane i: base and sum of part i, i + 32, ... (a row has at most kLatentMaxCtas)
    constexpr int kRounds = (kLatentMaxCtas + 31) / 32;
    float top = -INFINITY, sum = 0.f, m[kRounds], l[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int i = 32 * k + lane;
      m[k] = i < np ? __ldcg(part_at(i) + h) : -INFINITY;
      l[k] = i < np ? __ldcg(part_at(i) + kHeads + h) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) top = fmaxf(top, m[k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float b0 = top == -INFINITY ? 0.f : top;
    float4 acc[kLaneVecs];
#pragma unroll
    for (int k = 0; k < kLaneVecs; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int rd = 0; rd < kRounds; ++rd) {
      if (32 * rd >= np) break;
      const float f = exp2_fast(m[rd] - b0);
      sum = fmaf(f, l[rd], sum);
      const int n = min(32, np - 32 * rd);
#pragma unroll 4
      for (int i = part0; i < n; i += parts_step) {
        const float w = __shfl_sync(0xffffffffu, f, i);
        const float4* src = reinterpret_cast<const float4*>(part_at(32 * rd + i) + 2 * kHeads + h * kLatentValue) + lane;
#pragma unroll
        for (int k = 0; k < kLaneVecs; ++k) {
          const float4 v = __ldcg(src + 32 * k);
          acc[k].x = fmaf(w, v.x, acc[k].x);
          acc[k].y = fmaf(w, v.y, acc[k].y);
          acc[k].z = fmaf(w, v.z, acc[k].z);
          acc[k].w = fmaf(w, v.w, acc[k].w);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!by_warp) {
      // the warps' sums, added in their order
#pragma unroll
      for (int k = 0; k < kLaneVecs; ++k) acc_s[warp][32 * k + lane] = acc[k];
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int k = 0; k < kLaneVecs; ++k)
          for (int w = 1; w < kJoinWarps; ++w) {
            const float4 v = acc_s[w][32 * k + lane];
            acc[k].x += v.x;
            acc[k].y += v.y;
            acc[k].z += v.z;
            acc[k].w += v.w;
          }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    if (h >= r.heads) continue;                           // (a last block of heads: its other parts were never written)
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int64_t row = int64_t(r.b) * p.heads + r.head0 + h;
#pragma unroll
    for (int k = 0; k < kLaneVecs; ++k)
      reinterpret_cast<uint2*>(p.out + row * kLatentValue)[32 * k + lane] =
          make_uint2(pack_bf16x2_rn(acc[k].x * inv, acc[k].y * inv), pack_bf16x2_rn(acc[k].z * inv, acc[k].w * inv));
    if (lane == 0 && p.lse != nullptr) p.lse[row] = (top + log2f(sum)) * 0.69314718055994531f;
  }
}

}  // namespace latent

using namespace latent;

size_t latent_part_bytes(int) {
  return kLatentMaxCtas * sizeof(Record) + size_t(kLatentMaxCtas) * 2 * kPartFloats * sizeof(float);
}

template <bool DIAG>
static cudaError_t launch(const AttnParams& p, Record* records, int grid, int device, cudaStream_t stream) {
  static bool attr_set[64] = {false};
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[device]) {
    const cudaError_t e =
        cudaFuncSetAttribute(latent_kernel<DIAG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set[device] = true;
  }
  latent_kernel<DIAG><<<grid, kThreads, kSmemBytes, stream>>>(p, records);
  return cudaGetLastError();
}

cudaError_t launch_latent_attention(const AttnParams& p0, int device, cudaStream_t stream) {
  AttnParams p = p0;
  Record* records = reinterpret_cast<Record*>(p.parts);
  p.parts = reinterpret_cast<float*>(records + kLatentMaxCtas);
  int grid = device_info(device).sm_count;
  if (grid > kLatentMaxCtas) grid = kLatentMaxCtas;
  cudaError_t e = p.wait_ns == kWaitLimitNs ? launch<false>(p, records, grid, device, stream)
                                            : launch<true>(p, records, grid, device, stream);
  if (e != cudaSuccess) return e;
  // the join may be set up while the first kernel runs; it waits for that kernel's end before it reads
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid * 8));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, latent_join_kernel, static_cast<const AttnParams&>(p), static_cast<const Record*>(records),
                         grid);
  note_launch(2);
  return e;
}

}  // namespace moe
