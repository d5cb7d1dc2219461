// Attention of a chunk of new tokens per sequence over a paged cache, grouped heads.
//
// The query rows of a cache head -- its `group` heads times the chunk's tokens -- are the rows of one product with each
// tile of 128 tokens:
//
//   S [rows x tokens] = Q [rows x D] . K^T          both operands in shared memory
//   O [rows x D]     += P [rows x tokens] . V       P = exp2(S - base) in tensor memory, over its own S
//
// so keys and values are read once for up to 256 rows (two streams of 128; 129 to 256 channels: 128 rows), and a prompt is
// bound by its products, drafts by HBM. Both products run on tcgen05 with FP32 accumulators in TMEM.
//
//   * A CTA has two streams, each with its rows' queries, scores and accumulator, an issuing warp and four softmax
//     warps, a thread a row. While one stream's softmax runs, the tensor pipe works for the other: O += P V of its last
//     tile and S of its next, the two streams in turns (in no order prompts take 1.12 times as long). Rows of a chunk that
//     fit one stream: both streams take the same rows and every other tile, and their accumulators are joined at the end.
//   * P is handed over in halves, so that the first half's products run while the second's exponentials are taken.
//   * 129 to 256 channels: one stream, as its accumulator takes half of TMEM; its scores have two buffers, and the next
//     tile's are computed during a tile's softmax, which has two threads a row.
//   * The base of a row's exponents moves when a score passes it by 2^8, not with every new maximum, so the accumulator is
//     seldom rescaled. BF16 probabilities keep their relative precision (2^-8) above the base, FP32 sums their range; what is lost
//     is a largest probability of one, which is not rounded (as in the attention of single tokens, which has the time for it).
//     Prompts' errors against 64 bits: 0.0021; against the exact maximum 0.0019, in 607 us for 550; the outputs' own 0.0016.
//   * Four warps bring the tiles into a ring of 128-byte swizzled ones, each 32 tokens: boxes of 8 to 32 tokens by TMA where
//     they lie behind each other in a page and all are seen, else token by token with cp.async. E4M3 comes to a buffer of
//     its own and is converted to FP16 on the way to the ring, exactly.
//   * Every CTA takes an equal share of one line of tiles over all sequences, heads and row blocks, whatever the lengths;
//     rows that cross CTAs are written as FP32 parts, which a second kernel joins in order.
//   * Unseen slots (past the end, freed pages) are not read: their rows are zero-filled and their scores -infinity.
//   * Nothing in this kernel takes longer than the tiles before it, as its waits are bounded: rows that a hidden value which is no
//     number reaches are flagged here and computed again by the third kernel.
//
// Measured (GB300; 64 query and 8 cache heads of 128 channels where not said otherwise; floors: HBM at 6.78 TB/s, products at
// 1919 TFLOP/s): prompts of 3 x up to 4096 tokens 546 us (338), a chunk of 1024 tokens over 32768 in E4M3 781 us (563), four
// drafts of each of 64 sequences of up to 8191 tokens 221 us (196), a window of 1024 over 256 channels 65 us (16).
// What bounds a prompt is the way of one stream's tile, about 3300 cycles for both streams' 2048 of products: scores,
// their maximum, the exponentials (512 of a softmax's 1900 cycles on the special-function pipe), the products' second half.
// Of registers there are 128 a thread, as 512 threads take all; a split by roles would free some, but the functions that stay
// out of line (copies of queries and of single tokens, rows that see nothing) cannot be called in a kernel that changes its
// registers, and code in line that the instruction cache does not hold is slow (163 KB took 1.14 to 1.17 times as long as 96).
#include <cuda.h>
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace chunk {

constexpr int kTile = 128;                    // tokens of a tile
constexpr int kRows = 128;                    // query rows of a stream (MMA M)
constexpr int kMaxCtas = 152;
// A block of rows costs about as much as kBlockTiles tiles on top of its own (queries, first scores, epilogue): the line that
// the CTAs share has as many places before its tiles. (A prompt's chunk among single tokens: 1 70.5 us, 2 63.7; prompts: 1 626,
// 2 590, 3 591 then.)
constexpr int kBlockTiles = 2;
// Places of the line that a CTA takes at least: a block of one tile has three, and is not cut. (20 tokens of 2 cache heads: 4
// 14.4 us, both blocks on one CTA, 2 10.4; 512 of 8: 24.4 and 21.6; 1512 of 8: 19.4 and 20.2, for more parts to join.)
constexpr int kMinPlaces = 2;
constexpr int kMaskBufs = 8;                  // tiles whose masks of seen tokens are kept
constexpr int kChunkBytes = 128 * 128;        // 64 channels of 128 rows, 128-byte swizzled

// warps: 0-3 and 4-7 the streams' softmax, 8-11 loaders, 12 and 13 issuers, 14 the list of pieces, 15 rows that see nothing
constexpr int kThreads = 512;

template <int DP, bool E4M3>
struct Cfg {
  static constexpr bool kWide = DP == 256;
  static constexpr int kStreams = kWide ? 1 : 2;
  static constexpr int kUnitCh = DP < 128 ? DP : 128;              // channels of a ring slot
  static constexpr int kHalves = DP / kUnitCh;                     // slots of a tile's keys, and of its values
  static constexpr int kUnitBytes = kUnitCh / 64 * kChunkBytes;
  static constexpr int kQBytes = DP / 64 * kChunkBytes;            // a stream's queries
  static constexpr int kSlots = DP == 64 ? 8 : kWide && !E4M3 ? 5 : 4;
  static constexpr int kLag = 1;                                   // E4M3: units in flight behind the newest
  static constexpr int kStages = kLag + 1;                         // raw units of a loader warp
  static_assert(kStages == 2, "barriers");
  static constexpr int kStageBytes = 32 * kUnitCh;
  static constexpr int kRingOff = kStreams * kQBytes;
  static constexpr int kRawOff = kRingOff + kSlots * kUnitBytes;
  static constexpr int kMiscOff = kRawOff + (E4M3 ? 4 * kStages * kStageBytes : 0);
  static constexpr int kPartRows = kStreams * kRows;
  static constexpr int kPartFloats = (2 + DP) * kPartRows;         // a part of a row block: bases, sums, O as [channel][row]
};

enum {
  kBarFull = 0,                  // [8] ring slot loaded
  kBarFree = 8,                  // [8] ring slot read by every product that takes it
  kBarQ = 16,                    // [2] a stream's queries loaded
  kBarScore = 18,                // [2] S of a tile computed (a stream's; wide: a buffer's)
  kBarProb = 20,                 // [2] P of a tile written, O rescaled if need be
  kBarOut = 22,                  // [2] O of a piece complete (wide: of a tile, even and odd ones)
  kBarOutFree = 24,              // [2] O of a piece read
  kBarPiece = 26,                // [4] piece listed
  kBarPieceFree = 30,            // [4] piece done with by all warps
  kBarBases = 34,                // bases and sums of a piece's two accumulators written, then read
  kBarTurn = 35,                 // [2] a stream's products issued: the other's turn
  kBarDrain = 37,                // [2]
  kBarHalf = 47,                 // [2] P of a tile's first 64 tokens
  kBarRaw = 39,                  // [4][2] E4M3: a loader warp's raw unit has come
  kBarPair = 49,                 // [4] wide: two softmax warps of the same rows have exchanged numbers
  kNumBars = 53
};
constexpr int kPieces = 4;       // pieces listed ahead
constexpr int kUsers = 14;       // warps that read them

// Where a CTA's share of the line begins.
struct Share {
  int64_t total, x, x_end, first, seq;       // seq: places of a work row of sequence b
  int ctas, b, r, qt, place;
  int64_t sums[kThreads / 32];
};
// Some tiles of one block of rows: `n` tokens of a sequence's chunk, work row r. (tiles = 0: the share is done.)
struct Piece {
  int token, pos, n, r;          // the first token's row of q and position
  int head, blk;                 // of the work row: cache head, block of its query heads
  int row, len;                  // row of the tables, tokens that the sequence has
  int j0, tiles;                 // token at which the first tile begins
  int np;                        // CTAs that the block's tiles fall to, if its first one is here; else 0
};
struct Misc {
  unsigned long long bars[kNumBars];
  uint32_t tmem;
  int abort_flag;
  uint32_t issued[4];                        // units that a loader warp has asked for
  alignas(16) uint32_t masks[kMaskBufs][4];  // seen tokens of a tile
  Piece pieces[kPieces];
  union {
    float2 ml[2][kRows];                     // [stream] bases and sums of a piece's rows
    float pair[2][2][kRows];                 // wide: what the two threads of a row exchange
    Share share;                             // (before the roles part)
  };
};

// How the rows of a chunk fall into blocks: `tokens` tokens of up to 128 heads of a cache head's group a stream.
struct Blocks {
  int heads;      // query heads of a block (of the last one of a cache head: fewer), rows of a token
  int count;      // blocks of a cache head
  int tokens;     // tokens of a stream
};
__host__ __device__ __forceinline__ Blocks blocks_of(int group) {
  if (group <= kRows) return Blocks{group, 1, kRows / group};
  return Blocks{kRows, (group + kRows - 1) / kRows, 1};
}

__device__ __forceinline__ int tiles_of(int lo, int hi) { return hi > lo ? (hi - 1) / kTile + 1 - lo / kTile : 0; }
// Seen tokens [lo, hi) of the n tokens from the i-th of a chunk on.
__device__ __forceinline__ void seen_by(const ChunkParams& p, const ChunkRange& c, int i, int n, int& lo, int& hi) {
  const int first = c.base + i;
  hi = first + n;
  lo = p.window > 0 && first >= p.window ? first - p.window + 1 : 0;
  if (c.row < 0 || hi < 0) hi = 0;
}
// Places on the line.
__device__ __forceinline__ int places_of(int tiles) { return tiles > 0 ? tiles + kBlockTiles : 0; }
__device__ __forceinline__ int64_t places_of_row(const ChunkParams& p, const ChunkRange& c, int step) {
  int64_t sum = 0;
  for (int64_t i = 0; i < c.n; i += step) {
    int lo, hi;
    seen_by(p, c, static_cast<int>(i), static_cast<int>(min(int64_t(step), c.n - i)), lo, hi);
    sum += places_of(tiles_of(lo, hi));
  }
  return sum;
}
// (A division of 64 bits takes some hundred cycles, and a CTA does nothing else meanwhile: 32 bits where they do.)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (a >> 32 == 0 && b >> 32 == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
__device__ __forceinline__ int64_t cta_begin(int64_t total, int ctas, int c) { return divide(total * c, ctas); }
__device__ __forceinline__ int cta_of(int64_t total, int ctas, int64_t x) {
  return static_cast<int>(divide((x + 1) * ctas - 1, total));
}

// Fills *sh for CTA `cta` of `grid` (every thread calls it): sequence after sequence, their `rows` work rows (cache heads x
// head blocks) one after the other, each the places of its blocks of `step` tokens. False: no work. (In line: arguments by
// reference out of line are read through memory, and the first tile of a cold call comes 5000 cycles later.)
static __device__ __forceinline__ bool find_share(const ChunkParams& p, int cta, int grid, int rows, int step, Share* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t line = 0;                                   // places of the sequences before these
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      const int64_t n = b < p.batch ? places_of_row(p, chunk_range(p, b), step) : 0;
      int64_t pre = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += y;
      }
      __syncthreads();
      if (lane == 31) sh->sums[warp] = pre;
      __syncthreads();
      int64_t before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sh->sums[w];
        all += sh->sums[w];
      }
      const int64_t at = line + (before + pre - n) * rows;
      line += all * rows;
      if (pass == 0 && b0 + kThreads >= p.batch) {
        if (threadIdx.x < 2) {                          // begin and end
          int64_t ctas = line / kMinPlaces;
          ctas = ctas < 1 ? 1 : ctas > grid ? grid : ctas;
          const bool work = line > 0 && cta < ctas;
          const int64_t x = work ? cta_begin(line, static_cast<int>(ctas), cta + threadIdx.x) : 0;
          if (threadIdx.x == 0) {
            sh->total = line;
            sh->ctas = static_cast<int>(ctas);
            sh->x = x;
          } else {
            sh->x_end = x;
          }
        }
        __syncthreads();
        if (sh->x >= sh->x_end) return false;
      }
      // the sequence in which the share begins (one round of sequences: without a second pass)
      if ((pass == 1 || p.batch <= kThreads) && n > 0 && sh->x >= at && sh->x < at + n * rows) {
        sh->b = b;
        sh->first = at;
        sh->seq = n;
      }
      if (pass == 1 && sh->x < line) break;
    }
    if (p.batch <= kThreads) break;
  }
  __syncthreads();
  if (warp == 0) {
    // the work row, the block of tokens and the place in it
    const ChunkRange c = chunk_range(p, sh->b);
    int64_t y = sh->x - sh->first;
    const int64_t seq = sh->seq;
    int r = 0;                                          // work rows before it
    for (int more = 32; more == 32; r += more)
      more = __popc(__ballot_sync(0xffffffffu, r + lane + 1 < rows && (r + lane + 1) * seq <= y));
    y -= r * seq;
    for (int q0 = 0; q0 * int64_t(step) < c.n; q0 += 32) {
      const int64_t i = (q0 + lane) * int64_t(step);
      int lo, hi, n = 0;
      if (i < c.n) {
        seen_by(p, c, static_cast<int>(i), min(step, c.n - static_cast<int>(i)), lo, hi);
        n = places_of(tiles_of(lo, hi));
      }
      int64_t pre = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += v;
      }
      if (y < pre && y >= pre - n) {
        sh->r = r;
        sh->qt = q0 + lane;
        sh->place = static_cast<int>(y - (pre - n));
      }
      const int64_t sum = __shfl_sync(0xffffffffu, pre, 31);
      if (y < sum) break;
      y -= sum;
    }
  }
  __syncthreads();
  return true;
}

// A walk through a CTA's share.
struct Walk {
  int64_t x, x_end, total;
  ChunkRange c;
  int b, r, qt, place, ctas;
  __device__ __forceinline__ void start(const ChunkParams& p, const Share& sh) {
    x = sh.x;
    x_end = sh.x_end;
    total = sh.total;
    ctas = sh.ctas;
    b = sh.b;
    r = sh.r;
    qt = sh.qt;
    place = sh.place;
    c = chunk_range(p, b);
  }
  __device__ __forceinline__ bool next(const ChunkParams& p, int rows, int step, int count, Piece& o) {
    while (x < x_end) {
      const int64_t i = qt * int64_t(step);
      if (i >= c.n) {                              // the next work row, or sequence
        qt = 0;
        if (++r >= rows || c.n == 0) {
          r = 0;
          if (++b >= p.batch) return false;
          c = chunk_range(p, b);
        }
        continue;
      }
      o.n = min(step, c.n - static_cast<int>(i));
      int lo, hi;
      seen_by(p, c, static_cast<int>(i), o.n, lo, hi);
      const int ntiles = tiles_of(lo, hi);
      ++qt;
      if (ntiles == 0) continue;
      const int64_t tile0 = x - place + kBlockTiles;   // line position of the block's first tile
      const int from = max(0, place - kBlockTiles);
      const int to = static_cast<int>(max(int64_t(0), min(int64_t(ntiles), x_end - tile0)));
      x = min(x_end, tile0 + ntiles);
      place = 0;
      if (to <= from) continue;                        // the share ends before its tiles
      o.token = c.first + static_cast<int>(i);
      o.pos = c.base + static_cast<int>(i);
      o.r = r;
      o.head = r / count;
      o.blk = r - o.head * count;
      o.row = c.row;
      o.len = c.base + c.n;
      o.j0 = (lo / kTile + from) * kTile;
      o.tiles = to - from;
      o.np = from > 0 ? 0 : tile0 + ntiles <= x_end ? 1 : cta_of(total, ctas, tile0 + ntiles - 1) - static_cast<int>(blockIdx.x) + 1;
      return true;
    }
    return false;
  }
};

// Pages as a tensor of (channels, heads, tokens of a page, pages), in boxes of 64 channels (E4M3: a unit's) of `rows` tokens
// (0: none, see page_maps).
struct PageMaps {
  CUtensorMap k, v;
  int rows;
};

// What a CTA left for the join: a block of rows that starts in it and goes on in the next np - 1.
struct Record {
  int32_t np, token, n, r;                        // first token of q, tokens, work row
  int32_t none;                                   // not 0: an output of this CTA is infinite or no number
};

// ---------------------------------------------------------------------------
// tensor memory and tcgen05
// ---------------------------------------------------------------------------
// One lane of the warp. (Behind this instruction, unlike a comparison of the lane's number, the compiler keeps addresses and
// descriptors in uniform registers: eight products issued beside two softmax warps take 413 cycles, else 699.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Operand tiles are rows of 128 bytes in 128-byte swizzle, 8-row groups of 1024 bytes. K-major (rows along M or N, 64
// channels of the reduction a row): groups follow each other along the rows. N-major (rows along the reduction, 64 channels
// of N a row): groups follow each other along the reduction, the next 64 channels are a chunk further.
// (A descriptor's upper word is the same for all; the lower one's address advances in 16 bytes.)
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr) { return (addr & 0x3FFFFu) >> 4 | static_cast<uint32_t>(kChunkBytes >> 4) << 16; }
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}
// A in tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}
// A thread's lane and N columns from `addr` on.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15"
      "}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
      "%28,%29,%30,%31"
      "}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
// 16 lanes x 32 columns as fragments: registers 4j, 4j + 1 hold lane t / 4, columns 8j + 2 (t % 4), + 1 (thread t),
// registers 4j + 2, 4j + 3 the same of lane t / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_frags(uint32_t (&r)[2][16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(r[k >> 4][k & 15]));
}
// Word w[k] of lane i of four goes to word w[i] of lane k.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4], int i) {
  const bool odd = i & 1, high = i & 2;
  uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1), b = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
  if (odd) w[0] = a, w[2] = b;
  else w[1] = a, w[3] = b;
  a = __shfl_xor_sync(0xffffffffu, high ? w[0] : w[2], 2), b = __shfl_xor_sync(0xffffffffu, high ? w[1] : w[3], 2);
  if (high) w[0] = a, w[1] = b;
  else w[2] = a, w[3] = b;
}
// tmem_ld32's loads are there: nothing reads them before.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32], uint32_t (&r2)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(r[k]), "+r"(r2[k]));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31,%32"
      "};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
        "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16"
      "};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
        "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// kind::f16, FP32 accumulator, M = 128; bit 16: B N-major.
__device__ __forceinline__ uint32_t instr_desc(bool f16, int n, bool n_major) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kRows >> 4) << 24) | (n_major ? 1u << 16 : 0u);
}

// d (+)= A B^T over `steps` (1 .. MOST) times 16 channels, both K-major. A thread issues a product every 67 cycles, with a
// branch before each every 147 (a product takes 64): each number of steps has a sequence of its own.
template <int STEPS>
__device__ __forceinline__ void score_products(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const uint32_t off = (k >> 2) * (kChunkBytes >> 4) + 2 * (k & 3);       // 16 channels = 32 bytes a step
    tc_mma(d, a + off, b + off, idesc, accumulate || k > 0 ? 1u : 0u);
  }
}
template <int MOST>
__device__ __forceinline__ void score_steps(int steps, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  if (steps == MOST) return score_products<MOST>(d, a, b, idesc, accumulate);
  if constexpr (MOST > 1) score_steps<MOST - 1>(steps, d, a, b, idesc, accumulate);
}

// ---------------------------------------------------------------------------
// arithmetic
// ---------------------------------------------------------------------------
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two FP32 numbers an instruction: the same pipe time, half the issue slots, for which the CTA's warps compete.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(x));
  lo = __uint_as_float(a);
  hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {           // (a NaN is passed over)
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t word, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(word));
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
// Bits below x of a word of 32.
__device__ __forceinline__ uint32_t bits_below(int x) { return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u; }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// A warp's 32 rows of queries on their way to shared memory (first row's chunk at qs); off: the lane's row in q, -1: zeros.
template <int DP>
static __device__ __noinline__ void load_queries(const uint16_t* q, int dim, uint32_t qs, int64_t off, bool any) {
  const int lane = threadIdx.x & 31;
  if (any) {
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
      const int r = j * 4 + (lane >> 3);
      const int64_t o = __shfl_sync(0xffffffffu, off, r);
      const uint32_t to = qs + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        const int ch = c * 64 + (lane & 7) * 8;
        if (ch < dim) cp_async16(to + c * kChunkBytes, q + (o >= 0 ? o + ch : 0), o >= 0 ? 16 : 0);
      }
    }
  }
  cp_async_commit();
}
// They have come: negated where the scale is negative; E4M3: in FP16, a row scaled by a power of two. -> the row's factor of
// the scores.
template <bool E4M3>
static __device__ __noinline__ float finish_queries(int dim, uint32_t qs, float abs_scale, bool negate) {
  const int lane = threadIdx.x & 31;
  cp_async_wait<0>();
  __syncwarp();
  float factor = abs_scale;
  const uint32_t row = qs + lane * 128;
  auto at = [&](int c16) { return row + (c16 >> 3) * kChunkBytes + (((c16 & 7) ^ (lane & 7)) << 4); };
  const uint32_t flip = negate ? 0x80008000u : 0u;
  if (E4M3) {
    float top = 0.f;
#pragma unroll 4
    for (int c = 0; c < dim / 8; ++c) {
      const uint4 v = lds128(at(c));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u))));
    }
    // top in [2^e, 2^(e+1)): scale by 2^(15-e) (two factors, each a normal number for any e), to below 2^16, where the FP16
    // range ends: channels keep their eight bits down to 2^-32 of the largest, and end at 2^-40 of it
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    if (top == 0.f || e > 127) e = 15;
    e = max(e, -126) - 15;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23);
    const float down2 = __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
    factor = fmaxf(abs_scale * __uint_as_float(static_cast<uint32_t>(127 + e / 2) << 23) *
                       __uint_as_float(static_cast<uint32_t>(127 + (e - e / 2)) << 23),
                   1.2e-38f);
#pragma unroll 2
    for (int c = 0; c < dim / 8; ++c) {
      const uint4 v = lds128(at(c));
      uint32_t w[4] = {v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack_f16x2_rn(__uint_as_float(w[j] << 16) * down * down2, __uint_as_float(w[j] & 0xffff0000u) * down * down2);
      sts128(at(c), w[0], w[1], w[2], w[3]);
    }
  } else if (negate) {
    for (int c = 0; c < dim / 8; ++c) {
      const uint4 v = lds128(at(c));
      sts128(at(c), v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  return factor;
}

// 32 tokens of a unit one by one: the lane's at off in the pages (elements, -1: zeros), to the rows from dst on. E4M3: as they
// are, row behind row.
template <int CHANNELS>
static __device__ __noinline__ void load_raw_tokens(const uint8_t* src, int dim, int ch0, int64_t off, uint32_t dst) {
  constexpr int kPer = CHANNELS / 16;
  const int lane = threadIdx.x & 31, ch = ch0 + lane % kPer * 16;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t o = __shfl_sync(0xffffffffu, off, k * (32 / kPer) + lane / kPer);
    const bool have = o >= 0 && ch < dim;
    cp_async16(dst + k * 512 + lane * 16, src + (have ? o + ch : 0), have ? 16 : 0);
  }
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
}
template <int CHANNELS>
static __device__ __noinline__ void load_tokens(const uint8_t* src, int dim, int ch0, int64_t off, uint32_t dst) {
  const int lane = threadIdx.x & 31;
  const uint32_t to = dst + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);                  // rows 4 k + lane / 8
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t o = __shfl_sync(0xffffffffu, off, k * 4 + (lane >> 3));
    // (row 4 k + i: its swizzle is row i's with bit 2 flipped for odd k)
    const uint32_t at = (to + k * 512) ^ ((k & 1) << 6);
#pragma unroll
    for (int c = 0; c < CHANNELS / 64; ++c) {
      const int ch = ch0 + c * 64 + (lane & 7) * 8;
      if (ch < dim) cp_async16(at + c * kChunkBytes, src + (o >= 0 ? (o + ch) * 2 : 0), o >= 0 ? 16 : 0);
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  fence_proxy_async_smem();
  __syncwarp();
}

// Rows that stand before their sequence's first token, or have none: zeros and -infinity, spread over the CTAs (a warp of each).
static __device__ __noinline__ void zero_unseeing(const ChunkParams& p) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const ChunkRange c = b0 + lane < p.batch ? chunk_range(p, b0 + lane) : ChunkRange{-1, 0, 0, 0};
    const int n = c.row < 0 ? c.n : c.base < 0 ? min(c.n, -c.base) : 0;
#pragma unroll 1
    for (uint32_t m = __ballot_sync(0xffffffffu, n > 0); m != 0; m &= m - 1) {
      const int first = __shfl_sync(0xffffffffu, c.first, __ffs(m) - 1), count = __shfl_sync(0xffffffffu, n, __ffs(m) - 1);
#pragma unroll 1
      for (int i = blockIdx.x; i < count; i += gridDim.x) {
        const int64_t row = int64_t(first + i) * p.heads;
        uint4* out = reinterpret_cast<uint4*>(p.out + row * p.dim);
#pragma unroll 1
        for (int e = lane; e < p.heads * (p.dim / 8); e += 32) out[e] = make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr)
          for (int h = lane; h < p.heads; h += 32) p.lse[row + h] = -INFINITY;
      }
    }
  }
}

// A row of this CTA's outputs has a channel that is infinite or no number (a call: rare, and out of the way of the code around it).
static __device__ __noinline__ void flag_none(Record* records) { atomicExch(&records[blockIdx.x].none, 1); }

template <int DP, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ PageMaps maps,
                                                            Record* records, float* parts) {
  using C = Cfg<DP, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& misc = *reinterpret_cast<Misc*>(smem + C::kMiscOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem), bars = smem_u32(misc.bars);
  auto bar = [&](int i) { return bars + 8 * i; };
  volatile int* abort_flag = &misc.abort_flag;
  const Blocks blocks = blocks_of(p.group);
  const int rows = p.kv_heads * blocks.count, step = C::kStreams * blocks.tokens;

  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    records[blockIdx.x].np = 0;
    records[blockIdx.x].none = 0;
  }
  // (set up while the others look for the share)
  if (warp == 12 && lane == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(bar(kBarFull + i), 4);
      mbar_init(bar(kBarFree + i), C::kStreams);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarQ + i), 4);
      mbar_init(bar(kBarScore + i), 1);
      mbar_init(bar(kBarProb + i), 4);
      mbar_init(bar(kBarHalf + i), 4);
      mbar_init(bar(kBarOut + i), 1);
      mbar_init(bar(kBarOutFree + i), 8);
      mbar_init(bar(kBarDrain + i), 1);
      mbar_init(bar(kBarTurn + i), 1);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(bar(kBarPiece + i), 1);
      mbar_init(bar(kBarPieceFree + i), C::kWide ? kUsers - 1 : kUsers);
    }
    mbar_init(bar(kBarBases), 8);
    for (int i = 0; i < 4; ++i) mbar_init(bar(kBarPair + i), 2);
    for (int i = 0; i < 8; ++i) mbar_init(bar(kBarRaw + i), 1);
    misc.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&misc.tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  const bool aligned = (base & 1023u) == 0;  // the swizzle is a function of address bits
  if (!aligned && threadIdx.x == 0) set_error(p.err, MOE_W4A16_ERR_CUDA);
  const bool work = find_share(p, blockIdx.x, gridDim.x, rows, step, &misc.share) && aligned;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&misc.tmem);
  if (!work) {
    if (warp == 15) zero_unseeing(p);
    if (warp == 13) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    return;
  }
  const uint32_t ring = base + C::kRingOff;
  auto wait = [&](int i, uint32_t parity) { return warp_wait(bar(i), parity, abort_flag, p.err, p.wait_ns); };
  // scores enter the exponentials as |scale| s, the queries negated where the scale is negative (zeroed where it is zero,
  // so that the factor itself is never zero: an unseen token's -infinity stays one)
  const bool flat = p.score_scale == 0.f, negate = p.score_scale < 0.f;
  const float abs_scale = flat ? 1.f : fmaxf(fabsf(p.score_scale), 1.2e-38f);
  constexpr int kAcc = 256;                              // columns: scores at 0 and 128, accumulators from 256 on

  Walk walk;
  if (warp == 14) walk.start(p, misc.share);
  __syncthreads();                                       // (the share's memory is the bases' from here on)
  // the k-th piece, listed by warp 14; freed once by each of the warps that read it
  auto piece = [&](uint32_t k) -> const Piece& { return misc.pieces[k % kPieces]; };
  auto piece_there = [&](uint32_t k) { return wait(kBarPiece + k % kPieces, (k / kPieces) & 1u); };
  auto piece_done = [&](uint32_t k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarPieceFree + k % kPieces));
  };

  if (warp < 8) {
    // ------------------------------------------------------------- softmax, a thread a row
    const int s = warp >> 2, rr = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    {
      const int trow = rr / blocks.heads, hrow = rr - trow * blocks.heads;   // token and head of the row
      const uint32_t qs = base + s * C::kQBytes + (warp & 3) * 32 * 128;     // this warp's 32 rows
      uint32_t n_score = 0, n_out[2] = {0, 0}, n_tile = 0, n_bases = 0, n_pair = 0, k = 0;
      auto split_of = [&](const Piece& x) { return C::kWide || x.n <= blocks.tokens; };
      // Whether this stream has tiles of a piece: queries and accumulators change hands for those alone (a phase that passes
      // without its issuer would be taken for the one before).
      auto has = [&](const Piece& x) { return x.tiles > (split_of(x) && !C::kWide ? s : 0); };
      // Wide: the two threads of a row trade x; false: a wait gave up.
      auto trade = [&](float& x) {
        misc.pair[n_pair & 1][s][rr] = x;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPair + (warp & 3)));
        if (!wait(kBarPair + (warp & 3), n_pair & 1u)) return false;
        x = misc.pair[n_pair++ & 1][s ^ 1][rr];
        return true;
      };
      // This thread's row of a block: token relative to the block's first (-1: none), query head.
      auto token_of = [&](const Piece& x) {
        const int t = trow + (s == 1 && !split_of(x) ? blocks.tokens : 0);   // (wide: both groups of warps have the same rows)
        return trow < blocks.tokens && t < x.n && x.blk * blocks.heads + hrow < p.group ? t : -1;
      };
      auto head_of = [&](const Piece& x) { return x.head * p.group + x.blk * blocks.heads + hrow; };
      // This thread's row as an offset in q (elements, -1: none), and its warp's rows on their way.
      auto load = [&](const Piece& x) {
        const int t = token_of(x);
        load_queries<DP>(p.q, p.dim, qs, t >= 0 && !flat ? int64_t(x.token + t) * p.q_stride + int64_t(head_of(x)) * p.dim : -1,
                         __any_sync(0xffffffffu, t >= 0));
      };
      auto finish = [&]() {
        const float factor = finish_queries<E4M3>(p.dim, qs, abs_scale, negate);
        if (lane == 0) mbar_arrive(bar(kBarQ + s));
        return factor;
      };

      bool ok = piece_there(0);
      float factor = 0.f;
      const bool loads = !C::kWide || s == 0;            // wide: the first group's warps bring the queries
      if (ok && has(piece(0)) && loads) {
        load(piece(0));
        factor = finish();
      }
      while (ok) {
        const int n = piece(k).tiles;
        if (n == 0 || !(ok = piece_there(k + 1))) break;
        const bool split = split_of(piece(k)), have_next = has(piece(k + 1)) && loads;
        const int token = token_of(piece(k)), pos = piece(k).pos + token, j_first = piece(k).j0;
        const bool active = __any_sync(0xffffffffu, token >= 0);
        const int stride = !C::kWide && split ? 2 : 1, first = stride == 2 ? s : 0;
        float m = -INFINITY, l = 0.f, next_factor = 0.f;
        if (C::kWide) {
          float x = factor;
          if (!(ok = trade(x))) break;
          if (s == 1) factor = x;
        }
        // what the exponents are taken against: a maximum that is taken when a score passes it by 2^kSlack. E4M3: FP16
        // probabilities of 2^kLift to 2^15, which keep their bits down to 2^-22 of the largest, and end at 2^-32 of it
        constexpr float kLift = E4M3 ? 8.f : 0.f, kSlack = E4M3 ? 7.f : 8.f;
        for (int i = first; i < n; i += stride, ++n_score) {
          const int buf = C::kWide ? n_score & 1 : s;
          const uint32_t par = C::kWide ? (n_score >> 1) & 1u : n_score & 1u;
          const uint32_t score = tmem + buf * 128 + lanes;
          if (!(ok = wait(kBarScore + buf, par))) break;
          tc_fence_after();
          if (i + stride >= n && have_next) load(piece(k + 1));      // the last product with these is done
          if (C::kWide) {
            // a thread has half of a row's tokens, in registers from the scores to the probabilities
            if (active) {
              uint32_t x[32], y[32];
              tmem_ld32(score + 64 * s, x);
              tmem_ld32(score + 64 * s + 32, y);
              const uint32_t* seen = misc.masks[(n_tile + i) % kMaskBufs] + 2 * s;
              const uint32_t seen0 = seen[0], seen1 = seen[1];
              const int j0 = j_first + i * kTile + 64 * s;
              const int above = pos - j0 + 1, below = p.window > 0 && pos >= p.window ? pos - p.window + 1 - j0 : 0;
              const bool part = __any_sync(0xffffffffu, above < 64 || below > 0 || (seen0 & seen1) != 0xffffffffu);
              tmem_wait_ld(x, y);
              if (part) {
                const uint32_t w0 = seen0 & bits_below(above) & ~bits_below(below);
                const uint32_t w1 = seen1 & bits_below(above - 32) & ~bits_below(below - 32);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  if (!(w0 >> j & 1u)) x[j] = 0xff800000u;
                  if (!(w1 >> j & 1u)) y[j] = 0xff800000u;
                }
              }
              float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int e = 0; e < 32; e += 4)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  top4[j] = max3(top4[j], __uint_as_float(x[e + 2 * j]), __uint_as_float(x[e + 2 * j + 1]));
                  top4[2 + j] = max3(top4[2 + j], __uint_as_float(y[e + 2 * j]), __uint_as_float(y[e + 2 * j + 1]));
                }
              const float mine = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
              float top = mine;
              // (from here on the other's scores have been read too: its probabilities may lie over them)
              if (!(ok = trade(top))) break;
              top = fmaxf(top, mine) * factor;
              const bool over = top > m + kSlack;
              if (__any_sync(0xffffffffu, over)) {
                float keep = 1.f;
                if (over) {
                  keep = exp2_fast(m - top);
                  m = top;
                }
                l *= keep;
                if (i != first) {
                  if (!(ok = wait(kBarOut + ((n_score - 1) & 1), ((n_score - 1) >> 1) & 1u))) break;
                  tc_fence_after();
#pragma unroll 1
                  for (int c = 16 * s; c < p.dim; c += 32) {                 // each thread half of the channels
                    uint32_t o[16];
                    tmem_ld16(tmem + kAcc + lanes + c, o);
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                    tmem_st16(tmem + kAcc + lanes + c, o);
                  }
                }
              }
              const float off = kLift - (m == -INFINITY ? 0.f : m);
              uint64_t sums[2] = {0, 0};
              const uint64_t factor2 = pack2(__float_as_uint(factor), __float_as_uint(factor)),
                             off2 = pack2(__float_as_uint(off), __float_as_uint(off));
              uint32_t packed[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const uint32_t a = j < 16 ? x[2 * j & 31] : y[2 * j & 31], b = j < 16 ? x[(2 * j + 1) & 31] : y[(2 * j + 1) & 31];
                float e0, e1;
                unpack2(fma2(pack2(a, b), factor2, off2), e0, e1);
                e0 = exp2_fast(e0);
                e1 = exp2_fast(e1);
                sums[j & 1] = add2(sums[j & 1], pack2(__float_as_uint(e0), __float_as_uint(e1)));
                packed[j] = E4M3 ? pack_f16x2_rn(e0, e1) : pack_bf16x2_rn(e0, e1);
              }
              tmem_st32(score + 32 * s, packed);
              tmem_wait_st();
              float sum_lo, sum_hi;
              unpack2(add2(sums[0], sums[1]), sum_lo, sum_hi);
              l += sum_lo + sum_hi;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar((s == 0 ? kBarHalf : kBarProb) + buf));
          } else if (active) {
            uint32_t x[32], y[32];
            // the second half for its maximum, then the first, which stays in registers for the exponentials
            tmem_ld32(score + 64, x);
            tmem_ld32(score + 96, y);
            const uint4 seen4 = lds128(smem_u32(misc.masks[(n_tile + i) % kMaskBufs]));
            const int j0 = j_first + i * kTile;
            const int above = pos - j0 + 1;                                  // tokens of the tile up to the row's own
            const int below = p.window > 0 && pos >= p.window ? pos - p.window + 1 - j0 : 0;
            const bool part = __any_sync(0xffffffffu, above < kTile || below > 0 ||
                                                          (seen4.x & seen4.y & seen4.z & seen4.w) != 0xffffffffu);
            float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto maxima = [&](const uint32_t (&r)[32]) {
#pragma unroll
              for (int e = 0; e < 32; e += 8)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  top4[j] = max3(top4[j], __uint_as_float(r[e + 2 * j]), __uint_as_float(r[e + 2 * j + 1]));
            };
            if (!part) {                                                     // (a straight line: 539 us for the prompts, else 549)
              tmem_wait_ld(x, y);
              maxima(x);
              tmem_ld32(score, x);
              maxima(y);
              tmem_ld32(score + 32, y);
              tmem_wait_ld(x, y);
              maxima(x);
              maxima(y);
            } else {                                                         // tokens that the row does not see at -infinity
#pragma unroll 1
              for (int half = 1; half >= 0; --half) {
                tmem_wait_ld(x, y);
                const uint32_t w0 = (half ? seen4.z : seen4.x) & bits_below(above - 64 * half) & ~bits_below(below - 64 * half);
                const uint32_t w1 = (half ? seen4.w : seen4.y) & bits_below(above - 64 * half - 32) & ~bits_below(below - 64 * half - 32);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  if (!(w0 >> j & 1u)) x[j] = 0xff800000u;
                  if (!(w1 >> j & 1u)) y[j] = 0xff800000u;
                }
                if (half) {
                  tmem_st32(score + 64, x);
                  tmem_st32(score + 96, y);
                  tmem_wait_st();
                }
                maxima(x);
                maxima(y);
                if (half) {
                  tmem_ld32(score, x);
                  tmem_ld32(score + 32, y);
                }
              }
            }
            const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * factor;
            const bool over = top > m + kSlack;                              // (m of -infinity: any seen score)
            if (__any_sync(0xffffffffu, over)) {
              float keep = 1.f;
              if (over) {
                keep = exp2_fast(m - top);
                m = top;
              }
              l *= keep;
              if (i != first) {
                const uint32_t acc = tmem + kAcc + s * 128 + lanes;
#pragma unroll 1
                for (int c = 0; c < p.dim; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(acc + c, o);
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                  tmem_st16(acc + c, o);
                }
              }
            }
            const float off = kLift - (m == -INFINITY ? 0.f : m);
            uint64_t sums[2] = {0, 0};
            const uint64_t factor2 = pack2(__float_as_uint(factor), __float_as_uint(factor)),
                           off2 = pack2(__float_as_uint(off), __float_as_uint(off));
            auto exponentials = [&](const uint32_t (&r)[32], int q) {
              uint32_t packed[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float e0, e1;
                unpack2(fma2(pack2(r[2 * j], r[2 * j + 1]), factor2, off2), e0, e1);
                e0 = exp2_fast(e0);
                e1 = exp2_fast(e1);
                sums[j & 1] = add2(sums[j & 1], pack2(__float_as_uint(e0), __float_as_uint(e1)));
                packed[j] = E4M3 ? pack_f16x2_rn(e0, e1) : pack_bf16x2_rn(e0, e1);
              }
              tmem_st16(score + 16 * q, packed);                             // (over scores that have been read)
            };
            exponentials(x, 0);
            tmem_ld32(score + 64, x);
            exponentials(y, 1);
            tmem_ld32(score + 96, y);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarHalf + buf));
            tmem_wait_ld(x, y);
            exponentials(x, 2);
            exponentials(y, 3);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarProb + buf));
            float sum_lo, sum_hi;
            unpack2(add2(sums[0], sums[1]), sum_lo, sum_hi);
            l += sum_lo + sum_hi;
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(kBarHalf + buf));
              mbar_arrive(bar(kBarProb + buf));
            }
          }
        }
        if (!ok) break;
        if (have_next && first < n) next_factor = finish();

        // ---- epilogue: O / l, or a part of it
        const Piece& pc = piece(k);
        const bool whole = pc.np == 1;
        const bool two = !C::kWide && split;             // both streams hold accumulators of the same rows
        float f0 = 1.f, f1 = 0.f;
        m -= kLift;
        if (C::kWide) {
          float other = l;
          if (!(ok = trade(other))) break;
          l += other;
        }
        if (two) {
          misc.ml[s][rr] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarBases));
          if (!(ok = wait(kBarBases, n_bases++ & 1u))) break;
          const float2 a = misc.ml[0][rr], b = misc.ml[1][rr];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarBases));
          if (!(ok = wait(kBarBases, n_bases++ & 1u))) break;                // read before the next piece's are written
          if (first >= n && have_next) load(piece(k + 1));
          m = fmaxf(a.x, b.x);
          const float at = m == -INFINITY ? 0.f : m;
          f0 = exp2_fast(a.x - at);
          f1 = exp2_fast(b.x - at);
          l = a.y * f0 + b.y * f1;
        }
        if (C::kWide) {                                  // (the last tile's product)
          ok = wait(kBarOut + ((n_score - 1) & 1), ((n_score - 1) >> 1) & 1u);
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (!two || q < n) {
              if (ok && (two || q == s)) ok = wait(kBarOut + q, n_out[q] & 1u);
              ++n_out[q];
            }
        }
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const bool valid = token >= 0;
          const int64_t out_row = int64_t(pc.token + token) * p.heads + head_of(pc);
          float* part = parts + (int64_t(blockIdx.x) * 2 + (pc.np > 0 ? 1 : 0)) * C::kPartFloats +
                        (two || C::kWide ? rr : s * kRows + rr);
          if (valid && ((!two && !C::kWide) || s == 0)) {
            if (!whole) {
              __stcg(part, m);
              __stcg(part + C::kPartRows, l);
            } else if (p.lse != nullptr) {
              p.lse[out_row] = (m + log2f(l)) * 0.69314718055994531f;
            }
          }
          const float inv = whole ? (l == 0.f ? 0.f : p.v_scale / l) : 1.f;
          f0 *= inv;
          f1 *= inv;
          const int half = (p.dim + 63) / 64 * 32;       // shared rows: half of the channels each
          const bool shared = two || C::kWide;
          const int from = shared && s == 1 ? half : 0, to = shared && s == 0 ? half : p.dim;
          const bool second = two && n > 1;
          if (whole) {
            // Fragments of 16 rows x 32 columns; the four lanes of a row trade words, so that each stores 16 bytes of the
            // 64 that are theirs (a thread a row stores to 32 lines at once, four times as long). A lane has rows lane / 4 + 8 q.
            float g0[4], g1[4];
            int64_t at[4];
            uint32_t none = 0u;             // of its channels: zeros, or no numbers (repair_kernel's)
            const int64_t off = valid ? out_row * p.dim : -1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int r = 8 * q + (lane >> 2);
              g0[q] = __shfl_sync(0xffffffffu, f0, r);
              g1[q] = __shfl_sync(0xffffffffu, f1, r);
              at[q] = __shfl_sync(0xffffffffu, off, r);
            }
#pragma unroll 1
            for (int c = from; c < to; c += 32) {
              uint32_t o[2][16];
              const uint32_t acc = tmem + kAcc + (shared ? 0 : s * 128) + c + lanes;
              tmem_ld_frag(acc, o[0]);
              tmem_ld_frag(acc + (16u << 16), o[1]);
              tmem_wait_frags(o);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                o[j >> 4][j & 15] = __float_as_uint(__uint_as_float(o[j >> 4][j & 15]) * g0[2 * (j >> 4) + (j >> 1 & 1)]);
              if (second) {
                uint32_t o1[2][16];
                tmem_ld_frag(acc + 128, o1[0]);
                tmem_ld_frag(acc + 128 + (16u << 16), o1[1]);
                tmem_wait_frags(o1);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  o[j >> 4][j & 15] = __float_as_uint(fmaf(__uint_as_float(o1[j >> 4][j & 15]), g1[2 * (j >> 4) + (j >> 1 & 1)],
                                                           __uint_as_float(o[j >> 4][j & 15])));
              }
              const int ch = c + 8 * (lane & 3);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  w[j] = pack_bf16x2_rn(__uint_as_float(o[q >> 1][4 * j + 2 * (q & 1)]), __uint_as_float(o[q >> 1][4 * j + 2 * (q & 1) + 1]));
                transpose4(w, lane & 3);
                if (at[q] >= 0 && ch < p.dim) {
                  *reinterpret_cast<uint4*>(p.out + at[q] + ch) = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
                  for (int j = 0; j < 4; ++j) none = fma_bf16x2(w[j], 0u, none);
                }
              }
            }
            if ((none & 0x7fff7fffu) != 0u) flag_none(records);
          } else {
            float zero = 0.f;
#pragma unroll 1
            for (int c = from; c < min(to, p.dim); c += 16) {
              uint32_t o[16];
              tmem_ld16(tmem + kAcc + (shared ? 0 : s * 128) + c + lanes, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f0);
              if (second) {
                uint32_t o1[16];
                tmem_ld16(tmem + kAcc + 128 + c + lanes, o1);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(fmaf(__uint_as_float(o1[j]), f1, __uint_as_float(o[j])));
              }
              if (valid) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  __stcg(part + (2 + c + j) * C::kPartRows, __uint_as_float(o[j]));
                  zero = fmaf(__uint_as_float(o[j]), 0.f, zero);
                }
              }
            }
            if (zero != 0.f) flag_none(records);
          }
        }
        if (pc.np > 1 && threadIdx.x == 0) {
          Record& rec = records[blockIdx.x];               // (but for the flag)
          rec.np = pc.np;
          rec.token = pc.token;
          rec.n = pc.n;
          rec.r = pc.r;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (C::kWide) {
            mbar_arrive(bar(kBarOutFree));
          } else if (two) {
            mbar_arrive(bar(kBarOutFree));
            if (n > 1) mbar_arrive(bar(kBarOutFree + 1));
          } else {
            mbar_arrive_n(bar(kBarOutFree + s), 2);
          }
        }
        if (have_next && first >= n) next_factor = finish();
        n_tile += n;
        piece_done(k);
        ++k;
        factor = next_factor;
      }
      cp_async_wait<0>();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------- loaders: 32 tokens of every tile a warp, a lane a token
    const int w = warp - 8;
    bool ok = true;
    uint32_t unit = 0, n_tile = 0;
    auto slot_free = [&](uint32_t u) { return u < C::kSlots || wait(kBarFree + u % C::kSlots, (u / C::kSlots - 1) & 1u); };
    // ---- E4M3: a unit comes to a buffer of the warp's own, kLag units ahead, and is converted on its way to the ring
    constexpr int kRawPer = C::kUnitCh / 16, kRawRows = 32 / kRawPer;        // lanes of a row, rows of an access
    const uint32_t raw = base + C::kRawOff + w * C::kStages * C::kStageBytes + lane * 16;
    auto raw_bar = [&](uint32_t u) { return kBarRaw + 2 * w + static_cast<int>(u % C::kStages); };
    auto convert = [&](uint32_t u) {
      if (!(ok = wait(raw_bar(u), (u / C::kStages) & 1u)) || !(ok = slot_free(u))) return;
      const uint32_t from = raw + u % C::kStages * C::kStageBytes, dst = ring + u % C::kSlots * C::kUnitBytes + w * 32 * 128;
      const int c = lane % kRawPer;                                          // 16 channels: half a 64-byte part of a chunk
      const bool swap = c >> 2 & 1;                                          // (the two stores on different banks)
      constexpr int kBatch = 4;                                              // reads in flight together
#pragma unroll 1
      for (int k0 = 0; k0 < 32 / kRawRows; k0 += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) v[k] = lds128(from + (k0 + k) * 512);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int r = (k0 + k) * kRawRows + lane / kRawPer;
          uint32_t h[8];
          const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) e4m3x4_to_f16x4(x[j], h[2 * j], h[2 * j + 1]);
          const uint32_t at = dst + (c >> 2) * kChunkBytes + r * 128 + (((2 * (c & 3)) ^ (r & 7)) << 4);
          if (swap) {                                                        // (the pair of a chunk of 16 bytes: bit 4)
            sts128(at ^ 16, h[4], h[5], h[6], h[7]);
            sts128(at, h[0], h[1], h[2], h[3]);
          } else {
            sts128(at, h[0], h[1], h[2], h[3]);
            sts128(at ^ 16, h[4], h[5], h[6], h[7]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarFull + u % C::kSlots));
    };
    // This lane's token of a tile: its page (-1: unseen) and place there; of the lane's box its first token's.
    struct Token {
      int page, at, box_page, box_at;
      bool all;                                                              // every lane's is seen
    };
    // Boxes of maps.rows tokens (8, 16 or 32), a lane a box (BF16: of 64 channels).
    const int boxes = maps.rows > 0 ? 32 / maps.rows : 1, box_row = (lane & (boxes - 1)) * maps.rows;
    // one unit: channels ch0 .. of the 32 tokens
    auto load_unit = [&](bool is_key, int head, int ch0, const Token& tok) {
      const bool by_box = tok.all && maps.rows > 0;
      const CUtensorMap* map = is_key ? &maps.k : &maps.v;
      auto offset = [&]() {
        return tok.page < 0 ? -1 : int64_t(tok.page) * p.page_stride + int64_t(tok.at) * p.token_stride + int64_t(head) * p.head_stride;
      };
      if (E4M3) {
        const uint32_t dst = raw - lane * 16 + unit % C::kStages * C::kStageBytes, there = bar(raw_bar(unit));
        if (by_box) {
          if (lane == 0) mbar_arrive_expect_tx(there, C::kStageBytes);
          __syncwarp();
          if (lane < boxes) tma_load_4d(dst + box_row * C::kUnitCh, map, ch0, head, tok.box_at, tok.box_page, there);
        } else {
          load_raw_tokens<C::kUnitCh>(static_cast<const uint8_t*>(is_key ? p.k : p.v), p.dim, ch0, offset(), dst);
          if (lane == 0) mbar_arrive(there);
        }
        if (unit >= C::kLag) convert(unit - C::kLag);
      } else {
        if (!(ok = slot_free(unit))) return;
        const uint32_t full = bar(kBarFull + unit % C::kSlots), dst = ring + unit % C::kSlots * C::kUnitBytes + w * 32 * 128;
        if (by_box) {
          const int chunks = min(C::kUnitCh / 64, (p.dim - ch0 + 63) / 64), c = lane / boxes;
          if (lane == 0) mbar_arrive_expect_tx(full, chunks * 32 * 128);
          __syncwarp();
          if (c < chunks) tma_load_4d(dst + c * kChunkBytes + box_row * 128, map, ch0 + c * 64, head, tok.box_at, tok.box_page, full);
        } else {
          load_tokens<C::kUnitCh>(static_cast<const uint8_t*>(is_key ? p.k : p.v), p.dim, ch0, offset(), dst);
          if (lane == 0) mbar_arrive(full);
        }
      }
      ++unit;
    };
    const int step_col = kTile / p.t.page_size, step_at = kTile % p.t.page_size;
    for (uint32_t piece_no = 0; ok; ++piece_no) {
      if (!(ok = piece_there(piece_no))) break;
      const Piece pc = piece(piece_no);
      const int n = pc.tiles;
      if (n == 0) break;
      const int32_t* table = p.t.tables + int64_t(pc.row) * p.t.table_stride;
      const int head = pc.head;
      // the lane's token, its column of the table and place in the page, a tile further with every step
      // (tokens behind the block's last are read with the others, its rows' masks hide them)
      int left = pc.len - (pc.j0 + 32 * w + lane);                           // tokens of the sequence from it on
      int col = (pc.j0 + 32 * w + lane) / p.t.page_size, at = (pc.j0 + 32 * w + lane) % p.t.page_size;
      int entry = left > 0 ? table[col] : -1;
      Token old{-1, 0, 0, 0, false};                                         // wide: of the tile before
      for (int i = 0; ok && i < n; ++i) {
        Token tok;
        tok.page = entry;
        tok.at = at;
        if (entry >= p.t.num_pages) {
          set_error(p.err, MOE_W4A16_ERR_BAD_INDEX);
          tok.page = -1;
        }
        left -= kTile;
        col += step_col;
        at += step_at;
        if (at >= p.t.page_size) {
          at -= p.t.page_size;
          ++col;
        }
        entry = i + 1 < n && left > 0 ? table[col] : -1;
        const uint32_t seen = __ballot_sync(0xffffffffu, tok.page >= 0);
        tok.all = seen == 0xffffffffu;
        tok.box_page = __shfl_sync(0xffffffffu, tok.page, box_row);
        tok.box_at = __shfl_sync(0xffffffffu, tok.at, box_row);
        if (lane == 0) misc.masks[(n_tile + i) % kMaskBufs][w] = seen;
        // in the order in which the products take them (wide: the next tile's keys before this one's values)
        const int values = C::kWide ? (i > 0) + (i == n - 1) : 1, units = C::kHalves * (1 + values);
#pragma unroll 1
        for (int k = 0; ok && k < units; ++k)
          load_unit(k < C::kHalves, head, k % C::kHalves * 128, C::kWide && i > 0 && k >= C::kHalves && k < 2 * C::kHalves ? old : tok);
        if (C::kWide) old = tok;
      }
      n_tile += n;
      piece_done(piece_no);
    }
    cp_async_wait<0>();
    if (lane == 0) misc.issued[w] = unit;
    if (E4M3 && unit > 0) {
      if (ok) convert(unit - 1);
      if (!ok)                                               // a wait gave up: what is in flight lands before the CTA ends
        for (uint32_t u = unit > 1 ? unit - 2 : 0; u < unit; ++u) mbar_drain(bar(raw_bar(u)), (u / C::kStages) & 1u);
    }
  } else {
    // ------------------------------------------------------------- issuers
    const int s = warp - 12;
    if (s < C::kStreams) {
      bool ok = true;
      const uint32_t score_desc = instr_desc(E4M3, kTile, false);
      uint32_t n_prob = 0, n_piece = 0, n_own = 0, n_tile = 0, unit = 0, n_turn = 0;
      const int steps = p.dim / 16;
      auto full = [&](uint32_t u) { return wait(kBarFull + u % C::kSlots, (u / C::kSlots) & 1u); };
      auto free_unit = [&](uint32_t u) { tc_commit(bar(kBarFree + u % C::kSlots)); };
      // the products of S = Q K^T with the unit u (half h of a tile's keys), into column d
      auto score = [&](uint32_t u, int h, uint32_t d) {
        const uint32_t a = smem_desc(base + s * C::kQBytes + h * 2 * kChunkBytes);
        const uint32_t b = smem_desc(ring + u % C::kSlots * C::kUnitBytes);
        score_steps<C::kUnitCh / 16>(min(C::kUnitCh / 16, steps - h * 8), d, a, b, score_desc, h > 0);
      };
      // the products of O (+)= P V with the unit u (half h of a tile's values)
      auto value = [&](uint32_t u, int h, uint32_t prob, bool accumulate, int half) {
        const uint32_t desc = instr_desc(E4M3, min(p.dim - 128 * h, 128), true);
        const uint32_t b = smem_desc(ring + u % C::kSlots * C::kUnitBytes) + half * 512;
#pragma unroll
        for (int k = 0; k < kTile / 32; ++k)                                 // 16 tokens = two 1024-byte groups a step
          tc_mma_ts(tmem + kAcc + s * 128 + h * 128, prob + 32 * half + 8 * k, b + k * 128, desc, accumulate || k > 0 ? 1u : 0u);
      };
      while (ok) {
        if (!(ok = piece_there(n_piece))) break;
        const int n = piece(n_piece).tiles;
        const bool split = piece(n_piece).n <= blocks.tokens;
        if (n == 0) break;
        const bool own = n > (split && !C::kWide ? s : 0);   // tiles of this stream
        if (own && !(ok = wait(kBarQ + s, n_own & 1u))) break;
        bool freed = n_own == 0;                             // the accumulator, read by the piece before
        auto acc_free = [&]() {
          if (!freed) ok = wait(kBarOutFree + s, (n_own - 1) & 1u);
          freed = true;
          return ok;
        };
        if (!C::kWide) {
          const int stride = split ? 2 : 1, first = split ? s : 0;
          const uint32_t score_col = tmem + s * 128;
          auto keys_of = [&](int i) { return 2 * (n_tile + i); };
          // A tile of the other stream: its units are waited for and given back all the same, so that every phase of a slot is
          // seen by both issuers (a parity tells two phases apart, not three).
          auto pass = [&](int i) {
            for (uint32_t u = keys_of(i); ok && u < keys_of(i) + 2; ++u) {
              ok = full(u);
              if (ok && lane == 0) mbar_arrive(bar(kBarFree + u % C::kSlots));
            }
            return ok;
          };
          // Both streams with the same tiles: their products are issued in turns, a tile's O += P V and next S of one, then of
          // the other. In no order, the tensor pipe takes them by turns one at a time, both streams get their scores
          // together and run their softmax against each other.
          auto my_turn = [&]() { return s == 0 ? n_turn == 0 || wait(kBarTurn + 1, (n_turn - 1) & 1u) : wait(kBarTurn, n_turn & 1u); };
          if (split && s == 1) pass(0);
          // Step i: O += P V of tile i (none in the first step), S of the next. A stream of its own tiles waits for all that
          // both take before P, and issues them together: the softmax waits for the second. With every other tile, what
          // a product does not take is not waited for: the slots are given back early.
          for (int i = first - stride; ok && i < n; i += stride) {
            const bool values = i >= first, scores = i + stride < n;
            const uint32_t v = keys_of(i) + 1, q = keys_of(i + stride);
            if (values && !(acc_free() && (ok = full(v)))) break;
            if (!split && scores && !(ok = full(q))) break;
            if (!split && !(ok = my_turn())) break;
            if (values) {
              if (!(ok = wait(kBarHalf + s, n_prob & 1u))) break;
              tc_fence_after();
              if (elect_one()) value(v, 0, score_col, i != first, 0);
              if (!(ok = wait(kBarProb + s, n_prob++ & 1u))) break;
              tc_fence_after();
              if (elect_one()) value(v, 0, score_col, true, 1);
            }
            tc_fence_after();
            if (split) {
              if (values && elect_one()) free_unit(v);
              if (values && !scores && elect_one()) tc_commit(bar(kBarOut + s));
              if (values && i + 1 < n && !pass(i + 1)) break;
              if (scores && !(ok = full(q))) break;
              tc_fence_after();
            }
            if (elect_one()) {
              if (scores) score(q, 0, score_col);
              if (!split) mbar_arrive(bar(kBarTurn + s));
              if (scores) {
                tc_commit(bar(kBarScore + s));
                free_unit(q);
              }
              if (values && !split) {
                free_unit(v);
                if (!scores) tc_commit(bar(kBarOut + s));
              }
            }
            __syncwarp();
            if (!split) ++n_turn;
          }
        } else {
          // scores one tile ahead; the units come in this order
          for (int i = 0; ok && i <= n; ++i) {
            if (i < n) {
              const uint32_t buf = (n_prob + (i > 0)) & 1;
#pragma unroll 1
              for (int h = 0; ok && h < C::kHalves; ++h, ++unit) {
                if (!(ok = full(unit))) break;
                tc_fence_after();
                if (elect_one()) {
                  score(unit, h, tmem + buf * 128);
                  if (h == C::kHalves - 1) tc_commit(bar(kBarScore + buf));
                  free_unit(unit);
                }
                __syncwarp();
              }
            }
            if (!ok || i == 0) continue;
            if (!acc_free() || !(ok = wait(kBarHalf + (n_prob & 1), (n_prob >> 1) & 1u)) || !(ok = wait(kBarProb + (n_prob & 1), (n_prob >> 1) & 1u))) break;
#pragma unroll 1
            for (int h = 0; ok && h < C::kHalves; ++h, ++unit) {
              if (!(ok = full(unit))) break;
              tc_fence_after();
              if (elect_one()) {
                value(unit, h, tmem + (n_prob & 1) * 128, i > 1, 0);
                value(unit, h, tmem + (n_prob & 1) * 128, true, 1);
                if (h == C::kHalves - 1) tc_commit(bar(kBarOut + (n_prob & 1)));
                free_unit(unit);
              }
              __syncwarp();
            }
            ++n_prob;
          }
        }
        if (!ok) break;
        n_tile += n;
        n_own += own;
        piece_done(n_piece);
        ++n_piece;
      }
      if (elect_one()) {
        tc_commit(bar(kBarDrain + s));
        mbar_drain(bar(kBarDrain + s), 0);
      }
    } else if (warp == 14) {
      // ----------------------------------------------------------- the list of pieces
      Piece pc;
      for (uint32_t k = 0;; ++k) {
        if (k >= kPieces && !wait(kBarPieceFree + k % kPieces, (k / kPieces - 1) & 1u)) break;
        const bool more = walk.next(p, rows, step, blocks.count, pc);
        if (!more) pc.tiles = 0;
        if (lane == 0) {
          misc.pieces[k % kPieces] = pc;
          mbar_arrive(bar(kBarPiece + k % kPieces));
        }
        __syncwarp();
        if (!more) break;
      }
    } else if (warp == 15) {
      zero_unseeing(p);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (!E4M3 && *abort_flag) {
    // a wait gave up: the boxes in flight land before the CTA ends (the loaders' missing arrivals made up for)
    if (warp >= 8 && warp < 12 && lane == 0) {
      const uint32_t last = max(max(misc.issued[0], misc.issued[1]), max(misc.issued[2], misc.issued[3]));
      for (uint32_t u = misc.issued[warp - 8]; u < last; ++u) mbar_arrive(bar(kBarFull + u % C::kSlots));
      for (uint32_t u = last > C::kSlots ? last - C::kSlots : 0; u < last; ++u)
        mbar_drain(bar(kBarFull + u % C::kSlots), (u / C::kSlots) & 1u);
    }
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the blocks of rows that cross CTAs: a thread a row and 16 channels, the parts in the order of their CTAs.
template <int DP, bool E4M3>
__global__ void __launch_bounds__(kRows) chunk_join_kernel(const ChunkParams p, const Record* records, const float* parts, int ctas) {
  using C = Cfg<DP, E4M3>;
  static_assert(kMaxCtas <= 2 * kRows, "a thread looks at two records");
  __shared__ int list[kMaxCtas], counts[2 * kRows / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool is[2];
  uint32_t found[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = i * kRows + threadIdx.x;
    is[i] = c < ctas && __ldcg(&records[c].np) > 1;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    found[i] = __ballot_sync(0xffffffffu, is[i]);
    if ((threadIdx.x & 31) == 0) counts[i * (kRows / 32) + threadIdx.x / 32] = __popc(found[i]);
  }
  __syncthreads();
  int count = 0;
#pragma unroll
  for (int g = 0; g < 2 * kRows / 32; ++g) {
    const int i = g / (kRows / 32);
    if (g % (kRows / 32) == threadIdx.x / 32 && is[i])
      list[count + __popc(found[i] & ((1u << (threadIdx.x & 31)) - 1u))] = i * kRows + threadIdx.x;
    count += counts[g];
  }
  __syncthreads();
  const Blocks blocks = blocks_of(p.group);
  const int cols = p.dim / 16;
  for (int item = blockIdx.x; item < count * C::kStreams * cols; item += gridDim.x) {
    const int c = list[item / (C::kStreams * cols)], rest = item % (C::kStreams * cols), s = rest / cols, ch = rest % cols * 16;
    const Record rec = records[c];
    if (s == 1 && rec.n <= blocks.tokens) continue;
    const int trow = threadIdx.x / blocks.heads, hrow = threadIdx.x % blocks.heads, t = trow + s * blocks.tokens;
    const int blk = rec.r % blocks.count, head = rec.r / blocks.count * p.group + blk * blocks.heads + hrow;
    const bool valid = trow < blocks.tokens && t < rec.n && blk * blocks.heads + hrow < p.group;
    const int64_t row = int64_t(rec.token + t) * p.heads + head;
    if (valid) {
      const int prow = s * kRows + threadIdx.x;
      auto part_at = [&](int i) { return parts + (int64_t(c + i) * 2 + (i == 0 ? 1 : 0)) * C::kPartFloats + prow; };
      float m = -INFINITY;
#pragma unroll 4
      for (int i = 0; i < rec.np; ++i) m = fmaxf(m, __ldcg(part_at(i)));
      const float at = m == -INFINITY ? 0.f : m;
      float l = 0.f, o[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = 0.f;
#pragma unroll 2
      for (int i = 0; i < rec.np; ++i) {
        const float* src = part_at(i);
        const float f = exp2_fast(__ldcg(src) - at);
        l = fmaf(f, __ldcg(src + C::kPartRows), l);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = fmaf(f, __ldcg(src + (2 + ch + k) * C::kPartRows), o[k]);
      }
      const float inv = l == 0.f ? 0.f : p.v_scale / l;
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
      uint4* dst = reinterpret_cast<uint4*>(p.out + row * p.dim + ch);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      if (ch == 0 && p.lse != nullptr) p.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

// ---------------------------------------------------------------------------
// values that are no numbers
// ---------------------------------------------------------------------------
// A product takes every token of a tile for every row, those that a row does not see with a probability of zero; a value there
// that is infinite or no number makes the row's sum one too. The first kernel flags such sums, and then the third looks
// through the outputs: if a token that some row of a block does not see has such a value, the rows that are none are computed
// again, token by token, 16 channels where one is, a CTA a row. That takes milliseconds for a long row, so it stands where nothing
// waits for it (GB300, one infinite value in the last token: 7.7 ms for 300 new of 65536 tokens, 8 heads of 128 channels, 0.12
// without it; 146 ms for 1024 new of 131072 in E4M3, 64 heads, 3.1 without; bound by the latency of the scores' reads).
// Where nothing is flagged its start and end are 0.8 us of the shortest call, 3 of drafts of 64 sequences, none of prompts (in
// the join, on a path that is not taken, the same code made calls 2 to 4 us longer), whatever its grid: one CTA an SM.
constexpr int kRepairThreads = 512, kRepairWarps = kRepairThreads / 32;
struct RepairShared {
  uint32_t channels[kRepairWarps];                       // of a row each: those to compute again, 16 a bit
  float q[MOE_W4A16_MAX_HEAD_DIM], prob[kRepairThreads], most[kRepairWarps], sum[kRepairWarps];
  int64_t at[kRepairThreads];
  float out[kRepairThreads * 8];
};

// Eight channels of a token, from element `at` of the pages on.
template <bool E4M3>
__device__ __forceinline__ void load8(const void* pages, int64_t at, float (&x)[8]) {
  if constexpr (E4M3) {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pages) + at);
    uint32_t h[4];
    e4m3x4_to_f16x4(v.x, h[0], h[1]);
    e4m3x4_to_f16x4(v.y, h[2], h[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
          : "=f"(x[2 * j]), "=f"(x[2 * j + 1])
          : "r"(h[j]));
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pages) + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
// Place of token j of a sequence in the pages (elements, its head's first channel), -1: not there.
__device__ __forceinline__ int64_t token_at(const ChunkParams& p, int row, int kvh, int j) {
  const int page = p.t.tables[row * p.t.table_stride + j / p.t.page_size];
  if (page < 0 || page >= p.t.num_pages) return -1;
  return int64_t(page) * p.page_stride + int64_t(j % p.t.page_size) * p.token_stride + int64_t(kvh) * p.head_stride;
}
// The tokens that the tiles of a block hold and not all its rows see: behind its first row's, and before its last row's window.
struct Hidden {
  int low, low_end, high, high_end;
};
__device__ __forceinline__ Hidden hidden_of(const ChunkParams& p, int pos, int n, int len) {
  Hidden h{0, 0, max(pos + 1, 0), 0};
  const int hi = pos + n;                                // the block's tokens
  h.high_end = static_cast<int>(min(int64_t(len), (int64_t(hi - 1) / kTile + 1) * kTile));
  if (p.window > 0 && hi - 1 >= p.window) {
    h.low_end = hi - p.window;
    h.low = (pos >= p.window ? pos - p.window + 1 : 0) / kTile * kTile;
  }
  return h;
}
// Whether one of them has such a value (every thread of the CTA calls it).
template <bool E4M3>
static __device__ bool hidden_values(const ChunkParams& p, int row, int kvh, int pos, int n, int len) {
  const Hidden h = hidden_of(p, pos, n, len);
  float zero = 0.f;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int from = part == 0 ? h.low : h.high, to = part == 0 ? h.low_end : h.high_end;
#pragma unroll 1
    for (int64_t j = int64_t(from) + threadIdx.x; j < to; j += kRepairThreads) {      // (lengths end less than a step below 2^31)
      const int64_t at = token_at(p, row, kvh, static_cast<int>(j));
      if (at < 0) continue;
#pragma unroll 1
      for (int c = 0; c < p.dim; c += 8) {
        float x[8];
        load8<E4M3>(p.v, at + c, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) zero = fmaf(x[k], 0.f, zero);
      }
    }
  }
  return __syncthreads_or(zero != 0.f);
}
// One row's channels again, 16 for every bit of `channels` (every thread calls it, a token each at a time).
template <bool E4M3>
static __device__ void repair_row(const ChunkParams& p, int token, int head, int row, int pos, uint32_t channels, RepairShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, kvh = head / p.group;
  const uint16_t* q = p.q + token * p.q_stride + int64_t(head) * p.dim;
  for (int d = tid; d < p.dim; d += kRepairThreads) sh.q[d] = bf16_to_f32(q[d]);
  const int lanes = p.dim / 8, groups = kRepairThreads / lanes, g = tid / lanes, ch = (tid - g * lanes) * 8;   // of the values
  float m = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  __syncthreads();
#pragma unroll 1
  for (int64_t j0 = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0; j0 <= pos; j0 += kRepairThreads) {
    const int64_t at = j0 + tid <= pos ? token_at(p, row, kvh, static_cast<int>(j0) + tid) : -1;
    float s = -INFINITY;
    if (at >= 0) {
      s = 0.f;
#pragma unroll 2
      for (int d = 0; d < p.dim; d += 8) {
        float x[8];
        load8<E4M3>(p.k, at + d, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(sh.q[d + k], x[k], s);
      }
      s *= p.score_scale;
    }
    float top = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (lane == 0) sh.most[warp] = top;
    __syncthreads();
    top = m;
#pragma unroll
    for (int w = 0; w < kRepairWarps; ++w) top = fmaxf(top, sh.most[w]);
    const float base = top == -INFINITY ? 0.f : top, keep = exp2_fast(m - base), e = at >= 0 ? exp2_fast(s - base) : 0.f;
    m = top;
    l = fmaf(l, keep, e);
    sh.prob[tid] = e;
    sh.at[tid] = at;
    __syncthreads();                                     // (the next tile's are written behind its first barrier)
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] *= keep;
    if (g < groups) {
#pragma unroll 2
      for (int t = g; t < kRepairThreads; t += groups) {
        const int64_t v = sh.at[t];
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (v >= 0) load8<E4M3>(p.v, v + ch, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = fmaf(sh.prob[t], x[k], o[k]);
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  if (lane == 0) sh.sum[warp] = l;
  if (g < groups)
#pragma unroll
    for (int k = 0; k < 8; ++k) sh.out[g * p.dim + ch + k] = o[k];
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kRepairWarps; ++w) l += sh.sum[w];
  const float inv = l == 0.f ? 0.f : p.v_scale / l;
  uint16_t* out = p.out + (int64_t(token) * p.heads + head) * p.dim;
  for (int d = tid; d < p.dim; d += kRepairThreads) {
    if (!(channels >> (d / 16) & 1u)) continue;
    float x = 0.f;
    for (int k = 0; k < groups; ++k) x += sh.out[k * p.dim + d];
    out[d] = f32_to_bf16_rn(x * inv);
  }
  __syncthreads();                                       // (read before the next row's)
}

// Behind the join: nothing, if no CTA has flagged an output; else all rows of the call, a warp a row until one is none.
template <int DP, bool E4M3>
__global__ void __launch_bounds__(kRepairThreads, 1) chunk_repair_kernel(const __grid_constant__ ChunkParams p, const Record* records,
                                                                         int ctas) {
  __shared__ RepairShared sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int flags = 0;
  for (int c = threadIdx.x; c < ctas; c += kRepairThreads) flags |= __ldcg(&records[c].none);
  if (!__syncthreads_or(flags)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int step = Cfg<DP, E4M3>::kStreams * blocks_of(p.group).tokens;
#pragma unroll 1
  for (int b = 0; b < p.batch; ++b) {
    const ChunkRange c = chunk_range(p, b);
    if (c.row < 0) continue;                             // (all zeros)
    const int64_t rows = int64_t(c.n) * p.heads;
#pragma unroll 1
    for (int64_t r0 = blockIdx.x; r0 < rows; r0 += int64_t(gridDim.x) * kRepairWarps) {
      const int64_t mine = r0 + int64_t(warp) * gridDim.x;
      bool none = false;                                 // 16 channels a lane
      if (mine < rows && lane < p.dim / 16) {
        const uint32_t* out = reinterpret_cast<const uint32_t*>(p.out + (int64_t(c.first) * p.heads + mine) * p.dim) + lane * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) none |= (out[k] & 0x7f80u) == 0x7f80u || (out[k] & 0x7f800000u) == 0x7f800000u;
      }
      const uint32_t found = __ballot_sync(0xffffffffu, none);
      if (lane == 0) sh.channels[warp] = found;
      if (!__syncthreads_or(found != 0)) continue;
#pragma unroll 1
      for (int w = 0; w < kRepairWarps; ++w) {
        const uint32_t channels = sh.channels[w];
        if (channels == 0) continue;
        const int64_t row = r0 + int64_t(w) * gridDim.x;
        const int i = static_cast<int>(row / p.heads), head = static_cast<int>(row - int64_t(i) * p.heads);
        const int i0 = i / step * step;                  // its block
        if (hidden_values<E4M3>(p, c.row, head / p.group, c.base + i0, min(step, c.n - i0), c.base + c.n))
          repair_row<E4M3>(p, c.first + i, head, c.row, c.base + i, channels, sh);
      }
      __syncthreads();                                   // (sh.channels has been read)
    }
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link needed).
static EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  return fn;
}
// A tile's 32 tokens of a loader warp are boxes of tokens that lie behind each other in a page: as many as divide its size,
// 8 at least (the swizzle's rows). Pages of other sizes, and of strides that a map cannot have, go token by token.
static void page_maps(const ChunkParams& p, bool e4m3, int unit_channels, PageMaps* maps) {
  maps->rows = 0;
  int rows = 32;
  while (rows >= 8 && p.t.page_size % rows != 0) rows /= 2;
  EncodeTiledFn enc = encode_tiled();
  if (rows < 8 || enc == nullptr) return;
  const int64_t head_stride = p.kv_heads > 1 ? p.head_stride : p.dim;
  const int64_t page_stride = p.t.num_pages > 1 ? p.page_stride : p.token_stride * p.t.page_size;
  const int64_t most = int64_t(1) << 39;                 // strides of a map end at 2^40 bytes
  if (page_stride < 1 || page_stride >= most || p.token_stride >= most || head_stride >= most) return;
  const cuuint64_t size = e4m3 ? 1 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.dim), static_cast<cuuint64_t>(p.kv_heads),
                              static_cast<cuuint64_t>(p.t.page_size), static_cast<cuuint64_t>(p.t.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(head_stride) * size, static_cast<cuuint64_t>(p.token_stride) * size,
                                 static_cast<cuuint64_t>(page_stride) * size};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(e4m3 ? unit_channels : 64), 1, static_cast<cuuint32_t>(rows), 1},
                   ones[4] = {1, 1, 1, 1};
  CUtensorMap* const map[2] = {&maps->k, &maps->v};
  for (int i = 0; i < 2; ++i)
    if (enc(map[i], e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(i == 0 ? p.k : p.v), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return;
  maps->rows = rows;
}

template <int DP, bool E4M3>
static cudaError_t launch(const ChunkParams& p, int device, cudaStream_t stream) {
  using C = Cfg<DP, E4M3>;
  constexpr int kSmem = C::kMiscOff + static_cast<int>(sizeof(Misc));
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static_assert(C::kMiscOff % 16 == 0 && C::kUnitBytes % 1024 == 0 && C::kQBytes % 1024 == 0, "swizzled tiles");
  static bool attr_set[64] = {false};
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[device]) {
    const cudaError_t e = cudaFuncSetAttribute(chunk_kernel<DP, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr_set[device] = true;
  }
  Record* records = static_cast<Record*>(p.scratch);
  float* parts = reinterpret_cast<float*>(records + kMaxCtas);
  int grid = device_info(device).sm_count;
  if (grid > kMaxCtas) grid = kMaxCtas;
  PageMaps maps;
  page_maps(p, E4M3, C::kUnitCh, &maps);
  chunk_kernel<DP, E4M3><<<grid, kThreads, kSmem, stream>>>(p, maps, records, parts);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the join may be set up while the first kernel runs; it waits for that kernel's end before it reads
  cudaLaunchConfig_t cfg{};
  // at most one block of rows of each CTA to join, and no more than there are
  const Blocks blocks = blocks_of(p.group);
  const int64_t most = (p.tokens / (C::kStreams * blocks.tokens) + int64_t(p.batch)) * p.kv_heads * blocks.count;
  cfg.gridDim = dim3(static_cast<unsigned>((most < grid ? most : grid) * (C::kStreams * (p.dim / 16))));
  cfg.blockDim = dim3(kRows);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, chunk_join_kernel<DP, E4M3>, p, static_cast<const Record*>(records),
                         static_cast<const float*>(parts), grid);
  if (e != cudaSuccess) return e;
  // the third waits for both
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kRepairThreads);
  e = cudaLaunchKernelEx(&cfg, chunk_repair_kernel<DP, E4M3>, p, static_cast<const Record*>(records), grid);
  note_launch(3);
  return e;
}

}  // namespace chunk

size_t chunk_scratch_bytes(int, int, int dim) {
  const size_t floats = dim <= 64 ? chunk::Cfg<64, false>::kPartFloats
                        : dim <= 128 ? chunk::Cfg<128, false>::kPartFloats
                                     : chunk::Cfg<256, false>::kPartFloats;
  return chunk::kMaxCtas * (sizeof(chunk::Record) + 2 * floats * sizeof(float));
}

cudaError_t launch_chunk_attention(const ChunkParams& p, int dtype, int device, cudaStream_t stream) {
  const bool e4m3 = dtype == MOE_W4A16_CACHE_E4M3;
  if (p.dim <= 64) return e4m3 ? chunk::launch<64, true>(p, device, stream) : chunk::launch<64, false>(p, device, stream);
  if (p.dim <= 128) return e4m3 ? chunk::launch<128, true>(p, device, stream) : chunk::launch<128, false>(p, device, stream);
  return e4m3 ? chunk::launch<256, true>(p, device, stream) : chunk::launch<256, false>(p, device, stream);
}

}  // namespace moe
