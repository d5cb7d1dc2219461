// Attention of one new token per sequence over a paged cache, grouped heads.
//
// For each sequence and cache head: scores s = q K^T of the query heads that share it, a softmax over the seen
// tokens with a running maximum and sum, and o = p V. Every key and value is read once (by groups above 16 heads once
// for each block of 16); at one flop a byte and query head (E4M3: two) the bound is HBM, so the kernel is built around
// keeping copies in flight:
//
//   * One CTA of four warps takes an equal share of all tiles of all sequences (split.cuh), whatever
//     the lengths; rows that cross a CTA's range are joined by the last CTA to arrive, in order, from
//     FP32 parts. One launch, no host knowledge of the lengths.
//   * Within a tile each warp owns its own tokens: its own ring of shared-memory stages filled by
//     its own cp.async, its own maximum, sum and accumulator. No barrier in the loop; the four
//     warps are joined once per row, in a buffer beside the ring, while the next rows' stages are on their way
//     (4096 rows of 128 tokens: 481 us against 756 with the ring drained at a row's end).
//   * Two CTAs an SM with 96 KB of stages each, 24 KB a warp, keep HBM busy (256 BF16 channels: one CTA with 192 KB). Three
//     or four CTAs with shorter rings are slower (230 to 445 us where two take 194).
//   * The query heads of a cache head share its keys and values as loaded from shared memory, by warp-level MMA
//     (m16n8k16; at full HBM speed its pipe is 10% busy, E4M3 18%). Groups of up to 8 heads are its 8 columns, tokens
//     (scores) and channels (output) its 16 rows; larger groups are the 16 rows, 16 heads at a time. With 8 heads in 16
//     rows, half of them idle, twice the MMAs and registers cost E4M3 much (256 channels 223 us against 173, 128: 183
//     against 174, 64: 244 against 224) and BF16 a little (128 channels 328 against 324).
//   * Unseen slots (past the end, before the window, freed pages) are not read: their rows are
//     zero-filled and their scores are -infinity, so nothing in them reaches the result.
//   * The probabilities enter the value product as BF16 (E4M3 pages: FP16, keys and values converted
//     exactly, queries scaled by a power of two per row: exact down to 2^-32 of the row's largest channel). Their sum is
//     taken in FP32 before that rounding.
//
// 96 sequences of up to 8191 tokens, 8 cache heads x 8 query heads x 128 channels, BF16: 324 us, 6.6 TB/s, 98% of a plain
// copy. 8 sequences of up to 131072 tokens, E4M3: 192 us, 6.1 TB/s. What E4M3 still lacks there goes to the conversions
// of its elements (64 channels: 5.7 TB/s, with as much softmax a token for half the bytes; groups of 16 heads 6.0 TB/s).
// With 256 channels and 16 heads registers spill, 40 bytes BF16 (6.1 TB/s, 6.7 with 8 heads) and 32 E4M3 (4.8, 6.0). Rows
// of 128 tokens: 4.5 TB/s BF16, 2.8 E4M3, bound by each row's start and join. Rows of 80 or 96 BF16 channels: 4.9 to 5.7
// TB/s; heads' rows that share DRAM bursts are read by CTAs that drift apart.
#include <cuda_runtime.h>

#include "block.h"
#include "common.cuh"
#include "split.cuh"

namespace moe {
namespace attn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;                // query heads of a work row (MMA M)

template <int DP, bool E4M3>
struct Cfg {
  static constexpr int kElem = E4M3 ? 1 : 2;
  static constexpr int kRowBytes = DP * kElem;
  static constexpr int kChunks = kRowBytes / 16;
  // tokens of a warp's stage: 8 KB of keys and values (16 KB for 256 BF16 channels)
  static constexpr int kTok = DP * kElem <= 128 ? 32 : 16;
  static constexpr uint32_t kAll = kTok == 32 ? 0xffffffffu : (1u << (kTok & 31)) - 1u;   // all of them seen
  static constexpr int kStageBytes = 2 * kTok * kRowBytes;
  static constexpr int kStages = kStageBytes <= 4096 ? 6 : 3;
  static constexpr int kTile = kWarps * kTok;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  // the warps' accumulators are joined 8 rows and up to 128 channels at a time, beside the ring
  static constexpr int kJoinCols = DP < 128 ? DP : 128;
  static constexpr int kSmemBytes = kRingBytes + kWarps * 8 * kJoinCols * 4;
};

// Position of 16-byte chunk c of token row r: rows r .. r+7 at one chunk (ldmatrix) fall on eight
// different 16-byte banks groups.
template <int CHUNKS>
__device__ __forceinline__ int swz(int r, int c) {
  if (CHUNKS >= 8) return r * CHUNKS + (c ^ (r & 7));
  return r * CHUNKS + (c ^ ((r >> 1) & 3));                               // 64-byte rows: two to a bank line
}
// 8-bit keys are read as 16-byte rows of four lanes, two token rows at a time.
template <int CHUNKS>
__device__ __forceinline__ int swz_key8(int r, int c) {
  if (CHUNKS >= 8) return r * CHUNKS + (c ^ ((r & 1) << 2));
  return r * CHUNKS + c;
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_16816(d, a, b0, b1);
}
// The transpose of an 8x8 matrix of 16-bit elements, a row's pair of columns a register.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(pair)));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A part of a row: M and L of its 16 heads, then the unnormalised accumulator [16][DP].
template <int DP>
constexpr int part_floats() { return 2 * kRows + kRows * DP; }

// 16 bytes that are there (cp_async16's zero-filling form costs more instructions).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int DP, bool E4M3, bool EIGHT>
__global__ void __launch_bounds__(kThreads) attention_kernel(const AttnParams p, float* parts, int* counters) {
  using C = Cfg<DP, E4M3>;
  constexpr int QR = EIGHT ? 1 : 2;              // query rows of a lane (g, and g + 8)
  constexpr int ST = EIGHT ? C::kTok / 16 : C::kTok / 8;     // score tiles: 16 tokens x 8 heads, or 16 heads x 8 tokens
  constexpr int OT = EIGHT ? DP / 16 : DP / 8;               // output tiles: 16 channels x 8 heads, or 16 heads x 8 channels
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Share share;
  __shared__ float part_m[kWarps][kRows], part_l[kWarps][kRows];
  __shared__ int last_flag;
  // the pieces that a warp's copies have reached and its work has not finished
  struct Ahead {
    int64_t row0;
    int b, r, n, ntiles;
  };
  constexpr int kAhead = C::kStages + 1;
  __shared__ Ahead pieces[kWarps][kAhead];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
  const int chunks = (p.group + kRows - 1) / kRows;
  // The work rows of a sequence (cache heads x blocks of 16 query heads): `lanes` of them go side by side, CTA
  // lane + lanes * i taking the i-th share of the tokens of row `lane`; the others follow each other on the line.
  // (Divisions are by far the longest instruction sequences of a short row: shifts or nothing in the usual cases.)
  const int page_shift = (p.t.page_size & (p.t.page_size - 1)) == 0 ? 31 - __clz(p.t.page_size) : -1;
  auto page_of = [&](int tok) { return page_shift >= 0 ? tok >> page_shift : tok / p.t.page_size; };
  auto head_of = [&](int r, int& block) {              // cache head and block of 16 query heads of work row r
    if (chunks == 1) {
      block = 0;
      return r;
    }
    block = r % chunks;
    return r / chunks;
  };
  const int lanes = p.lanes, lane_row = blockIdx.x % lanes, rows = p.kv_heads * chunks / lanes;

  zero_empty<kThreads>(p, p.dim);
  // A part of a split row costs its join about 0.13 us a vector that a thread adds up, a tile 0.8 us, and a split as such
  // 2.5 us: where no row has more than three tiles each share is as long as the longest row, so that few rows are cut (those
  // that a share's end falls into), and a few longer rows are cut into about 2.8 sqrt(tiles / vectors) parts, no more.
  // (One sequence, 8 heads a cache head: 20000 tokens of one cache head 51 -> 20 us against a part for every CTA, 8192
  // tokens of 8 cache heads 20 -> 17, 100 tokens 8.3 -> 6.0. With 4 or 5.6 in place of 2.8 long rows take 2 to 18% longer.)
  const int items = (min(kRows, p.group) * p.dim + 511) / 512;
  const auto ctas_of = [items](int64_t tiles, int longest) -> int64_t {
    if (longest <= 3) return tiles / max(longest, 1);
    const int64_t most = static_cast<int64_t>(static_cast<float>(tiles) * 2.8f * rsqrtf(static_cast<float>(longest) * items)) + 1;
    return tiles <= most ? tiles : (tiles + (tiles + most - 1) / most - 1) / ((tiles + most - 1) / most);
  };
  if (!find_share<kThreads>(p, blockIdx.x / lanes, gridDim.x / lanes, rows, C::kTile, ctas_of, &share)) return;
  const int64_t total = share.total;
  const int ctas = share.ctas;
  // a stage's tokens never straddle a page, and every chunk of their rows holds channels
  const bool one_run = p.t.page_size % C::kTok == 0 && p.dim == DP;
  // scores enter the exponentials as |scale| s, the queries negated where the scale is negative
  // (zeroed where it is zero, so that the factor itself is never zero: an unseen token's -infinity stays one)
  const uint32_t negate = p.score_scale < 0.f ? 0x80008000u : 0u;
  const float abs_scale = p.score_scale == 0.f ? 1.f : fmaxf(fabsf(p.score_scale), 1.2e-38f);
  const bool flat = p.score_scale == 0.f;
  // ---- copies run ahead of the work by kStages - 1 stages, across the pieces of the share: a walk of their own
  PieceWalk ahead;
  ahead.start(p, &share);
  int ahead_tok = 0, ahead_left = 0, ahead_lo = 0, ahead_hi = 0, entry = -1;   // of the warp's next stage
  int64_t ahead_head = 0;
  const int32_t* ahead_table = nullptr;
  // this lane's page in the next stage, read a stage early
  auto next_entry = [&]() {
    const int tok = ahead_tok + (lane & (C::kTok - 1));
    entry = tok >= ahead_lo && tok < ahead_hi ? ahead_table[page_of(tok)] : -1;
  };
  int found = 0, found_slot = 0;
  auto next_piece = [&]() {
    Piece pc;
    if (!ahead.next(p, rows, C::kTile, pc)) return;
    if (lane == 0) pieces[warp][found_slot] = {pc.row0, pc.b, pc.r, pc.tile1 - pc.tile0, pc.ntiles};
    ++found;
    found_slot = found_slot + 1 == kAhead ? 0 : found_slot + 1;
    int block;
    const int kvh = head_of(pc.r * lanes + lane_row, block), head0 = kvh * p.group + block * kRows;
    ahead_table = p.t.tables + int64_t(pc.seq) * p.t.table_stride;
    ahead_head = int64_t(kvh) * p.head_stride;
    ahead_tok = (pc.lo / C::kTile + pc.tile0) * C::kTile + warp * C::kTok;
    ahead_left = pc.tile1 - pc.tile0;
    ahead_lo = pc.lo;
    ahead_hi = pc.hi;
    next_entry();
    // its queries to L2 (warp 0: one line a lane; up to 16 heads x 256 channels are two)
    if (warp == 0) {
      const uint8_t* q = reinterpret_cast<const uint8_t*>(p.q + int64_t(pc.b) * p.q_stride + int64_t(head0) * p.dim);
      const int bytes = min(kRows, p.group - block * kRows) * p.dim * 2;
      for (int i = lane * 128; i < bytes; i += 32 * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i));
    }
  };
  auto issue = [&](int slot) -> uint32_t {
    uint32_t seen = 0;
    if (ahead_left > 0) {
      const int tok = ahead_tok + (lane & (C::kTok - 1));
      if (entry >= p.t.num_pages) {
        set_error(p.err, MOE_W4A16_ERR_BAD_INDEX);
        entry = -1;
      }
      int64_t off = -1;
      if (entry >= 0)
        off = int64_t(entry) * p.page_stride + int64_t(tok - page_of(tok) * p.t.page_size) * p.token_stride + ahead_head;
      seen = __ballot_sync(0xffffffffu, off >= 0) & C::kAll;
      if (seen != 0) {
        const uint32_t kd = ring + slot * C::kStageBytes, vd = kd + C::kTok * C::kRowBytes;
        const uint8_t* kb = static_cast<const uint8_t*>(p.k);
        const uint8_t* vb = static_cast<const uint8_t*>(p.v);
        constexpr int kCopies = C::kTok * C::kChunks / 32;
        const auto key_at = [](int tr, int c) { return 16 * (E4M3 ? swz_key8<C::kChunks>(tr, c) : swz<C::kChunks>(tr, c)); };
        if (seen == C::kAll && one_run) {
          // the stage's tokens lie behind each other in one page: lane's row and chunk advance by whole rows
          const int64_t o = (__shfl_sync(0xffffffffu, off, 0) + int64_t(lane / C::kChunks) * p.token_stride) * C::kElem +
                            lane % C::kChunks * 16;
          const uint8_t* ks = kb + o;
          const uint8_t* vs = vb + o;
          const int64_t step = int64_t(32 / C::kChunks) * p.token_stride * C::kElem;
#pragma unroll
          for (int j = 0; j < kCopies; ++j) {
            const int idx = j * 32 + lane, tr = idx / C::kChunks, c = idx % C::kChunks;
            copy16(kd + key_at(tr, c), ks);
            copy16(vd + 16 * swz<C::kChunks>(tr, c), vs);
            ks += step;
            vs += step;
          }
        } else {
#pragma unroll
          for (int j = 0; j < kCopies; ++j) {
            const int idx = j * 32 + lane, tr = idx / C::kChunks, c = idx % C::kChunks;
            const int64_t o = __shfl_sync(0xffffffffu, off, tr);
            const bool ok = o >= 0 && c * 16 < p.dim * C::kElem;
            const int64_t at = ok ? o * C::kElem + c * 16 : 0;
            cp_async16(kd + key_at(tr, c), kb + at, ok ? 16 : 0);
            cp_async16(vd + 16 * swz<C::kChunks>(tr, c), vb + at, ok ? 16 : 0);
          }
        }
      }
      if (--ahead_left > 0) {
        ahead_tok += C::kTile;
        next_entry();
      } else {
        next_piece();
      }
    }
    cp_async_commit();
    return seen;
  };
  // A piece's queries. BF16: (row, k 2t..2t+1) and (row, k 2t+8..2t+9) of each 16-channel step. E4M3: the channels in
  // the order in which a lane reads 8-bit keys: step s of a 64-channel block takes channels 16 t + 4 s .. + 3 of lane t.
  // Up to 128 channels they are asked for while the piece before is being joined (4096 rows of 128 tokens: BF16 540 ->
  // 495 us, E4M3 465 -> 430); with 256, and 16 heads of E4M3, registers are wanting (186 us for a long row against 191).
  constexpr int KS = DP / 16;
  constexpr bool kEarly = DP <= 128 && (EIGHT || !E4M3);
  uint2 raw[KS][QR];
  auto load_queries = [&](const Ahead& pc) {
    int block;
    const int head0 = head_of(pc.r * lanes + lane_row, block) * p.group + block * kRows;
    const int heads = min(kRows, p.group - block * kRows);
#pragma unroll
    for (int hh = 0; hh < QR; ++hh) {
      const int row = g + 8 * hh;
      const uint16_t* src = p.q + int64_t(pc.b) * p.q_stride + int64_t(head0 + row) * p.dim;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int d = E4M3 ? (ks >> 2) * 64 + 16 * t + 4 * (ks & 3) : ks * 16 + 2 * t;
        raw[ks][hh] = make_uint2(0u, 0u);
        if (row < heads && d < p.dim && !flat) {
          if (E4M3) raw[ks][hh] = *reinterpret_cast<const uint2*>(src + d);
          else raw[ks][hh] = make_uint2(*reinterpret_cast<const uint32_t*>(src + d), *reinterpret_cast<const uint32_t*>(src + d + 8));
        }
      }
    }
  };
  next_piece();
  __syncwarp();
  if (kEarly) load_queries(pieces[warp][0]);      // (a CTA that gets here has a piece)
  uint32_t masks[C::kStages];                     // seen tokens of the stages in flight
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) masks[s] = issue(s);
  int slot = 0;

  for (int done = 0, done_slot = 0; done < found; ++done, done_slot = done_slot + 1 == kAhead ? 0 : done_slot + 1) {
    __syncwarp();
    const Ahead& pc = pieces[warp][done_slot];
    int block;
    const int head0 = head_of(pc.r * lanes + lane_row, block) * p.group + block * kRows;
    const int heads = min(kRows, p.group - block * kRows);
    const int n = pc.n, b = pc.b;

    // ---- queries as MMA fragments: A (16 rows), or B (8 columns: the same elements as rows 0-7 of A)
    if (!kEarly) load_queries(pc);
    uint32_t qa[KS][2 * QR];
    float qscale[2];
#pragma unroll
    for (int hh = 0; hh < QR; ++hh) {
      qscale[hh] = abs_scale;
      if (!E4M3) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qa[ks][hh] = raw[ks][hh].x ^ negate;
          qa[ks][QR + hh] = raw[ks][hh].y ^ negate;
        }
      } else {
        // scaled into the FP16 range by a power of two
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t w[2] = {raw[ks][hh].x, raw[ks][hh].y};
#pragma unroll
          for (int j = 0; j < 2; ++j)
            top = fmaxf(top, fmaxf(fabsf(bf16_to_f32(static_cast<uint16_t>(w[j]))),
                                   fabsf(bf16_to_f32(static_cast<uint16_t>(w[j] >> 16)))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // top in [2^e, 2^(e+1)): scale by 2^(15-e) (two factors, each a normal number for any e), to below 2^16, where the
        // FP16 range ends: channels keep their eight bits down to 2^-32 of the largest, and end at 2^-40 of it
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        if (top == 0.f || e > 127) e = 15;
        e = max(e, -126) - 15;
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23);
        const float down2 = __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
        qscale[hh] = fmaxf(abs_scale * __uint_as_float(static_cast<uint32_t>(127 + e / 2) << 23) *
                               __uint_as_float(static_cast<uint32_t>(127 + (e - e / 2)) << 23),
                           1.2e-38f);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t w[2] = {raw[ks][hh].x ^ negate, raw[ks][hh].y ^ negate};
#pragma unroll
          for (int half = 0; half < 2; ++half)
            qa[ks][QR * half + hh] =
                pack_f16x2_rn(bf16_to_f32(static_cast<uint16_t>(w[half])) * down * down2,
                              bf16_to_f32(static_cast<uint16_t>(w[half] >> 16)) * down * down2);
        }
      }
    }

    // statistics of a lane's two heads: g, g + 8, or with heads as columns 2 t, 2 t + 1
    if (EIGHT && E4M3) {
      const float of_g = qscale[0];
      qscale[0] = __shfl_sync(0xffffffffu, of_g, 8 * t);
      qscale[1] = __shfl_sync(0xffffffffu, of_g, 8 * t + 4);
    } else if (EIGHT) {
      qscale[1] = abs_scale;
    }
    // m: what the exponents are taken against. 16 heads: the maximum seen so far (E4M3: 15 below it, so that FP16
    // probabilities reach 2^15, keep their bits down to 2^-29 of the largest and end at 2^-39 of it). Up to 8 heads, where
    // a maximum over the tokens crosses eight lanes: a maximum that is only taken when a score passes it by 2^kSlack. BF16:
    // by anything, so that the largest probability is 1 and not rounded (error of 96 ragged sequences 0.0008 against 0.0009
    // with a slack of 2^8, for 0.3% of the time). E4M3: FP16 probabilities of 2^kLift to 2^15, which keep their bits down to
    // 2^-22 of the largest or further, and end at 2^-32 of it or below.
    constexpr float kLift = !E4M3 ? 0.f : EIGHT ? 8.f : 15.f, kSlack = E4M3 ? 7.f : 0.f;
    float top_of[2], m[2], l[2], o[OT][4];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      top_of[hh] = -INFINITY;
      m[hh] = -INFINITY;
      l[hh] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;

    for (int i = 0; i < n; ++i) {
      {
        const int to = slot == 0 ? C::kStages - 1 : slot - 1;
        const uint32_t seen = issue(to);
#pragma unroll
        for (int s = 0; s < C::kStages; ++s)
          if (s == to) masks[s] = seen;
      }
      cp_async_wait<C::kStages - 1>();
      __syncwarp();
      uint32_t seen = 0;
#pragma unroll
      for (int s = 0; s < C::kStages; ++s)
        if (s == slot) seen = masks[s];
      if (seen != 0) {
        const uint32_t ks0 = ring + slot * C::kStageBytes, vs0 = ks0 + C::kTok * C::kRowBytes;
        float s[ST][4];
#pragma unroll
        for (int j = 0; j < ST; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[j][k] = 0.f;
        if constexpr (EIGHT) {
          // ---- scores, tokens x heads
          if (!E4M3) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int j = 0; j < ST; ++j) {
                uint32_t a4[4];
                const int tr = j * 16 + (lane & 15), c = ks * 2 + (lane >> 4);
                ldsm_x4(ks0 + 16 * swz<C::kChunks>(tr, c), a4[0], a4[1], a4[2], a4[3]);
                mma<false>(s[j], a4, qa[ks][0], qa[ks][1]);
              }
          } else {
#pragma unroll
            for (int kb = 0; kb < DP / 64; ++kb)
#pragma unroll
              for (int j = 0; j < ST; ++j) {
                const uint4 x4 = lds128(ks0 + 16 * swz_key8<C::kChunks>(j * 16 + g, kb * 4 + t));
                const uint4 y4 = lds128(ks0 + 16 * swz_key8<C::kChunks>(j * 16 + 8 + g, kb * 4 + t));
                const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w}, y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
                for (int st = 0; st < 4; ++st) {
                  const uint32_t a4[4] = {e4m3x2_to_f16x2(x[st] & 0xffffu), e4m3x2_to_f16x2(y[st] & 0xffffu),
                                          e4m3x2_to_f16x2(x[st] >> 16), e4m3x2_to_f16x2(y[st] >> 16)};
                  mma<true>(s[j], a4, qa[kb * 4 + st][0], qa[kb * 4 + st][1]);
                }
              }
          }
          // ---- running softmax, exponents in units of log 2: scale s - m
          if (seen != C::kAll) {
#pragma unroll
            for (int j = 0; j < ST; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!(seen >> (j * 16 + (k >> 1) * 8 + g) & 1u)) s[j][k] = -INFINITY;
          }
          bool over = false;                               // (m of -infinity: any seen score)
#pragma unroll
          for (int j = 0; j < ST; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) over |= fmaf(s[j][k], qscale[k & 1], -m[k & 1]) > kLift + kSlack;
          if (__any_sync(0xffffffffu, over)) {
            float keep[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = -INFINITY;
#pragma unroll
              for (int j = 0; j < ST; ++j) top = fmaxf(top, fmaxf(s[j][e], s[j][2 + e]));
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              const float base = top * qscale[e] - kLift;
              keep[e] = 1.f;
              if (base > m[e]) {
                keep[e] = exp2_fast(m[e] - base);
                m[e] = base;
              }
              l[e] *= keep[e];
            }
#pragma unroll
            for (int i2 = 0; i2 < OT; ++i2)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[i2][k] *= keep[k & 1];
          }
          const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
          for (int j = 0; j < ST; ++j) {
            // ---- probabilities as the 16 x 8 operand: its columns are heads, a register two tokens
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              s[j][k] = exp2_fast(fmaf(s[j][k], qscale[k & 1], -base[k & 1]));
              l[k & 1] += s[j][k];
            }
            const uint32_t p0 = transpose8(E4M3 ? pack_f16x2_rn(s[j][0], s[j][1]) : pack_bf16x2_rn(s[j][0], s[j][1]));
            const uint32_t p1 = transpose8(E4M3 ? pack_f16x2_rn(s[j][2], s[j][3]) : pack_bf16x2_rn(s[j][2], s[j][3]));
            // ---- values, channels x tokens
#pragma unroll
            for (int c = 0; c < C::kChunks; c += 2) {
              uint32_t v4[4];
              if (!E4M3) {
                const int tr = j * 16 + (lane & 7) + ((lane >> 4) << 3), cc = c + ((lane >> 3) & 1);
                ldsm_x4_t(vs0 + 16 * swz<C::kChunks>(tr, cc), v4[0], v4[1], v4[2], v4[3]);
                mma<false>(o[c / 2], v4, p0, p1);
              } else {
                // a 16-bit element is two channels of one token: bytes 0, 2 and 1, 3 pair two tokens' even and odd
                // channels, rows g and g + 8 of the tile
                const int tr = j * 16 + (lane & 15), cc = c + (lane >> 4);
                ldsm_x4_t(vs0 + 16 * swz<C::kChunks>(tr, cc), v4[0], v4[1], v4[2], v4[3]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const uint32_t a4[4] = {e4m3x2_to_f16x2(__byte_perm(v4[2 * q], 0u, 0x4420u)),
                                          e4m3x2_to_f16x2(__byte_perm(v4[2 * q], 0u, 0x4431u)),
                                          e4m3x2_to_f16x2(__byte_perm(v4[2 * q + 1], 0u, 0x4420u)),
                                          e4m3x2_to_f16x2(__byte_perm(v4[2 * q + 1], 0u, 0x4431u))};
                  mma<true>(o[c + q], a4, p0, p1);
                }
              }
            }
          }
        } else {
          // ---- scores
          if (!E4M3) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int j = 0; j < ST; j += 2) {
                uint32_t b4[4];
                const int tr = j * 8 + (lane & 7) + ((lane >> 4) << 3), c = ks * 2 + ((lane >> 3) & 1);
                ldsm_x4(ks0 + 16 * swz<C::kChunks>(tr, c), b4[0], b4[1], b4[2], b4[3]);
                mma<false>(s[j], qa[ks], b4[0], b4[1]);
                mma<false>(s[j + 1], qa[ks], b4[2], b4[3]);
              }
          } else {
#pragma unroll
            for (int kb = 0; kb < DP / 64; ++kb)
#pragma unroll
              for (int j = 0; j < ST; ++j) {
                const uint4 w4 = lds128(ks0 + 16 * swz_key8<C::kChunks>(j * 8 + g, kb * 4 + t));
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int st = 0; st < 4; ++st) {
                  const uint32_t b0 = e4m3x2_to_f16x2(w[st] & 0xffffu), b1 = e4m3x2_to_f16x2(w[st] >> 16);
                  mma<true>(s[j], qa[kb * 4 + st], b0, b1);
                }
              }
          }
          // ---- running softmax, exponents in units of log 2: scale s - m
          if (seen != C::kAll) {
#pragma unroll
            for (int j = 0; j < ST; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!(seen >> (j * 8 + 2 * t + (k & 1)) & 1u)) s[j][k] = -INFINITY;
          }
          bool moved = false;
          float keep[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float top = top_of[hh];
#pragma unroll
            for (int j = 0; j < ST; ++j) top = fmaxf(top, fmaxf(s[j][2 * hh], s[j][2 * hh + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float base = top == -INFINITY ? 0.f : top * qscale[hh] - kLift;
            keep[hh] = exp2_fast(m[hh] - base);
            moved |= top != top_of[hh];
            top_of[hh] = top;
            m[hh] = top == -INFINITY ? -INFINITY : base;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < ST; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float e = exp2_fast(fmaf(s[j][2 * hh + k], qscale[hh], -base));
                s[j][2 * hh + k] = e;
                sum += e;
              }
            l[hh] = l[hh] * keep[hh] + sum;
          }
          if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int i2 = 0; i2 < OT; ++i2)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[i2][k] *= keep[k >> 1];
          }
          // ---- values
#pragma unroll
          for (int kt = 0; kt < ST / 2; ++kt) {
            uint32_t pa[4];
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const float lo = s[2 * kt + half][2 * hh], hi = s[2 * kt + half][2 * hh + 1];
                pa[2 * half + hh] = E4M3 ? pack_f16x2_rn(lo, hi) : pack_bf16x2_rn(lo, hi);
              }
#pragma unroll
            for (int c = 0; c < C::kChunks; c += 2) {
              uint32_t v4[4];
              const int tr = kt * 16 + (lane & 15), cc = c + (lane >> 4);
              ldsm_x4_t(vs0 + 16 * swz<C::kChunks>(tr, cc), v4[0], v4[1], v4[2], v4[3]);
              if (!E4M3) {
                mma<false>(o[c], pa, v4[0], v4[1]);
                mma<false>(o[c + 1], pa, v4[2], v4[3]);
              } else {
                // a 16-bit element is two channels of one token: bytes 0, 2 and 1, 3 pair two tokens' even and
                // odd channels, which become two tiles of eight channels
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                  for (int odd = 0; odd < 2; ++odd) {
                    const uint32_t sel = odd ? 0x4431u : 0x4420u;
                    const uint32_t b0 = e4m3x2_to_f16x2(__byte_perm(v4[2 * q], 0u, sel));
                    const uint32_t b1 = e4m3x2_to_f16x2(__byte_perm(v4[2 * q + 1], 0u, sel));
                    mma<true>(o[2 * (c + q) + odd], pa, b0, b1);
                  }
              }
            }
          }
        }
      }
      __syncwarp();
      slot = slot + 1 == C::kStages ? 0 : slot + 1;
    }
    if (kEarly && done + 1 < found) {
      __syncwarp();
      load_queries(pieces[warp][done_slot + 1 == kAhead ? 0 : done_slot + 1]);
    }
    // ---- join the warps: unnormalised accumulators through shared memory, beside the copies in flight. Row `row` of
    // 8, block i of 8 channels at (row * blocks + at_block(row, i)) * 8: a fragment's rows fall on different banks.
    constexpr int kBlocks = C::kJoinCols / 8;
    auto at_block = [](int row, int i) { return i ^ (EIGHT ? row >> 1 : row & (kBlocks - 1)); };
    float* buf = reinterpret_cast<float*>(smem + C::kRingBytes);
    // first and last CTA of the row, as blocks of the grid
    const bool whole = n == pc.ntiles;
    const int c0 = whole ? 0 : cta_of(total, ctas, pc.row0) * lanes + lane_row;
    const int c1 = whole ? 0 : cta_of(total, ctas, pc.row0 + pc.ntiles - 1) * lanes + lane_row;
    float* part = parts + (int64_t(blockIdx.x) * 2 + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0)) * part_floats<DP>();
    const int vecs = p.dim / 4;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float sum = l[hh];
#pragma unroll
      for (int x = EIGHT ? 4 : 1; x < (EIGHT ? 32 : 4); x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      if (EIGHT ? g == 0 : t == 0) {
        part_m[warp][EIGHT ? 2 * t + hh : g + 8 * hh] = m[hh];
        part_l[warp][EIGHT ? 2 * t + hh : g + 8 * hh] = sum;
      }
    }
#pragma unroll
    for (int hh = 0; hh < QR; ++hh) {
#pragma unroll
      for (int cb = 0; cb < DP / C::kJoinCols; ++cb) {
        if constexpr (EIGHT) {
          // tile i: heads 2 t, 2 t + 1, channels 16 i + g, + 8 (E4M3: 16 i + 2 g, + 1)
#pragma unroll
          for (int j = 0; j < kBlocks; j += 2)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = 2 * t + e, i = (cb * kBlocks + j) / 2;
              float* dst = buf + (warp * 8 + row) * C::kJoinCols;
              if (!E4M3) {
                dst[at_block(row, j) * 8 + g] = o[i][e];
                dst[at_block(row, j + 1) * 8 + g] = o[i][2 + e];
              } else {
                *reinterpret_cast<float2*>(dst + at_block(row, j + (g >> 2)) * 8 + 2 * (g & 3)) = make_float2(o[i][e], o[i][2 + e]);
              }
            }
        } else {
          float* dst = buf + (warp * 8 + g) * C::kJoinCols;
#pragma unroll
          for (int j = 0; j < kBlocks; ++j) {
            const int i = cb * kBlocks + j;
            if (!E4M3) {
              *reinterpret_cast<float2*>(dst + at_block(g, j) * 8 + 2 * t) = make_float2(o[i][2 * hh], o[i][2 * hh + 1]);
            } else if ((i & 1) == 0) {
              // channels 16 (i / 2) + 4 t ..: the half of a pair of blocks that t / 2 names
              *reinterpret_cast<float4*>(dst + at_block(g, j + (t >> 1)) * 8 + 4 * (t & 1)) =
                  make_float4(o[i][2 * hh], o[i + 1][2 * hh], o[i][2 * hh + 1], o[i + 1][2 * hh + 1]);
            }
          }
        }
        __syncthreads();
        const int here = min(8, heads - 8 * hh);           // rows of this half (may be <= 0)
        constexpr int kVecs = C::kJoinCols / 4;
#pragma unroll 2
        for (int e = threadIdx.x; e < 8 * kVecs; e += kThreads) {
          const int row8 = e / kVecs, row = 8 * hh + row8, dc = e % kVecs * 4, d = cb * C::kJoinCols + dc;
          if (row8 >= here || d >= p.dim) continue;
          float top = part_m[0][row];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) top = fmaxf(top, part_m[w][row]);
          const float base = top == -INFINITY ? 0.f : top;
          float sum2 = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_fast(part_m[w][row] - base);
            const float4 v = *reinterpret_cast<const float4*>(buf + (w * 8 + row8) * C::kJoinCols +
                                                              at_block(row8, dc >> 3) * 8 + (dc & 7));
            sum2 = fmaf(f, part_l[w][row], sum2);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
          }
          if (whole) {
            const float inv = sum2 > 0.f ? p.v_scale / sum2 : 0.f;
            const int64_t h = int64_t(b) * p.heads + head0 + row;
            *reinterpret_cast<uint2*>(p.out + h * p.dim + d) =
                make_uint2(pack_bf16x2_rn(acc.x * inv, acc.y * inv), pack_bf16x2_rn(acc.z * inv, acc.w * inv));
            if (d == 0 && p.lse != nullptr) p.lse[h] = (top + log2f(sum2)) * 0.69314718055994531f;
          } else {
            __stcg(reinterpret_cast<float4*>(part + 2 * kRows + row * DP + d), acc);
            if (d == 0) {
              __stcg(part + row, top);
              __stcg(part + kRows + row, sum2);
            }
          }
        }
        __syncthreads();                                   // the buffer is free again
      }
    }

    // ---- join the CTAs of a row: the last one to arrive adds the parts in order
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int before = atomicAdd(counters + c0, 1), others = (c1 - c0) / lanes;
        const bool last = before == others;
        if (last) counters[c0] = 0;
        if (before < 0 || before > others) set_error(p.err, MOE_W4A16_ERR_WORKSPACE);   // not a zeroed workspace's
        last_flag = last;
      }
      __syncthreads();
      if (last_flag) {
        __threadfence();
        const int np = (c1 - c0) / lanes + 1;
        // part of CTA c0 + i: its last row for the first one, its first row for the others
        auto part_at = [&](int i) { return parts + (int64_t(c0 + i * lanes) * 2 + (i == 0 ? 1 : 0)) * part_floats<DP>(); };
        float* row_top = part_m[0];                       // read by nobody any more
        float* row_sum = part_l[0];
        for (int row = warp; row < heads; row += kWarps) {
          float top = -INFINITY;
          for (int i = lane; i < np; i += 32) top = fmaxf(top, __ldcg(part_at(i) + row));
#pragma unroll
          for (int o2 = 16; o2 > 0; o2 >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2));
          const float base = top == -INFINITY ? 0.f : top;
          float sum = 0.f;
          for (int i = lane; i < np; i += 32) {
            const float f = exp2_fast(__ldcg(part_at(i) + row) - base);
            sum = fmaf(f, __ldcg(part_at(i) + kRows + row), sum);
          }
#pragma unroll
          for (int o2 = 16; o2 > 0; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
          if (lane == 0) {
            row_top[row] = top;
            row_sum[row] = sum;
          }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < heads * vecs; e += kThreads) {
          const int row = e / vecs, d = e % vecs * 4;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          const float base = row_top[row] == -INFINITY ? 0.f : row_top[row];
          // (always kFlight parts in flight: a loop's remainder would wait for each of its parts)
          constexpr int kFlight = 8;
          for (int i0 = 0; i0 < np; i0 += kFlight) {
            float f[kFlight];
            float4 v[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
              const float* from = part_at(min(i0 + i, np - 1));
              f[i] = __ldcg(from + row);
              v[i] = __ldcg(reinterpret_cast<const float4*>(from + 2 * kRows + row * DP + d));
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
              const float w = i0 + i < np ? exp2_fast(f[i] - base) : 0.f;
              acc.x = fmaf(w, v[i].x, acc.x);
              acc.y = fmaf(w, v[i].y, acc.y);
              acc.z = fmaf(w, v[i].z, acc.z);
              acc.w = fmaf(w, v[i].w, acc.w);
            }
          }
          const float sum = row_sum[row], inv = sum > 0.f ? p.v_scale / sum : 0.f;
          const int64_t h = int64_t(b) * p.heads + head0 + row;
          *reinterpret_cast<uint2*>(p.out + h * p.dim + d) =
              make_uint2(pack_bf16x2_rn(acc.x * inv, acc.y * inv), pack_bf16x2_rn(acc.z * inv, acc.w * inv));
          if (d == 0 && p.lse != nullptr) p.lse[h] = (row_top[row] + log2f(sum)) * 0.69314718055994531f;
        }
      }
    }
    if (!whole) __syncthreads();                          // the flag and the totals are free again
  }
  cp_async_wait<0>();
}

template <int DP, bool E4M3, bool EIGHT>
cudaError_t launch(const AttnParams& p, int device, cudaStream_t stream) {
  using C = Cfg<DP, E4M3>;
  const void* fn = reinterpret_cast<const void*>(attention_kernel<DP, E4M3, EIGHT>);
  static bool attr_set[64] = {false};
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[device]) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set[device] = true;
  }
  int grid = device_info(device).sm_count * (2 * (C::kSmemBytes + 2048) <= 228 * 1024 ? 2 : 1);
  if (grid > kAttnMaxCtas) grid = kAttnMaxCtas;
  // As many rows of a sequence side by side as divide them and idle at most one CTA in four: the heads of a token lie
  // next to each other in the usual cache, and read at about the same time they share DRAM pages. (64 sequences of 4096
  // tokens against one row after another: 64 heads of 64 E4M3 channels 645 -> 421 us, 56 of 128 578 -> 543, 64 of 128 BF16
  // channels, where a sixth of the CTAs idles, 1219 -> 1185.)
  AttnParams q = p;
  const int rows = p.kv_heads * ((p.group + kRows - 1) / kRows);
  for (q.lanes = rows < grid ? rows : grid; rows % q.lanes != 0 || grid / q.lanes * q.lanes * 4 < grid * 3; --q.lanes) {
  }
  attention_kernel<DP, E4M3, EIGHT><<<grid / q.lanes * q.lanes, kThreads, C::kSmemBytes, stream>>>(q, p.parts, p.counters);
  note_launch();
  return cudaGetLastError();
}
template <int DP>
cudaError_t launch_dim(const AttnParams& p, bool e4m3, int device, cudaStream_t stream) {
  const bool eight = p.group <= 8;
  if (e4m3) return eight ? launch<DP, true, true>(p, device, stream) : launch<DP, true, false>(p, device, stream);
  return eight ? launch<DP, false, true>(p, device, stream) : launch<DP, false, false>(p, device, stream);
}

}  // namespace attn

size_t attention_part_bytes(int, int, int dim) {
  const int floats = dim <= 64 ? attn::part_floats<64>() : dim <= 128 ? attn::part_floats<128>() : attn::part_floats<256>();
  return size_t(kAttnMaxCtas) * 2 * floats * sizeof(float);
}

cudaError_t launch_attention(const AttnParams& p, int dtype, int device, cudaStream_t stream) {
  const bool e4m3 = dtype == MOE_W4A16_CACHE_E4M3;
  if (p.dim <= 64) return attn::launch_dim<64>(p, e4m3, device, stream);
  if (p.dim <= 128) return attn::launch_dim<128>(p, e4m3, device, stream);
  return attn::launch_dim<256>(p, e4m3, device, stream);
}

}  // namespace moe
