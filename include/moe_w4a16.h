/*
 * moe_w4a16.h -- C ABI of a W4A16 mixture-of-experts grouped GEMM for one
 * GB300 (sm_103a) GPU.
 *
 * Source of the method: the page "vLLM x Novita AI launch Chord: an INT4 MoE
 * operator that speeds up Kimi K2.x by up to 2.15x" (aihot.vn), called "the
 * Chord page" below. It describes a CUDA MoE operator for BF16 activations,
 * INT4 (uint4) weights and BF16 scales per group of 32 along K (TL;DR), with
 * an indexed and two grouped layouts (section "Grouped SM90 kernels",
 * Figure 3), a schedule chosen from the tokens routed per expert (TL;DR and
 * section "H200 prefill and TP8"), and subtract-then-scale dequantisation
 * (section "H200 and Blackwell indexed decode"). The page prints no
 * signatures; the entry points below are this library's own design.
 *
 * Conventions shared by every entry point
 *   - Every pointer is a DEVICE pointer owned by the caller unless the
 *     comment says "host". The library allocates no device memory.
 *   - BF16 tensors are passed as uint16_t bit patterns, row-major, dense.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and runs asynchronously; a return of MOE_W4A16_OK means the
 *     arguments were accepted and the kernels were launched.
 *   - Functions never throw, never abort and never print (unless the
 *     environment variable MOE_W4A16_LOG=1 asks for plan logging). Invalid
 *     arguments are rejected on the host before any launch.
 *   - Index arrays are also checked on the device: an out-of-range expert id,
 *     row id or count is skipped and recorded in the workspace error word
 *     (read it with moe_w4a16_get_device_error); a kernel never reads or
 *     writes outside the buffers it was given, and every wait inside a
 *     kernel gives up after about two seconds (moe_w4a16_set_wait_limit_ns)
 *     and records MOE_W4A16_ERR_DEVICE_TIMEOUT instead of hanging.
 *   - `ws` is a caller-owned workspace of at least moe_w4a16_workspace_size()
 *     bytes (always >= 256: its first bytes hold the device error word and the
 *     decode kernel's unit hand-out counters). Zero it once after allocation
 *     (moe_w4a16_workspace_init); every call leaves its counters at zero, but a
 *     call that recorded a device error may not, so zero it again after one.
 *     Calls that share a workspace must be ordered on one stream. Indexed GEMM
 *     calls with block_m <= 32 and masked ones keep their counters at one place:
 *     they may share a workspace whatever their shapes. A GEMM call with
 *     block_m > 32 or of the contiguous layout keeps other data there, so it
 *     shares one only with calls like itself (or zero it in between). A call
 *     that finds a counter which cannot be right records
 *     MOE_W4A16_ERR_WORKSPACE; part of its output may then not be written.
 */
#ifndef MOE_W4A16_H_
#define MOE_W4A16_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_W4A16_API __attribute__((visibility("default")))
#else
#define MOE_W4A16_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* moe_w4a16_stream_t; /* same type as cudaStream_t */

typedef enum moe_w4a16_status {
  MOE_W4A16_OK = 0,
  MOE_W4A16_ERR_INVALID_ARG = 1,    /* null pointer, bad size, inconsistent flags */
  MOE_W4A16_ERR_UNSUPPORTED = 2,    /* quantisation scheme or shape outside what the kernels handle */
  MOE_W4A16_ERR_MODE_MISMATCH = 3,  /* prepared weight's recorded mode/version does not fit the call */
  MOE_W4A16_ERR_WORKSPACE = 4,      /* workspace missing or too small; device: its counters were not left at zero */
  MOE_W4A16_ERR_CAPACITY = 5,       /* device: an expert holds more rows than the masked budget */
  MOE_W4A16_ERR_DEVICE_TIMEOUT = 6, /* device: a pipeline wait gave up */
  MOE_W4A16_ERR_CUDA = 7,           /* a CUDA runtime call failed */
  MOE_W4A16_ERR_BAD_INDEX = 8,      /* device: an index array held an out-of-range value */
  MOE_W4A16_ERR_SCRATCH_LIMIT = 9   /* the call needs more scratch than the static array holds */
} moe_w4a16_status;

/* Activation layouts (the Chord page, section "Grouped SM90 kernels", Figure 3). */
enum {
  MOE_W4A16_LAYOUT_INDEXED = 0,    /* activations unpadded; sorted_ids carry the padding sentinels */
  MOE_W4A16_LAYOUT_CONTIGUOUS = 1, /* each expert's rows padded to a 128-row boundary */
  MOE_W4A16_LAYOUT_MASKED = 2      /* fixed row budget max_m per expert, masked_m valid counts */
};

/* Prepared-weight modes, recorded in the prepared weight and checked at dispatch
 * (the Chord page, section "Grouped SM90 kernels": the mode is stored with the
 * prepared weight so a mismatched call fails loudly). */
enum {
  MOE_W4A16_MODE_PLAIN = 1,  /* output channels in logical order */
  MOE_W4A16_MODE_GATE_UP = 2 /* N = 2*I: gate = channels [0, I), up = [I, 2I); packed so that a
                                tile holds matching gate and up channels (needed for SWIGLU) */
};

/* Epilogue / input flags of the GEMM entry points. */
enum {
  MOE_W4A16_FLAG_SWIGLU = 1u,   /* out[r, i] = bf16(silu(bf16(y[r, i])) * bf16(y[r, I + i])), width N/2;
                                    needs a MODE_GATE_UP weight */
  MOE_W4A16_FLAG_COMBINE = 2u,  /* out[t, :] = bf16(sum_j w[t, j] * bf16(y[t*top_k + j, :])), j ascending;
                                    needs a MODE_PLAIN weight, topk_weights and a workspace */
  MOE_W4A16_FLAG_A_PER_ROW = 4u, /* indexed only: A holds one row per routed row (row f = t*top_k + j),
                                    as for the down projection; default: one row per token (row f / top_k) */
  MOE_W4A16_FLAG_A_SORTED = 8u,  /* indexed only: A holds one row per sorted_ids slot, [max_sorted, k]
                                    (the output of a call with MOE_W4A16_FLAG_OUT_SORTED) */
  MOE_W4A16_FLAG_OUT_SORTED = 16u, /* indexed only: output row = sorted_ids slot instead of flat id,
                                    c is [max_sorted, n] (or n/2 with SWIGLU); padding slots are not written */
  MOE_W4A16_FLAG_SPLIT = 32u      /* indexed only, block_m <= 32, not with COMBINE or A_SORTED: experts with
                                    more than 32 routed rows run on the tcgen05 kernel (their rows gathered
                                    in slot order, blocks of up to 192 rows), the others on the decode
                                    kernel; the token-count rule applied per expert instead of per call */
};

/* GEMM kernel families (selected by moe_w4a16_plan or forced). */
enum {
  MOE_W4A16_KERNEL_AUTO = 0,
  MOE_W4A16_KERNEL_DECODE = 1, /* warp-level MMA, dequantised weights as the MMA M operand, <= 32 rows/block */
  MOE_W4A16_KERNEL_PREFILL = 2, /* tcgen05 MMA with TMEM accumulators, <= 256 rows/block */
  MOE_W4A16_KERNEL_SPLIT = 3    /* both, split per expert: indexed calls with MOE_W4A16_FLAG_SPLIT (block_m 32);
                                   masked calls by themselves */
};

/* Element type of a cache's pages. */
enum {
  MOE_W4A16_CACHE_BF16 = 0,
  MOE_W4A16_CACHE_E4M3 = 1 /* 8-bit float (4 exponent, 3 mantissa bits, no infinities); value = element * scale */
};
/* Element type of the residual stream of moe_w4a16_block_norm. */
enum { MOE_W4A16_RESIDUAL_BF16 = 0, MOE_W4A16_RESIDUAL_F32 = 1 };

#define MOE_W4A16_MAGIC 0x34413457u /* "W4A4" little-endian tag */
#define MOE_W4A16_VERSION 1u
#define MOE_W4A16_MAX_EXPERTS 1024
#define MOE_W4A16_WS_HEADER_BYTES 256
#define MOE_W4A16_STATIC_SCRATCH_BYTES (64u << 20) /* scratch of moe_w4a16_indexed_noalloc */
#define MOE_W4A16_WAIT_LIMIT_NS 2000000000ull      /* default limit of a device pipeline wait */
#define MOE_W4A16_ROUTED_MAX_ROWS 4096             /* routed rows of a moe_w4a16_indexed_routed call */

#define MOE_W4A16_LATENT_DIM 576                   /* channels of a latent cache row ... */
#define MOE_W4A16_LATENT_VALUE_DIM 512             /* ... of which the first are the values */
#define MOE_W4A16_MAX_HEAD_DIM 256                 /* head_dim of moe_w4a16_paged_attention: 16, 32, ... 256 */
#define MOE_W4A16_MAX_PAGE_SIZE 4096               /* tokens of a cache page */
#define MOE_W4A16_MAX_NORM_WIDTH 32768             /* row length of moe_w4a16_block_norm */
#define MOE_W4A16_MAX_ROTARY_DIM 1024              /* channels of a head that moe_w4a16_rotary turns */

/* Host-side description of a prepared weight, filled by moe_w4a16_prepare and
 * passed by address to every GEMM call (host pointer). */
typedef struct moe_w4a16_desc {
  uint32_t magic;       /* MOE_W4A16_MAGIC */
  uint32_t version;     /* MOE_W4A16_VERSION */
  uint32_t mode;        /* MOE_W4A16_MODE_* */
  uint32_t num_experts; /* E */
  uint32_t n;           /* output channels per expert */
  uint32_t k;           /* reduction length */
  uint32_t group_size;  /* 32 */
  uint32_t reserved;
  uint64_t bytes;       /* size of the prepared device buffer */
} moe_w4a16_desc;

/* Schedule chosen from the routed rows per expert (host pointer). */
typedef struct moe_w4a16_schedule {
  int32_t kernel;  /* MOE_W4A16_KERNEL_DECODE, _PREFILL or (indexed) _SPLIT */
  int32_t block_m; /* rows per block the indexed align step must use */
  int32_t tok_e;   /* routed rows per expert the choice was made from */
  int32_t grid;    /* CTAs the GEMM launches (persistent, a multiple of the SM count) */
} moe_w4a16_schedule;

/* ---------------------------------------------------------------------------
 * Library information
 * ------------------------------------------------------------------------- */

/* Static, NUL-terminated description of a status code (never NULL). */
MOE_W4A16_API const char* moe_w4a16_status_string(moe_w4a16_status status);

/* Library ABI version (MOE_W4A16_VERSION). */
MOE_W4A16_API uint32_t moe_w4a16_abi_version(void);

/* Number of CUDA kernels this library has launched in this process (all devices). */
MOE_W4A16_API uint64_t moe_w4a16_launch_count(void);

/* ---------------------------------------------------------------------------
 * Weight preparation (the Chord page, sections "Indexed kernels" and
 * "Grouped SM90 kernels": weights are packed once at model load, the forward
 * path sees permuted INT4 bytes and MN-major scales, and the mode is recorded
 * in the prepared weight). One prepared layout serves both kernel families.
 * ------------------------------------------------------------------------- */

/* Bytes of the prepared buffer for E experts of [n, k] weights.
 * Requirements: group_size == 32 (else UNSUPPORTED, the page's load-time schema
 * check), k % 64 == 0, n % 256 == 0 (MODE_GATE_UP: n % 256 == 0 as well),
 * 1 <= num_experts <= MOE_W4A16_MAX_EXPERTS. `bytes` is a host pointer. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_prepare_size(int num_experts, int n, int k, int group_size, int mode, size_t* bytes);

/* Packs logical weights into the private prepared layout.
 *   qweight  int32  [E, n, k/8]  word w of row r holds k = 8w..8w+7, nibble i in bits 4i..4i+3
 *   scales   bf16   [E, n, k/32] one scale per 32 consecutive k of a row
 *   prepared device buffer of prepared_bytes >= moe_w4a16_prepare_size(), 256-byte aligned
 *   desc     host; filled on success
 * The weights are dequantised as bf16_rne((q - 8) * s). The input buffers may be
 * freed once the stream has passed this call. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_prepare(const int32_t* qweight, const uint16_t* scales, int num_experts, int n, int k,
                                   int group_size, int mode, void* prepared, size_t prepared_bytes,
                                   moe_w4a16_desc* desc, moe_w4a16_stream_t stream);

/* Writes expert `expert`'s dequantised weights, bf16 [n, k] in logical order,
 * through the same device dequantisation routine the GEMM kernels use (the
 * subtract-then-scale rule of the Chord page, section "H200 and Blackwell
 * indexed decode"). For bit-exact checks. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_dequant_check(const moe_w4a16_desc* desc, const void* prepared, int expert, uint16_t* out,
                                         moe_w4a16_stream_t stream);

/* ---------------------------------------------------------------------------
 * Routing layouts (the Chord page, Figure 3)
 * ------------------------------------------------------------------------- */

/* Capacities for moe_w4a16_align: sorted_ids needs max_sorted int32 entries,
 * expert_ids max_blocks entries (host pointers out). */
MOE_W4A16_API moe_w4a16_status moe_w4a16_align_size(int num_tokens, int top_k, int num_experts, int block_m, size_t* max_sorted,
                                      size_t* max_blocks);

/* Indexed layout from routing.
 *   topk_ids        int32 [T, top_k], expert ids in [0, E) (distinct per token)
 *   sorted_ids      int32 [max_sorted] out: per expert in ascending expert order, the flat ids
 *                   f = t*top_k + j routed to it in ascending order, padded to a multiple of
 *                   block_m with the sentinel R = T*top_k; experts with no rows get no blocks
 *   expert_ids      int32 [max_blocks] out: expert of each block of block_m entries
 *   num_post_padded int32 [1] out: entries used in sorted_ids
 *   expert_counts   int32 [E] out (nullable): rows per expert
 * Ids outside [0, E) are skipped and recorded as MOE_W4A16_ERR_BAD_INDEX in `ws`.
 * Bit-exact: the result is unique. 1 <= block_m <= 256. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_align(const int32_t* topk_ids, int num_tokens, int top_k, int num_experts, int block_m,
                                 int32_t* sorted_ids, int32_t* expert_ids, int32_t* num_post_padded,
                                 int32_t* expert_counts, void* ws, size_t ws_bytes, moe_w4a16_stream_t stream);

/* Contiguous layout from an align result made with block_m = 128.
 *   m_pad      rows of the contiguous layout = max_sorted of that align call
 *   m_indices  int32 [m_pad] out: expert of the row, -1 on padding rows
 *   row_ids    int32 [m_pad] out: flat id t*top_k+j of the row, -1 on padding rows */
MOE_W4A16_API moe_w4a16_status moe_w4a16_contiguous_layout(const int32_t* sorted_ids, const int32_t* expert_ids,
                                             const int32_t* num_post_padded, int num_rows, int m_pad,
                                             int32_t* m_indices, int32_t* row_ids, moe_w4a16_stream_t stream);

/* Masked layout from routing.
 *   masked_m  int32 [E] out: rows routed to each expert (the true count)
 *   row_ids   int32 [E, max_m] out: flat ids per expert in ascending order, -1 past the count
 * An expert with more than max_m rows records MOE_W4A16_ERR_CAPACITY in `ws`
 * (its extra rows are dropped). */
MOE_W4A16_API moe_w4a16_status moe_w4a16_masked_layout(const int32_t* topk_ids, int num_tokens, int top_k, int num_experts,
                                         int max_m, int32_t* masked_m, int32_t* row_ids, void* ws, size_t ws_bytes,
                                         moe_w4a16_stream_t stream);

/* Row gather used to build contiguous / masked activations:
 * dst[i, :] = src[row_ids[i] / row_div, :] for row_ids[i] >= 0, zeros otherwise.
 *   src bf16 [src_rows, k], dst bf16 [num_rows, k], row_ids int32 [num_rows]; k % 8 == 0.
 * Out-of-range ids are written as zero rows and recorded in `ws` (nullable). */
MOE_W4A16_API moe_w4a16_status moe_w4a16_gather_rows(const uint16_t* src, int src_rows, int k, const int32_t* row_ids, int num_rows,
                                       int row_div, uint16_t* dst, void* ws, size_t ws_bytes,
                                       moe_w4a16_stream_t stream);

/* Activation rows in sorted_ids slot order, for MOE_W4A16_FLAG_A_SORTED calls:
 * dst[slot, :] = src[sorted_ids[slot] / row_div, :] for every slot below
 * *num_post_padded whose id is not the sentinel; padding slots are not written.
 *   src bf16 [src_rows, k]; dst bf16 [max_sorted, k]; sorted_ids from moe_w4a16_align
 *   num_rows = T*top_k (the sentinel); row_div = top_k (A per token) or 1 (A per routed row)
 * Whole rows are copied once, so the prefill kernel then reads consecutive rows. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_gather_sorted(const uint16_t* src, int src_rows, int k,
                                                      const int32_t* sorted_ids, const int32_t* num_post_padded,
                                                      int max_sorted, int num_rows, int row_div, uint16_t* dst,
                                                      void* ws, size_t ws_bytes, moe_w4a16_stream_t stream);

/* ---------------------------------------------------------------------------
 * Schedule and workspace (the Chord page, TL;DR: the schedule is chosen from
 * the tokens routed per expert, not the total; section "H200 prefill and TP8":
 * about 80 routed tokens per expert is where the block-M heuristic switches;
 * section "Grouped SM90 kernels": resolution is memoised per descriptor).
 * ------------------------------------------------------------------------- */

/* Chooses the kernel family and block_m from the routed rows per expert:
 * tok_e = T*top_k/E (indexed), m_pad/E (contiguous) or expected_m (masked,
 * a positive count used only to choose the launch; results never depend on
 * it). The environment variable MOE_W4A16_FORCE_KERNEL=decode|prefill|split
 * overrides the family (read on every call, part of the memo key; split is
 * prefill for contiguous calls). Indexed
 * block_m: 16 for the decode family at tok_e <= 4, 32 for the rest of the
 * decode family, 192 for the prefill family. Indexed calls with
 * 8 <= tok_e < 128 (without a forced family) get MOE_W4A16_KERNEL_SPLIT with
 * block_m 32: under skewed routing such calls mix experts of a few rows and
 * experts of hundreds, and each family serves its own (the caller passes
 * MOE_W4A16_FLAG_SPLIT; a call that also combines uses the decode family).
 * Masked calls with 24 <= expected_m < 128 get MOE_W4A16_KERNEL_SPLIT and
 * moe_w4a16_masked runs it itself: experts with masked_m <= 32 on the decode
 * kernel, the others on the tcgen05 kernel, each reading the experts' rows in
 * place (a combining call stays on the tcgen05 family).
 * `plan` is host. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_plan(int layout, int num_tokens, int top_k, int num_experts, int n, int k, int expected_m,
                                moe_w4a16_schedule* plan);

/* Workspace bytes for a GEMM call of the given layout and shape: 256 bytes of
 * header; for an indexed call on the prefill kernel (block_m > 32, or with
 * MOE_W4A16_FLAG_SPLIT) whose A is not already sorted, a bf16 [max_sorted, k]
 * buffer into which the routed
 * activation rows are gathered in sorted_ids order (whole rows, once) so the
 * GEMM reads consecutive rows; for MOE_W4A16_FLAG_COMBINE an arrival counter
 * per (token, 256 output channels, slice) and a bf16 [num_tokens*top_k, n]
 * staging buffer for the routed rows; for calls that may run the decode kernel
 * (indexed block_m <= 32, masked), the counters (behind the header, whatever
 * the shape) and FP32 partial tiles of the units it cuts into k-ranges: the last min(units, 304) units of a call with
 * at most 2048 (row block, 256-channel) units (304 units x 4 parts: 19.9 MB for
 * block_m <= 16, 39.9 MB for 32-row blocks and masked calls); with
 * MOE_W4A16_FLAG_SPLIT also the table of the tcgen05 kernel's blocks (int4
 * [1 + R/192 + R/33]), a per-expert int32 flag [num_experts] and the decode
 * kernel's block list (int32 [1 + max_blocks]).
 * block_m is ignored for the other grouped layout. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_workspace_size(int layout, int num_tokens, int top_k, int num_experts, int n,
                                                        int k, int block_m, uint32_t flags, size_t* bytes);

/* Zeroes a workspace (run once after allocating it). */
MOE_W4A16_API moe_w4a16_status moe_w4a16_workspace_init(void* ws, size_t ws_bytes, moe_w4a16_stream_t stream);

/* Synchronises `stream`, then copies the device error word of `ws` to *code
 * (host): MOE_W4A16_OK or the first device-detected error since the last clear. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_get_device_error(const void* ws, moe_w4a16_stream_t stream, int32_t* code);

/* Diagnostics and tests: sets, for the current device, the limit after which a
 * pipeline wait of a GEMM, the latent or the chunk attention kernel gives up (default MOE_W4A16_WAIT_LIMIT_NS, about
 * two seconds; larger values are INVALID_ARG). A wait that runs out records
 * MOE_W4A16_ERR_DEVICE_TIMEOUT in the workspace error word; the kernel then
 * stops its CTA's pipeline, lets copies already in flight land (those drains
 * keep the default limit), releases its tensor memory and returns. Below 20 us
 * the waits poll without suspending, so with a limit of 0 the first wait for
 * data that has not arrived yet gives up at once. Applies to the calls
 * made after it on that device, from any thread, until set again. Recover from
 * the error with moe_w4a16_workspace_init on the workspace (counters may be
 * left non-zero). */
MOE_W4A16_API moe_w4a16_status moe_w4a16_set_wait_limit_ns(uint64_t ns);

/* Resets the device error word (async on stream). */
MOE_W4A16_API moe_w4a16_status moe_w4a16_clear_device_error(void* ws, moe_w4a16_stream_t stream);

/* ---------------------------------------------------------------------------
 * Grouped GEMM entry points. Each computes, for every valid routed row r with
 * expert e, y[r, :] = A[row(r), :] . W_e^T (FP32 accumulation of BF16 products
 * of the dequantised weights), rounds to BF16 and applies the epilogue of
 * `flags`. Output tolerance against an exact reference: |err| <= 2e-2*(1+|ref|);
 * for COMBINE outputs plus sum_j |w[t, j]| * ulp_bf16(y[t*top_k + j]), because
 * each routed row y is rounded to BF16 from an FP32 sum whose order differs from
 * the reference's, so it may land one BF16 ulp away before it is weighted.
 * The kernel family follows moe_w4a16_plan (indexed: from block_m).
 * Errors: INVALID_ARG / UNSUPPORTED / MODE_MISMATCH / WORKSPACE before launch.
 * ------------------------------------------------------------------------- */

/* Indexed layout (the Chord page, Figure 3: unpadded activations, sentinels in
 * the routing index; section "Indexed kernels").
 *   a          bf16 [a_rows, k]: a_rows = T, or T*top_k with MOE_W4A16_FLAG_A_PER_ROW
 *   sorted_ids, expert_ids, num_post_padded: from moe_w4a16_align with this block_m
 *   block_m    1..32 runs the decode kernel (1..16: its 16-row variant), 33..192 the prefill kernel
 *              (33..128: its 128-row variant, four weight stages in tensor memory instead of two)
 *   topk_weights float32 [T, top_k] (COMBINE only, else may be NULL)
 *   c          plain: bf16 [T*top_k, n] at row f; SWIGLU: [T*top_k, n/2]; COMBINE: [T, n] */
MOE_W4A16_API moe_w4a16_status moe_w4a16_indexed(const uint16_t* a, int a_rows, int k, const moe_w4a16_desc* desc,
                                   const void* prepared, const int32_t* sorted_ids, const int32_t* expert_ids,
                                   const int32_t* num_post_padded, int num_tokens, int top_k, int block_m,
                                   const float* topk_weights, uint32_t flags, uint16_t* c, void* ws, size_t ws_bytes,
                                   moe_w4a16_stream_t stream);

/* Indexed layout straight from the router's output, in one launch (the Chord
 * page, sections "H200 and Blackwell indexed decode": the token-tile schedule is
 * resolved mostly up front and refined by the actual token counts, and "Grouped
 * SM90 kernels": repeated host-side resolution is what memoisation removes).
 * Every CTA of the decode kernel builds, in its own shared memory, the block
 * layout that moe_w4a16_align would build (experts in ascending order, each
 * expert's routed rows in ascending flat id, blocks of block_m rows), so the
 * call needs neither an align launch nor sorted_ids / expert_ids arrays. The
 * result is the one of moe_w4a16_align + moe_w4a16_indexed with the same
 * block_m, bit for bit.
 *   topk_ids   int32 [T, top_k], expert ids in [0, E); an id outside is skipped and
 *              recorded as MOE_W4A16_ERR_BAD_INDEX in `ws`
 *   block_m    1..32 (the decode kernel), else INVALID_ARG
 *   flags      as for moe_w4a16_indexed except A_SORTED, OUT_SORTED and SPLIT (INVALID_ARG)
 *   T*top_k    at most MOE_W4A16_ROUTED_MAX_ROWS (4096), else UNSUPPORTED
 *   ws         at least moe_w4a16_workspace_size(MOE_W4A16_LAYOUT_INDEXED, ..., block_m, flags)
 * Other arguments and outputs as for moe_w4a16_indexed. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_indexed_routed(const uint16_t* a, int a_rows, int k,
                                                        const moe_w4a16_desc* desc, const void* prepared,
                                                        const int32_t* topk_ids, int num_tokens, int top_k,
                                                        int block_m, const float* topk_weights, uint32_t flags,
                                                        uint16_t* c, void* ws, size_t ws_bytes,
                                                        moe_w4a16_stream_t stream);

/* Contiguous layout (the Chord page, Figure 3: each expert padded to a 128-row
 * boundary; valid rows of a segment come first).
 *   a          bf16 [m_pad, k], m_pad % 128 == 0
 *   m_indices  int32 [m_pad]: expert of each row, -1 for padding rows
 *   row_ids    int32 [m_pad]: flat id of each row (COMBINE only, else may be NULL)
 *   c          plain: bf16 [m_pad, n]; SWIGLU: [m_pad, n/2]; COMBINE: [num_tokens, n].
 *              Padding rows of c are not written. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_contiguous(const uint16_t* a, int m_pad, int k, const int32_t* m_indices,
                                      const moe_w4a16_desc* desc, const void* prepared, const int32_t* row_ids,
                                      int num_tokens, int top_k, const float* topk_weights, uint32_t flags,
                                      uint16_t* c, void* ws, size_t ws_bytes, moe_w4a16_stream_t stream);

/* Indexed layout on the decode kernel with NO caller workspace and NO allocation.
 * The paper has no counterpart: this entry point exists for callers that cannot
 * allocate device memory at call time (a custom allocator or memory pool that
 * forbids side allocations, a runtime whose device heap is sized once at
 * start-up, an embedding without a caching allocator to lend a workspace).
 * It computes exactly what moe_w4a16_indexed computes for block_m 1..32, with
 * the same arguments except the workspace, and takes its scratch (device error
 * word, combine counters, combine staging rows, decode partial tiles) from one statically reserved
 * device array of MOE_W4A16_STATIC_SCRATCH_BYTES (64 MiB) per device.
 *   block_m    1..32 (decode kernel only), else INVALID_ARG
 *   flags      as for moe_w4a16_indexed, except MOE_W4A16_FLAG_SPLIT (INVALID_ARG: it
 *              would also run the tcgen05 kernel)
 *   scratch    optional host pointer; receives the device address of the array,
 *              whose first int32 is this call's device error word (read it with
 *              moe_w4a16_get_device_error). Owned by the library: never free it.
 * A call whose moe_w4a16_workspace_size exceeds MOE_W4A16_STATIC_SCRATCH_BYTES
 * (19.9 MB of decode partial tiles at block_m <= 16, 39.9 MB above; with
 * COMBINE also 2*num_tokens*top_k*n bytes of staging: at top-8 and n = 7168
 * up to 408 tokens at block_m <= 16, 235 above) returns
 * MOE_W4A16_ERR_SCRATCH_LIMIT before any CUDA call. No cudaMalloc, cudaFree or
 * allocating library routine is called.
 * Set-up: the first call on a device, with that device current, resolves the
 * array's address (cudaGetSymbolAddress) and caches it; make that first call
 * before any stream capture. The cached address is stale after a
 * cudaDeviceReset of that device: reload the library before calling again.
 * Sharing: all calls on a device share the array. Each call clears, on
 * `stream` before its kernel, every counter a call may leave behind (the
 * error word, the unit hand-out, combine and cut-unit counters), so a call
 * after one that recorded a device error needs no recovery step. Calls whose
 * kernels overlap on the GPU race on the array (undefined results), so order
 * them on one stream or with events. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_indexed_noalloc(const uint16_t* a, int a_rows, int k, const moe_w4a16_desc* desc,
                                          const void* prepared, const int32_t* sorted_ids,
                                          const int32_t* expert_ids, const int32_t* num_post_padded, int num_tokens,
                                          int top_k, int block_m, const float* topk_weights, uint32_t flags,
                                          uint16_t* c, void** scratch, moe_w4a16_stream_t stream);

/* Masked layout (the Chord page, section "grouped operator entry points":
 * expected_m is a positive count used only to choose the launch, masked_m
 * holds the valid rows per expert, and the output is flat even though the
 * input is 3-D; rows past masked_m[e] are not written). With 24 <= expected_m
 * < 128 the call is split per expert (see moe_w4a16_plan): two launches.
 *   a3         bf16 [E, max_m, k]
 *   masked_m   int32 [E]; a count above max_m records MOE_W4A16_ERR_CAPACITY
 *   row_ids    int32 [E*max_m]: flat id of each row (COMBINE only, else may be NULL)
 *   c          plain: bf16 [E*max_m, n]; SWIGLU: [E*max_m, n/2]; COMBINE: [num_tokens, n] */
MOE_W4A16_API moe_w4a16_status moe_w4a16_masked(const uint16_t* a3, int num_experts, int max_m, int k, const int32_t* masked_m,
                                  int expected_m, const moe_w4a16_desc* desc, const void* prepared,
                                  const int32_t* row_ids, int num_tokens, int top_k, const float* topk_weights,
                                  uint32_t flags, uint16_t* c, void* ws, size_t ws_bytes, moe_w4a16_stream_t stream);

/* ---------------------------------------------------------------------------
 * Paged cache and the attention that reads it: the half of a decoder layer's
 * decode step beside the MoE FFN.
 *
 * A cache is a pool of pages of page_size tokens. Which pages a sequence owns is
 * its row of `tables` (int32 [num_seqs, table_stride], the first max_pages
 * columns): token j of the sequence sits in page tables[seq][j / page_size] at
 * offset j % page_size. A negative entry is no page: its tokens (freed ones, as
 * behind a sliding window) are not seen. `lens` (int32 [num_seqs]) holds the
 * token counts, `refs` (int32 [num_pages]) how many table rows hold each page; a
 * page is free when its count is 0. Pages are always taken lowest free id first,
 * in the order of the call's entries, so every result is unique.
 * Lengths above max_pages * page_size, page ids at or above num_pages and sequence
 * ids outside [0, num_seqs) are skipped (lengths: cut) and recorded in `ws` as
 * MOE_W4A16_ERR_BAD_INDEX.
 * ------------------------------------------------------------------------- */

/* A layer's pages (host pointer; `k` and `v` are device pointers). Element (page p,
 * token t, head h, channel c) sits at p * page_stride + t * token_stride +
 * h * head_stride + c, in elements; the strides are the same for k and v. k, v and
 * the strides are multiples of 16 bytes. */
typedef struct moe_w4a16_pages {
  void* k;
  void* v;              /* NULL for a latent cache */
  int32_t dtype;        /* MOE_W4A16_CACHE_* */
  int32_t num_pages;
  int32_t page_size;    /* 1 .. MOE_W4A16_MAX_PAGE_SIZE tokens */
  int32_t reserved;     /* 0 */
  int64_t page_stride, token_stride, head_stride;
  float k_scale, v_scale; /* E4M3: an element stands for element * scale; BF16: 1 */
} moe_w4a16_pages;

/* The attention, cache_* and page calls may share a workspace of the largest of their sizes (ordered on one stream), but
 * not with a GEMM call, which keeps data where the attention calls' counters have to be zero, and the other way round.
 *
 * Workspace bytes of the two attention calls for num_heads query heads over
 * num_kv_heads cache heads of head_dim channels (latent: 1 head of
 * MOE_W4A16_LATENT_DIM). Independent of batch and lengths. Zero it once
 * (moe_w4a16_workspace_init); every call leaves its counters at zero. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_attention_workspace_size(int num_heads, int num_kv_heads, int head_dim,
                                                                  size_t* bytes);

/* Attention of one new token per sequence over a paged cache, grouped heads: query
 * head h reads cache head h / (num_heads / num_kv_heads).
 *   s[j] = scale * k_scale * <q, K_j> over the seen tokens j, max(0, len - window) <= j < len
 *   (window 0: all), whose table entry is a page;
 *   out = v_scale * sum_j exp(s[j] - m) V_j / l,  lse = m + ln l,  m = max s, l = sum_j exp(s[j] - m);
 *   nothing seen: out = 0, lse = -infinity.
 * Scores, maxima, sums and outputs are FP32 (the products take the probabilities
 * rounded to BF16, or to FP16 over E4M3 pages); the output is rounded once. Over E4M3
 * pages the queries of a head are taken into FP16 by a power of two: exact, but for
 * channels below 2^-32 of the head's largest, which lose bits and below 2^-40 count as
 * zero. What lies in unseen slots, NaN included, does not reach the result.
 *   q    bf16 [batch, num_heads, head_dim], q_stride elements between sequences; 16-byte aligned
 *   head_dim  a multiple of 16, at most MOE_W4A16_MAX_HEAD_DIM (else UNSUPPORTED)
 *   seq_ids  int32 [batch]: the row of tables and lens of each query (NULL: query b reads row b)
 *   out  bf16 [batch, num_heads, head_dim] dense; lse float [batch, num_heads] or NULL */
MOE_W4A16_API moe_w4a16_status moe_w4a16_paged_attention(const uint16_t* q, int64_t q_stride, int batch, int num_heads,
                                                         int num_kv_heads, int head_dim, const moe_w4a16_pages* cache,
                                                         const int32_t* tables, int64_t table_stride, int max_pages,
                                                         const int32_t* lens, const int32_t* seq_ids, int num_seqs,
                                                         float scale, int window, uint16_t* out, float* lse, void* ws,
                                                         size_t ws_bytes, moe_w4a16_stream_t stream);

/* The same over a latent cache, BF16 only: one row of MOE_W4A16_LATENT_DIM channels per
 * token (cache->k; cache->v is NULL) is every head's key, its first
 * MOE_W4A16_LATENT_VALUE_DIM channels every head's value.
 *   q    bf16 [batch, num_heads, MOE_W4A16_LATENT_DIM] (queries already taken into the latent space)
 *   out  bf16 [batch, num_heads, MOE_W4A16_LATENT_VALUE_DIM] */
MOE_W4A16_API moe_w4a16_status moe_w4a16_latent_attention(const uint16_t* q, int64_t q_stride, int batch, int num_heads,
                                                          const moe_w4a16_pages* cache, const int32_t* tables,
                                                          int64_t table_stride, int max_pages, const int32_t* lens,
                                                          const int32_t* seq_ids, int num_seqs, float scale, int window,
                                                          uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                                                          moe_w4a16_stream_t stream);

/* Writes new tokens' rows into their pages. Row i goes to token positions[i] of sequence
 * seq_ids[i]; a negative position is skipped, a position without a page recorded as
 * MOE_W4A16_ERR_BAD_INDEX. E4M3 pages: the element nearest to k / k_scale (ties to even, cut to
 * +-448, NaN stays NaN). Two rows for one slot: either may win.
 *   k, v   bf16 [num_tokens, num_heads, head_dim], k_stride / v_stride elements between tokens,
 *          16-byte aligned; v NULL with cache->v NULL (a latent cache)
 *   head_dim  a multiple of 8 (E4M3: 16)
 *   ws     at least MOE_W4A16_WS_HEADER_BYTES */
MOE_W4A16_API moe_w4a16_status moe_w4a16_cache_append(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                                      int64_t v_stride, int num_tokens, int num_heads, int head_dim,
                                                      const moe_w4a16_pages* cache, const int32_t* tables,
                                                      int64_t table_stride, int max_pages, int num_seqs,
                                                      const int32_t* seq_ids, const int32_t* positions, void* ws,
                                                      size_t ws_bytes, moe_w4a16_stream_t stream);

/* Workspace bytes of the calls below for a pool of num_pages pages and `count` entries. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_cache_workspace_size(int num_pages, int count, size_t* bytes);

/* Grows sequences: entry i adds counts[i] tokens (counts NULL: one) to sequence seq_ids[i],
 * taking free pages where the new length needs them, and returns the old length (the first
 * new token's position) in positions[i]. An entry whose pages are no longer there, or whose
 * new length passes max_pages * page_size, is left as it was, positions[i] = -1, and recorded
 * as MOE_W4A16_ERR_CAPACITY: entry i gets its pages if the entries up to and including it
 * need no more than are free. Sequence ids of a call are distinct. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_cache_extend(int32_t* refs, int num_pages, int32_t* tables,
                                                      int64_t table_stride, int max_pages, int32_t* lens, int num_seqs,
                                                      const int32_t* seq_ids, const int32_t* counts, int count,
                                                      int page_size, int32_t* positions, void* ws, size_t ws_bytes,
                                                      moe_w4a16_stream_t stream);

/* A pool's storage as the page copies see it (host pointer): plane i (a layer's keys, a
 * layer's values, ...) holds page p as page_bytes consecutive bytes at base + i * plane_stride
 * + p * page_stride. All byte counts and addresses are multiples of 16. */
typedef struct moe_w4a16_pool {
  void* base;
  int32_t num_planes, num_pages;
  int64_t plane_stride, page_stride, page_bytes;
} moe_w4a16_pool;

/* Forks: sequence children[i] (empty) becomes a copy of parents[i]. Full pages are shared
 * (refs + 1); a partly filled last page is copied, in every plane, into a free page of the
 * child's own. Freed entries of the parent stay freed. A fork whose page is no longer there
 * is left empty and recorded as MOE_W4A16_ERR_CAPACITY; a child that is not empty as
 * MOE_W4A16_ERR_BAD_INDEX. Children are distinct and none is a parent of the same call. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_cache_fork(const moe_w4a16_pool* pool, int32_t* refs, int32_t* tables,
                                                    int64_t table_stride, int max_pages, int32_t* lens, int num_seqs,
                                                    const int32_t* parents, const int32_t* children, int count,
                                                    int page_size, void* ws, size_t ws_bytes,
                                                    moe_w4a16_stream_t stream);

/* Frees: keep NULL: every page of sequence seq_ids[i] (refs - 1, table entries -1) and its
 * length becomes 0. Otherwise only the pages wholly before its newest keep[i] tokens, and its
 * length stays unless keep[i] <= 0. A sequence named twice is freed once. A count that is already 0
 * is recorded as MOE_W4A16_ERR_BAD_INDEX and stays 0. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_cache_free(int32_t* refs, int num_pages, int32_t* tables,
                                                    int64_t table_stride, int max_pages, int32_t* lens, int num_seqs,
                                                    const int32_t* seq_ids, const int32_t* keep, int count,
                                                    int page_size, void* ws, size_t ws_bytes,
                                                    moe_w4a16_stream_t stream);

/* Copies page src[i] to page dst[i] in every plane. No dst is a src or another dst of the call. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_cache_copy(const moe_w4a16_pool* pool, const int32_t* src, const int32_t* dst,
                                                    int count, void* ws, size_t ws_bytes, moe_w4a16_stream_t stream);

/* Compacts: with L pages in use, the used pages with ids >= L move, in ascending order, into
 * the free ids below L, in every plane; refs and tables follow.
 *   refs_out   int32 [num_pages] (may be refs); tables_out int32 [num_seqs, table_stride] (may be
 *              tables), of which the first max_pages columns are written
 *   page_map   int32 [num_pages] out: new id of each page, -1 for free ones
 *   num_live   int32 [1] out: L */
MOE_W4A16_API moe_w4a16_status moe_w4a16_cache_compact(const moe_w4a16_pool* pool, const int32_t* refs,
                                                       const int32_t* tables, int64_t table_stride, int max_pages,
                                                       int num_seqs, int32_t* refs_out, int32_t* tables_out,
                                                       int32_t* page_map, int32_t* num_live, void* ws, size_t ws_bytes,
                                                       moe_w4a16_stream_t stream);

/* Workspace bytes of moe_w4a16_paged_chunk_attention, independent of batch, chunks and lengths; another attention,
 * cache_* or page call may share it (see above). */
MOE_W4A16_API moe_w4a16_status moe_w4a16_paged_chunk_workspace_size(int num_heads, int num_kv_heads, int head_dim,
                                                                    size_t* bytes);

/* Attention of a chunk of new tokens per sequence over a paged cache, grouped heads, causal: a prompt or a piece of
 * one, drafts to verify, or both beside sequences that decode. The chunk of sequence b is the rows starts[b] <= t <
 * starts[b + 1] of q, n of them; its keys and values are in the cache already, as the last n of the sequence's lens
 * tokens. Row t stands at position p = lens - n + (t - starts[b]) and sees the tokens j, max(0, p - window + 1) <= j <= p
 * (window 0: all up to p), whose table entry is a page. Scores, outputs, unseen slots and what is refused or recorded
 * are those of moe_w4a16_paged_attention; a row that sees nothing (a chunk longer than its sequence, freed pages) gives
 * zeros and -infinity. Rows before starts[0] and from starts[batch] on are left as they were.
 *   q        bf16 [num_tokens, num_heads, head_dim], q_stride elements between tokens; 16-byte aligned
 *   starts   int32 [batch + 1], ascending, 0 .. num_tokens; a chunk that does not lie within them is skipped and recorded as
 *            MOE_W4A16_ERR_BAD_INDEX
 *   seq_ids  int32 [batch]: the row of tables and lens of each chunk (NULL: chunk b reads row b)
 *   out      bf16 [num_tokens, num_heads, head_dim] dense; lse float [num_tokens, num_heads] or NULL; q, out and lse do not
 *            overlap (INVALID_ARG; out may lie between q's rows) */
MOE_W4A16_API moe_w4a16_status moe_w4a16_paged_chunk_attention(
    const uint16_t* q, int64_t q_stride, int num_tokens, const int32_t* starts, int batch, int num_heads,
    int num_kv_heads, int head_dim, const moe_w4a16_pages* cache, const int32_t* tables, int64_t table_stride,
    int max_pages, const int32_t* lens, const int32_t* seq_ids, int num_seqs, float scale, int window, uint16_t* out,
    float* lse, void* ws, size_t ws_bytes, moe_w4a16_stream_t stream);

/* The same for chunks that may not have fitted into the cache (moe_w4a16_cache_extend):
 *   positions int32 [num_tokens], as moe_w4a16_cache_append takes them, or NULL: a chunk whose first token's is negative was not
 *            appended, so that the sequence's last tokens are others; its rows give zeros and -infinity, and nothing is
 *            recorded here */
MOE_W4A16_API moe_w4a16_status moe_w4a16_paged_chunk_attention_at(
    const uint16_t* q, int64_t q_stride, int num_tokens, const int32_t* starts, const int32_t* positions, int batch,
    int num_heads, int num_kv_heads, int head_dim, const moe_w4a16_pages* cache, const int32_t* tables,
    int64_t table_stride, int max_pages, const int32_t* lens, const int32_t* seq_ids, int num_seqs, float scale,
    int window, uint16_t* out, float* lse, void* ws, size_t ws_bytes, moe_w4a16_stream_t stream);

/* ---------------------------------------------------------------------------
 * Rotation of positions. Of a head's channels, `dim` from `offset` on turn in pairs: at position p pair i becomes
 *   a' = magnitude * (a cos w - b sin w),  b' = magnitude * (a sin w + b cos w),  w = p * f_i,
 * with (a, b) the channels offset + i and offset + i + dim / 2, or, interleaved, offset + 2i and offset + 2i + 1. The
 * other channels are copied. A frequency f_i (radians a token, in double precision) is kept in whole 2^-64 turns, off by
 * one of them and 2^-52 of itself at most, and p * f_i modulo a turn is taken in whole numbers: at position p (a negative
 * one turns back) the angle is off by |p| (2^-64 + 2^-52 f_i / 2 pi) turns at most (one radian a token at p = 2^27:
 * less than 2^-27 of a turn), before it is rounded to FP32; sines, cosines and products are FP32, the result is rounded once.
 * ------------------------------------------------------------------------- */

/* Frequencies for contexts longer than the trained one (`trained_length` tokens), by a factor >= 1, in double
 * precision: with g_i = theta^(-2i/dim) and n_i = trained_length * g_i / 2 pi turns within that length,
 *   NONE    g_i
 *   LINEAR  g_i / factor
 *   BASE    (theta * factor^(dim / (dim - 2)))^(-2i/dim): the slowest pair turns `factor` times slower, the first as before
 *   TURNS   s g_i + (1 - s) g_i / factor, s = (n_i - low) / (high - low) cut to 0 .. 1
 *   INDEX   the same with 1 - s = (i - i_high) / max(i_low - i_high, 0.001) cut to 0 .. 1, i_high = floor and i_low = ceil of
 *           dim ln(trained_length / (2 pi n)) / (2 ln theta) at n = high and low, cut to 0 .. dim - 1
 *   GIVEN   given[i]
 * LINEAR and BASE take factor; TURNS and INDEX also trained_length and 0 < low < high (INDEX: theta != 1). Host only:
 * turns[dim / 2] is host memory, to be copied to the device by the caller. */
enum { MOE_W4A16_ROTARY_NONE = 0, MOE_W4A16_ROTARY_LINEAR = 1, MOE_W4A16_ROTARY_BASE = 2, MOE_W4A16_ROTARY_TURNS = 3,
       MOE_W4A16_ROTARY_INDEX = 4, MOE_W4A16_ROTARY_GIVEN = 5 };
MOE_W4A16_API moe_w4a16_status moe_w4a16_rotary_frequencies(int dim, double theta, int scaling, double factor,
                                                            int trained_length, double low, double high,
                                                            const double* given, uint64_t* turns);

typedef struct moe_w4a16_rotary_desc {
  const uint64_t* turns;  /* device, [dim / 2], 8-byte aligned */
  int32_t dim;            /* channels that turn: even, 2 .. MOE_W4A16_MAX_ROTARY_DIM */
  int32_t offset;         /* the first of them */
  int32_t interleaved;    /* 0: pairs dim / 2 apart, 1: side by side */
  float magnitude;
} moe_w4a16_rotary_desc;

/* out = x turned by its positions.
 *   x, out   bf16 [num_tokens, num_heads, head_dim] with any strides (elements) between tokens and between heads; out may be
 *            x (the same address and strides: turned in place), else the two do not overlap (INVALID_ARG; their rows may lie
 *            between each other's). Rows of out do not overlap.
 *            The wider the power of two, up to 8, that divides head_dim, offset, dim / 2 (interleaved: dim) and the strides, with
 *            pointers aligned alike, the wider the accesses.
 *   positions int32 [num_tokens] */
MOE_W4A16_API moe_w4a16_status moe_w4a16_rotary(const uint16_t* x, int64_t x_stride, int64_t x_head_stride,
                                                const int32_t* positions, int num_tokens, int num_heads, int head_dim,
                                                const moe_w4a16_rotary_desc* rotary, uint16_t* out, int64_t out_stride,
                                                int64_t out_head_stride, moe_w4a16_stream_t stream);

/* moe_w4a16_cache_append with the rotation on the way, in one launch: k is turned by its position, then written (E4M3: the
 * element nearest to the turned key / k_scale, without a rounding to BF16 between); v is written as it is; q, turned by the
 * same positions, goes to q_out. Query rows are turned whatever becomes of their key: a negative position turns back.
 *   q, q_out bf16 [num_tokens, num_q_heads, head_dim], strides between tokens, 16-byte aligned; both NULL: keys and values
 *            alone. q_out may be q (the same address and stride), else the two do not overlap; it does not overlap k or v
 *            (INVALID_ARG; rows may lie between each other's, as queries and keys of one buffer do).
 *   rotary   offset and dim multiples of 8, dim of 16 unless interleaved (else UNSUPPORTED); offset + dim <= head_dim
 * Other arguments as for moe_w4a16_cache_append. */
MOE_W4A16_API moe_w4a16_status moe_w4a16_cache_append_rotary(
    const uint16_t* q, int64_t q_stride, int num_q_heads, uint16_t* q_out, int64_t q_out_stride, const uint16_t* k,
    int64_t k_stride, const uint16_t* v, int64_t v_stride, int num_tokens, int num_heads, int head_dim,
    const moe_w4a16_rotary_desc* rotary, const moe_w4a16_pages* cache, const int32_t* tables, int64_t table_stride,
    int max_pages, int num_seqs, const int32_t* seq_ids, const int32_t* positions, void* ws, size_t ws_bytes,
    moe_w4a16_stream_t stream);

/* ---------------------------------------------------------------------------
 * Norms around a block (attention or FFN) on the residual stream, in one pass:
 *   u = x, or x / sqrt(mean(x^2) + eps) * w_post       (w_post NULL: x itself)
 *   h' = residual_scale * h + block_scale * gate * u     (gate NULL: 1)
 *   y = h' / sqrt(mean(h'^2) + eps) * w_pre             (the next block's input)
 * in FP32, each output rounded once (y from the unrounded h').
 *   x      bf16 [rows, n], the block's output; NULL: h' = residual_scale * h
 *   h      [rows, n] of residual_dtype (MOE_W4A16_RESIDUAL_*); h_out the same or NULL, may be h
 *   gate   bf16 [gate_rows, n] dense or NULL; gate_rows divides rows, row t takes gate row
 *          t / (rows / gate_rows): one for all tokens, one per sequence, one per token
 *   w_post, w_pre  bf16 [n]; w_pre and y both or neither; x NULL needs gate and w_post NULL
 *   n      1 .. MOE_W4A16_MAX_NORM_WIDTH; strides in elements between rows, any from n on (the wider the power of two,
 *          up to 8, that divides n and the strides, with pointers aligned alike, the wider the accesses) */
MOE_W4A16_API moe_w4a16_status moe_w4a16_block_norm(const uint16_t* x, int64_t x_stride, const void* h, int64_t h_stride,
                                                    int residual_dtype, const uint16_t* gate, int gate_rows,
                                                    const uint16_t* w_post, const uint16_t* w_pre, int rows, int n,
                                                    float eps, float residual_scale, float block_scale, void* h_out,
                                                    int64_t h_out_stride, uint16_t* y, int64_t y_stride,
                                                    moe_w4a16_stream_t stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* MOE_W4A16_H_ */
