/*
 * pkv_attn.h: C ABI of the GB300 (sm_103a) paged / causal attention library.
 *
 * Every call computes scaled-dot-product attention, softmax(Q K^T * scale) V
 * ("FlashInfer内核库：利用CUDA Warp-Level Primitives加速级联推理的Attention计算",
 * section 1). The score matrix is never written to memory: scores, softmax and
 * the weighted sum of V stay on chip ("快速注意力内核与算子融合", Q&A on
 * FlashAttention; the FMHA page "TensorRT-LLM深度优化", section 2).
 *
 * Conventions common to every call
 * --------------------------------
 * - Pointers named q, k*, v*, out*, lse*, block_table*, kv_lens*, *_lens,
 *   workspace and err_flag are DEVICE pointers. The caller owns them. The
 *   library never allocates or frees device memory, copies to the host or
 *   synchronises (attn_decode_cascade keeps one side stream and two events per
 *   device, created on first use).
 * - `stream` is a cudaStream_t passed as void*; NULL means the legacy default
 *   stream. All work is enqueued on it asynchronously. Outputs are valid once
 *   the caller has synchronised with that stream.
 * - Element types: PKV_F32 (float) or PKV_BF16 (bfloat16). Softmax statistics
 *   and partial states are always fp32. Outputs are rounded to the input type
 *   with round-to-nearest-even.
 * - lse is the natural logarithm of sum_j exp(scale * q . k_j), in fp32. It is
 *   -inf when there is no key; the output row is then 0.
 * - GQA: query head h reads KV head h / (n_qo_heads / n_kv_heads).
 *   n_qo_heads must be a multiple of n_kv_heads.
 * - Return value: PKV_OK (0) or a negative PKV_ERR_* code. A non-zero code
 *   means nothing was enqueued, except PKV_ERR_LAUNCH, which reports the CUDA
 *   launch error. Arguments are checked on the host before any launch. No call
 *   aborts the process.
 * - Every compute call runs inside an NVTX range named after it (for example
 *   "attn_decode_paged"), so that Nsight Systems or `ncu --nvtx` can attribute
 *   kernels to calls; without a tool attached a range costs a pointer test.
 * - err_flag (nullable, int32 in device memory) collects problems that only
 *   the device can see, as a bitwise OR of PKV_DEVERR_* bits: a block-table
 *   entry outside [0, num_pages), a length above the table's capacity, or a
 *   pipeline wait that timed out. The rows affected are written as NaN. The
 *   caller clears the flag; the library only ORs bits into it.
 *
 * Paged KV layout
 * ---------------
 *   k_pages, v_pages : [num_pages][n_kv_heads][page_size][head_dim]
 *   block_table      : int32 [batch][max_blocks_per_seq], row-major
 *   kv_lens          : int32 [batch]
 * Token t of sequence b lives in physical page block_table[b][t / page_size],
 * slot t % page_size ("快速注意力内核与算子融合", Q&A on paged attention: a block
 * table maps logical blocks to physical blocks). Table entries at or past
 * ceil(kv_len / page_size), and the slots of the last page past kv_len, are
 * never read.
 */
#ifndef PKV_ATTN_H
#define PKV_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define PKV_F32 0
#define PKV_BF16 1
#define PKV_FP8_E4M3 2 /* page pools of attn_decode_paged_fp8 (planning and workspace queries) */
#define PKV_FP4_E2M1 3 /* 4-bit page pools (planning and workspace queries of attn_decode_paged_fp4) */

/* activations of attn_linear */
#define PKV_ACT_NONE 0
#define PKV_ACT_RELU 1
#define PKV_ACT_GELU 2      /* y/2 (1 + erf(y / sqrt 2)) */
#define PKV_ACT_GELU_TANH 3 /* y/2 (1 + tanh(sqrt(2/pi) (y + 0.044715 y^3))) */
#define PKV_ACT_SILU 4      /* y / (1 + exp(-y)) */

/* status codes */
#define PKV_OK 0
#define PKV_ERR_INVALID_ARG (-1) /* null pointer, negative size, inconsistent shape */
#define PKV_ERR_UNSUPPORTED (-2) /* valid but not built: head_dim, page_size, group size, dtype */
#define PKV_ERR_WORKSPACE (-3)   /* workspace missing or smaller than the *_workspace_size call says */
#define PKV_ERR_LAUNCH (-4)      /* a CUDA launch or attribute call failed */
#define PKV_ERR_DEVICE (-5)      /* no usable sm_100-family device is current */

/* device-side error bits ORed into *err_flag */
#define PKV_DEVERR_BAD_PAGE 1 /* a block-table entry outside [0, num_pages) */
#define PKV_DEVERR_BAD_LEN 2  /* a length < 0 or > max_blocks * page_size */
#define PKV_DEVERR_TIMEOUT 4  /* a bounded pipeline wait gave up (nothing hung) */
#define PKV_DEVERR_BAD_AXIS 8 /* attn_qk_norm_rope_append: a pair_axis entry outside [0, n_axes) */
#define PKV_DEVERR_NO_PAGES 16 /* attn_cache_reserve: fewer free pages than asked for */

#define PKV_MAX_POOLS 256 /* pools of one attn_cache_reserve or attn_cache_compact call */

/* Support set of this build (others return PKV_ERR_UNSUPPORTED):
 *   decode / cascade : head_dim 64 or 128; page_size 16; group size 1, 2, 4 or 8;
 *                      PKV_F32 or PKV_BF16 (cascade: PKV_BF16, head_dim 128)
 *   prefill          : head_dim 128; PKV_BF16; any seq_len >= 1
 *   flat GEMM        : PKV_BF16; 1 <= m <= 64; k a multiple of 8
 *   append           : head_dim 64 or 128; page_size 16; PKV_F32 or PKV_BF16; any head counts
 *   accumulated weights, eviction : as decode (eviction: any head count); over a chunk as the
 *                      chunked prefill: PKV_BF16, head_dim 128, page_size 16, groups dividing 128
 *   linear           : PKV_BF16; any m and n; k a multiple of 8
 *   accumulated weights over a chunk, eviction : up to 2^30 tokens per sequence
 *   append, accumulated weights of a step, eviction : batch up to 65535; KV heads up to 65535
 *                      (append: 2^20); over a chunk batch times KV heads below 2^30
 *   FP8 pages: attn_decode_paged_fp8 only. A page has one scale per KV head, so a token written to
 *                      it, or gathered beside tokens of another page, would re-quantise the page
 *   4-bit pages : head_dim 64 or 128; page_size 16; batch up to 65535; decode: bf16 queries, group
 *                      sizes 1 to 8, KV heads up to 65535, up to 2^30 tokens per sequence; pack, unpack:
 *                      PKV_F32 or PKV_BF16 on the other side, KV heads up to 2^20
 *   page reservation, compaction : page_size up to 32767; batch up to 65535; num_pages up to 2^30; batch
 *                      times max_blocks below 2^31; up to PKV_MAX_POOLS pools of any element type
 */

/* Human-readable name of a status code. Static storage; never NULL. */
const char* attn_status_string(int status);

/* Text of the CUDA error behind the most recent PKV_ERR_LAUNCH returned on the
 * calling host thread ("no error" if there was none). Static storage; never NULL.
 * A diagnostic for callers; the pages define no counterpart. */
const char* attn_last_cuda_error_string(void);

/*
 * Number of KV splits the decode calls use for this shape and dtype. num_splits > 0
 * is taken as asked (capped at max_blocks_per_seq); 0 lets the library choose from
 * the shape, the SM count of the current device and how many decode CTAs fit on an
 * SM, as the split count that minimises (waves of CTAs) x (pages per CTA + 4), plus 24
 * for the split merge when there is more than one split (so small problems get one
 * split and no merge launch). A split covers a contiguous range of
 * ceil(max_blocks_per_seq / splits) pages of a sequence.
 * FlashDecoding computes each partial softmax independently and combines them
 * all at the end ("【FlashAttention-V4，非官方】FlashDecoding++", section 1).
 * Returns the split count (>= 1) or a negative PKV_ERR_* code.
 */
int attn_decode_num_splits(int batch, int max_blocks_per_seq, int n_qo_heads, int n_kv_heads,
                           int head_dim, int page_size, int num_splits, int dtype);

/*
 * Workspace bytes attn_decode_paged and attn_decode_paged_unified_max need for
 * this shape: the fp32 partial states O[batch][n_qo_heads][splits][head_dim] and
 * LSE[batch][n_qo_heads][splits]. It is 0 when one split suffices. Returns
 * (size_t)-1 for invalid arguments.
 */
size_t attn_decode_workspace_size(int batch, int max_blocks_per_seq, int n_qo_heads,
                                  int n_kv_heads, int head_dim, int page_size, int num_splits,
                                  int dtype);

/*
 * Single-token decode over a paged KV cache.
 *
 *   q     : [batch][n_qo_heads][head_dim], dtype
 *   out   : [batch][n_qo_heads][head_dim], dtype (must not alias an input)
 *   lse   : [batch][n_qo_heads] fp32 (nullable: not written)
 *   scale : multiplies q . k before the softmax (1/sqrt(head_dim) for the
 *           textbook form)
 *
 * The pages read K and V through a block table that maps a sequence's logical
 * blocks to physical pages ("快速注意力内核与算子融合", Q&A on paged attention), and
 * split the keys into partial softmax states that are combined at the end
 * ("【FlashAttention-V4，非官方】FlashDecoding++", section 1, on FlashDecoding).
 * One unit of work is (sequence, KV head, split): that split's K/V pages are
 * streamed through the block table into a shared-memory ring, with a running max
 * and sum (online softmax), and a partial (O, LSE) state is written. A merge kernel
 * (one CTA per output row, launched on `stream` as a programmatic dependent of the
 * decode so that it is placed while the decode's last CTAs run) then combines the
 * partials by log-sum-exp. Sequences whose pages fit in one split are written directly. With 1 or 2 query heads per KV head (and for fp32) the dot
 * products and sums run on the CUDA cores, one CTA per unit, the group's queries in
 * registers. For bf16, head_dim 128 and 4 or 8 query heads per KV head they run on
 * the tcgen05 tensor cores: 128-key tiles (8 pages) against the group's queries,
 * padded to 16, with fp32 accumulators in tensor memory; CTAs take units from the
 * grid until none is left, and with one split per sequence (batch <= 2048) the longest
 * sequences' units are handed out first. The workspace (device, >= attn_decode_workspace_size bytes,
 * 256-byte aligned) holds the partials; its contents on entry do not matter.
 */
int attn_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                      const int32_t* block_table, const int32_t* kv_lens, void* out, float* lse,
                      int batch, int max_blocks_per_seq, int num_pages, int n_qo_heads,
                      int n_kv_heads, int head_dim, int page_size, float scale, int num_splits,
                      int dtype, void* workspace, size_t workspace_bytes, int32_t* err_flag,
                      void* stream);

/*
 * Allocation-free variant of attn_decode_paged (the pages have no counterpart;
 * this is a convenience of the library).
 *
 * Some callers cannot allocate device memory when they call in. Examples are an
 * inference runtime's plugin or enqueue hook that is not allowed to allocate
 * while it runs, and a process that reserved all device memory up front for its
 * own pool. Those callers cannot supply the workspace that attn_decode_paged
 * wants. This entry point keeps the split partial states in a scratch array
 * that the library owns instead: PKV_NOALLOC_SCRATCH_BYTES bytes of static
 * device memory, held on every GPU that loads the library until the process
 * exits. It calls no cudaMalloc, cudaFree or other allocating routine.
 *
 * - Arguments, layouts and results are those of attn_decode_paged, minus the
 *   workspace. The output equals attn_decode_paged's for the same split count.
 * - Returns PKV_ERR_WORKSPACE when the shape needs more than
 *   PKV_NOALLOC_SCRATCH_BYTES of partial states, i.e. when
 *   attn_decode_workspace_size(...) > PKV_NOALLOC_SCRATCH_BYTES. Fewer splits
 *   (num_splits) or a smaller batch fit.
 * - The first call on a device looks up the scratch array's device address
 *   (cudaGetSymbolAddress) with that device current, and caches it with the
 *   unique id of the current context (cuCtxGetId). Make that first call before
 *   any stream capture on that device. cudaDeviceReset destroys the array with
 *   the device's context; the first call in the context that replaces it sees
 *   another context id and looks the address up again (again outside a
 *   capture). Where the driver gives no context id, every call looks it up.
 * - Every call on a device shares the one array. Calls whose kernels overlap on
 *   the GPU (different streams, no ordering between them) race on it and give
 *   wrong results; order them, e.g. on one stream. The array keeps the last
 *   call's contents. Nothing in it needs to start at zero: every partial state
 *   that a call reads was written by the same call.
 */
#define PKV_NOALLOC_SCRATCH_BYTES (8u << 20) /* 8 MiB of fp32 partial states */

int attn_decode_paged_noalloc(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* block_table, const int32_t* kv_lens, void* out,
                              float* lse, int batch, int max_blocks_per_seq, int num_pages,
                              int n_qo_heads, int n_kv_heads, int head_dim, int page_size,
                              float scale, int num_splits, int dtype, int32_t* err_flag,
                              void* stream);

/*
 * Decode with FlashDecoding++'s asynchronised softmax with a unified maximum
 * value ("【FlashAttention-V4，非官方】FlashDecoding++", sections 1 and 3).
 * Scaled logits are exponentiated against the preset value `phi` (natural-log
 * units, same units as lse), not against a running maximum. There is no per-tile
 * max synchronisation, and partial states that share phi add up without
 * rescaling. The pages leave the bound and the fallback open. This library's
 * reading:
 *   - when a tile holds a logit above phi + 60, the CTA raises its reference
 *     value to that tile's max and rescales what it has accumulated;
 *   - when a tile lies wholly below phi - 60 before anything was accumulated,
 *     the reference value drops to the tile's max.
 * Either event adds 1 to *fallback_count (nullable, int32 device counter,
 * caller-cleared). The result equals attn_decode_paged up to rounding. Arguments,
 * workspace and errors are as for attn_decode_paged.
 */
int attn_decode_paged_unified_max(const void* q, const void* k_pages, const void* v_pages,
                                  const int32_t* block_table, const int32_t* kv_lens, void* out,
                                  float* lse, int batch, int max_blocks_per_seq, int num_pages,
                                  int n_qo_heads, int n_kv_heads, int head_dim, int page_size,
                                  float scale, int num_splits, int dtype, float phi,
                                  int32_t* fallback_count, void* workspace,
                                  size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * Decode over FP8 page pools. FP8 cuts attention's memory traffic ("TensorRT-LLM
 * 深度优化：利用FMHA（Fused Multi-Head Attention）内核加速Hopper架构推理", section 4);
 * the page names neither a format nor a scaling, and this library's reading is:
 *   - k_pages, v_pages hold E4M3 codes (the OCP 8-bit floating-point format: bias 7,
 *     3 mantissa bits, no infinities), one byte per element, in the paged layout;
 *   - k_scale, v_scale : fp32 [num_pages][n_kv_heads], one scale per (page, KV head)
 *     tile; an element's value is e4m3(code) * scale;
 *   - q and out are bf16 (dtype PKV_BF16 implied); lse, workspace, splits and
 *     err_flag are as for attn_decode_paged, with the workspace size from
 *     attn_decode_workspace_size(..., PKV_FP8_E4M3).
 * The result is the attention of attn_decode_paged over the dequantised values, with
 * the per-tile scales applied to the dot products and to the softmax weights.
 * Arithmetic: codes become f16 exactly; q is scaled per head by a power of two that
 * brings its largest magnitude to [2^14, 2^15) and converted to f16 (exact for bf16 q,
 * whatever its range, except for elements more than 2^24 below the head's largest);
 * dot products and the weighted sums of V accumulate in fp32. A softmax weight times the
 * tile's V scale enters the V sum as an f16 value (11-bit significand, normal from 2^-14
 * to 65504): V scales above 65504 are not supported, and below about 2^-14 such a weight
 * keeps an absolute precision of 2^-24. Pools
 * must be 16-byte aligned, and n_kv_heads must be even (the CUDA-core kernel's CTA takes two
 * adjacent KV heads). Built for head_dim 64 and 128, page_size 16 and GQA groups 1, 2, 4 and
 * 8; other shapes return PKV_ERR_UNSUPPORTED. At head_dim 128 with 4 or 8 query heads per KV
 * head the products run on the tcgen05 tensor cores: converter warps take each tile's codes
 * to f16 in shared memory (exactly), q goes to f16 as above, the K scale multiplies each
 * logit and a weight times its page's V scale enters the V product as f16, with fp32
 * accumulation; the other shapes run on the CUDA cores.
 */
int attn_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages,
                          const float* k_scale, const float* v_scale, const int32_t* block_table,
                          const int32_t* kv_lens, void* out, float* lse, int batch,
                          int max_blocks_per_seq, int num_pages, int n_qo_heads, int n_kv_heads,
                          int head_dim, int page_size, float scale, int num_splits,
                          void* workspace, size_t workspace_bytes, int32_t* err_flag,
                          void* stream);

/*
 * Chunked prefill over the paged cache: each sequence b already holds prefix_lens[b]
 * tokens and appends chunk_len new ones, whose K and V the caller has already written
 * into the pages at positions prefix_lens[b] .. prefix_lens[b] + chunk_len - 1. New
 * token i attends to keys 0 .. prefix_lens[b] + i of its own sequence (the causal mask
 * with an offset), read through the block table ("快速注意力内核与算子融合", Q&A on
 * paged attention and on FlashAttention; the pages do not describe the combination).
 * The V of a masked key enters a query's product with weight 0, so all of those slots must
 * hold finite values, also where a shorter chunk is padded to chunk_len.
 *
 *   q, out      : bf16 [batch][chunk_len][n_qo_heads][head_dim], contiguous
 *   k_pages, v_pages, block_table : the paged layout above (bf16 pools)
 *   prefix_lens : int32 [batch]; prefix_lens[b] + chunk_len must fit the table's
 *                 max_blocks_per_seq pages (else PKV_DEVERR_BAD_LEN, computed on a
 *                 clamped length)
 *   lse         : fp32 [batch][n_qo_heads][chunk_len] (nullable)
 * Both products run on the tcgen05 tensor cores (the prefill kernel's paged mode). Built
 * for bf16, head_dim 128, page_size 16 and GQA groups dividing 128; all pointers 16-byte
 * aligned.
 */
int attn_prefill_paged_chunk(const void* q, const void* k_pages, const void* v_pages,
                             const int32_t* block_table, const int32_t* prefix_lens, void* out,
                             float* lse, int batch, int chunk_len, int max_blocks_per_seq,
                             int num_pages, int n_qo_heads, int n_kv_heads, int head_dim,
                             int page_size, float scale, int dtype, int32_t* err_flag,
                             void* stream);

/*
 * Merge two partial softmax states over disjoint key sets into one
 * ("【FlashAttention-V4，非官方】FlashDecoding++", section 1: partial softmax
 * results are updated at the end):
 *   M = max(lse_a, lse_b), w_x = exp(lse_x - M),
 *   out = (w_a out_a + w_b out_b) / (w_a + w_b), lse = M + ln(w_a + w_b).
 * Two -inf sides give out = 0, lse = -inf.
 *
 *   out_a, out_b : fp32 [n_rows][head_dim];  lse_a, lse_b : fp32 [n_rows]
 *   out          : out_dtype [n_rows][head_dim]; with out_dtype PKV_F32 it may
 *                  alias out_a or out_b exactly
 *   lse          : fp32 [n_rows] (nullable); may alias lse_a or lse_b exactly
 * n_rows is every leading dimension flattened (e.g. batch * heads).
 */
int attn_merge_states(const float* out_a, const float* lse_a, const float* out_b,
                      const float* lse_b, void* out, float* lse, int n_rows, int head_dim,
                      int out_dtype, void* stream);

/*
 * Causal self-attention for prefill: query i of a sequence attends to keys
 * 0..i of the same sequence. The query length equals the key length.
 *
 *   q, out : [batch][seq_len][n_qo_heads][head_dim], dtype, contiguous
 *   k, v   : [batch][seq_len][n_kv_heads][head_dim], dtype, contiguous
 *   lse    : fp32 [batch][n_qo_heads][seq_len] (nullable)
 *
 * The work is tiled as in FlashAttention: per tile, compute the scores,
 * update the softmax statistics and accumulate the output on chip, so the
 * T x T score matrix never reaches HBM ("快速注意力内核与算子融合", Q&A on
 * FlashAttention). Both products run on the tcgen05 tensor cores with fp32
 * accumulators in tensor memory, fed by TMA. All pointers must be 16-byte
 * aligned.
 */
int attn_prefill_causal(const void* q, const void* k, const void* v, void* out, float* lse,
                        int batch, int seq_len, int n_qo_heads, int n_kv_heads, int head_dim,
                        float scale, int dtype, int32_t* err_flag, void* stream);

/* Workspace bytes attn_decode_cascade needs (fp32 partial states). (size_t)-1 on bad args. */
size_t attn_cascade_workspace_size(int n_requests, int prefix_len, int max_suffix_blocks,
                                   int n_qo_heads, int n_kv_heads, int head_dim, int page_size);

/*
 * Cascade (shared-prefix) decode. Every request's sequence is one shared prefix,
 * whose pages are listed once in prefix_block_table, followed by that request's
 * own suffix pages. Two readings meet here: "级联推理", which splits attention
 * into stages that each handle part of the data (FlashInfer page, sections 2
 * and 4), and prefix sharing in the paged cache ("快速注意力内核与算子融合", Q&A
 * on paged attention). The prefix is attended once per KV head for the queries
 * of all requests and that KV head's query heads, as one tensor-core product.
 * The suffix is attended per request. The two partial states are merged by
 * log-sum-exp.
 *
 *   q, out             : [n_requests][n_qo_heads][head_dim], dtype
 *   lse                : fp32 [n_requests][n_qo_heads] (nullable)
 *   prefix_block_table : int32 [ceil(prefix_len / page_size)]
 *   suffix_block_table : int32 [n_requests][max_suffix_blocks]
 *   suffix_lens        : int32 [n_requests] (0 allowed)
 *   workspace          : >= attn_cascade_workspace_size bytes, 256-byte aligned
 * The result equals attn_decode_paged over the concatenated sequences, up to
 * rounding.
 *
 * With 4 or 8 query heads per KV head (bf16, head_dim 128) the suffix runs on the
 * tensor-core decode, one unit per (request, KV head), launched on `stream` right after
 * the prefix product so that it starts while the prefix product finishes (programmatic
 * dependent launch); each unit waits for the prefix grid only before it merges the
 * prefix's partial states with its own and writes the request's rows. Other groups run
 * the prefix product on a side stream of the library's (one per device, created with two
 * events on first use and kept for the life of the process), forked from and joined back
 * into `stream` with events, so that it overlaps the CUDA-core suffix decode, and a merge
 * kernel combines the states. Either way the call completes in `stream` order and may be
 * captured.
 */
int attn_decode_cascade(const void* q, const void* k_pages, const void* v_pages,
                        const int32_t* prefix_block_table, int prefix_len,
                        const int32_t* suffix_block_table, const int32_t* suffix_lens, void* out,
                        float* lse, int n_requests, int max_suffix_blocks, int num_pages,
                        int n_qo_heads, int n_kv_heads, int head_dim, int page_size, float scale,
                        int dtype, void* workspace, size_t workspace_bytes, int32_t* err_flag,
                        void* stream);

/*
 * Flat GEMM of the decode phase: y = x w^T for a few tokens ("【FlashAttention-V4，非官方】
 * FlashDecoding++", section 4, Flat GEMM Optimization with Double Buffering; the problem is
 * stated in sections 1 and 2). In decode the projections either side of attention see only
 * a few tokens at a time, so the GEMM is flat (with one token, a GEMV); the page pads the
 * token dimension with zeros to 8 instead of the libraries' 64 and overlaps the loads of
 * the next tile with the products of the current one with two shared-memory buffers.
 *
 *   x : bf16 [m][k], the m tokens, row-major
 *   w : bf16 [n][k], the k x n weight operand passed transposed (each of its n columns
 *       contiguous, as projection weights are stored)
 *   y : bf16 [m][n] = x w^T, fp32 accumulation, rounded to nearest even; must not alias
 *       x or w
 * Built for dtype PKV_BF16, 1 <= m <= 64, k >= 1 a multiple of 8 (16-byte rows), any n;
 * x and w 16-byte aligned. m = 0 or n = 0 does nothing. Other shapes return
 * PKV_ERR_UNSUPPORTED. err_flag (nullable) gets PKV_DEVERR_TIMEOUT if a bounded wait gave
 * up; the 128 columns of y that CTA group owns are then NaN.
 *
 * The weights stream through the tcgen05 tensor cores 128 rows at a time (the product's M
 * dimension); the tokens are the product's N dimension, padded with zeros to 16, 32 or 64
 * by the TMA loads (16 is the narrowest product with 128 rows). A ring of shared-memory
 * stages, fed by TMA, overlaps the loads of the next 64-column slice of K with the
 * products of the current one (the page's double buffering, with more than two buffers).
 * K is split over a thread-block cluster of up to 8 CTAs, whose partial tiles are summed
 * through distributed shared memory: one launch, and no workspace.
 */
int attn_flat_gemm(const void* x, const void* w, void* y, int m, int n, int k, int dtype,
                   int32_t* err_flag, void* stream);

/*
 * Write of new tokens into the paged cache, with the per-head norms and the rotary position
 * rotation of queries and keys in the same pass: what runs between the QKV projection and
 * attn_decode_paged (chunk_len 1) or attn_prefill_paged_chunk. New token i of sequence b
 * goes to cache position prefix_lens[b] + i. For every query and key head row x:
 *   y = x * rsqrt(mean(x^2) + norm_eps) * norm[head_dim]      (q_norm / k_norm; NULL: y = x)
 *   a pair (a, b) of y turns by t = position[axis] * inv_freq[pair]:
 *   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
 * in fp32, rounded once. Values are copied. Elements from rotary_dim on are not rotated.
 *
 *   q, k, v      : dtype; token t = b * chunk_len + i at q + t * q_stride (k_stride, v_stride;
 *                  in elements), its [n_qo_heads] ([n_kv_heads]) rows of head_dim contiguous
 *                  from there, so q, k and v may be slices of one fused projection. Strides
 *                  are multiples of 4 elements, at least heads * head_dim; pointers aligned
 *                  to 4 elements (16 bytes for PKV_F32, 8 for PKV_BF16)
 *   q_norm, k_norm : dtype [head_dim], or NULL for no norm; aligned like q
 *   inv_freq     : fp32 [rotary_dim / 2], radians per position (finite; another value makes
 *                  its pair NaN); may be NULL when rotary_dim is 0
 *   rotary_dim   : 0 (no rotation) or a multiple of 8, at most head_dim
 *   interleaved  : 0: pair p is elements (p, p + rotary_dim / 2); 1: (2 p, 2 p + 1)
 *   positions    : int32 [n_axes][batch][chunk_len] (any value, also negative), or NULL:
 *                  prefix_lens[b] + i on every axis. They are separate from the cache
 *                  positions, which fall behind once attn_cache_evict has shortened a cache
 *   pair_axis    : int32 [rotary_dim / 2], the axis (0 .. n_axes - 1) that each pair turns
 *                  by, e.g. time, height and width; NULL: axis 0. 1 <= n_axes <= 4. An entry
 *                  outside the range sets PKV_DEVERR_BAD_AXIS and makes its pair NaN
 *   chunk_lens   : int32 [batch], new tokens of each sequence (0 .. chunk_len), the rest of
 *                  its row being padding; NULL: chunk_len each
 *                  (attn_prefill_paged_chunk takes none: for ragged chunks its padding queries
 *                  read the slots behind a sequence, up to prefix_lens[b] + chunk_len, which this
 *                  call leaves as they were. The table needs pages for them and they must hold
 *                  finite values, as in a pool that was zeroed when it was made; the rows of the
 *                  queries that count then do not depend on them. A NaN there reaches those rows)
 *   q_out        : dtype [batch][chunk_len][n_qo_heads][head_dim], contiguous, aligned like
 *                  q; may be q itself when q_stride = n_qo_heads * head_dim, and must not overlap
 *                  another input or a pool (their addresses are refused). Padding rows are
 *                  left as they were
 *   k_pages, v_pages, block_table : the paged layout above (two pools, 16-byte aligned; one for both is
 *                  refused)
 * A sequence with prefix_lens[b] < 0, chunk_lens[b] outside its range, or prefix_lens[b] +
 * chunk_lens[b] past the table sets PKV_DEVERR_BAD_LEN, a bad table entry
 * PKV_DEVERR_BAD_PAGE; the q_out rows of such tokens are NaN and their K and V are not
 * written. Two new tokens must not share a cache slot. Angles are taken modulo a turn exactly
 * (fixed point), so far positions lose no precision.
 */
int attn_qk_norm_rope_append(const void* q, const void* k, const void* v, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, const void* q_norm,
                             const void* k_norm, float norm_eps, const float* inv_freq,
                             int rotary_dim, int interleaved, const int32_t* positions, int n_axes,
                             const int32_t* pair_axis, const int32_t* block_table,
                             const int32_t* prefix_lens, const int32_t* chunk_lens, void* q_out,
                             void* k_pages, void* v_pages, int batch, int chunk_len,
                             int max_blocks_per_seq, int num_pages, int n_qo_heads, int n_kv_heads,
                             int head_dim, int page_size, int dtype, int32_t* err_flag,
                             void* stream);

/*
 * Accumulated attention weights: how much softmax weight every cached token has received,
 * summed over decode steps (and prompt chunks) per KV head, which is what
 * attn_cache_evict ranks tokens by.
 *
 *   sums : fp32 [batch][n_kv_heads][max_blocks_per_seq * page_size], row b in step with row b
 *          of the block table; 16-byte aligned
 *
 * attn_decode_paged_weights is attn_decode_paged that also adds the step's weights:
 *   sums_out[b][g][t] = decay * sums_in[b][g][t] + sum_{h in group g} exp(scale q_h . k_t - lse_h)
 * for t < kv_lens[b]; slots at or past the length are neither read nor written, so the sums of
 * the newest token must have been set (to 0) before. sums_out may be sums_in (in place), and
 * must not overlap it otherwise. decay is finite (1: plain accumulation). out, lse, splits and
 * errors are as for attn_decode_paged (out is closer to the exact value than that call's where
 * the tensor cores take the weights: two bf16 parts of each, 2^-17 of the weight, not one; infinite V
 * makes infinite out, as there); a row that came out
 * NaN makes its group's sums NaN, and a bad length leaves the sequence's sums as they were. workspace: at least
 * attn_decode_weights_workspace_size bytes, 256-byte aligned: the split partials, the call's
 * logits (fp32 [batch][n_qo_heads][max_blocks_per_seq * page_size]) and log-sum-exps.
 */
size_t attn_decode_weights_workspace_size(int batch, int max_blocks_per_seq, int n_qo_heads,
                                          int n_kv_heads, int head_dim, int page_size,
                                          int num_splits, int dtype);

int attn_decode_paged_weights(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* block_table, const int32_t* kv_lens, void* out,
                              float* lse, const float* sums_in, float* sums_out, int batch,
                              int max_blocks_per_seq, int num_pages, int n_qo_heads,
                              int n_kv_heads, int head_dim, int page_size, float scale, float decay,
                              int num_splits, int dtype, void* workspace, size_t workspace_bytes,
                              int32_t* err_flag, void* stream);

/*
 * The same accumulation for a chunk of queries whose log-sum-exps are known (the lse of
 * attn_prefill_paged_chunk on the same q, pages, table and prefix_lens):
 *   sums_out[b][g][t] = decay * sums_in[b][g][t]
 *                       + sum_{i} sum_{h in group g} exp(scale q_ih . k_t - lse_h(i))
 * over the queries i >= t - prefix_lens[b] (the causal mask) among the last `window` of the
 * sequence's new tokens (window 0: all of them), for t < prefix_lens[b] + n; other slots are
 * neither read nor written. n = chunk_lens[b] where given (0 .. chunk_len; the rest of the
 * chunk is padding whose q and lse do not matter), else chunk_len. Without queries (n = 0, also by
 * chunk_len = 0, where q and lse may be NULL) the sums of the prefix_lens[b] keys decay. (A call
 * with chunk_len 0, decay 1 and sums in place has nothing to do and does not look at the lengths.)
 *
 *   q    : bf16 [batch][chunk_len][n_qo_heads][head_dim]
 *   lse  : fp32 [batch][n_qo_heads][chunk_len]
 *   sums : as above; sums_out may be sums_in; q and k_pages 16-byte aligned
 * A bad length sets PKV_DEVERR_BAD_LEN and leaves the sequence's sums as they were; a bad table
 * entry sets PKV_DEVERR_BAD_PAGE and makes its keys' sums NaN. bf16, head_dim 128, page_size 16,
 * groups dividing 128. The product runs on the tcgen05 tensor cores.
 */
int attn_chunk_weights(const void* q, const void* k_pages, const int32_t* block_table,
                       const int32_t* prefix_lens, const int32_t* chunk_lens, const float* lse,
                       const float* sums_in, float* sums_out, int batch, int chunk_len, int window,
                       int max_blocks_per_seq, int num_pages, int n_qo_heads, int n_kv_heads,
                       int head_dim, int page_size, float scale, float decay, int dtype,
                       int32_t* err_flag, void* stream);

/*
 * Eviction from the paged cache: every sequence is cut to at most `budget` tokens per KV head.
 * A KV head of a sequence with n = kv_lens[b] > budget tokens keeps the first n_sink, the last
 * n_recent and, of those between, the budget - n_sink - n_recent with the largest sums (equal
 * sums: the lower index first; NaN counts as the largest), in their order; with n <= budget it
 * keeps all. The kept rows of K and V are copied into the pages of new_block_table, in the same
 * pools, and the caller then goes on with the new table, lengths and sums and frees the old
 * pages. Heads keep different tokens, so cache positions say nothing about token positions
 * any more: attn_qk_norm_rope_append takes those separately.
 *
 *   block_table     : int32 [batch][max_blocks_per_seq], kv_lens: int32 [batch]
 *   sums            : fp32 [batch][n_kv_heads][max_blocks_per_seq * page_size], 16-byte aligned
 *   new_block_table : int32 [batch][new_max_blocks]; new_max_blocks * page_size >= budget. The
 *                     first ceil(min(n, budget) / page_size) entries of a row are used; those
 *                     pages must not occur in the old pages in use, nor twice (a page that does
 *                     is left with mixed contents). Old pages may be shared between sequences
 *   kept            : int32 [batch][n_kv_heads][budget], out: old index of new token j, -1 at
 *                     and past the new length
 *   new_lens        : int32 [batch], out: min(n, budget)
 *   new_sums        : fp32 [batch][n_kv_heads][new_max_blocks * page_size], out: the kept
 *                     tokens' sums, 0 at and past the new length
 * Outputs must not overlap inputs or one another (the same address is refused). A length < 0 or past the
 * table sets PKV_DEVERR_BAD_LEN and counts as 0. A bad entry of block_table sets
 * PKV_DEVERR_BAD_PAGE and makes the rows NaN; a bad entry of new_block_table sets it too and
 * its rows are not copied.
 */
int attn_cache_evict(void* k_pages, void* v_pages, const int32_t* block_table,
                     const int32_t* kv_lens, const float* sums, const int32_t* new_block_table,
                     int32_t* kept, int32_t* new_lens, float* new_sums, int batch,
                     int max_blocks_per_seq, int new_max_blocks, int num_pages, int n_kv_heads,
                     int head_dim, int page_size, int budget, int n_sink, int n_recent, int dtype,
                     int32_t* err_flag, void* stream);

/*
 * Linear layer with its epilogue: y = act(x w^T + bias) + residual, for any number of tokens:
 * the projections on either side of the attention, with what follows them in the same pass.
 *
 *   x : bf16 [m][k];  w : bf16 [n][k] (16-byte aligned both)
 *   bias : bf16 [n], or NULL;  residual : bf16 [m][n], or NULL (2-byte aligned both)
 *   activation : PKV_ACT_*
 *   y : bf16 [m][n]; may be residual itself, and must not overlap an input otherwise (the
 *     address of x, w or bias is refused)
 * The product accumulates in fp32; bias, activation and residual are applied in fp32 and the
 * result is rounded once. k >= 1 a multiple of 8. m = 0 or n = 0 does nothing. err_flag
 * (nullable) gets PKV_DEVERR_TIMEOUT if a bounded wait gave up; the outputs affected are NaN.
 * Small results keep their relative precision, down to the smallest numbers of bf16. Few tokens
 * (at most 64) run as attn_flat_gemm does where the weights' stream is most of the time, the rest
 * on a tiled kernel.
 */
int attn_linear(const void* x, const void* w, const void* bias, const void* residual, void* y,
                int m, int n, int k, int activation, int dtype, int32_t* err_flag, void* stream);

/*
 * 4-bit pages. A pool holds E2M1 codes (a sign, two bits of exponent, one of fraction: 0, 0.5, 1, 1.5,
 * 2, 3, 4, 6 and their negatives), 16 consecutive elements of a token sharing one E4M3 scale, and there
 * is a float scale for each KV head: value = e2m1(code) * e4m3(scale) * head scale. That is 4.5 bits an
 * element. The scales belong to tokens, so new tokens can join a page that holds others already.
 *
 *   k_pages, v_pages : bytes [num_pages][n_kv_heads][9 * head_dim]; the tile of a (page, KV head) is
 *                      codes [16][head_dim / 2] (element 2 i of a token in the low half of byte i,
 *                      2 i + 1 in the high half), then scales [head_dim / 16][16] (by group, then by
 *                      token); 16-byte aligned
 *   k_scale, v_scale : fp32 [n_kv_heads], finite and at least 2^-126 in magnitude, or NULL (1 for every head). A
 *                      head's largest magnitude over 2688 (6 * 448) uses the whole range of the scales
 *
 * attn_cache_pack_fp4 writes tokens of ordinary pages into 4-bit pages: new tokens that
 * attn_qk_norm_rope_append has put into the pages of a step, or a prompt after its prefill. Token i of
 * sequence b, i < counts[b], goes from position src_first[b] + i of src_table's pages to position
 * first[b] + i of block_table's. For each 16 elements x, with one rounding (to nearest even) a step:
 *   y = x * (1 / head scale);  s = e4m3(max |y| * (1 / 6)), at most 448;  code = e2m1(y * (1 / s)), at most 6
 * s = 0 has codes 0. An element whose y is not finite makes its group's scale NaN: all 16 read as NaN.
 *
 * attn_cache_unpack_fp4 reads tokens back into ordinary pages, where attn_prefill_paged_chunk and the
 * other calls take them: x = (e2m1(code) * e4m3(s)) * head scale, rounded once more to the type of the pages.
 *
 *   k_src, v_src, k_dst, v_dst : src_dtype / dst_dtype [src_num_pages / dst_num_pages][n_kv_heads]
 *                      [page_size][head_dim], 32-byte aligned
 *   src_table, dst_table : int32 [batch][src_max_blocks / dst_max_blocks]
 *   block_table      : int32 [batch][max_blocks_per_seq]
 *   first, src_first, dst_first : int32 [batch], positions of the first tokens, or NULL: 0
 *   counts           : int32 [batch], 0 .. max_count
 *   max_count        : no count is above it (it bounds the launch); 0: what the smaller table holds
 * Slots of other tokens keep what they hold. A sequence with a bad count or position sets
 * PKV_DEVERR_BAD_LEN and nothing of it is written. A bad table entry sets PKV_DEVERR_BAD_PAGE: tokens
 * that would go there, or would be packed from there, are not written; what is unpacked from there is NaN.
 * Two tokens of a call must not share a slot. Outputs must not overlap inputs (their addresses are refused).
 */
int attn_cache_pack_fp4(const void* k_src, const void* v_src, const int32_t* src_table,
                        const int32_t* src_first, void* k_pages, void* v_pages,
                        const int32_t* block_table, const int32_t* first, const int32_t* counts,
                        const float* k_scale, const float* v_scale, int batch, int max_count,
                        int src_max_blocks, int src_num_pages, int max_blocks_per_seq, int num_pages,
                        int n_kv_heads, int head_dim, int page_size, int src_dtype, int32_t* err_flag,
                        void* stream);

int attn_cache_unpack_fp4(const void* k_pages, const void* v_pages, const int32_t* block_table,
                          const int32_t* first, void* k_dst, void* v_dst, const int32_t* dst_table,
                          const int32_t* dst_first, const int32_t* counts, const float* k_scale,
                          const float* v_scale, int batch, int max_count, int max_blocks_per_seq,
                          int num_pages, int dst_max_blocks, int dst_num_pages, int n_kv_heads,
                          int head_dim, int page_size, int dst_dtype, int32_t* err_flag, void* stream);

/*
 * Decode over 4-bit pages: the attention of attn_decode_paged over the values that the pages stand for.
 * q and out are bf16 and 16-byte aligned, lse, splits, workspace (attn_decode_workspace_size and
 * attn_decode_num_splits with PKV_FP4_E2M1) and err_flag as there. Group sizes 1 to 8.
 * Arithmetic: a code times its scale is exact in f16; q is scaled per head by a power of two and held in f16 as
 * in attn_decode_paged_fp8; a softmax weight enters the sum over V rounded to f16, off by 2^-11 of itself or by 2^-32 of the
 * largest (2^-25 where logits pass 2^20 in magnitude) before the division by their sum, which has them
 * unrounded; sums and statistics are fp32. A row with logits past 2^23, where fp32 is in whole steps, may be NaN.
 * Slots behind a sequence's length do not matter, whatever bytes they hold. Both products run on the tensor
 * cores; there is no bounded wait in this call, so attn_debug_decode_stall does not act on it.
 */
int attn_decode_paged_fp4(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                          const float* v_scale, const int32_t* block_table, const int32_t* kv_lens,
                          void* out, float* lse, int batch, int max_blocks_per_seq, int num_pages,
                          int n_qo_heads, int n_kv_heads, int head_dim, int page_size, float scale,
                          int num_splits, void* workspace, size_t workspace_bytes, int32_t* err_flag,
                          void* stream);

/*
 * Pages of the pools. A page is in use if a row of the block table lists it among the first
 * ceil(kv_lens[b] / page_size) entries, or if the caller holds it; every other page is free. Nothing is
 * kept between calls: a sequence's pages are freed by setting its length to 0, and a sequence is forked
 * by copying its row and length to another row (ends of both may differ); the pages are then shared.
 *
 *   block_table     : int32 [batch][max_blocks_per_seq];  kv_lens : int32 [batch]
 *   new_block_table : the same shape, out; may be block_table itself, and must not overlap it otherwise
 *   held            : uint8 [num_pages], not 0: the caller holds the page; or NULL: none
 *   pools           : host array of n_pools pools with one table: K and V of every layer, scales too.
 *                     page_bytes bytes a page, [num_pages] pages from base; both multiples of 4
 *   workspace       : at least attn_cache_pages_workspace_size bytes, 256-byte aligned
 *
 * attn_cache_reserve gives every sequence the pages for the tokens kv_lens[b] .. new_lens[b] - 1 that
 * are to be written next: an entry for each block past its last, and, where its last block is not
 * full and others use that page too, a page of its own with the contents copied. Of the sequences that
 * share such a page the one with the most tokens in it goes on writing it (equal: the lower row), unless
 * the page is held: what it writes lies behind what the others read. Free pages are taken in order, lowest
 * first, by row and block. new_lens[b] <= kv_lens[b]: nothing. Entries that are not given keep their values.
 *   new_lens : int32 [batch]
 *   n_free   : int32 [1], out: the free pages left; below 0: so many are missing, PKV_DEVERR_NO_PAGES is set
 *              and the table stays as it was; or NULL
 *
 * attn_cache_compact moves pages so that the pages in use (their number is n) become 0 .. n - 1: the k-th
 * used page behind them moves to the k-th free one among them, in every pool, and the rest stay. Table
 * entries behind a length keep their values, and may name pages that have moved.
 *   page_map : int32 [num_pages], out: where each page went, -1 for a free one (held pages move, too)
 *   n_used   : int32 [1], out: n; or NULL
 *
 * A length below 0 or past the table, or a new length past it, sets PKV_DEVERR_BAD_LEN: the sequence gets
 * nothing (a length past the table counts as the whole row, below 0 as none). An entry in use that is
 * no page sets PKV_DEVERR_BAD_PAGE and is left as it is.
 */
typedef struct {
  void* base;
  int64_t page_bytes;
} attn_pool_t;

size_t attn_cache_pages_workspace_size(int batch, int max_blocks_per_seq, int num_pages);

int attn_cache_reserve(const int32_t* block_table, const int32_t* kv_lens, const int32_t* new_lens,
                       const uint8_t* held, int32_t* new_block_table, int32_t* n_free,
                       const attn_pool_t* pools, int n_pools, int batch, int max_blocks_per_seq,
                       int num_pages, int page_size, void* workspace, size_t workspace_bytes,
                       int32_t* err_flag, void* stream);

int attn_cache_compact(const int32_t* block_table, const int32_t* kv_lens, const uint8_t* held,
                       int32_t* new_block_table, int32_t* page_map, int32_t* n_used,
                       const attn_pool_t* pools, int n_pools, int batch, int max_blocks_per_seq,
                       int num_pages, int page_size, void* workspace, size_t workspace_bytes,
                       int32_t* err_flag, void* stream);

/*
 * Failure-handling hook for tests (the pages have no counterpart). It lets a test make a
 * bounded wait inside the decode kernel run out, without faulting or hanging anything:
 * after attn_debug_decode_stall(page, wait_limit_ns) with page >= 0, every launch of
 * attn_decode_paged, attn_decode_paged_unified_max, attn_decode_paged_weights,
 * attn_decode_paged_fp8 and attn_decode_paged_noalloc in this process has the producer warp of each CTA withhold
 * the copies of the page-th page of its split (on the tensor-core path: the K copies of
 * the 128-key tile that holds it) and the arrival that would announce them, and every
 * pipeline wait of those launches gives up after wait_limit_ns nanoseconds (0 keeps the
 * default of 2 s). The consumer waiting for that page then times out: the kernel ORs
 * PKV_DEVERR_TIMEOUT into err_flag, waits (within the same limit) for the copies it did
 * issue, writes the rows (or split partials) of the unit it was working on, and of any
 * later unit it had taken, as NaN and returns, so the context stays usable. attn_debug_decode_stall(-1, 0) turns it off. Not for use
 * beside production calls: the setting is process-wide. Returns PKV_OK, or
 * PKV_ERR_INVALID_ARG for page < -1 or a limit above 10 s.
 */
int attn_debug_decode_stall(int page, unsigned long long wait_limit_ns);

/* How many CTAs (the cluster size, 1..8) share K for this shape on the current device;
 * a negative PKV_ERR_* code for shapes attn_flat_gemm rejects. */
int attn_flat_gemm_num_splits(int m, int n, int k);

#ifdef __cplusplus
}
#endif

#endif /* PKV_ATTN_H */
