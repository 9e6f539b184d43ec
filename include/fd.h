/*
 * fd.h -- C ABI of libfd.so: length-aware GQA decode attention over a
 * preallocated KV cache, for NVIDIA GB300 (sm_103a).
 *
 * What the calls compute.  For sequence b, query row i, query head h and
 * kv head hk = h / (Hq / Hkv):
 *
 *     out[b,i,h,:] = sum_{j in V} softmax_j(scale * q[b,i,h,:] . k[b,hk,j,:]) v[b,hk,j,:]
 *
 * over the visible cache positions V, and 0 where V is empty.
 *   - fd_decode / fd_decode_int8: V = the filled prefix 0 .. L-1 with
 *     L = kv_lengths[b] read on the device, so the call never touches the
 *     unused tail of the cache ("Qwen3.5 text generation attends over the
 *     full KV capacity", ComfyUI #16509: problem statement and the
 *     length-aware FixedKV path).  With causal != 0 the n_q query rows are
 *     the newest n_q positions of the cache (the decode token plus MTP
 *     drafts already written at L-n_q .. L-1) and row i sees 0 .. L-n_q+i
 *     (same issue, list item 2 and "Existing Solutions": a bottom-right
 *     aligned causal window, up to 6 rows).
 *     fd_decode_paged computes the same over a paged cache,
 *     fd_decode_append after writing the step's new rows into the cache, and
 *     fd_decode_masked with an additive mask over the prefix.
 *   - fd_decode_gather: V = the cells listed for that (b, i) in idx
 *     ("attend the selected cells instead of masking the window",
 *     llama.cpp #28244, Conversation; "gather-based sparse attention for
 *     QSA decode", llama.cpp #28213: per-token lists for multi-row verify);
 *     fd_decode_gather_bias adds a bias per list entry, and fd_topk_blocks
 *     builds the lists from block scores.
 *   - fd_decode_fp4: the dense prefix over a cache held in 4 bits, flat or
 *     paged; fd_append_fp4 writes such a cache and fd_read_fp4 reads rows of
 *     it back.
 *   - fd_append writes new rows into a bf16 or int8 cache, flat or paged, and
 *     rotates keys and queries to their positions; fd_prefill attends a chunk
 *     of many new tokens over such a cache.
 *   - fd_pages_*: who holds which page of a paged cache, and copies of pages.
 *   - fd_beam_select: the best continuations of a beam search, whose rows of
 *     the block table fd_pages_reorder then puts in place.
 * The prefix is split across thread blocks and the last block to finish a
 * (sequence, kv head) combines the splits inside the same launch
 * (comfy-kitchen #239, "GQA decode"); the query heads of one GQA group share
 * each K/V tile.
 *
 * Conventions shared by every call.
 *   - Tensors are described by fd_tensor: a data pointer, a dtype, 4 sizes
 *     and 4 strides counted in ELEMENTS.  The innermost (head_dim) stride
 *     must be 1.  Device pointers unless stated otherwise.
 *   - q      : [B, n_q, Hq, d] bf16.
 *   - caches : [B, Hkv, cap, d] bf16 (fd_decode, fd_decode_gather) or int8
 *              (fd_decode_int8); any strides that are multiples of 16 bytes,
 *              so the canonical [B, Hkv, cap, d] and the token-major
 *              [B, cap, Hkv, d] (seen through a transpose) both work; the
 *              data pointer must be 16-byte aligned.
 *   - out    : [B, n_q, Hq, d] bf16 or fp32 (round to nearest even for bf16).
 *   - d (head_dim) is 128 or 256; 1 <= n_q <= 6; Hq % Hkv == 0;
 *     (Hq / Hkv) * n_q <= 64 query rows share one kv head per launch unit.
 *   - The caller owns every tensor, kv_lengths and idx.  The library owns
 *     only the workspace (fd_workspace_create) and never allocates, frees or
 *     synchronises inside a decode call, and never reads device data on the
 *     host, so the calls can be captured in a CUDA graph and replayed with
 *     new lengths or index lists written on the device.
 *   - Work is queued on opts->stream (a cudaStream_t; NULL = the legacy
 *     default stream).  One workspace serves one stream at a time.
 *   - Return value: FD_OK, or a negative FD_ERR_* code.  Every argument is
 *     checked on the host before any CUDA call; on error nothing is
 *     launched.  FD_ERR_CUDA reports a launch failure (cudaGetLastError).
 *   - Bad device-side data (a length outside [0, cap], an index >= cap) never
 *     faults: the value is clamped or the cell skipped, and a sticky bit is
 *     set in the workspace status word (fd_get_device_status).
 */
#ifndef FD_H
#define FD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define FD_OK 0
#define FD_ERR_ARG (-1)          /* null pointer, bad shape/dtype/stride   */
#define FD_ERR_UNSUPPORTED (-2)  /* head_dim, n_q or group size not served */
#define FD_ERR_ALIGN (-3)        /* pointer or stride not 16-byte aligned  */
#define FD_ERR_WORKSPACE (-4)    /* missing or too small workspace         */
#define FD_ERR_CUDA (-5)         /* CUDA runtime error                     */
#define FD_ERR_SCRATCH (-6)      /* problem exceeds fd_decode_noalloc's fixed scratch */

/* dtypes */
#define FD_BF16 0
#define FD_F32 1
#define FD_I8 2
#define FD_I32 3
#define FD_U8 4                  /* bytes; two e2m1 codes each in a 4-bit cache */
#define FD_E4M3 5                /* 8-bit floats, the scales of a 4-bit cache  */

/* sticky device status bits (fd_get_device_status) */
#define FD_DEV_BAD_LENGTH 1      /* some kv_lengths[b] outside [0, cap]    */
#define FD_DEV_BAD_INDEX 2       /* some idx entry >= cap (skipped)        */
#define FD_DEV_INTERNAL 4        /* a bounded internal wait gave up; the
                                    call's output is not valid              */
#define FD_DEV_NO_PAGES 8        /* fd_pages_reserve: fewer free pages than
                                    wanted; nothing was reserved            */

/* kernel selection (fd_opts.kernel); AUTO takes the tensor-core kernel for
 * the calls it serves when q's base pointer and strides are 16-byte aligned
 * (q is read through a TMA tensor map there), the CUDA-core kernel
 * otherwise */
#define FD_KERNEL_AUTO 0
#define FD_KERNEL_SIMT 1         /* CUDA-core kernel, every mode           */
#define FD_KERNEL_TC 2           /* tensor-core (tcgen05) kernel: bf16
                                    caches (head_dim 128/256, up to 64
                                    rows) and int8 caches (head_dim
                                    128/256, up to 32 rows; flat dense
                                    int8 with more rows in parts, see
                                    fd_decode_int8), flat or paged
                                    (pools whose rows form one strided 2-D
                                    array), the fused append and the
                                    masked prefix over flat bf16 caches,
                                    and gather over bf16 or int8 caches
                                    whose rows form one strided 2-D array;
                                    16-byte aligned q (else
                                    FD_ERR_UNSUPPORTED)                    */

#define FD_MAX_ROWS 64           /* query rows per kv head per launch unit */

typedef struct fd_tensor {
    void *data;
    int32_t dtype;               /* FD_BF16, FD_F32, FD_I8, FD_I32          */
    int32_t ndim;                /* 1 .. 4                                  */
    int64_t shape[4];
    int64_t stride[4];           /* in elements                             */
} fd_tensor;

/* Opaque device workspace: per-split partial results, one completion counter
 * per (sequence, kv head) and the sticky status word. */
typedef struct fd_workspace fd_workspace;

typedef struct fd_opts {
    void *stream;                /* cudaStream_t, NULL = legacy default      */
    fd_workspace *ws;            /* required                                 */
    int32_t num_ctas;            /* 0 = auto (from the SM count); > 0 forces
                                    the number of thread blocks, which sets
                                    the split count                          */
    int32_t kernel;              /* FD_KERNEL_*                              */
    float scale;                 /* fd_decode_gather only: 0 = 1/sqrt(d)     */
    int32_t wait_limit_us;       /* tensor-core kernel: bound on each of its
                                    internal waits, in microseconds; 0 = the
                                    default of 2 s.  A wait that runs out sets
                                    FD_DEV_INTERNAL and the launch ends (its
                                    output is then not valid).  Tests of that
                                    path shorten it; 1 .. 2e6.              */
    int32_t reserved[2];         /* must be zero                             */
} fd_opts;

/*
 * Dense prefix decode (bf16 cache).
 *   q [B, n_q, Hq, d] bf16; k_cache, v_cache [B, Hkv, cap, d] bf16;
 *   kv_lengths: device int32[B], L_b = number of filled positions;
 *   n_q: query rows (must equal q->shape[1]); causal: 0 or 1;
 *   scale: multiplies q.k (usually 1/sqrt(d));
 *   out [B, n_q, Hq, d] bf16 or fp32.
 */
int fd_decode(const fd_tensor *q, const fd_tensor *k_cache,
              const fd_tensor *v_cache, const int32_t *kv_lengths,
              int32_t n_q, int32_t causal, float scale, const fd_tensor *out,
              const fd_opts *opts);

/*
 * Dense prefix decode over an int8 cache with one fp32 scale per
 * (sequence, kv head, position): k = k_code * k_scale[b, hk, j], likewise v
 * (comfy-kitchen #239, commit list: bounded paged INT8 decode cache; the
 * cache here is not paged).  k_scale, v_scale: fp32 [B, Hkv, cap] with any
 * strides.  Other arguments as fd_decode.
 * On the tensor-core kernel the products run on fp16 operands: the codes
 * convert exactly, q is rounded to fp16 (exact for bf16 values of magnitude
 * 2^-14 .. 65504; larger ones saturate at 65504), and each softmax weight
 * (at most 16 before normalisation) times the position's v scale is held
 * in fp16 with about 2^-22 relative error, saturating at 65504 (a v scale
 * above 4094, i.e. dequantised |v| above about 5.2e5, can saturate).  The
 * CUDA-core kernel has no such range limit.  The same holds for every
 * int8 call (paged and gather).
 * The tensor-core kernel takes up to 32 rows (n_q * g) at once.  With more,
 * it serves each kv head's query heads in k parts of g / k heads, k the
 * fewest dividing g that bring n_q * g / k to 32 or fewer, each part a
 * segment of its own that reads the kv head's prefix again (k times the
 * cache bytes); the workspace then needs B * Hkv * k segments (B * Hq always
 * suffices).  Under FD_KERNEL_AUTO a workspace without that room, or a
 * shape with no such k (g = 1), takes the CUDA-core kernel, which reads the
 * prefix once; FD_KERNEL_TC returns FD_ERR_WORKSPACE or FD_ERR_UNSUPPORTED.
 */
int fd_decode_int8(const fd_tensor *q, const fd_tensor *k_cache,
                   const fd_tensor *v_cache, const fd_tensor *k_scale,
                   const fd_tensor *v_scale, const int32_t *kv_lengths,
                   int32_t n_q, int32_t causal, float scale,
                   const fd_tensor *out, const fd_opts *opts);

/*
 * Index-gather decode (bf16 cache).
 *   idx: device int32 [B, n_q, idx_len], contiguous (may be NULL when idx_len
 *   is 0: every output row is then 0); one list per (sequence,
 *   query row), shared by all heads of that row.  Entries < 0 are padding;
 *   entries >= cap are skipped and flag FD_DEV_BAD_INDEX.  Lists are read as
 *   given: a cell listed twice counts twice (distinct cells reproduce the
 *   masked path exactly).  No length and no causal mask apply: the list is
 *   the visible set.  Scale: opts->scale, or 1/sqrt(d) when 0.
 *   On the tensor-core kernel with opts->num_ctas = 0, lists of 2 to 16
 *   tiles of 128 entries whose (sequence, query row, kv head) lists all fit
 *   the device at once run as thread-block clusters, one per list, whose
 *   blocks merge their partial results through distributed shared memory
 *   instead of the workspace (the list length alone decides).
 */
int fd_decode_gather(const fd_tensor *q, const fd_tensor *k_cache,
                     const fd_tensor *v_cache, const int32_t *idx,
                     int32_t idx_len, const fd_tensor *out,
                     const fd_opts *opts);

/*
 * Gather lists from block scores (no counterpart call in the pages; the
 * step they ask for next): for each (sequence b, query row i), top_k of the
 * blocks are selected by score and only the winners are expanded to cells
 * ("qwen4exp : gather-based sparse attention for QSA decode", llama.cpp
 * #28213, review discussion: take top-k over blocks and expand only the
 * winners, instead of selecting over every cell).
 *   scores: device fp32 [B, n_q, n_blocks], contiguous; block j covers cells
 *     j*block_size .. (j+1)*block_size - 1.  Scores must not be NaN.
 *   kv_lengths: device int32 [B]; L_b clamped to [0, n_blocks*block_size].
 *     The candidates of row (b, i) are the blocks whose first cell is below
 *     L_b; the top_k highest scores win, ties going to the lower index
 *     (-0 and +0 tie).
 *   idx: device int32 [B, n_q, top_k*block_size], contiguous, written: the
 *     winners in increasing block order, each as its block_size cells, cells
 *     at or past L_b as -1, padded with -1 when fewer than top_k blocks are
 *     candidates.  The result feeds fd_decode_gather (idx_len =
 *     top_k*block_size).
 *   n_blocks <= 32768 (FD_ERR_UNSUPPORTED beyond); n_blocks*block_size below
 *   2^31.  Queued on `stream`; allocates nothing, reads nothing back,
 *   graph-capturable.  Returns FD_OK or a negative FD_ERR_* code.
 */
int fd_topk_blocks(const float *scores, int32_t B, int32_t n_q,
                   int32_t n_blocks, const int32_t *kv_lengths,
                   int32_t block_size, int32_t top_k, int32_t *idx,
                   void *stream);
/*
 * Index-gather decode over an int8 cache with per-position fp32 scales: as
 * fd_decode_gather, with k = k_code * k_scale[b, hk, cell] and v likewise,
 * k_scale / v_scale as in fd_decode_int8.  The gather measurements of
 * "qwen4exp : gather-based sparse attention for QSA decode" (llama.cpp
 * #28213, Additional information and review discussion) all run over a q8_0
 * (8-bit) KV cache.  The tensor-core kernel serves head_dim 128 / 256 with up
 * to 32 query rows per list (fetching each listed cell's codes with
 * tile::gather4); the CUDA-core kernel serves the rest.
 */
int fd_decode_gather_int8(const fd_tensor *q, const fd_tensor *k_cache,
                          const fd_tensor *v_cache, const fd_tensor *k_scale,
                          const fd_tensor *v_scale, const int32_t *idx, int32_t idx_len,
                          const fd_tensor *out, const fd_opts *opts);
/*
 * Index-gather decode with a per-entry score bias: as fd_decode_gather, and
 * bias[b, i, t] (fp32, device, [B, n_q, idx_len] contiguous, aligned with
 * idx) is added to the scaled score of list entry t ("qwen4exp :
 * gather-based sparse attention for QSA decode", llama.cpp #28213, Overview:
 * the mask entries are gathered with the cells).  An entry whose bias is
 * -inf is dropped, exactly as if it were padding; every other bias must be
 * finite.  bias = NULL is fd_decode_gather.
 */
int fd_decode_gather_bias(const fd_tensor *q, const fd_tensor *k_cache,
                          const fd_tensor *v_cache, const int32_t *idx,
                          const float *bias, int32_t idx_len,
                          const fd_tensor *out, const fd_opts *opts);
/*
 * Dense prefix decode with an additive mask, skipping hidden chunks: as
 * fd_decode, and mask[b, i, j] (fp32, device, [B, n_q, cap], positions
 * contiguous) is added to the scaled score of query row i at position j;
 * -inf hides the position.  A 32-position chunk that the mask and the window
 * hide for every query row of a sequence is not read at all: the masked scan
 * whose cost follows the visible chunks ("qwen4exp : gather-based sparse
 * attention for QSA decode", llama.cpp #28213, Metal measurements: the
 * FA-vec kernel skips fully masked 32-cell chunks).  Mask values must be
 * finite or -inf.  Both kernels serve it: the CUDA-core kernel skips a
 * hidden chunk (its tiles are 32 positions); the tensor-core kernel, whose
 * tiles are 128 positions, loads each tile as four 32-position chunks and
 * copies only the chunks some query row sees.  When the workspace holds
 * fd_masked_list_bytes(B, cap) bytes past the call's split partials
 * ((B*Hkv + num_ctas) slots of slot_floats(rows, d) floats, rows = (Hq/Hkv)
 * * n_q, as fd_workspace_bytes counts them), a first pass on the stream lists
 * each sequence's visible chunks in that room and the tensor-core launch
 * walks only the listed chunks, four to a 128-position tile, so its time
 * follows the visible chunks, not the length; with less room each tile of the
 * prefix finds its visible chunks in place.  Positions the mask hides must
 * hold finite values (they lie in the filled prefix).  Other arguments as
 * fd_decode.
 */
int fd_decode_masked(const fd_tensor *q, const fd_tensor *k_cache,
                     const fd_tensor *v_cache, const int32_t *kv_lengths,
                     const fd_tensor *mask, int32_t n_q, int32_t causal,
                     float scale, const fd_tensor *out, const fd_opts *opts);
/*
 * Dense prefix decode with a fused K/V append (bf16 caches): one launch
 * writes the step's new rows into the caches and attends over the prefix
 * including them, as flash_attn_with_kvcache does with k / v and
 * cache_seqlens ("Qwen3.5 text generation attends over the full KV
 * capacity", ComfyUI #16509: Existing Solutions).  For sequence b with
 * base_b = kv_lengths[b] (clamped to [0, cap]):
 *   - k_new[b, i, hk, :] and v_new[b, i, hk, :] are written to cache
 *     positions base_b + i, i = 0 .. n_q - 1 (positions at or past cap are
 *     not written, and FD_DEV_BAD_LENGTH is set);
 *   - the result is fd_decode's with L_b = min(base_b + n_q, cap): the n_q
 *     query rows are the new tokens, and with causal != 0 row i sees
 *     positions 0 .. base_b + i;
 *   - with update_lengths = 1, kv_lengths[b] becomes L_b when the launch
 *     ends (0 leaves it unchanged).
 *   k_new, v_new: [B, n_q, Hkv, d] bf16, device, 16-byte aligned base and
 *   strides, inner stride 1 (the [B, n_q, Hkv, d] layout of q's new tokens).
 *   k_cache, v_cache and kv_lengths are written by the call (caller-owned).
 *   The tensor-core kernel runs it as a cooperative launch (every block
 *   resident; an explicit opts->num_ctas above that returns
 *   FD_ERR_UNSUPPORTED) and meets once at a grid-wide barrier after the
 *   writes; its launch counters live in the workspace, so calls sharing a
 *   workspace must not overlap.  Other arguments as fd_decode.
 */
int fd_decode_append(const fd_tensor *q, const fd_tensor *k_cache,
                     const fd_tensor *v_cache, const fd_tensor *k_new,
                     const fd_tensor *v_new, int32_t *kv_lengths,
                     int32_t update_lengths, int32_t causal, float scale,
                     const fd_tensor *out, const fd_opts *opts);
/*
 * Dense prefix decode over a paged cache: the same visible set, causal
 * window and result as fd_decode / fd_decode_int8, but cache position j of
 * sequence b lives in a pool of fixed-size pages, at row j % page_size of
 * page block_table[b * max_pages + j / page_size] (comfy-kitchen #239,
 * commit list and Description: a bounded paged int8 decode cache with
 * rollback).  Rolling a sequence back needs only a smaller kv_lengths[b];
 * pages past the length are never read.
 *   k_pages, v_pages: [num_pages, Hkv, page_size, d] bf16 or int8 (both the
 *     same), any strides that are multiples of 16 bytes, so the token-major
 *     pool [num_pages, page_size, Hkv, d] works through a transpose.
 *   k_scale, v_scale: NULL for bf16 pools; for int8 pools fp32
 *     [num_pages, Hkv, page_size] (any strides), one scale per cached row.
 *   block_table: device int32 [B, max_pages], contiguous, caller-owned.
 *     The logical capacity is cap = max_pages * page_size (below 2^31);
 *     kv_lengths[b] is clamped to [0, cap] (FD_DEV_BAD_LENGTH).  Only the
 *     entries of pages that hold positions < kv_lengths[b] are read; such an
 *     entry outside [0, num_pages) skips that page's positions and sets
 *     FD_DEV_BAD_INDEX.
 *   Other arguments as fd_decode.  The tensor-core kernel serves pools whose
 *   three outer strides are multiples of the smallest, itself at least d
 *   (every contiguous layout), with the row limits of the flat caches.
 */
int fd_decode_paged(const fd_tensor *q, const fd_tensor *k_pages,
                    const fd_tensor *v_pages, const fd_tensor *k_scale,
                    const fd_tensor *v_scale, const int32_t *block_table,
                    int32_t max_pages, const int32_t *kv_lengths, int32_t n_q,
                    int32_t causal, float scale, const fd_tensor *out,
                    const fd_opts *opts);
/*
 * Dense prefix decode that allocates nothing (no counterpart in the paper).
 *
 * For callers that cannot call cudaMalloc: an application whose own allocator
 * owns all device memory, a process under a hard device-memory cap, or a
 * plugin inside an engine that forbids allocation after start-up.  Computes
 * exactly what fd_decode computes (bf16 cache, optional causal window) on
 * `stream`, with the same arguments minus the workspace; num_ctas = 0 picks
 * the block count automatically.
 *
 * Its scratch (split partials, per-(sequence, kv head) completion counters
 * and an internal status word, which this call does not report) is a fixed
 * 8 MiB array in device memory that every GPU which loads libfd.so holds
 * until the process exits.  Limits: at most 4096
 * (sequence, kv head) pairs, and the split partials must fit: the block count
 * is lowered to fit, and a problem that cannot fit even with one block per
 * (sequence, kv head), or an explicit num_ctas that does not fit, returns
 * FD_ERR_SCRATCH before anything is launched.  Each call clears the counters
 * and status word on `stream` first (cudaMemsetAsync, which allocates
 * nothing).  All calls share the one array: calls that overlap on the GPU
 * race and must not be issued.  Every call whose stream is not being
 * captured looks up the array's device address (with the caller's device
 * current); a captured call reuses the address the last uncaptured call on
 * that device found.  So the first call on a device, and the first after a
 * device reset or in another context, must come before any stream capture
 * (a captured first call returns FD_ERR_CUDA).  Returns FD_OK or a negative
 * FD_ERR_* code.
 */
int fd_decode_noalloc(const fd_tensor *q, const fd_tensor *k_cache,
                      const fd_tensor *v_cache, const int32_t *kv_lengths,
                      int32_t n_q, int32_t causal, float scale,
                      const fd_tensor *out, void *stream, int32_t num_ctas);

/*
 * A cache held in 4 bits.  A row of d values (one position of one kv head) is
 * d/2 bytes of e2m1 codes (sign, two exponent bits, one mantissa bit: 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6 and their negatives), value 2j in the low nibble of byte
 * j and value 2j+1 in its high nibble, and d/16 e4m3 scales, one for each 16
 * consecutive values.  Value x stands for code * scale * global, with one
 * fp32 factor per call for K and one for V (1 where the scales' own range,
 * 2^-9 .. 448, is enough).  These arguments are the same in the three calls
 * below:
 *   k_cache, v_cache: FD_U8 [B, Hkv, cap, d/2], or with a block_table pools
 *     [num_pages, Hkv, page_size, d/2]; both of one shape; 16-byte aligned
 *     base, strides that are multiples of 16 bytes, innermost stride 1.
 *   k_scale, v_scale: FD_E4M3 [.., .., .., d/16], as the caches; base and
 *     strides multiples of d/16 bytes.
 *   k_global, v_global: finite, 2^-64 .. 2^64.
 *   block_table: NULL for flat caches, else device int32 [B, max_pages],
 *     contiguous, as in fd_decode_paged; max_pages is 0 for flat caches.
 *   d is 128 or 256.
 */

/*
 * Dense prefix decode over a 4-bit cache: the visible set, causal window and
 * output of fd_decode (flat) or fd_decode_paged.  Up to 64 rows
 * ((Hq / Hkv) * n_q) share a kv head; more than 32 are served in two halves,
 * each of which reads the prefix and needs a segment of the workspace:
 * 2 * B * Hkv of them.
 * The scores and all sums are fp32 over exact products of the codes, the
 * scales and q (an entry of q below 2^-14 of its row's largest is off by up
 * to 2^-25 of that); each softmax weight is rounded to fp16, i.e. by up to
 * 2^-11 of itself or 2^-29 of the row's largest weight, or for an fp32 output
 * to two fp16 numbers, by up to 2^-22 or 2^-37.  Scores are finite where
 * |scale| * k_global * sum |code * scale * q| stays within fp32.  A NaN scale
 * (fd_append_fp4 writes one for a row that is not finite) makes NaN of what
 * it stands for in the query rows that see its position, and reaches no
 * other.  Positions at or past the length and pages past it are never read.
 * opts->kernel must be FD_KERNEL_AUTO.  The work of a
 * call is counted in 32 bits: FD_ERR_UNSUPPORTED where B * Hkv * cap / 96 (for
 * both halves, where there are two) comes near 2^31.
 */
int fd_decode_fp4(const fd_tensor *q, const fd_tensor *k_cache, const fd_tensor *v_cache,
                  const fd_tensor *k_scale, const fd_tensor *v_scale, float k_global,
                  float v_global, const int32_t *block_table, int32_t max_pages,
                  const int32_t *kv_lengths, int32_t n_q, int32_t causal, float scale,
                  const fd_tensor *out, const fd_opts *opts);
/*
 * Writes new rows into a 4-bit cache.  For sequence b with base_b =
 * kv_lengths[b] (clamped to [0, cap]), row i of k_new / v_new
 * [B, n, Hkv, d] (bf16; 16-byte aligned base and strides, innermost stride
 * 1) goes to position base_b + i, for i below new_lengths[b] (device int32[B],
 * clamped to [0, n]; NULL: n).  Rows past that are padding and are not read;
 * positions at or past cap are not written.
 *   16 values x share s = e4m3(max|x| / (6 * global)), rounded to nearest even
 *   and at most 448; their codes are e2m1(x / (s * global)), to nearest, ties
 *   to the even code, at most 6 (with the quotient's sign; s = 0 gives zero
 *   codes).  6 * global, s * global and both quotients are rounded to fp32
 *   first.  Where one of the values is a NaN or an infinity the scale is NaN
 *   and the codes are 0.
 *   lengths_out: device int32[B], gets min(base_b + new_b, cap); may be
 *   kv_lengths itself (but overlap it in no other way), or NULL.
 * FD_DEV_BAD_LENGTH is set where a length, a new length or base_b + new_b is
 * out of range, FD_DEV_BAD_INDEX where a page's table entry names no page
 * (its rows are not written).  A page must not be reached through two
 * sequences' write ranges (fd_pages_reserve sees to that).  opts supplies the
 * stream and the workspace's status word; opts->kernel must be
 * FD_KERNEL_AUTO, and opts->num_ctas is not used.
 */
int fd_append_fp4(const fd_tensor *k_new, const fd_tensor *v_new, const int32_t *new_lengths,
                  const fd_tensor *k_cache, const fd_tensor *v_cache, const fd_tensor *k_scale,
                  const fd_tensor *v_scale, float k_global, float v_global,
                  const int32_t *block_table, int32_t max_pages, const int32_t *kv_lengths,
                  int32_t *lengths_out, const fd_opts *opts);
/*
 * Reads rows of a 4-bit cache: k_out / v_out [B, n, Hkv, d] (both bf16 or both
 * fp32; 16-byte aligned base and strides, innermost stride 1) get positions
 * start_b .. start_b + n - 1 of every sequence (start: device int32[B], or
 * NULL for 0), and zeros for positions below 0, at or past kv_lengths[b]
 * (clamped to [0, cap]) or on a page whose table entry names none
 * (FD_DEV_BAD_INDEX).  A value is code * scale, exactly, times global in
 * fp32, rounded to the output's type.  opts as in fd_append_fp4.
 */
int fd_read_fp4(const fd_tensor *k_cache, const fd_tensor *v_cache, const fd_tensor *k_scale,
                const fd_tensor *v_scale, float k_global, float v_global,
                const int32_t *block_table, int32_t max_pages, const int32_t *start,
                const int32_t *kv_lengths, const fd_tensor *k_out, const fd_tensor *v_out,
                const fd_opts *opts);

/*
 * Rows of a bf16 or int8 cache.  These arguments are the same in fd_append and
 * fd_prefill:
 *   k_cache, v_cache: [B, Hkv, cap, d], or with a block_table pools
 *     [num_pages, Hkv, page_size, d]; both bf16 or both int8 and of one shape;
 *     16-byte aligned base, strides that are multiples of 16 bytes, innermost
 *     stride 1.
 *   k_scale, v_scale: NULL for bf16; for int8 fp32 [B, Hkv, cap] or
 *     [num_pages, Hkv, page_size], any strides: one scale a row, as in
 *     fd_decode_int8 and fd_decode_paged.
 *   block_table: NULL for flat caches, else device int32 [B, max_pages],
 *     contiguous, as in fd_decode_paged; max_pages is 0 for flat caches.
 *   d is 128 or 256; cap (max_pages * page_size) below 2^31.
 *
 * fd_append writes new rows.  For sequence b with base_b = kv_lengths[b]
 * (clamped to [0, cap]), row i of k_new / v_new [B, n, Hkv, d] (bf16; 16-byte
 * aligned base and strides, innermost stride 1) goes to position base_b + i,
 * for i below new_lengths[b] (device int32[B], clamped to [0, n]; NULL: n).
 * Rows past that are padding and are not read; positions at or past cap are
 * not written.
 *   rope: NULL, or fp32 [positions, r], 16-byte aligned base and row stride,
 *     innermost stride 1, r a multiple of 16 up to d: the first r/2 numbers of
 *     row p are the cosines of position p's angles, the others their sines.
 *     The first r values of a key are then turned in pairs (a, b) ->
 *     (a cos - b sin, b cos + a sin), where pair j is values j and j + r/2, or
 *     with interleaved != 0 values 2j and 2j+1; the rest stay.  fp32, each
 *     product rounded, then their sum, then once to bf16.  A position past the
 *     table sets FD_DEV_BAD_INDEX, and its row is neither written nor turned.
 *   q, q_out: NULL, or the queries of the same tokens [B, n, Hq, d] (bf16,
 *     aligned as k_new) and where they go, turned the same way (copied without
 *     rope).  q_out may be q itself (then of the same strides), but may
 *     overlap q, k_new or v_new in no other way.  Padding rows of q_out are left as
 *     they were.
 *   int8: s = max|x| / 127 over the d values of a row in fp32, code =
 *     x / s rounded to nearest even (both quotients correctly rounded), at
 *     most 127 in magnitude; s = 0 gives zero codes.  Where a value is a NaN
 *     or an infinity the scale is NaN and the codes are 0.
 *   lengths_out: device int32[B], gets min(base_b + new_b, cap); may be
 *     kv_lengths itself (but overlap it in no other way), or NULL.
 * FD_DEV_BAD_LENGTH is set where a length, a new length or base_b + new_b is
 * out of range, FD_DEV_BAD_INDEX where a page's table entry names no page (its
 * rows are not written).  A page must not be reached through two sequences'
 * write ranges (fd_pages_reserve sees to that).  opts supplies the stream and
 * the workspace; opts->kernel must be FD_KERNEL_AUTO, and opts->num_ctas is not
 * used.
 */
int fd_append(const fd_tensor *k_new, const fd_tensor *v_new, const int32_t *new_lengths,
              const fd_tensor *q, const fd_tensor *q_out, const fd_tensor *rope,
              int32_t interleaved, const fd_tensor *k_cache, const fd_tensor *v_cache,
              const fd_tensor *k_scale, const fd_tensor *v_scale, const int32_t *block_table,
              int32_t max_pages, const int32_t *kv_lengths, int32_t *lengths_out,
              const fd_opts *opts);
/*
 * Attention of a chunk of new tokens over a bf16 or int8 cache that holds
 * them already (fd_append, then this).  q [B, n, Hq, d] (bf16, 16-byte aligned
 * base and strides, innermost stride 1); sequence b has L_b = kv_lengths[b]
 * positions (clamped to [0, cap]), the newest new_b of which are its query
 * rows: new_b = new_lengths[b] (device int32[B], clamped to [0, n]; NULL: n).
 * Row i < new_b sees positions 0 .. L_b - 1, with causal != 0 positions 0 ..
 * L_b - new_b + i; a row that sees none gives zeros.  Rows past new_b are
 * padding: they are not used, and out keeps what it held there.
 *   out [B, n, Hq, d] bf16, 16-byte aligned base and strides, innermost
 *     stride 1; overlaps nothing else.
 *   n >= 1, Hq / Hkv up to 128; any number of rows.
 *   Scores and sums are fp32; a softmax weight (for int8 times its position's v
 *     scale) is rounded to bf16, i.e. by up to 2^-8 of itself.  Positions below
 *     L_b must hold finite values where some row does not see them; those at
 *     or past L_b and pages past it are never read.
 * FD_DEV_BAD_LENGTH is set where a length or new length is out of range;
 * FD_DEV_BAD_INDEX where the entry of a page below L_b names none, whose
 * positions nobody sees.
 *   An int8 position whose K or V scale is NaN makes NaN of the rows that see it.
 *   opts->kernel: FD_KERNEL_AUTO; FD_KERNEL_TC (the tcgen05 kernel; scale > 0,
 *     q and a flat cache of strides that a tensor map can describe, and
 *     B * Hkv * tiles * blocks below 2^31, where a tile is 128 / (Hq / Hkv) tokens of
 *     n and a block 128 positions of cap + n.  K and V of int8 pools must also have
 *     the same strides, the outer three multiples of the smallest, itself at least
 *     d, and so must those of bf16 pools at d = 128 with n more than one tile and a
 *     page_size of 64 or a multiple of 128; FD_ERR_UNSUPPORTED otherwise), or
 *     FD_KERNEL_SIMT (warp-level matrix instructions, every call), which AUTO falls
 *     back to.
 *   opts->num_ctas: 0, or the number of thread blocks that share the work of the
 *     tcgen05 kernel.  opts->wait_limit_us bounds its waits; one that runs out sets
 *     FD_DEV_INTERNAL, and the outputs are then undefined.
 * Long contexts of few rows are split over thread blocks, which takes
 * fd_prefill_scratch_bytes(num_ctas, d) bytes of the workspace's room for split
 * partials (num_ctas 0: of an automatic launch on the current device; see
 * fd_pages_scratch_bytes' room below).
 */
size_t fd_prefill_scratch_bytes(int32_t num_ctas, int32_t head_dim);
int fd_prefill(const fd_tensor *q, const fd_tensor *k_cache, const fd_tensor *v_cache,
               const fd_tensor *k_scale, const fd_tensor *v_scale, const int32_t *block_table,
               int32_t max_pages, const int32_t *kv_lengths, const int32_t *new_lengths,
               int32_t causal, float scale, const fd_tensor *out, const fd_opts *opts);

/*
 * One step of a beam search: the n_out best of a request's K beams times V
 * words.  logits [B, K, V] (bf16 or fp32, innermost stride 1), scores fp32
 * [B, K] (contiguous; the beams' sums of log-probabilities so far; -inf: no
 * beam).  With lse = log sum exp of a beam's logits as an fp32 number (off by at
 * most half a step of its own and 2^-15, by less than 2^-20 beside the half step on
 * logits of every spread measured; the same for beams of the same logits), word v of
 * beam k scores scores[b,k] + (logit - lse), compared exactly; higher scores
 * win, equal ones go to the lower beam, then the lower word.
 *   finished: NULL, or device int32 [B, K]: a beam whose entry is not 0 has
 *     ended, and goes on only by the word end_token (0 .. V-1; not used
 *     without finished), at a log-probability of 0; its logits are not used.
 *   scores_out (fp32), beams_out, tokens_out (int32), [B, n_out] each: the
 *     winners by falling score; beams_out holds the row b*K + k of the winner's
 *     beam, as fd_pages_reorder's src takes it.  Candidates of -inf or NaN
 *     score are none; where too few are left, the rest are -inf, -1 and -1.
 *     They overlap none of the inputs and not one another (FD_ERR_ARG where they do
 *     scores, finished or one another).
 *   K <= 128, n_out <= 64, V < 2^24 (FD_ERR_UNSUPPORTED beyond).
 * opts supplies the stream and the workspace, whose room for split partials
 * holds fd_beam_scratch_bytes(B, K, V, n_out) bytes; opts->kernel must be
 * FD_KERNEL_AUTO, and opts->num_ctas is not used.
 */
size_t fd_beam_scratch_bytes(int64_t B, int32_t K, int64_t V, int32_t n_out);
int fd_beam_select(const fd_tensor *logits, const float *scores, const int32_t *finished,
                   int32_t end_token, int32_t n_out, float *scores_out, int32_t *beams_out,
                   int32_t *tokens_out, const fd_opts *opts);

/*
 * Pages of a paged cache, shared between sequences by reference counts.  The
 * books are caller-owned device memory:
 *   block_table int32 [B, max_pages], contiguous; -1 where a row holds no
 *     page; kv_lengths int32 [B]; refs int32 [num_pages]: how many table
 *     entries name the page, 0 for a free one.
 * B * max_pages below 2^31; num_pages 1 .. 2^30; page_size >= 1.
 * Choices go by number: the lowest free pages are taken, sequences and their
 * pages in increasing order, so equal books give equal books.  A listed
 * sequence or page that does not exist is skipped and FD_DEV_BAD_INDEX set; a
 * length outside [0, max_pages * page_size] is clamped and FD_DEV_BAD_LENGTH
 * set.  The calls only queue work on opts->stream, so they can be captured.
 * opts supplies the stream and the workspace; opts->kernel must be
 * FD_KERNEL_AUTO, and opts->num_ctas is not used.
 *
 * fd_pages_reserve makes sure that every page in which positions
 *   kv_lengths[b] .. kv_lengths[b] + n_b - 1 lie (n_b: n_new[b], or n_each
 *   where n_new is NULL; a negative one counts as 0) is sequence b's alone.  An
 *   entry that names no page gets a free one; an entry whose page others name
 *   too is moved to a free one, except that the first of them (in order of
 *   sequences, then pages) keeps it when all of them write.  Where such a
 *   page holds positions below kv_lengths[b], (old, new) is put into pairs
 *   (int32 [B, 2]; the rest stays as it was) for fd_pages_copy.  count
 *   (int32[1]) gets the number of pairs.  With too few free pages nothing is
 *   reserved, count gets minus the missing pages and FD_DEV_NO_PAGES is set.
 *   kv_lengths is not changed.
 * fd_pages_fork: for each i < n, row dst[i] releases its pages and takes those
 *   that hold the first L positions of row src[i], L = kv_lengths[src[i]], or
 *   lengths[i] where that is given and smaller; kv_lengths[dst[i]] = L.  An
 *   entry whose dst is an earlier entry's dst, or another entry's src, is
 *   skipped and flagged as above; src[i] = dst[i] changes nothing.
 * fd_pages_reorder: every row b of the block table takes, all at once, the
 *   pages that hold the first L positions of the row that was src[b] (int32
 *   [B]), L that row's length, and kv_lengths[b] = L; a row that is its own
 *   source stays as it is, and a negative src[b] empties the row.  A source
 *   past the last row leaves row b as it is and is flagged as above.  B up to
 *   49152 (FD_ERR_UNSUPPORTED beyond).
 * fd_pages_free: for each i < n, the length of sequence seqs[i] (seqs NULL:
 *   sequence i, n = B) becomes 0, or lengths[i] where lengths is given and
 *   smaller than the length, and the row's pages past it are released.
 *   A sequence listed twice ends at the smaller length.
 * n = 0 lists nothing: fork and free then do nothing.
 * fd_pages_compact moves the pages in use to the numbers 0 .. used - 1: the
 *   i-th page in use at or past `used` goes to the i-th free page below it.
 *   block_table and refs are renumbered, pairs (int32 [num_pages / 2, 2])
 *   lists (from, to) and count their number; the contents follow by
 *   fd_pages_copy.
 * fd_pages_copy copies, in each of n_pools pools (1 .. 256) [num_pages, ...]
 *   of any dtype and 1 to 4 dimensions, page pairs[2i] to page pairs[2i+1] for
 *   i < count[0] (at most max_pairs; nothing for a negative count).  A page's
 *   elements must fill one block of memory, in any order of dimensions.  No
 *   page may be both copied from and copied to, nor be copied to twice.
 *
 * reserve and compact use fd_pages_scratch_bytes(num_pages) bytes of the
 * workspace's room for split partials (the room is at least
 * fd_workspace_bytes(segments, rows, head_dim, ctas) less 8 * segments + 4 *
 * ctas + 1024 bytes).
 */
size_t fd_pages_scratch_bytes(int64_t num_pages);
int fd_pages_reserve(int32_t *block_table, int32_t B, int32_t max_pages,
                     const int32_t *kv_lengths, const int32_t *n_new, int32_t n_each,
                     int32_t page_size, int32_t *refs, int32_t num_pages, int32_t *pairs,
                     int32_t *count, const fd_opts *opts);
int fd_pages_fork(int32_t *block_table, int32_t B, int32_t max_pages, int32_t *kv_lengths,
                  int32_t page_size, int32_t *refs, int32_t num_pages, const int32_t *src,
                  const int32_t *dst, const int32_t *lengths, int32_t n, const fd_opts *opts);
int fd_pages_reorder(int32_t *block_table, int32_t B, int32_t max_pages, int32_t *kv_lengths,
                     int32_t page_size, int32_t *refs, int32_t num_pages, const int32_t *src,
                     const fd_opts *opts);
int fd_pages_free(int32_t *block_table, int32_t B, int32_t max_pages, int32_t *kv_lengths,
                  int32_t page_size, int32_t *refs, int32_t num_pages, const int32_t *seqs,
                  const int32_t *lengths, int32_t n, const fd_opts *opts);
int fd_pages_compact(int32_t *block_table, int32_t B, int32_t max_pages, int32_t *refs,
                     int32_t num_pages, int32_t *pairs, int32_t *count, const fd_opts *opts);
int fd_pages_copy(const fd_tensor *pools, int32_t n_pools, const int32_t *pairs,
                  const int32_t *count, int32_t max_pairs, const fd_opts *opts);

/*
 * Workspace.  A launch unit ("segment") is one (sequence, kv head) in the
 * dense modes and one (sequence, query row, kv head) in gather mode; rows is
 * the number of query rows sharing it ((Hq/Hkv) * n_q dense, Hq/Hkv gather).
 * Size for the largest segment count, row count, head_dim and num_ctas any
 * call will use.  fd_workspace_create allocates device memory (cudaMalloc)
 * and zeroes the counters on `stream`; it is the only allocating call.
 * A workspace serves the calls of one stream at a time, in stream order: the
 * scratch of the split combine belongs to one stream-ordered launch at a
 * time, the rule comfy-kitchen #239 adopts for its GEMM workspace (commit
 * list: the workspace is tied to each launch in stream order).  Two streams
 * that may run decode calls at once need two workspaces.  Host threads may
 * share one with the stream: a call's launches follow one another without
 * another call's between them.  Calls that do
 * overlap on one workspace can leave its counters inconsistent (results of
 * later calls are then wrong: a merge is skipped, or a masked call keeps an
 * older chunk list) until fd_workspace_reset.
 */
size_t fd_workspace_bytes(int64_t max_segments, int32_t max_rows,
                          int32_t head_dim, int32_t max_ctas);
int fd_workspace_create(int64_t max_segments, int32_t max_rows,
                        int32_t head_dim, int32_t max_ctas, void *stream,
                        fd_workspace **ws);
/* Clears the completion counters and the status word on `stream` (needed
 * only after a launch was aborted part-way; every completed launch leaves the
 * counters at zero). */
int fd_workspace_reset(fd_workspace *ws, void *stream);
/* Test hook for the failure path: sets every per-segment completion counter
 * to `value` on `stream`.  A negative value stands for counters an aborted
 * launch left behind: the next call whose blocks share the merge of a split
 * segment (the tensor-core kernel's cooperative launches over few segments)
 * then waits for pieces that never arrive, gives up after opts->wait_limit_us
 * and sets FD_DEV_INTERNAL, recording the wait in fd_get_device_diagnostics;
 * fd_workspace_reset restores the zeros.  Never needed in normal use. */
int fd_workspace_fill_counters(fd_workspace *ws, int32_t value, void *stream);
int fd_workspace_destroy(fd_workspace *ws);
/* Synchronously reads the sticky status word (FD_DEV_* bits). */
int fd_get_device_status(fd_workspace *ws, int32_t *status);
/* Synchronously reads 13 words: the status word; then, if FD_DEV_INTERNAL was
 * set by the tensor-core kernel, the id, tile counter and piece index of the
 * first internal wait that gave up; then the same three for the first wait
 * that gave up in each role (TMA producer, MMA issuer, softmax).  Zero where
 * nothing gave up.  Cleared by fd_workspace_reset. */
int fd_get_device_diagnostics(fd_workspace *ws, int32_t *words);

/* Number of thread blocks an auto launch of a dense call with this cache
 * dtype would use on the current device (host query; 0 on error).  max_units
 * bounds the launch's work units (tiles for the capacity plus fd_seg_units
 * per segment); 0 for no bound. */
int32_t fd_auto_num_ctas(int32_t kernel, int32_t head_dim, int32_t kv_dtype,
                         int32_t rows, int64_t max_units);
/* Cache positions per K/V tile for a kernel / head_dim / cache dtype. */
int32_t fd_tile_tokens(int32_t kernel, int32_t head_dim, int32_t kv_dtype);
/* Workspace bytes the tensor-core kernel's chunk list of a masked call over
 * B sequences of capacity cap takes past the call's split partials (the
 * list, the counts and the listing pass's staging area); 0 for B or cap
 * outside [1, 65535] or [1, 2^23], where no list is made. */
size_t fd_masked_list_bytes(int64_t B, int64_t cap);

/*
 * Host mirror of the device split partitioner, for inspection and tests.
 * The split is over work units: each non-empty segment holds seg_units units
 * (the fixed cost of a piece boundary, mapped to no tile) followed by one
 * unit per tile; num_ctas blocks take balanced consecutive unit ranges.
 * For segment lengths seg_len[0..nseg) (positions), tile size, num_ctas and
 * seg_units, writes for every segment the first thread block that works on
 * its tiles and the number of blocks that share them (0 for an empty
 * segment).  Returns the total unit count, or a negative FD_ERR_* code.
 */
int64_t fd_plan(const int64_t *seg_len, int64_t nseg, int32_t tile_tokens,
                int32_t num_ctas, int32_t seg_units, int32_t *first_cta,
                int32_t *n_pieces);
/* seg_units a launch of this kernel, head_dim and cache dtype uses (0 for
 * the CUDA-core kernel; AUTO is not resolved here). */
int32_t fd_seg_units(int32_t kernel, int32_t head_dim, int32_t kv_dtype);

const char *fd_status_string(int status);
int32_t fd_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FD_H */
