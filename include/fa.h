/*
 * fa.h — C ABI of the GB300 (sm_103a) FlashAttention-style attention forward.
 *
 * Operation (non-causal scaled-dot-product attention with row log-sum-exp):
 *
 *   S = scale * Q K^T (+ mask broadcast over heads and query rows)
 *   O = softmax_row(S) V,   LSE_i = ln sum_j exp(S_ij)
 *
 * computed block by block with an online softmax (running row max m, running
 * denominator l, rescaled accumulator), so the Nq x Nk score matrix never
 * reaches device memory.  Sources:
 *  - "算子加速：注意力、编译与融合" (anrans.github.io ai-infra-handbooks, perf/kernels),
 *    section "注意力：从O(N²)显存到分块": the figure (per K/V block: S_ij = Q_i K_j^T,
 *    update m and l, O_i <- O_i e^(m_old - m) + P V_j, only O_i is written
 *    back) and the `blocked` worked example (the m / l / acc recurrence);
 *  - "FlashAttention原理与工业实战" (sheratonhq.com) §2.3: the forward kernel
 *    writes Out and a per-row Lse; §4.3: inputs must be contiguous [B,H,N,D];
 *  - "Step 3.7 Flash" (pwwt.cn) §2.3 and §3.1: scale first, then add the
 *    additive attention mask; non-causal (is_causal=False).
 *
 * All functions are thread-safe.  The library allocates no device memory.
 */
#ifndef UNET_FA_FWD_GB300_FA_H
#define UNET_FA_FWD_GB300_FA_H

#include <stddef.h>

/* The library exports these functions only; everything else is hidden. */
#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARGUMENT = 1, /* NULL pointer, bad size, misaligned or overlapping buffer, non-finite scale */
    FA_ERR_UNSUPPORTED = 2,      /* head dimension D not in {32, 64, 128}; device not sm_103 */
    FA_ERR_CUDA = 3,             /* a CUDA runtime/driver call failed (launch, attribute, tensor map) */
    FA_ERR_TIMEOUT = 4,          /* a kernel wait ran past its time limit (read with fa_read_device_status) */
    FA_ERR_DEBUG_CHECK = 5,      /* debug builds: a device-side bounds or schedule check failed
                                    (read with fa_read_device_status; details: fa_debug_report) */
    FA_ERR_INDEX = 6             /* a page number, length or position in device memory was out of range
                                    (read with fa_read_device_status) */
} fa_status;

/*
 * fa_fwd — attention forward on the GPU.
 *
 *   q     device pointer, bf16 [B, H, Nq, D], contiguous row-major
 *   k, v  device pointers, bf16 [B, H, Nk, D], contiguous row-major
 *   mask  device pointer to an fp32 additive key mask [B, Nk] (0 = keep,
 *         -inf = ignore; any finite value is added to the scaled score), or
 *         NULL for no mask.  Broadcast over heads and query rows.
 *   out   device pointer, bf16 [B, H, Nq, D]: O
 *   lse   device pointer, fp32 [B, H, Nq]: natural-log row log-sum-exp of the
 *         scaled, masked scores
 *   B, H, Nq, Nk  >= 1;  D in {32, 64, 128}
 *   scale finite; multiplies Q K^T before the mask is added
 *   stream  cudaStream_t (as void*), NULL = the legacy default stream
 *
 * A row whose keys are all masked gives O = 0 and LSE = -inf.
 *
 * Ownership: the caller owns every buffer; nothing is retained after the call
 * returns (TMA descriptors are encoded per call and passed by value).  Every
 * pointer must be 16-byte aligned (a TMA requirement); out and lse must not
 * overlap q, k, v, mask or each other.
 *
 * Errors: arguments are validated before any CUDA call; an invalid call
 * returns FA_ERR_INVALID_ARGUMENT or FA_ERR_UNSUPPORTED and launches nothing.
 * FA_ERR_CUDA means a launch or set-up call failed.  FA_OK means the kernel
 * was enqueued on `stream` (the call is asynchronous); a kernel that ran out
 * of time on an internal wait records FA_ERR_TIMEOUT in the device status
 * word (see fa_read_device_status) and exits without hanging.
 */
FA_API int fa_fwd(const void* q, const void* k, const void* v, const float* mask, void* out, float* lse,
           int B, int H, int Nq, int Nk, int D, float scale, void* stream);

/* Kinds of mask fa_fwd_ex accepts. */
typedef enum {
    FA_MASK_NONE = 0,
    FA_MASK_KEY_PADDING = 1, /* fp32 [B, Nk], added to every query row (as fa_fwd's mask) */
    FA_MASK_ADDITIVE = 2,    /* fp32 [B, heads, Nq, Nk], added to each scaled score */
    FA_MASK_BOOL = 3         /* uint8 [B, heads, Nq, Nk]: nonzero keeps the pair, 0 excludes it */
} fa_mask_kind;

/* A mask for fa_fwd_ex: `data` is a contiguous device array of the kind's
 * layout; `heads` (ADDITIVE and BOOL) is 1 to broadcast over heads, or H. */
typedef struct fa_mask {
    int kind;
    const void* data;
    int heads;
} fa_mask;

/*
 * fa_fwd_ex — fa_fwd with general masks and an optional causal triangle.
 *
 * A per-(query, key) additive mask is added after the scale, like the
 * key-padding mask ("Step 3.7 Flash" §2.3, where ignored positions carry a
 * large negative); a boolean mask excludes the pairs where it is 0, i.e. it
 * is the additive mask 0 / -inf ("FlashAttention原理与工业实战" §2.1,
 * masked_fill(mask == 0, -inf)).  causal != 0 also excludes key j > query i
 * (top-left aligned: row i sees keys 0..i, the lower-triangular mask of that
 * page's §4.3 causal example); key blocks entirely above the diagonal are not
 * computed.
 *
 *   mask  NULL or kind FA_MASK_NONE: no mask; otherwise as fa_mask above.  An
 *         ADDITIVE mask must be 4-byte aligned; a mask must not overlap out or lse.
 *         Speed, not results, depends on alignment: an ADDITIVE mask whose rows
 *         start 16-byte aligned (16-byte aligned data, Nk a multiple of 4) is
 *         copied tile by tile into shared memory by TMA; a BOOL mask with
 *         16-byte aligned rows is read 16 bytes at a time; other masks are
 *         read element by element.
 *   other arguments as fa_fwd.
 *
 * Rows left with no key give O = 0, LSE = -inf.  Errors as fa_fwd, plus
 * FA_ERR_INVALID_ARGUMENT for an unknown kind, NULL data, heads not 1 or H,
 * or a misaligned or overlapping mask.
 */
FA_API int fa_fwd_ex(const void* q, const void* k, const void* v, const fa_mask* mask, int causal,
              void* out, float* lse, int B, int H, int Nq, int Nk, int D, float scale,
              void* stream);

/*
 * fa_fwd_fp8 — the forward with Q K^T in FP8 (e4m3), SageAttention-style
 * ("算子加速：注意力、编译与融合", section "SageAttention": smooth K by
 * subtracting its mean, quantise, run the low-precision product; P and V stay
 * 16-bit, as in its first version).
 *
 * A pre-pass subtracts from K its per-channel mean over the keys of each head
 * (this moves every score of row i by the same q_i . mean, so the softmax is
 * unchanged and LSE is corrected by scale * q_i . mean), then quantises Q and
 * the smoothed K to e4m3 with one scale per 128-row block (block max / 448).
 * S = Q K^T runs on the tensor cores as kind::f8f6f4 (twice the bf16 rate,
 * half the MMA instructions); the block scales are folded into the softmax's
 * exp2 multiplier; P (bf16) V (bf16) is unchanged.  Results are close to, not
 * equal to, the bf16 forward: the error budget is looser (see the tests).
 *
 *   arguments as fa_fwd (mask: fp32 key padding [B, Nk] or NULL), plus
 *   workspace  device scratch, 16-byte aligned, at least
 *              fa_fp8_workspace_bytes(B, H, Nq, Nk, D) bytes, owned by the caller
 *              and not shared with a concurrent call.
 *
 * Four kernels are enqueued on `stream` (column sums of K, their means, the
 * quantisation of K and Q, attention).  Errors as fa_fwd, plus FA_ERR_INVALID_ARGUMENT for
 * a missing, misaligned, small or overlapping workspace.
 */
FA_API int fa_fwd_fp8(const void* q, const void* k, const void* v, const float* mask, void* out,
               float* lse, int B, int H, int Nq, int Nk, int D, float scale, void* workspace,
               size_t workspace_bytes, void* stream);

/* Workspace bytes fa_fwd_fp8 needs (0 for invalid sizes). */
FA_API size_t fa_fp8_workspace_bytes(int B, int H, int Nq, int Nk, int D);

/*
 * fa_fwd_split — the same forward with the key axis cut into `num_splits`
 * ranges computed by separate work units, then merged.
 *
 * Each range r yields its own normalised partial output O_r and LSE_r; the
 * merge is exact: LSE = ln sum_r e^(LSE_r), O = sum_r e^(LSE_r - LSE) O_r.
 * This is the exchange step of ring (sequence-parallel) attention in
 * "FlashAttention原理与工业实战" §6.2, here on one GPU: it fills the SMs when
 * B*H*ceil(Nq/256) work units are fewer than the SM count (few heads, short
 * query sets, long key sets).
 *
 *   q, k, v, mask, out, lse, B, H, Nq, Nk, D, scale, stream: as in fa_fwd.
 *   num_splits  >= 1 requested ranges; the library uses min(num_splits, nkv)
 *               balanced ranges of whole 128-key blocks, nkv = ceil(Nk / 128).
 *               1 behaves exactly as fa_fwd.
 *   workspace   device scratch, 16-byte aligned, at least
 *               fa_split_workspace_bytes(B, H, Nq, D, num_splits) bytes; holds
 *               fp32 partial O [ranges][B*H][Nq][D] and LSE [ranges][B*H][Nq].
 *               Owned by the caller; may be NULL when one range is used.  It
 *               must not overlap any other buffer and must not be used by
 *               another call in flight at the same time.
 *
 * Errors: as fa_fwd, plus FA_ERR_INVALID_ARGUMENT for num_splits < 1 or a
 * missing, misaligned, too small or overlapping workspace.  Two kernels are
 * enqueued on `stream` (the split forward, then the merge).
 */
FA_API int fa_fwd_split(const void* q, const void* k, const void* v, const float* mask, void* out,
                 float* lse, int B, int H, int Nq, int Nk, int D, float scale, int num_splits,
                 void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes fa_fwd_split needs for these sizes (0 for invalid sizes). */
FA_API size_t fa_split_workspace_bytes(int B, int H, int Nq, int D, int num_splits);

/*
 * A key-range count for fa_fwd_split on a GPU with `num_sms` SMs: 1 when the
 * unsplit work units already cover every SM, else enough ranges to do so,
 * each range at least four 128-key blocks long.  Pure arithmetic; no CUDA call.
 */
FA_API int fa_split_count(int B, int H, int Nq, int Nk, int num_sms);

/*
 * fa_fwd_window — window / shifted-window attention on an img_h x img_w token
 * grid: every token attends only to the tokens of its own win_h x win_w window
 * of the grid cyclically shifted by (shift_h, shift_w) (the token at (r, c)
 * moves to ((r - shift_h) mod img_h, (c - shift_w) mod img_w)).  Computed as in
 * "Step 3.7 Flash" §3.2: the windows form a batch of
 * B * (img_h/win_h) * (img_w/win_w) attention problems of win_h*win_w tokens.
 * Here the batch is never materialised: the attention kernel reads each
 * window's rows of q, k, v from their grid positions and writes O and LSE
 * back to them.  Windows of up to 64 tokens are packed several to a batch
 * entry, each row seeing only its own window's keys.  No mask is applied
 * across the wrap-around of a shifted grid (the pages name none).
 *
 *   q, k, v, out  device bf16 [B, H, img_h*img_w, D], tokens in row-major grid order
 *   lse           device fp32 [B, H, img_h*img_w]
 *   win_h, win_w  >= 1 and dividing img_h, img_w;  shift_h, shift_w any integers
 *   workspace,    not used (fa_window_workspace_bytes returns 0); any value,
 *   workspace_bytes  NULL and 0 included, is accepted
 *   other arguments as fa_fwd
 *
 * One kernel is enqueued on `stream`.  Errors as fa_fwd, plus
 * FA_ERR_INVALID_ARGUMENT for windows that do not tile the grid or more than
 * 2^31 - 1 rows (B * H * img_h * img_w).
 */
FA_API int fa_fwd_window(const void* q, const void* k, const void* v, void* out, float* lse, int B, int H,
                  int img_h, int img_w, int D, int win_h, int win_w, int shift_h, int shift_w,
                  float scale, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes fa_fwd_window needs: 0 (kept for callers that size one). */
FA_API size_t fa_window_workspace_bytes(int B, int H, int img_h, int img_w, int D);

/* Bytes of the fixed device scratch that fa_fwd_split_noalloc uses. */
#define FA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/*
 * fa_fwd_split_noalloc — fa_fwd_split for callers that cannot allocate device
 * memory (a plugin whose host application owns every device allocation, or a
 * latency-critical path that cannot afford cudaMalloc's implicit device
 * synchronisation).  The pages have no counterpart of this entry point.
 *
 * Arguments as fa_fwd_split, without the workspace: the partial results live
 * in a fixed array of FA_NOALLOC_SCRATCH_BYTES inside the library, which every
 * GPU that loads the library holds until the process exits.  The call
 * allocates nothing (no cudaMalloc, cudaFree or allocating library routine).
 * Sizes whose workspace (fa_split_workspace_bytes with the range count used)
 * exceeds FA_NOALLOC_SCRATCH_BYTES are rejected with FA_ERR_INVALID_ARGUMENT
 * before anything is enqueued.
 *
 * The first call on each device looks up the array's device address (with
 * that device current) and caches it; make that first call before capturing
 * a stream.  All calls on a device share the one array, which keeps the last
 * call's contents: calls that overlap on the GPU (other streams, or before the
 * previous call finished) race on it and must be serialised by the caller.
 */
FA_API int fa_fwd_split_noalloc(const void* q, const void* k, const void* v, const float* mask, void* out,
                         float* lse, int B, int H, int Nq, int Nk, int D, float scale,
                         int num_splits, void* stream);

/* A strided tensor [B, H, N, D]: strides in elements, the last axis contiguous.
 * A stride is >= 0 (0 broadcasts an input); strides of axes of size 1 are not used. */
typedef struct fa_tensor {
    void* data;
    long long stride_b, stride_h, stride_n;
} fa_tensor;

/* Element types of fa_rope. */
typedef enum { FA_DTYPE_BF16 = 0, FA_DTYPE_FP16 = 1, FA_DTYPE_FP32 = 2 } fa_dtype;

/* Which elements of a row form the pairs that turn. */
typedef enum {
    FA_ROPE_ADJACENT = 0, /* (2i, 2i + 1) */
    FA_ROPE_HALVES = 1    /* (i, i + D/2) */
} fa_rope_pairing;

#define FA_ROPE_MAX_AXES 4

/* The axes of fa_rope: dims[a] (even, >= 2) of the row's D elements belong to
 * axis a, in order, and sum to D; theta[a] > 0; scale[a] multiplies the
 * positions (1 for none). */
typedef struct fa_rope_axes {
    int count;
    int dims[FA_ROPE_MAX_AXES];
    double theta[FA_ROPE_MAX_AXES];
    double scale[FA_ROPE_MAX_AXES];
} fa_rope_axes;

/*
 * fa_rope — rotary positions over several axes (time, height, width) on q and
 * k, ahead of the attention.
 *
 * The D/2 pairs of a row are dealt to the axes in order, dims[a]/2 each; pair j
 * of axis a of token n turns by pos[b][n][a] * scale[a] * theta[a]^(-2j/dims[a]):
 * (x0, x1) -> (x0 cos - x1 sin, x0 sin + x1 cos).  A token at position 0 on
 * every axis is unchanged (one with numbers that are not finite: 0 times those
 * is NaN).  inverse != 0 turns the other way, which is also the gradient:
 * dx = fa_rope(dy, inverse).  (For a broadcast input the caller sums the
 * gradient over the broadcast axis.)
 *
 *   pos       device int32 [B, N, count], batch stride pos_stride_b elements
 *             (0: one set of positions for every batch entry); any int32
 *             value: the turns per unit of position, f, are held to
 *             |f| (5 + |ln theta|) 2^-53 and 2^-64, and their product with the
 *             position is reduced exactly
 *   q, q_out  [B, Hq, N, D] of `dtype`; k, k_out [B, Hk, N, D], or both NULL.
 *             Inputs may have any strides (slices of a token-major projection
 *             among them); outputs too, as long as no element is written
 *             twice.  An output may be exactly its input (in place); else the
 *             outputs share no element with the inputs or each other.
 *             (Rows of axes that do not nest, millions of which interleave, are
 *             refused where a bounded search does not tell them apart.)
 *   D in {32, 64, 128}.  Speed, not results, depends on alignment: rows that
 *   start 16-byte aligned are read and written 16 bytes at a time.
 *
 * One kernel is enqueued on `stream`.  Arithmetic is fp32, rounded once to
 * `dtype`.  Errors as fa_fwd; pointers aligned to their element.
 */
FA_API int fa_rope(const fa_rope_axes* axes, const int* pos, long long pos_stride_b, const fa_tensor* q,
                   const fa_tensor* q_out, int Hq, const fa_tensor* k, const fa_tensor* k_out, int Hk, int B,
                   int N, int D, int dtype, int pairing, int inverse, void* stream);

/*
 * A paged key/value cache in 8 bits.  A page holds page_tokens consecutive
 * tokens of a sequence for every head; which pages a sequence owns, in order,
 * is the caller's int32 table [B, table_width].
 *
 *   k, v              device, e4m3 codes [num_pages, H, page_tokens, D], 16-byte aligned
 *   k_scale, v_scale  device fp32 [num_pages, H]: an element is code * scale.
 *                     The scale is the least power of two s in [2^-117, 2^119]
 *                     with max |x| <= 448 s over the page's tokens of the head
 *                     (tokens that a later, smaller start takes back count while
 *                     earlier ones of their page are kept).
 *   page_tokens in {32, 64, 128};  D in {32, 64, 128}
 *
 * Nothing needs clearing: a page's scale and codes are read only where tokens
 * have been written.
 */
typedef struct fa_cache {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int num_pages, H, page_tokens, D;
} fa_cache;

/*
 * fa_cache_write — quantise new tokens and append them to the cache.
 *
 * Token i < count[b] of sequence b goes to position start[b] + i, i.e. to page
 * table[b][position / page_tokens].  start[b] is the number of tokens the
 * sequence holds: positions before it in the first page written are kept
 * (multiplied by the ratio of the scales, a power of two, and rounded again
 * where the page's scale has to grow), positions after the last token written
 * are left as they were and hold nothing.  Non-finite elements are stored as
 * NaN and take no part in the scale.
 *
 *   k, v   bf16 [B, H, N, D], any strides
 *   table  device int32 [B, table_width]
 *   start  device int32 [B];  count  device int32 [B], 0 <= count[b] <= N, or
 *          NULL for N each
 *
 * The pages written must be distinct: a page listed for two sequences of the
 * call may be read by the attention but not written by both (its contents are
 * then undefined).  A page number outside [0, num_pages), a start or count
 * below 0, a count above N and a position past the table record FA_ERR_INDEX
 * in the device status word; tokens that have no valid place are not written.
 * One kernel is enqueued on `stream`.
 */
FA_API int fa_cache_write(const fa_cache* cache, const fa_tensor* k, const fa_tensor* v, const int* table,
                          int table_width, const int* start, const int* count, int B, int N, void* stream);

/*
 * fa_cache_read — read tokens first[b] .. first[b] + N - 1 of each sequence back
 * as bf16 (exact: code * scale is a bf16 number); positions from lens[b] on
 * give zeros.
 *
 *   lens   device int32 [B]: tokens the sequence holds
 *   first  device int32 [B], or NULL for 0
 *   k_out, v_out  device bf16 [B, H, N, D], contiguous, 16-byte aligned
 *
 * An index out of range records FA_ERR_INDEX in the device status word (a page
 * outside the cache is read as page 0, a length or position is clamped).  One
 * kernel is enqueued on `stream`.
 */
FA_API int fa_cache_read(const fa_cache* cache, const int* table, int table_width, const int* lens,
                         const int* first, void* k_out, void* v_out, int B, int N, void* stream);

/*
 * fa_fwd_cache — attention of new queries to the cache, prompts, chunks and
 * single tokens alike.
 *
 * As fa_fwd (scale, O, LSE), with K and V read from the cache: sequence b has
 * the keys 0 .. lens[b] - 1.  causal != 0: query row i sees the keys
 * j <= q_start[b] + i only; q_start NULL means lens[b] - Nq (the queries are
 * the last Nq tokens).  Hq is a multiple of the cache's H: query head h reads
 * key head h / (Hq / H).  A row that sees no key (an empty sequence, a row
 * before the first key) gives O = 0, LSE = -inf.
 *
 * The cache's codes are used as they are; q is held to 2^-17.8 of its row's
 * largest element (2^-110 if that is more) or better, the probabilities to 11
 * bits or 2^-25 of the row's largest (times the ratio between the scales of V of
 * the pages it sees), sums are fp32.  A row's results follow from its q and the
 * keys that it sees alone (in the pages as they are: a later token may have grown
 * its page's scale).  A row of q, or a key that it sees, that holds a number that
 * is not finite gives NaN for the row; such a number in V gives NaN in O (in its
 * channel, perhaps in others) for the rows that see its key.  Scores are fp32
 * numbers: past 2^16 in magnitude a probability may be off by the part 2^-23 of
 * its score, and past 2^24 results mean nothing.
 *
 *   q, out   device bf16 [B, Hq, Nq, D], lse fp32 [B, Hq, Nq], as fa_fwd's
 *   table, lens, q_start  as above; pages may be shared between sequences.
 *            Table entries past a sequence's length are not read.
 *   workspace  device scratch, 16-byte aligned, at least
 *            fa_cache_workspace_bytes(...) bytes (may be NULL when that is 0),
 *            not shared with a concurrent call.
 *
 * One kernel is enqueued on `stream`, and where a sequence may be longer than
 * 128 tokens a second that joins what the first left in parts.  An index out of
 * range records FA_ERR_INDEX (see fa_cache_read), a wait that ran out
 * FA_ERR_TIMEOUT.
 */
FA_API int fa_fwd_cache(const void* q, const fa_cache* cache, const int* table, int table_width,
                        const int* lens, const int* q_start, int causal, void* out, float* lse, int B, int Hq,
                        int Nq, float scale, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes fa_fwd_cache needs (0 for none, and for invalid sizes). */
FA_API size_t fa_cache_workspace_bytes(int B, int Hq, int Hk, int Nq, int D, int table_width, int page_tokens);

/*
 * fa_read_device_status — read, and reset to FA_OK, the status word that
 * kernels on the current device write when an internal wait times out or an
 * index in device memory is out of range.  Synchronises `stream` first.
 * Writes FA_OK or the first error recorded (FA_ERR_TIMEOUT, FA_ERR_INDEX;
 * FA_ERR_DEBUG_CHECK in debug builds) to *status.
 * Returns FA_OK, FA_ERR_INVALID_ARGUMENT (status NULL) or FA_ERR_CUDA.
 */
FA_API int fa_read_device_status(void* stream, int* status);

/*
 * fa_measure_ex2_rate — throughput of the exponential the forward takes once
 * per score (ex2.approx.ftz.f32 on the special-function unit): runs a short
 * probe kernel on `stream` (4 CTAs of 256 threads per SM, 16 independent
 * chains per thread, each CTA timed with clock64) and writes the exponentials
 * one SM completes per SM clock, bounded by its slowest CTA, to
 * *ex2_per_clock_per_sm.  The exp-bound time of a launch is then
 * B·H·Nq·Nk / (rate · SMs · clock).  ("算子加速：注意力、编译与融合",
 * section "注意力：从O(N²)显存到分块": one exponential per score in the
 * softmax.)  Diagnostic, blocking: synchronises `stream`.  Uses static device
 * storage of the library; allocates nothing.  Returns FA_OK,
 * FA_ERR_INVALID_ARGUMENT (NULL output), FA_ERR_UNSUPPORTED (more than 1024
 * SMs) or FA_ERR_CUDA.
 */
FA_API int fa_measure_ex2_rate(void* stream, double* ex2_per_clock_per_sm);

/*
 * Debug build (libfa_fwd_debug.so, compiled with FA_DEBUG; no counterpart on
 * the pages): every kernel checks its unit schedule and the index of every
 * global-memory access before using it.  A failed check skips the access,
 * records the first violation, sets FA_ERR_DEBUG_CHECK in the device status
 * word and makes its CTA drain and exit as after a wait timeout; nothing traps.
 * It stands in for a memory checker where none can run.
 * (The cache's kernels check the page numbers, lengths and positions that they
 * read from device memory in both builds.)
 *
 * fa_debug_build — 1 in the debug build, 0 in the release build.
 *
 * fa_debug_report — synchronise `stream`, copy the first recorded violation
 *   to record[8] and clear it: {check id (0 = none; 1 unit schedule, 2
 *   producer/MMA unit mismatch, 3 mask row, 4 e4m3 scale index, 5 output
 *   store, 6 output row and 7 partial results of the cached attention), CTA, thread, value a, value b, 0, 0, number of failed checks}.
 *   The release build writes zeros.  Returns FA_OK, FA_ERR_INVALID_ARGUMENT
 *   (record NULL) or FA_ERR_CUDA.
 */
FA_API int fa_debug_build(void);
FA_API int fa_debug_report(void* stream, int* record);

/* Human-readable name of a status code (static storage; never NULL). */
FA_API const char* fa_status_string(int status);

/* Library version string, e.g. "unet_fa_fwd_gb300 0.1.0 sm_103a" (static storage). */
FA_API const char* fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* UNET_FA_FWD_GB300_FA_H */
