/*
 * lrkv.h — C ABI of the GB300 (sm_103a) LRKV factored-cache attention library.
 *
 * Low-Rank Key-Value attention writes each head's key/value projection as a
 * shared dense matrix plus a per-head rank-r residual, W_h = W_s + U_h B_h^T
 * ("Low-Rank Key Value Attention：中文研读笔记", §2.1, Eqs. (2)-(5)).  A token
 * therefore caches one shared row k_s, v_s (d_h each) plus per-head latents
 * z_k,h = x U_h^K and z_v,h = x U_h^V (r each) (same page, §2.3), and attention
 * runs directly on that factored cache by associativity (same page, §2.4,
 * Eqs. (6)-(7); "Low-Rank Key Value Attention | What a shared cache can
 * preserve", §3, Algorithm 2):
 *
 *   score_{h,j} = (q_h . k_s,j + (q_h B_h^K) . z_k,h,j) / sqrt(d_h)
 *   a_h        = softmax over the visible j of the summed scores (ONE softmax)
 *   o_h        = sum_j a_{h,j} v_s,j + (sum_j a_{h,j} z_v,h,j) (B_h^V)^T
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  * Memory.  Every pointer argument except `dims`, `bytes` and `out_status`
 *    is a DEVICE pointer on the current CUDA device.  The caller owns and
 *    allocates every buffer, including the workspace; the library allocates
 *    nothing and keeps no state between calls.  All work is enqueued on
 *    `stream` (a cudaStream_t passed as void*; NULL is the legacy default
 *    stream) and the calls return without synchronising.
 *  * Element types.  `dims->dtype` fixes the storage type of q, the cache
 *    (k_s, v_s, z_k, z_v), the bases (b_k, b_v) and the append inputs:
 *    LRKV_F32 (IEEE binary32) or LRKV_BF16 (bfloat16).  Accumulation is fp32.
 *    Outputs `out` and `lse` are always fp32.
 *  * Layouts (row-major, C order):
 *      k_s, v_s   [batch][max_len][head_dim]
 *      z_k, z_v   [batch][max_len][heads][rank]
 *      b_k, b_v   [heads][head_dim][rank]       (B_h is d_h x r; K_h = S + R_h B_h^T)
 *      seq_lens   [batch] int32, visible history length of each sequence
 *  * Alignment.  Cache pointers, q, x and the append weights must be 16-byte
 *    aligned, and head_dim*sizeof(elem) and heads*rank*sizeof(elem) must be
 *    multiples of 16 bytes (every row is moved by the Tensor Memory
 *    Accelerator, which copies 16-byte-aligned spans).  Keep b_k and b_v
 *    16-byte aligned as well: the calls refuse a base that lies where their
 *    kernels' wide reads of it cannot start.
 *  * Errors.  Arguments are checked on the host before anything is enqueued;
 *    a failed check returns a status and enqueues nothing.  A CUDA launch
 *    failure returns LRKV_ERR_CUDA.  Problems only the device can see (a
 *    seq_lens entry outside [0, max_len], a bounded wait that ran out) never
 *    trap: the kernels clamp, finish, and record the status in the workspace,
 *    readable with lrkv_read_device_status().  A wait of the kernels that
 *    keep copies or MMAs in flight (the bf16 decode scan, the RoPE, 8-bit and
 *    comparison decodes, lrkv_prefill_weights, lrkv_evict) gives up after
 *    LRKV_WAIT_LIMIT_CYCLES SM cycles (an environment variable read at each
 *    call; default 2e9, about 1 s); the kernel then skips the work that
 *    depended on it, still waits at the full bound for all that it issued,
 *    and records LRKV_ERR_TIMEOUT: the call's outputs are then not to be used.
 *    Set the variable only to exercise that path.
 *  * Order on the stream.  The calls' kernels use programmatic dependent
 *    launch.  A decode (lrkv_decode and its forms, the weighted, RoPE, 8-bit
 *    and comparison decodes) reads its inputs before it waits for the launch
 *    before it: they must be complete when that launch lets its dependents
 *    start.  A kernel that does not do so explicitly lets them start when it
 *    ends; so do all calls here that write a decode's input, but for
 *    lrkv_decode_step, whose new rows are sure to be seen by its own decode
 *    and by calls that wait (the next lrkv_decode_step, lrkv_append,
 *    lrkv_evict, lrkv_prefill_weights, lrkv_quantize, lrkv_pages_*).  A kernel
 *    of the caller's that signals early must not write q, positions, lengths,
 *    tables or rows afterwards.
 *  * Planning.  Launch grids and workspace sizes follow the current device's
 *    SM count, or LRKV_SM_COUNT when that environment variable holds a
 *    positive number (read at each call: workspace sizes without a device;
 *    results are the same for any value).
 *  * Scale.  dims->scale <= 0 selects 1/sqrt(head_dim), the scale of the
 *    summed score (technical review, §3 "Associative decode").
 *  * Positions.  Without RoPE the decode and prefill carry no position
 *    encoding; lrkv_decode_rope applies full RoPE to the keys exactly.
 */
#ifndef LRKV_H_
#define LRKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LRKV_ABI_VERSION 1

typedef enum {
  LRKV_OK = 0,
  LRKV_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, bad dtype          */
  LRKV_ERR_UNSUPPORTED = 2,   /* valid but outside the shapes the kernels implement */
  LRKV_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required          */
  LRKV_ERR_CUDA = 4,          /* a CUDA runtime call or kernel launch failed         */
  LRKV_ERR_TIMEOUT = 5,       /* device: a bounded wait ran out (reported, not trapped) */
  LRKV_ERR_DEVICE_BOUNDS = 6, /* device: a length, position or page out of range; clamped or skipped */
  LRKV_ERR_NO_PAGES = 7       /* device: fewer free pages than lrkv_pages_extend needs; nothing done */
} lrkv_status;

typedef enum { LRKV_F32 = 0, LRKV_BF16 = 1 } lrkv_dtype;

typedef struct {
  int batch;       /* B >= 1                                                  */
  int heads;       /* H >= 1                                                  */
  int head_dim;    /* d_h >= 1                                                */
  int rank;        /* r >= 0; r = 0 is MQA-style sharing (notes §2.1)         */
  int max_len;     /* token capacity of each sequence's cache rows            */
  lrkv_dtype dtype;
  float scale;     /* <= 0 selects 1/sqrt(head_dim)                           */
} lrkv_dims;

typedef void* lrkv_stream_t; /* a cudaStream_t */

/* ABI version of the loaded library (LRKV_ABI_VERSION). */
int lrkv_abi_version(void);

/* Human-readable name of a status code; never NULL. */
const char* lrkv_status_string(lrkv_status status);

/* Cache elements one token adds per layer: 2 (d_h + H r)
 * ("Low-Rank Key Value Attention：中文研读笔记", §2.5, Eq. (8)).
 * Returns 0 if any argument is negative. */
size_t lrkv_cache_elems_per_token(int heads, int head_dim, int rank);

/* Bytes of device workspace lrkv_decode needs for `dims` on the current
 * device (the split-KV partials depend on its SM count).  The workspace may
 * hold anything on entry; only its first 16 bytes (the device status word)
 * keep meaning after a call. */
lrkv_status lrkv_decode_workspace_size(const lrkv_dims* dims, size_t* bytes);

/*
 * One decode step of every head of every sequence against its factored
 * history ("Low-Rank Key Value Attention | What a shared cache can preserve",
 * §3, Algorithm 2, and the fused online-softmax paragraph after it;
 * "Low-Rank Key Value Attention：中文研读笔记", §2.4, Eqs. (6)-(7)).
 *
 *   q        [batch][heads][head_dim]  query of the new token (dtype)
 *   k_s, v_s, z_k, z_v                 the factored cache (layouts above); the
 *                                       new token's rows must already be in it
 *   b_k, b_v [heads][head_dim][rank]   reconstruction bases (dtype)
 *   seq_lens [batch] int32             sequence b attends rows [0, seq_lens[b]);
 *                                       0 gives out = 0 and lse = -inf
 *   out      [batch][heads][head_dim]  fp32 result o_h (heads not concatenated,
 *                                       no output projection)
 *   lse      [batch][heads] fp32 or NULL: natural-log log-sum-exp of the scaled
 *                                       scores
 *   ws, ws_bytes                        workspace of at least
 *                                       lrkv_decode_workspace_size() bytes
 * z_k, z_v, b_k, b_v may be NULL when rank == 0.
 * Supported: dtype BF16 with head_dim a multiple of 16 (<= 256) and rank <= 64,
 * ceil(heads/16) * head_dim / 8 <= 32; dtype F32 with rank <= 64,
 * head_dim <= 8 * (lanes per head); batch <= 4096.  Others return
 * LRKV_ERR_UNSUPPORTED.
 * Its inputs must be complete when the launch before it on the stream lets its
 * dependents start ("Order on the stream" above).
 */
lrkv_status lrkv_decode(const lrkv_dims* dims, const void* q, const void* k_s, const void* v_s,
                        const void* z_k, const void* z_v, const void* b_k, const void* b_v,
                        const int32_t* seq_lens, float* out, float* lse, void* ws, size_t ws_bytes,
                        lrkv_stream_t stream);

/*
 * lrkv_decode, plus two CUDA events (cudaEvent_t passed as void*, created by
 * the caller) recorded on `stream` immediately before and after the split-KV
 * kernel, the HBM-bound scan that dominates a decode step.  Used to time that
 * kernel alone; with the events in place the kernels of the step run
 * strictly one after another instead of overlapping their launch.  While
 * `stream` is being captured into a CUDA graph the events are recorded as
 * external event-record nodes, so that graph replays can be timed with them.
 * Both events are required (LRKV_ERR_INVALID_ARG otherwise).
 */
lrkv_status lrkv_decode_profiled(const lrkv_dims* dims, const void* q, const void* k_s,
                                 const void* v_s, const void* z_k, const void* z_v, const void* b_k,
                                 const void* b_v, const int32_t* seq_lens, float* out, float* lse,
                                 void* ws, size_t ws_bytes, lrkv_stream_t stream,
                                 void* ev_split_begin, void* ev_split_end);

/*
 * Size of the workspace array built into the library for
 * lrkv_decode_static_scratch: 16 MiB of device memory on every GPU that loads
 * the library, held until the process exits.
 */
#define LRKV_STATIC_SCRATCH_BYTES (16u * 1024u * 1024u)

/*
 * lrkv_decode for callers that cannot allocate device memory.  The LRKV pages
 * have no counterpart of this entry point: it only changes where the decode
 * workspace comes from.
 *
 * Some callers cannot hand lrkv_decode a workspace: a plugin inside a host
 * runtime that owns all device memory through its own pool, or a serving path
 * that must not allocate (and so possibly synchronise or fail) in the middle
 * of a request.  This call takes the workspace from a fixed array of
 * LRKV_STATIC_SCRATCH_BYTES compiled into the library and allocates nothing
 * (no cudaMalloc, cudaFree or allocating library routine).  Arguments and
 * results are those of lrkv_decode, without ws/ws_bytes.
 *
 *  * Shapes whose workspace (lrkv_decode_workspace_size) exceeds
 *    LRKV_STATIC_SCRATCH_BYTES return LRKV_ERR_WORKSPACE and enqueue nothing.
 *  * The first call on a device looks up the array's device address with the
 *    device current; make that first call before any stream capture.
 *  * All calls on a device share the array and it keeps the last call's
 *    contents; nothing in it has to start at zero.  Calls whose kernels
 *    overlap on the GPU (unordered streams) race on it.
 *  * The device status word lives at offset 0 of that array;
 *    lrkv_read_static_scratch_status reads it back (the last call's).
 */
lrkv_status lrkv_decode_static_scratch(const lrkv_dims* dims, const void* q, const void* k_s,
                                       const void* v_s, const void* z_k, const void* z_v,
                                       const void* b_k, const void* b_v, const int32_t* seq_lens,
                                       float* out, float* lse, lrkv_stream_t stream);

/*
 * The device status of the last lrkv_decode_static_scratch call on the
 * current device, as lrkv_read_device_status reports a workspace's: waits
 * for `stream` to drain, then sets *out_status to LRKV_OK,
 * LRKV_ERR_DEVICE_BOUNDS or LRKV_ERR_TIMEOUT.  Returns LRKV_ERR_INVALID_ARG
 * for a null out_status, LRKV_ERR_CUDA when the copy fails.  Allocates nothing.
 */
lrkv_status lrkv_read_static_scratch_status(lrkv_stream_t stream, lrkv_status* out_status);

/*
 * Append new tokens to the factored cache ("Low-Rank Key Value Attention |
 * What a shared cache can preserve", §3, Algorithm 1; "Low-Rank Key Value
 * Attention：中文研读笔记", §2.3): for every new token row x of sequence b,
 *   k_s = x W_sK^T, v_s = x W_sV^T (d_h each), and for every head h
 *   z_k,h = x U_h^K, z_v,h = x U_h^V (r each),
 * stored at cache row start_pos[b] + t.  One GEMM on the tensor cores with
 * fp32 accumulation; results rounded to bf16.
 *
 *   x          [batch][n_new][d_model]            layer input (bf16)
 *   w_sk, w_sv [head_dim][d_model]                shared projections, stored
 *                                                  output-major (row = output
 *                                                  column, like a Linear weight)
 *   u_k, u_v   [heads * rank][d_model]            per-head residual factors,
 *                                                  output-major; row h*r + c is
 *                                                  column c of U_h
 *   start_pos  [batch] int32 (device)             first cache row written
 *   k_s, v_s, z_k, z_v                            the cache (layouts above)
 *   ws, ws_bytes >= 16                            device status word
 * Supported: dtype BF16; d_model, head_dim and heads*rank multiples of 64.
 * Rows with start_pos[b] + t outside [0, max_len) are not written and set
 * LRKV_ERR_DEVICE_BOUNDS in the status word.
 */
lrkv_status lrkv_append(const lrkv_dims* dims, int d_model, int n_new, const void* x, const void* w_sk,
                        const void* w_sv, const void* u_k, const void* u_v, const int32_t* start_pos,
                        void* k_s, void* v_s, void* z_k, void* z_v, void* ws, size_t ws_bytes,
                        lrkv_stream_t stream);

/*
 * Causal attention of q_len new queries per sequence against the factored
 * cache, on the tensor cores ("Low-Rank Key Value Attention：中文研读笔记",
 * §2.4, Eqs. (6)-(7); "Low-Rank Key Value Attention | What a shared cache can
 * preserve", §3): logits [q_h | q_h B_h^K] . [k_s | z_k,h] / sqrt(d_h), one
 * causal softmax, values sum_j a_j v_s,j + (sum_j a_j z_v,h,j) (B_h^V)^T.
 *
 *   q        [batch][q_len][heads][head_dim]   queries (dtype)
 *   cache    rows [0, seq_lens[b]) hold the history including the q_len new
 *            tokens (append them first); query i sits at position
 *            seq_lens[b] - q_len + i and sees keys j <= that position
 *   out      [batch][q_len][heads][head_dim] fp32
 *   lse      [batch][heads][q_len] fp32 or NULL (natural log)
 *   ws, ws_bytes >= lrkv_prefill_workspace_size()  device status word (16-byte
 *                                              aligned)
 * q_h B_h^K enters its tensor-core contraction with the latents as the sum
 * of two bf16 parts (about 16 significant bits).  Supported: dtype BF16,
 * head_dim 128, rank 64.  seq_lens[b]
 * outside [q_len, max_len] is clamped and sets LRKV_ERR_DEVICE_BOUNDS.
 */
lrkv_status lrkv_prefill(const lrkv_dims* dims, int q_len, const void* q, const void* k_s, const void* v_s,
                         const void* z_k, const void* z_v, const void* b_k, const void* b_v,
                         const int32_t* seq_lens, float* out, float* lse, void* ws, size_t ws_bytes,
                         lrkv_stream_t stream);

/*
 * Bytes of device workspace lrkv_prefill, lrkv_prefill_normed and
 * lrkv_prefill_paged need for `dims` and `q_len` queries per sequence
 * ("Low-Rank Key Value Attention | What a shared cache can preserve", §3: the
 * prefill is Algorithm 2 for a block of causal queries).  The workspace holds
 * the device status word; the prefill kernel keeps its partial results on
 * chip and needs no other scratch memory.  Returns LRKV_ERR_INVALID_ARG or
 * LRKV_ERR_UNSUPPORTED for the shapes lrkv_prefill rejects (the same checks,
 * without the pointers); a prefill given fewer bytes returns
 * LRKV_ERR_WORKSPACE and enqueues nothing.
 */
lrkv_status lrkv_prefill_workspace_size(const lrkv_dims* dims, int q_len, size_t* bytes);

/*
 * One decode step of a layer: the new token's cache rows from its layer
 * input x, then attention over the cache that now holds them ("Low-Rank Key
 * Value Attention | What a shared cache can preserve", §3, Algorithm 1 for
 * one token, then Algorithm 2; "Low-Rank Key Value Attention：中文研读笔记",
 * §2.3-§2.4).  For every sequence b the token's
 *   k_s = x W_sK^T, v_s = x W_sV^T, z_k,h = x U_h^K, z_v,h = x U_h^V
 * (fp32 accumulation, rounded to bf16) are written at cache row
 * seq_lens[b] - 1, then the call decodes exactly like lrkv_decode over rows
 * [0, seq_lens[b]).  Two launches chained by programmatic dependent launch
 * (the decode's set-up overlaps the projection), plus the decode's merge.
 *
 *   x          [batch][d_model]               the new token's layer input
 *   w_sk, w_sv [head_dim][d_model]            as in lrkv_append (output-major)
 *   u_k, u_v   [heads * rank][d_model]        as in lrkv_append
 *   q, k_s, v_s, z_k, z_v, b_k, b_v, seq_lens, out, lse, ws, ws_bytes: as in
 *              lrkv_decode; seq_lens[b] counts the new token (seq_lens[b] = 0:
 *              no row is written and that sequence decodes as empty)
 * Supported: dtype BF16, rank >= 1, d_model a multiple of 8 (16-byte rows);
 * the decode's own limits.  Lengths outside [0, max_len] write no row and
 * set LRKV_ERR_DEVICE_BOUNDS through the decode.
 */
lrkv_status lrkv_decode_step(const lrkv_dims* dims, int d_model, const void* x, const void* w_sk,
                             const void* w_sv, const void* u_k, const void* u_v, const void* q, void* k_s,
                             void* v_s, void* z_k, void* z_v, const void* b_k, const void* b_v,
                             const int32_t* seq_lens, float* out, float* lse, void* ws, size_t ws_bytes,
                             lrkv_stream_t stream);

/*
 * Post-projection RMSNorm of the keys ("Low-Rank Key Value Attention | What a
 * shared cache can preserve", §8, "Post-projection normalization has a cache
 * cost"): the key of head h at token j, k = s_j + z_j B_h^T, is divided by its
 * joint RMS n = sqrt(mean_d k[d]^2 + eps) (never the two parts apart).  In a
 * kernel without RoPE the exact treatment caches one reciprocal scale per
 * head and token and multiplies the summed score by it; a per-head gain of
 * the norm is folded into q by the caller.
 *
 * lrkv_key_scales writes key_scale[b][h][t] = 1 / n (fp32) for the rows
 * t = start_pos[b] .. start_pos[b] + n_new - 1 of every sequence, from the
 * cached k_s, z_k (bf16, as stored) and B^K; rows outside [0, max_len) are
 * skipped.  Call it after appending the rows.
 *   key_scale  [batch][heads][max_len] fp32 (device), caller-allocated
 * Supported: dtype BF16, 1 <= rank <= 64, head_dim a multiple of 32 (at most
 * 256); k_s 16-byte aligned (else LRKV_ERR_INVALID_ARG).
 *
 * lrkv_decode_normed is lrkv_decode with every summed score multiplied by
 * key_scale[b][h][j] before the softmax (values are not normalised).
 * Supported: the shapes on which lrkv_decode streams bf16 (others return
 * LRKV_ERR_UNSUPPORTED).
 *
 * lrkv_prefill_normed is lrkv_prefill with the same per-key multiplication
 * of the summed scores (before the causal mask and the softmax); key_scale
 * must hold rows [0, seq_lens[b]) of every sequence.  key_scale NULL returns
 * LRKV_ERR_INVALID_ARG.  Supported: the shapes of lrkv_prefill.
 */
lrkv_status lrkv_key_scales(const lrkv_dims* dims, float eps, int n_new, const void* k_s, const void* z_k,
                            const void* b_k, const int32_t* start_pos, float* key_scale, lrkv_stream_t stream);
lrkv_status lrkv_decode_normed(const lrkv_dims* dims, const void* q, const void* k_s, const void* v_s,
                               const void* z_k, const void* z_v, const void* b_k, const void* b_v,
                               const float* key_scale, const int32_t* seq_lens, float* out, float* lse, void* ws,
                               size_t ws_bytes, lrkv_stream_t stream);
lrkv_status lrkv_prefill_normed(const lrkv_dims* dims, int q_len, const void* q, const void* k_s,
                                const void* v_s, const void* z_k, const void* z_v, const void* b_k,
                                const void* b_v, const float* key_scale, const int32_t* seq_lens, float* out,
                                float* lse, void* ws, size_t ws_bytes, lrkv_stream_t stream);

/*
 * Decode over a paged factored cache (page boundaries as a serving concern:
 * "Low-Rank Key Value Attention | What a shared cache can preserve", §4 and
 * §9; the pages give no layout).  The rows of every sequence live in pages
 * of page_size rows drawn from one pool per cache tensor:
 *   k_s, v_s     [num_pages][page_size][head_dim]
 *   z_k, z_v     [num_pages][page_size][heads][rank]
 *   block_table  [batch][max_len / page_size] int32 (device): logical row t
 *                of sequence b is row t % page_size of page
 *                block_table[b][t / page_size]; entries of blocks at or past
 *                seq_lens[b] are not read
 * dims->max_len is the logical capacity of a sequence (a multiple of
 * page_size).  Everything else (q, b_k, b_v, seq_lens, out, lse, ws, the
 * workspace size from lrkv_decode_workspace_size(dims)) is as in lrkv_decode,
 * and so is the result over the logical rows [0, seq_lens[b]).
 * page_size: a power of two >= 16 (a 16-token tile never spans two pages);
 * num_pages * page_size < 2^31.  A block table entry outside [0, num_pages)
 * reads as zero rows and sets LRKV_ERR_DEVICE_BOUNDS in the status word.
 * Supported: the shapes on which lrkv_decode streams bf16 (others return
 * LRKV_ERR_UNSUPPORTED).
 */
lrkv_status lrkv_decode_paged(const lrkv_dims* dims, int page_size, int num_pages, const int32_t* block_table,
                              const void* q, const void* k_s, const void* v_s, const void* z_k, const void* z_v,
                              const void* b_k, const void* b_v, const int32_t* seq_lens, float* out, float* lse,
                              void* ws, size_t ws_bytes, lrkv_stream_t stream);

/*
 * Appends into a paged cache (pools, block table and page_size as in
 * lrkv_decode_paged): after a prefill, at any position, across page
 * boundaries.
 *
 * lrkv_append_paged is lrkv_append writing logical row start_pos[b] + t of
 * sequence b through the block table; a row whose block names no page of the
 * pool is not written and sets LRKV_ERR_DEVICE_BOUNDS in the status word
 * (as a row past max_len does).
 *
 * lrkv_decode_step_paged is lrkv_decode_step over a paged cache: the token's
 * rows go to logical row seq_lens[b] - 1 through the block table (a page
 * outside the pool: no row; the decode flags it), then lrkv_decode_paged.
 */
/*
 * Causal prefill over a paged cache (pools, block table as in
 * lrkv_decode_paged): lrkv_prefill over the logical rows [0, seq_lens[b]);
 * the chunk's own rows are appended first (lrkv_append_paged), the rows
 * before them are the cached prefix.  page_size: a power of two >= 128 (a
 * 128-key tile never spans two pages).  A block table entry outside the pool
 * reads as zero rows and sets LRKV_ERR_DEVICE_BOUNDS.  Supported: the shapes
 * of lrkv_prefill.
 */
lrkv_status lrkv_prefill_paged(const lrkv_dims* dims, int q_len, const void* q, int page_size, int num_pages,
                               const int32_t* block_table, const void* k_s, const void* v_s, const void* z_k,
                               const void* z_v, const void* b_k, const void* b_v, const int32_t* seq_lens,
                               float* out, float* lse, void* ws, size_t ws_bytes, lrkv_stream_t stream);
lrkv_status lrkv_append_paged(const lrkv_dims* dims, int d_model, int n_new, const void* x, const void* w_sk,
                              const void* w_sv, const void* u_k, const void* u_v, const int32_t* start_pos,
                              int page_size, int num_pages, const int32_t* block_table, void* k_s, void* v_s,
                              void* z_k, void* z_v, void* ws, size_t ws_bytes, lrkv_stream_t stream);
lrkv_status lrkv_decode_step_paged(const lrkv_dims* dims, int d_model, const void* x, const void* w_sk,
                                   const void* w_sv, const void* u_k, const void* u_v, const void* q,
                                   int page_size, int num_pages, const int32_t* block_table, void* k_s, void* v_s,
                                   void* z_k, void* z_v, const void* b_k, const void* b_v, const int32_t* seq_lens,
                                   float* out, float* lse, void* ws, size_t ws_bytes, lrkv_stream_t stream);

/*
 * Decode with full rotary position embedding (RoPE) of the keys, exactly
 * ("Low-Rank Key Value Attention | What a shared cache can preserve", §8,
 * "Full RoPE needs a stronger identity"; "Low-Rank Key Value
 * Attention：中文研读笔记", §2.7).  A key rotation cannot be moved into the
 * rank-r latent for a generic basis, so the cache keeps unrotated rows and the
 * decode rebuilds each key, k_j = s_j + z_j B_h^T, turns it by the rotation of
 * its position j and takes the dot product with the query, which the caller
 * passes already rotated to its own position (the review's q~).  Values are
 * not rotated.  For head h and row j of sequence b:
 *   score = scale * q~_h . (k_j D_j),  D_j: each pair (2k, 2k+1) turned by the
 *   angle j theta_k (as the complex number x_2k + i x_2k+1 times
 *   exp(i j theta_k)), theta_k = base^(-2k / head_dim);
 * one softmax over the rows [0, seq_lens[b]); o_h as in lrkv_decode.  Row j
 * of the cache sits at position j.
 *
 * lrkv_rope_table writes the rotation table cos_sin [max_pos][head_dim] fp32
 * (device, caller-allocated): cos_sin[j][2k] = cos(j theta_k),
 * cos_sin[j][2k+1] = sin(j theta_k), with the angle and both functions in
 * fp64, rounded once to fp32.  Compute it once per model; base > 1, head_dim
 * even.
 *
 * lrkv_decode_rope takes the arguments of lrkv_decode (q is q~, [B][H][d_h]
 * in the cache dtype) plus the table and its row count max_pos (at least
 * dims->max_len, else LRKV_ERR_INVALID_ARG), and a workspace of
 * lrkv_decode_rope_workspace_size() bytes.  Supported: dtype BF16,
 * head_dim 64 or 128, rank 16, 32, 48 or 64, heads a multiple of 8, a
 * contiguous cache; others return LRKV_ERR_UNSUPPORTED.  The rebuild costs
 * head_dim x rank multiply-adds per (row, head) on the tensor cores beyond
 * lrkv_decode.
 */
lrkv_status lrkv_rope_table(int max_pos, int head_dim, float base, float* cos_sin, lrkv_stream_t stream);
lrkv_status lrkv_decode_rope_workspace_size(const lrkv_dims* dims, size_t* bytes);
lrkv_status lrkv_decode_rope(const lrkv_dims* dims, const void* q_rot, const void* k_s, const void* v_s,
                             const void* z_k, const void* z_v, const void* b_k, const void* b_v,
                             const float* cos_sin, int max_pos, const int32_t* seq_lens, float* out, float* lse,
                             void* ws, size_t ws_bytes, lrkv_stream_t stream);

/*
 * A cache inside a token budget.  Four calls: the attention weights that each
 * cache row gathers, from decode steps (lrkv_decode_weighted) and from a
 * prompt's queries (lrkv_prefill_weights); the eviction of the rows that
 * gathered least (lrkv_evict); and, since a row then no longer sits at its
 * position, a full-RoPE decode whose rows carry their positions
 * (lrkv_decode_rope_axes, below).  The pages have no counterpart: eviction
 * shortens the same cache that the factorisation narrows.  A row's shared part
 * serves every head, so a token is kept or dropped for all heads at once and
 * its weight is the sum over them.
 *
 * Weights are fp32, [batch][max_len].  A call reads `weights` and writes
 * `weights_out` (the same array for an update in place) on the rows [0, L_b)
 * of each sequence and leaves the others as they were:
 *   weights_out[j] = decay * weights[j] + what the call's queries gave row j
 * where the rows of the call's own new tokens have no earlier weight: their
 * slots in `weights` are not read and may hold anything, so nothing has to be
 * cleared when a row is appended.  decay >= 0 and finite, else
 * LRKV_ERR_INVALID_ARG; 1 accumulates, less forgets, 0 reads no earlier weight
 * at all (`weights` may then be NULL).  Sums are fp32, in a fixed order.
 *
 * lrkv_decode_weighted is one decode step as lrkv_decode (page_size,
 * num_pages and block_table as in lrkv_decode_paged, block_table NULL: a
 * contiguous cache; key_scale as in lrkv_decode_normed, or NULL) that also
 * accumulates
 *   sum over the heads of a_{h,j}
 * into row j; its new token is row L_b - 1.  The cache is read once.  out is
 * held to fp32 accuracy (q B^K and the probabilities enter their products as
 * three bf16 parts).  lse must not be NULL.  Supported: the shapes on which
 * lrkv_decode streams bf16 (others return LRKV_ERR_UNSUPPORTED).  Workspace:
 * lrkv_decode_weighted_workspace_size() bytes (the decode's and the scores,
 * 4 batch heads max_len).
 *
 * lrkv_prefill_weights accumulates what the last `window` of a prompt's q_len
 * queries looked at,
 *   sum over those queries i and the heads of exp(score_{h,i,j} - lse_{h,i}),
 * from q [batch][q_len][heads][head_dim], the keys' half of the cache and the
 * lse [batch][heads][q_len] that lrkv_prefill (lrkv_prefill_normed with
 * key_scale, lrkv_prefill_paged with block_table) wrote; a query with lse -inf
 * gives nothing, whatever it holds (padding).  Query i sits at row seq_lens[b] - q_len + i and sees the rows
 * up to its own; the prompt's q_len rows are the call's new tokens, so call it
 * once per chunk.  seq_lens[b] outside [q_len, max_len] is clamped and sets
 * LRKV_ERR_DEVICE_BOUNDS.  1 <= window <= q_len (else LRKV_ERR_INVALID_ARG),
 * q_len <= max_len.  q B^K enters the scores as two bf16 parts (the decode's
 * as three): a score is off by up to 2^-16 of sum |q B^K| |z_k| more than
 * fp32 arithmetic makes it, a weight by that much of itself.  Supported:
 * dtype BF16, head_dim 64 or 128, rank a multiple of 8 up to 64, heads <=
 * 256; page_size a power of two >= 16. z_k and b_k may be NULL when rank ==
 * 0.  Workspace: lrkv_prefill_weights_workspace_size() bytes; its status
 * word is set afresh.
 */
lrkv_status lrkv_decode_weighted_workspace_size(const lrkv_dims* dims, size_t* bytes);
lrkv_status lrkv_decode_weighted(const lrkv_dims* dims, const void* q, int page_size, int num_pages,
                                 const int32_t* block_table, const void* k_s, const void* v_s, const void* z_k,
                                 const void* z_v, const void* b_k, const void* b_v, const float* key_scale,
                                 const int32_t* seq_lens, float decay, const float* weights, float* weights_out,
                                 float* out, float* lse, void* ws, size_t ws_bytes, lrkv_stream_t stream);
lrkv_status lrkv_prefill_weights_workspace_size(const lrkv_dims* dims, int window, size_t* bytes);
lrkv_status lrkv_prefill_weights(const lrkv_dims* dims, int q_len, int window, const void* q, int page_size,
                                 int num_pages, const int32_t* block_table, const void* k_s, const void* z_k,
                                 const void* b_k, const float* key_scale, const float* lse,
                                 const int32_t* seq_lens, float decay, const float* weights, float* weights_out,
                                 void* ws, size_t ws_bytes, lrkv_stream_t stream);

/*
 * Eviction.  Sequence b keeps n = min(L_b, budget) of its L_b = seq_lens[b]
 * rows:
 *   - the held rows: age < sink (the first tokens) or age >= newest - recent,
 *     where the age of a row is order[b][j] (its token's number, >= 0; NULL:
 *     the row index) and newest is one past the largest age;
 *   - then the rows of the largest weights, equal weights by the lower row,
 *     NaN as -infinity.  (If the ages given hold more than n rows, these
 *     compete by weight among themselves.)
 * Attention does not depend on the order of the rows, so none is shifted: a
 * kept row below n stays, and the k-th kept row at or past n moves into the
 * k-th dropped row below n (both counted upwards).  Moved with it: k_s, v_s,
 * z_k, z_v (in place), key_scale [batch][heads][max_len] and positions
 * [batch][max_len][axes] when given (in place), its weight and its age.
 *   weights [batch][max_len] -> weights_out (may be the same array)
 *   order   [batch][max_len] or NULL -> order_out or NULL (may be the same)
 *   seq_lens -> new_lens [batch] = n (may be the same)
 *   kept    [batch][budget] int32 or NULL: the former row of row i < n, -1
 *           past n
 * Rows at or past n are left as they were, in every array.  With order, number
 * the tokens appended afterwards on (order[b][new row] = tokens seen so far):
 * after an eviction the row index no longer tells the age.
 * block_table as in lrkv_decode_paged (NULL: contiguous), here with any
 * power-of-two page_size; pages past a sequence's last kept row are free after
 * the call.  Pages that are written must belong to one sequence only (not to
 * several after lrkv_pages_fork).  A row whose block names no page of the pool is not moved (its weight, age and
 * kept entry are) and sets LRKV_ERR_DEVICE_BOUNDS, as a length outside
 * [0, max_len], which is clamped, does.
 * dtype BF16 or F32; rows of a multiple of 16 bytes; batch max_len at most
 * 2^31 - 2^16 (for lrkv_prefill_weights too); 1 <= budget <= max_len;
 * sink, recent >= 0 and sink + recent <= budget; axes 1 .. 4 with positions, 0
 * without.  z_k, z_v may be NULL when rank == 0.  Workspace:
 * lrkv_evict_workspace_size() bytes, its status word set afresh.  The call
 * works in place: after LRKV_ERR_TIMEOUT some rows have moved and others have
 * not, and the sequences have to be built anew.
 */
lrkv_status lrkv_evict_workspace_size(int batch, int max_len, int budget, size_t* bytes);
lrkv_status lrkv_evict(const lrkv_dims* dims, int budget, int sink, int recent, const float* weights,
                       const int32_t* order, const int32_t* seq_lens, int page_size, int num_pages,
                       const int32_t* block_table, void* k_s, void* v_s, void* z_k, void* z_v, float* key_scale,
                       int32_t* positions, int axes, float* weights_out, int32_t* order_out, int32_t* new_lens,
                       int32_t* kept, void* ws, size_t ws_bytes, lrkv_stream_t stream);

/*
 * Rotary positions with several axes.  A head's pairs (2k, 2k+1) are cut into
 * consecutive sections, sections[a] pairs for axis a (time, height, width;
 * host array, `axes` of them, 1 .. 4, none negative, adding up to head_dim/2):
 * pair k turns by p_a theta_k with the position p_a on its axis, theta_k and
 * the table cos_sin [max_pos][head_dim] as in lrkv_rope_table.  One axis whose
 * positions are the row indices is the rotation of lrkv_decode_rope.
 * Positions are int32; one outside [0, max_pos) is clamped and sets
 * LRKV_ERR_DEVICE_BOUNDS.
 *
 * lrkv_rope_rotate turns x [batch][n][heads][head_dim] (dims->dtype, BF16 or
 * F32; dims->batch, heads and head_dim used) by positions [batch][n][axes]
 * into out (may be x): the rotated queries of the calls below.  fp32
 * arithmetic, rounded once.  head_dim * sizeof(elem) a multiple of 16, at most
 * 1024 elements; x, out 16-byte aligned.  ws: NULL, or 16 bytes whose status
 * word the call ORs its bits into (the caller clears it).
 *
 * lrkv_decode_rope_axes is lrkv_decode_rope with the keys of row j turned by
 * positions[b][j][axis] (positions [batch][max_len][axes]; rows at or past
 * seq_lens[b] are not read), so that rows may have been moved or evicted, and
 * with the accumulation of lrkv_decode_weighted when weights_out is not NULL
 * (then lse must not be NULL either).  out is held to fp32 accuracy.
 * Supported: the shapes of lrkv_decode_rope, which are fewer than lrkv_evict
 * moves: contiguous bf16 caches without key scales.  Workspace:
 * lrkv_decode_rope_axes_workspace_size() bytes (the scores of the accumulation
 * among them, also for a call without it).
 */
lrkv_status lrkv_rope_rotate(const lrkv_dims* dims, int n, const void* x, const int32_t* positions, int axes,
                             const int* sections, const float* cos_sin, int max_pos, void* out, void* ws,
                             size_t ws_bytes, lrkv_stream_t stream);
lrkv_status lrkv_decode_rope_axes_workspace_size(const lrkv_dims* dims, size_t* bytes);
lrkv_status lrkv_decode_rope_axes(const lrkv_dims* dims, const void* q_rot, const void* k_s, const void* v_s,
                                  const void* z_k, const void* z_v, const void* b_k, const void* b_v,
                                  const float* cos_sin, int max_pos, const int32_t* positions, int axes,
                                  const int* sections, const int32_t* seq_lens, float decay, const float* weights,
                                  float* weights_out, float* out, float* lse, void* ws, size_t ws_bytes,
                                  lrkv_stream_t stream);

/*
 * The factored cache in 8 bits.  Every element of k_s, v_s, z_k, z_v is an
 * e4m3 number (sign, 4 bits of exponent, 3 of mantissa, largest 448, no
 * infinity; one byte) times the scale of its block: LRKV_BLOCK8 consecutive
 * rows of a sequence share one fp32 scale per tensor and head (the shared rows
 * count as one head),
 *   value = scale[block][head] * e4m3,
 * so a token costs half of what it costs in bf16, and 8 (1 + heads) / 16 bytes
 * of scales.  The pages have no counterpart.  Layouts, contiguous (rows =
 * max_len, lead = batch) or pools of pages (rows = page_size, lead =
 * num_pages; block_table as in lrkv_decode_paged), with
 * blocks = ceil(rows / LRKV_BLOCK8):
 *   k_s, v_s              [lead][rows][head_dim]     e4m3
 *   z_k, z_v              [lead][rows][heads][rank]  e4m3 (NULL when rank == 0)
 *   k_s_scale, v_s_scale  [lead][blocks]             fp32
 *   z_k_scale, z_v_scale  [lead][blocks][heads]      fp32 (NULL when rank == 0)
 * The eight pointers are 16-byte aligned.
 */
#define LRKV_BLOCK8 16

typedef struct {
  void *k_s, *v_s, *z_k, *z_v;
  float *k_s_scale, *v_s_scale, *z_k_scale, *z_v_scale;
} lrkv_cache8;

/*
 * lrkv_quantize stores n_new rows of every sequence in an 8-bit cache, at rows
 * start_pos[b] + t: the rows of a prompt, or the one of a decode step.
 *   k_s, v_s [batch][n_new][head_dim], z_k, z_v [batch][n_new][heads][rank]
 *            dtype rows, as lrkv_append writes them into a cache of n_new rows
 *   start_pos [batch] int32; new_lens [batch] int32 or NULL: sequence b brings
 *            new_lens[b] <= n_new rows only (a padded batch; NULL: n_new each)
 * For each block of rows, tensor and head that gets rows: with `need` the
 * smallest power of two, 2^-126 at least, for which the largest finite
 * magnitude of the new rows is at most 448 need,
 *   scale = max(need, the block's scale if rows before start_pos[b] lie in it)
 * (a power of two keeps what a larger scale leaves of a number's bits, and no
 * finer scale makes an e4m3 number more exact).  New elements are x / scale
 * rounded to nearest even; magnitudes past 448 scale (infinities) become 448
 * scale and NaN stays NaN.  Where the scale has grown the earlier rows of the
 * block are rounded to it anew; a power of two only takes bits off numbers
 * that become small.  Rows at or past start_pos[b] + n are left as they were,
 * and so are blocks without a new row.  Only the block of start_pos[b] is read.
 * start_pos[b] + t outside [0, max_len), new_lens[b] outside [0, n_new] or a
 * page outside the pool: those rows are skipped, LRKV_ERR_DEVICE_BOUNDS.  Blocks
 * that are written must belong to one sequence only.  ws: NULL, or 16 bytes
 * whose status word the call ORs its bits into (the caller clears it).
 * dims->dtype (BF16 or F32) is that of the rows.  Supported: head_dim a
 * multiple of 16 up to 256, rank even up to 64, heads rank a multiple of 16,
 * heads <= 256, batch <= 4096; batch max_len, batch n_new and num_pages
 * page_size below 2^31 (batch max_len of a paged cache too, where max_len is
 * the width of its table in rows); page_size a power of two >= 16; block_table
 * NULL: contiguous.
 *
 * lrkv_decode8 is lrkv_decode over an 8-bit cache (block_table NULL:
 * contiguous).  The cache's numbers enter the products as they are; what
 * multiplies them is split into e4m3 parts that hold 24 bits, but that what is
 * small beside the largest of its kind is off by up to 2^-29 (q of a head),
 * 2^-37 (q B^K of a head) and 2^-30 (probability times value scale, of 128 rows
 * that begin at a multiple of 128) of that largest one.  Scales: any finite
 * positive numbers; where a score, the largest q or q B^K times a key scale or
 * a sum of values leaves fp32's range, so do outputs.  Rows at or past
 * seq_lens[b] and the scales of blocks past them may hold anything; a NaN in a
 * visible row may make any output of its sequence NaN.  Supported: dtype BF16
 * (of q and the bases), and the shapes of lrkv_quantize; b_k and b_v 4-byte
 * aligned, faster at 16 bytes.  Workspace: lrkv_decode8_workspace_size()
 * bytes; errors as in lrkv_decode_paged.
 */
lrkv_status lrkv_quantize(const lrkv_dims* dims, int n_new, const void* k_s, const void* v_s, const void* z_k,
                          const void* z_v, const int32_t* start_pos, const int32_t* new_lens, int page_size,
                          int num_pages, const int32_t* block_table, const lrkv_cache8* cache, void* ws,
                          size_t ws_bytes, lrkv_stream_t stream);
lrkv_status lrkv_decode8_workspace_size(const lrkv_dims* dims, size_t* bytes);
lrkv_status lrkv_decode8(const lrkv_dims* dims, const void* q, int page_size, int num_pages,
                         const int32_t* block_table, const lrkv_cache8* cache, const void* b_k, const void* b_v,
                         const int32_t* seq_lens, float* out, float* lse, void* ws, size_t ws_bytes,
                         lrkv_stream_t stream);

/*
 * The pages of a paged cache, managed on the device: which page holds which
 * rows is decided by kernels on the call's stream, from arrays in device
 * memory, so that a serving step of forks, appends and decodes can be captured
 * whole.  The pages have no counterpart of it.
 *
 *   block_table [batch][max_blocks], seq_lens [batch] int32: as in
 *       lrkv_decode_paged.  Entry j of sequence b is in use when
 *       j < ceil(seq_lens[b] / page_size).
 *   refs [num_pages] int32: how many entries in use name the page, and whatever
 *       the caller adds to hold a page that no sequence names (a prompt kept
 *       for later).  A page is free when refs is 0 (or less).
 * Each call reads these and writes table_out, lens_out, refs_out, which may be
 * the same arrays (else they do not overlap).  All numbering is fixed: the
 * lowest free pages, in the order of the sequences.  page_size: a power of two
 * >= 16.  Lengths outside [0, max_blocks page_size] are clamped; these, and an
 * entry in use that names no page of the pool, set LRKV_ERR_DEVICE_BOUNDS (such
 * an entry stays as it is; lrkv_pages_extend looks only at those that its new
 * rows begin inside of).  ws: lrkv_pages_workspace_size() bytes, its status
 * word set afresh.  num_pages and batch * max_blocks at most 2^30, batch <= 4096.
 *
 * lrkv_pages_fork: sequence b becomes the first keep[b] rows of sequence
 * parent[b] as it was before the call, on the same pages: beams that go on
 * from other beams, samples of one prompt; keep[b] below its own length cuts
 * b back (after lrkv_evict: keep = new_lens), 0 frees it.  parent NULL: each
 * its own; -1: empty.  keep NULL: all rows; keep[b] past the parent's length
 * means all.  refs gains the entries in use after the call and loses those
 * before.  Entries not in use become -1.  Other values of parent, or a
 * negative keep, empty the sequence (LRKV_ERR_DEVICE_BOUNDS).  A sequence that
 * shares pages after a fork cannot be evicted: lrkv_evict moves rows inside of
 * pages that must be one sequence's own, and lrkv_pages_extend copies only the
 * page that new rows begin inside of.
 *
 * lrkv_pages_extend: room for the rows [seq_lens[b], new_lens[b]) of every
 * sequence (new_lens[b] <= seq_lens[b]: none), before they are appended.
 * Blocks without a page take free ones.  A page that the new rows begin inside
 * of and that others use too (refs > 1) is copied first: the rows before
 * seq_lens[b] of every pool go to a free page, and b leaves the shared one; of
 * sequences that would be its only users and all write, the last one keeps it.
 * Pages are taken in the order of the sequences, the copy's page first.  All or
 * nothing: when the free pages do not suffice, tables, lengths, refs and
 * pools stay as they were and *missing is the number of pages that lack
 * (LRKV_ERR_NO_PAGES in the status word), else 0.  lens_out = new_lens, refs 1
 * for each page taken.
 *
 * lrkv_pages_compact: the n pages in use (refs > 0) move to pages [0, n): the
 * k-th used page at or past n goes whole into the k-th free page below it, in
 * every pool; the tables' entries in use follow.  moved [num_pages] or NULL:
 * the new number of every page, -1 for free ones (for pages held outside the
 * tables).  *live = n.  refs_out moves with the pages.
 *
 * Pools: the arrays that the pages consist of, host array of n_pools (0 .. 16)
 * entries: page p of a pool is page_size / rows pieces of `bytes` bytes from
 * data + p * (page_size / rows) * bytes on, one piece for every `rows` rows (1:
 * a row of a cache tensor; LRKV_BLOCK8: the scales of a block of an 8-bit
 * cache).  data and bytes are multiples of 4; rows divides page_size; all pools
 * have num_pages pages.  Pools do not overlap.
 */
typedef struct {
  void* data;
  int rows;
  int bytes;
} lrkv_pool;

#define LRKV_MAX_POOLS 16

lrkv_status lrkv_pages_workspace_size(int batch, int max_blocks, int num_pages, size_t* bytes);
lrkv_status lrkv_pages_fork(int batch, int max_blocks, int page_size, int num_pages, const int32_t* parent,
                            const int32_t* keep, const int32_t* block_table, const int32_t* seq_lens,
                            const int32_t* refs, int32_t* table_out, int32_t* lens_out, int32_t* refs_out, void* ws,
                            size_t ws_bytes, lrkv_stream_t stream);
lrkv_status lrkv_pages_extend(int batch, int max_blocks, int page_size, int num_pages, const int32_t* new_lens,
                              const int32_t* block_table, const int32_t* seq_lens, const int32_t* refs,
                              int32_t* table_out, int32_t* lens_out, int32_t* refs_out, int32_t* missing,
                              const lrkv_pool* pools, int n_pools, void* ws, size_t ws_bytes, lrkv_stream_t stream);
lrkv_status lrkv_pages_compact(int batch, int max_blocks, int page_size, int num_pages, const int32_t* block_table,
                               const int32_t* seq_lens, const int32_t* refs, int32_t* table_out, int32_t* refs_out,
                               int32_t* moved, int32_t* live, const lrkv_pool* pools, int n_pools, void* ws,
                               size_t ws_bytes, lrkv_stream_t stream);

/*
 * Comparison decodes on the same box ("Low-Rank Key Value Attention | What a
 * shared cache can preserve", §4 "Weight count and the two decode regimes"
 * and §5: a fair serving comparison runs optimized GQA, dense MHA and
 * absorbed MLA beside the factored kernel at the same batch, length and
 * dtype).  They are not part of the LRKV method; they measure the layouts it
 * replaces.
 *
 * lrkv_dense_decode: one decode step over materialised K/V (bf16),
 *   q [batch][heads][head_dim], k, v [batch][max_len][kv_heads][head_dim];
 *   query head h attends KV head h / (heads / kv_heads) over rows
 *   [0, seq_lens[b]) with one softmax (MHA: kv_heads = heads; GQA; MQA:
 *   kv_heads = 1); out [batch][heads][head_dim] fp32, lse [batch][heads] or
 *   NULL.  No position encoding.  Supported: head_dim 64 or 128,
 *   heads / kv_heads in {1, 2, 4, 8}.  Workspace:
 *   lrkv_dense_decode_workspace_size() bytes; status word and errors as in
 *   lrkv_decode.
 */
typedef struct {
  int batch;       /* B >= 1                                 */
  int heads;       /* query heads H >= 1                     */
  int kv_heads;    /* KV heads, dividing H                   */
  int head_dim;    /* d                                      */
  int max_len;     /* rows per sequence in k and v           */
  float scale;     /* <= 0 selects 1/sqrt(head_dim)          */
} lrkv_dense_dims;

lrkv_status lrkv_dense_decode_workspace_size(const lrkv_dense_dims* dims, size_t* bytes);
lrkv_status lrkv_dense_decode(const lrkv_dense_dims* dims, const void* q, const void* k, const void* v,
                              const int32_t* seq_lens, float* out, float* lse, void* ws, size_t ws_bytes,
                              lrkv_stream_t stream);

/*
 * lrkv_mla_decode: absorbed multi-head latent attention over one latent row
 * per token for all heads (review §5: the head computes (q_h A_h) Z^T instead
 * of materialising its keys; the values likewise), bf16 storage:
 *   q [batch][heads][head_dim], c [batch][max_len][latent_dim],
 *   w_uk, w_uv [heads][head_dim][latent_dim] (K_h = C W_uk[h]^T,
 *   V_h = C W_uv[h]^T), score q_h . k_h,j * scale (scale <= 0:
 *   1/sqrt(head_dim)), one softmax, out [batch][heads][head_dim] fp32, lse as
 *   in lrkv_decode.  Three launches: q_h W_uk[h] (fp32, in the workspace),
 *   the scan over c (q_c split into two bf16 parts for the tensor cores), and
 *   the merge, which lifts the latent sum through W_uv[h]^T.  Supported:
 *   latent_dim 256 or 512, heads 8, 16 or 32, head_dim <= 128; c 16-byte
 *   aligned.  Workspace: lrkv_mla_decode_workspace_size() bytes.
 */
typedef struct {
  int batch;
  int heads;
  int head_dim;    /* d_h of q and of the output                          */
  int latent_dim;  /* d_c of the cached latent rows                       */
  int max_len;
  float scale;     /* <= 0 selects 1/sqrt(head_dim)                       */
} lrkv_mla_dims;

lrkv_status lrkv_mla_decode_workspace_size(const lrkv_mla_dims* dims, size_t* bytes);
lrkv_status lrkv_mla_decode(const lrkv_mla_dims* dims, const void* q, const void* c, const void* w_uk,
                            const void* w_uv, const int32_t* seq_lens, float* out, float* lse, void* ws,
                            size_t ws_bytes, lrkv_stream_t stream);

/*
 * Read the device status word that the kernels of the last call(s) using
 * `ws` recorded (LRKV_OK, LRKV_ERR_TIMEOUT, LRKV_ERR_NO_PAGES or
 * LRKV_ERR_DEVICE_BOUNDS).
 * Synchronises `stream`.  Each lrkv_decode/lrkv_prefill call sets the word
 * afresh: a decode writes the bits its kernels recorded (no clearing needed
 * before a call), a prefill clears it when it starts.
 */
lrkv_status lrkv_read_device_status(const void* ws, lrkv_stream_t stream, lrkv_status* out_status);

#ifdef __cplusplus
}
#endif

#endif /* LRKV_H_ */
