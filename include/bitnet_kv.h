/*
 * bitnet_kv.h -- C ABI of the paged 8-bit key/value cache and the attention
 * that reads it, part of the B200 (sm_100a) BitLinear library.
 *
 * These calls stand between the q / k / v projections (bitnet_linear and its
 * variants, see bitnet.h) and the output projection of a decoder layer (BitNet
 * model page: "Architecture" -- rotary position embeddings, grouped-query
 * attention; BitNetConfig: 20 query heads, 5 key/value heads of 128, context
 * 4096).  The page gives no formulas and no cache layout; both are defined
 * here.
 *
 * The cache holds keys and values as int8 codes in pages of page_size tokens,
 * with one fp32 step per (page, kv head):
 *
 *   k, v            [num_pages][n_kv_heads][page_size][head_dim] int8
 *   k_step, v_step  [num_pages][n_kv_heads] fp32, not negative;  value = code * step
 *
 * A batch of sequences is described on the device:
 *
 *   page_table  [n_seqs][table_width] int32: page of tokens j * page_size ..
 *               (j + 1) * page_size - 1 of sequence b at [b][j].  Entries
 *               behind a sequence's last token are never read.
 *   seq_lens    [n_seqs] int32: tokens of each sequence in the cache, the new
 *               ones included
 *   q_start     [n_seqs + 1] int32, q_start[0] >= 0, not decreasing: the new
 *               tokens of sequence b are rows q_start[b] .. q_start[b + 1] - 1
 *               of q, k, v and out, at positions seq_lens[b] - n_b ..
 *               seq_lens[b] - 1 (n_b = q_start[b + 1] - q_start[b], which may
 *               be 0).  Rows outside [q_start[0], q_start[n_seqs]) (padding)
 *               are not written, and what they hold has no effect.
 *
 * The conventions of bitnet.h hold (device pointers, caller-owned memory, no
 * allocation, no synchronisation, host-side validation before any launch,
 * 16-byte alignment of q, k, v, out, the codes, the rotation table and the
 * workspace, finite inputs), except that page_table, seq_lens, q_start and the
 * steps need only their natural 4-byte alignment.  Nothing is read before
 * earlier work on the same stream has finished.  The device of the stream must
 * be the current one.
 *
 * What only the device can see -- page ids, lengths, offsets, positions -- is
 * checked there: a page id outside [0, num_pages), a seq_lens[b] that is
 * negative, larger than table_width * page_size or (append only) smaller than
 * n_b, a q_start that decreases or leaves [0, T], a position beyond the rotation
 * table, or more new tokens than max_new makes the kernels skip what they would
 * have had to access and record BITNET_ERR_INVALID_ARG in the batch status word
 * (see bitnet_batch_status).  The outputs of the sequences concerned are then
 * unspecified; nothing outside the caller's buffers is touched.  A q_start that
 * decreases may leave sequences that look sound and claim the same rows: if all
 * together claim more than T, the attention for prompts computes none of them.
 */
#ifndef BITNET_KV_H
#define BITNET_KV_H

#include "bitnet.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct bitnet_kv_cache {
    int8_t *k, *v;          /* [num_pages][n_kv_heads][page_size][head_dim] */
    float *k_step, *v_step; /* [num_pages][n_kv_heads] */
    int64_t num_pages;      /* 1 .. 2^31 - 1 */
    int32_t n_kv_heads;     /* >= 1 */
    int32_t page_size;      /* 16, 32, 64 or 128 */
    int32_t head_dim;       /* 64 or 128 */
} bitnet_kv_cache_t;

typedef struct bitnet_kv_batch {
    const int32_t *page_table; /* [n_seqs][table_width] */
    const int32_t *seq_lens;   /* [n_seqs] */
    const int32_t *q_start;    /* [n_seqs + 1] */
    int64_t table_width;       /* pages per row of page_table; table_width * page_size < 2^31 */
    int32_t n_seqs;            /* 1 .. 65536 */
    int32_t T;                 /* rows of q, k, v and out (padding included): 1 .. 2^24 */
} bitnet_kv_batch_t;

/*
 * Table of the position rotation (page: "Architecture" -- rotary position
 * embeddings; BitNetConfig rope_theta = 500000), made once:
 *   table [max_pos][head_dim] fp32: row p holds cos(p w_j) for j = 0 ..
 *   head_dim / 2 - 1, then sin(p w_j), with w_j = theta^(-2 j / head_dim),
 * angles, cosines and sines in fp64, each rounded once.
 *   theta     > 0, finite;  max_pos 1 .. 2^24;  head_dim 64 or 128
 */
bitnet_status_t bitnet_rope_table(double theta, int64_t max_pos, int32_t head_dim, float *table, cudaStream_t stream);

/*
 * Rotates the new queries and keys by their positions, quantises the new keys
 * and values and writes them into the pages of their sequences.
 *
 *   q, k, v   rows t = 0 .. T - 1 of n_heads (k, v: n_kv_heads) heads of
 *             head_dim elements of type dtype; row t starts at element
 *             t * q_stride (k_stride, v_stride), so they may be parts of one
 *             fused projection's rows.  Strides are multiples of 16 bytes and
 *             at least the row's length.  q may be NULL (then q_out too):
 *             only the cache is written.
 *   rope      [rope_len][head_dim] fp32 table of bitnet_rope_table, or NULL: no
 *             rotation.  With (c, s) = cos, sin of the position:
 *               y[j]         = x[j] c_j - x[j + D/2] s_j
 *               y[j + D / 2] = x[j + D/2] c_j + x[j] s_j        (j < D / 2)
 *             in fp32, each product and sum rounded.
 *   q_out     [T][n_heads][head_dim] bf16, rows q_out_stride elements apart:
 *             the rotated queries rounded to nearest even.  It may be q itself
 *             (bf16, same stride) and lie between k and v in their rows, but
 *             must not overlap q, k or v otherwise, nor the cache, rope or the
 *             batch.
 *
 * The cache's four arrays lie apart from one another and from everything that
 * the call reads.
 *
 * For each page that gets new tokens, each kv head, and each of K (rotated) and
 * V, with x the new tokens' values there:
 *   t     = max |x| * fl(1 / 127)
 *   old   = the stored step if the page holds tokens before the first new one,
 *           else 0 (what the page held before is of no account)
 *   step  = max(old, t)                             (stored)
 *   codes before the first new token become rne(code * (old / step)) if step
 *   has grown; new codes are clamp(rne(x / step), -127, 127), 0 if step = 0.
 * All in fp32, each operation rounded, with IEEE division, so the codes are reproducible bit for bit and
 * do not depend on how the other sequences are batched.  Slots behind the last
 * token keep their bytes.  A page that gets new tokens must belong to one
 * sequence only (full pages may be shared).  Appending the same rows at the
 * same positions again is allowed; steps never shrink while a page keeps
 * earlier tokens.
 */
bitnet_status_t bitnet_kv_append(const bitnet_kv_cache_t *cache, const bitnet_kv_batch_t *batch,
                                 const void *q, const void *k, const void *v, bitnet_dtype_t dtype,
                                 int32_t n_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                 const float *rope, int64_t rope_len, void *q_out, int64_t q_out_stride,
                                 cudaStream_t stream);

/*
 * Attention of the new tokens over the cache, grouped-query, causal: row i of
 * sequence b, query head h (kv head h / (n_heads / n_kv_heads)) gives
 *   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale (q . k_j) - max),
 * over the cached tokens j <= seq_lens[b] - n_b + i of the sequence: every
 * earlier token and itself.  A row that sees no token (seq_lens[b] = 0, or less
 * than n_b for the first ones; allowed here, not in the append) gives zeros.
 *
 *   q          [T][n_heads][head_dim] bf16, rows q_stride elements apart
 *              (multiple of 8, at least n_heads * head_dim)
 *   n_heads    multiple of the cache's n_kv_heads, at most 128 per kv head
 *   max_new    at least the largest n_b, 1 .. T; it chooses the kernel: up to
 *              48 rows (max_new times query heads per kv head) the one for few
 *              new tokens, above that the one for prompts.  Either takes any
 *              n_b <= max_new, 0 included.
 *   scale      finite, > 0; 1 / sqrt(head_dim) in BitNet
 *   out        [T][n_heads][head_dim] bf16, rows out_stride elements apart
 *              (written); must not overlap the cache, the batch, nor q, except
 *              that it may be q itself with the same stride
 *   workspace  device scratch of at least bitnet_attention_workspace_size
 *              bytes, any contents, apart from q, out, the cache and the batch;
 *              calls that may overlap on the GPU need separate ones
 *
 * Weights and sums of the softmax are fp32; its weights enter the tensor cores in
 * fp16 (11 bits), the codes exactly, the queries in fp16 scaled by a power of two
 * per row (few new tokens) or as they are (prompts); products are summed in fp32
 * and the result is rounded to bf16 once.  Results do not depend on timing: the
 * same call gives the same bits.
 *
 * Ranges.  For prompts a sum of D products of a query's elements and codes has to
 * be finite in fp32 (always so below 2e34); for few tokens only the scores have
 * to.  A sum of 2^8 |v| over the tokens has to be finite.  Steps of one sequence
 * may lie any number of powers of two apart; what a page adds whose v_step is
 * below 2^-90 of the sequence's largest, or below 2^-35 of the largest within the
 * same 128 tokens, may be off by that fraction of the largest value.
 */
bitnet_status_t bitnet_attention(const bitnet_kv_cache_t *cache, const bitnet_kv_batch_t *batch, const void *q,
                                 int64_t q_stride, int32_t n_heads, int32_t max_new, float scale, void *out,
                                 int64_t out_stride, void *workspace, size_t ws_bytes, cudaStream_t stream);

/* Workspace of bitnet_attention for these sizes; 0 for sizes that it refuses. */
size_t bitnet_attention_workspace_size(int32_t n_seqs, int32_t T, int32_t n_heads, int32_t n_kv_heads,
                                       int32_t head_dim, int32_t max_new);

/*
 * Reads and resets (clear != 0) the batch status word of the current device:
 * BITNET_OK, or BITNET_ERR_INVALID_ARG once a call above met a batch it had to
 * refuse on the device.  Synchronises `stream`.
 */
bitnet_status_t bitnet_batch_status(int clear, bitnet_status_t *status_out, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BITNET_KV_H */
