/*
 * kvattend.h - operators that use a cache while an agent generates, AMD
 * Instinct MI355X (gfx950). Same library, conventions and error codes as
 * kvcodec.h (libkvcodec.so, C ABI):
 *
 *  - kvc_norm_rotate: norms of queries and keys for each head and the position
 *    rotation, in one pass over the projection's rows;
 *  - kvpage_write, kvpage_read: a paged cache of one layer, quantised as it is
 *    written, and read back;
 *  - kvpage_attend: attention of one new token per sequence over its pages;
 *  - kvpool_attend: attention of one new token of each of n agents over one
 *    layer of the shared pool (PolyKV section 2.A: every agent reads the same
 *    compressed document), without decompressing it, together with the pages
 *    that each agent filled itself.
 *
 * Conventions besides those of kvcodec.h:
 *  - Queries, keys, values and outputs are bf16 rows (kvc_rows): element
 *    (token n, head h, channel c) is data[n * token_stride + h * head_stride
 *    + c]. Strides are in elements and multiples of 8, data is 16-byte
 *    aligned, head_dim is 64 or 128. A stride whose count is 1 is not used.
 *    Rows that are read may repeat (stride 0) and may lie in one buffer (the
 *    rows of a fused projection). Rows that are written must be apart from
 *    one another and from everything that is read. Two sets of rows may lie
 *    in one buffer, between one another: the heads of a token (or the tokens of
 *    a head) of each together at places of their own within an equal stride, or
 *    single vectors at places of their own within the greatest common divisor of
 *    the strides, as of [tokens][heads][3][head_dim]. What lies between rows is
 *    neither read nor written.
 *  - Sizes of 0 (tokens, sequences, agents) enqueue nothing and return KVC_OK.
 *  - Sums, maxima and sums of the softmax, and norms are binary32.
 *  - A workspace needs no clearing and holds nothing between calls. Calls
 *    that overlap in time (other streams, replayed graphs) need workspaces of
 *    their own.
 *  - `stream` belongs to the device that is current.
 */
#ifndef KVATTEND_H
#define KVATTEND_H

#include "kvcodec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bf16 head vectors in memory (see above). */
typedef struct kvc_rows {
    void* data;
    uint64_t token_stride; /* elements from token n to n + 1 */
    uint64_t head_stride;  /* elements from head h to h + 1 */
} kvc_rows;

/* A paged cache of one layer: num_pages pages of page_tokens tokens. */
typedef struct kvc_pages {
    uint32_t num_pages;    /* >= 1 */
    uint32_t num_kv_heads; /* >= 1 */
    uint32_t page_tokens;  /* 16, 32, 64, 128 or 256 */
    uint32_t head_dim;     /* 64 or 128 */
    uint32_t format;       /* KVC_PAGE_* */
} kvc_pages;

#define KVC_PAGE_BF16 0u /* the values as they are */
#define KVC_PAGE_INT8 1u /* int8 codes, one binary32 step for each head vector */
#define KVC_PAGE_FP8 2u  /* e4m3 codes (OCP, no infinities), one binary32 step for each head vector */

/* Further bits of *dev_status. */
enum {
    KVC_DEV_BAD_SLOT = 16,  /* a slot is not below num_pages * page_tokens */
    KVC_DEV_BAD_PAGE = 32,  /* a page number of a table is not a page */
    KVC_DEV_BAD_LENGTH = 64 /* a length is negative or longer than its table's row */
};

/* ------------------------------------------------------ norm and rotation */

/* Norm of each query and key head vector and the rotation to its position,
 * in one pass:
 *     y = x * (1 / sqrt(mean(x^2) + eps)) * weight       (weight given)
 *     pair j of y turned by positions[n] * inv_freq[j]   (first 2 * n_pairs channels)
 * Pair j is (j, j + n_pairs) or (2j, 2j + 1) (KVC_ROPE_*); channels from
 * 2 * n_pairs on are not turned. The angle is the binary64 product, reduced
 * to a turn in binary64; everything else is binary32, rounded once to bf16. So
 * mean(x^2) + eps has to be a normal binary32 number: values up to 2^60, and with
 * eps = 0 vectors whose largest value is 2^-59 or more (a zero vector gives NaN).
 *   q_in, k_in     rows of n_tokens x q_heads and n_tokens x kv_heads;
 *                  n_tokens <= 2^26 - 4
 *   q_weight, k_weight  device bf16 [head_dim], 16-byte aligned, or NULL: no norm
 *   eps            >= 0 and finite
 *   positions      device int64 [n_tokens], 8-byte aligned (not used, may be
 *                  NULL, if n_pairs is 0)
 *   inv_freq       host, n_pairs floats; n_pairs a multiple of 8, at most head_dim / 2
 *   q_out, k_out   rows; the same as q_in / k_in turns in place
 * kv_heads may be 0 (then k_in, k_out are not used), and so may q_heads.
 * Errors: KVC_E_NULL, KVC_E_SHAPE, KVC_E_RANGE (pairing, n_pairs, eps),
 * KVC_E_ALIGN, KVC_E_ALIAS, KVC_E_HIP. */
int kvc_norm_rotate(uint32_t n_tokens, uint32_t q_heads, uint32_t kv_heads, uint32_t head_dim,
                    const kvc_rows* q_in, const kvc_rows* k_in, const void* q_weight, const void* k_weight,
                    float eps, const int64_t* positions, const float* inv_freq, uint32_t n_pairs,
                    uint32_t pairing, const kvc_rows* q_out, const kvc_rows* k_out, hipStream_t stream);

/* ------------------------------------------------------------- paged cache */

/* Bytes of a paged cache; 0 if the description is invalid. Layout: pages one
 * after another, each on a 256-byte boundary:
 *   codes  [2][num_kv_heads][page_tokens][head_dim]  keys, then values (bf16,
 *          int8 or e4m3)
 *   steps  f32 [2][num_kv_heads][page_tokens]        (8-bit formats) */
size_t kvpage_bytes(const kvc_pages* spec);

/* Write keys and values of n_tokens tokens into their slots.
 *   k, v     rows of n_tokens x num_kv_heads; n_tokens < 2^26
 *   slots    device int64 [n_tokens], 8-byte aligned: page * page_tokens +
 *            offset; a negative slot is skipped (padding). Slots of one call
 *            are distinct: a slot that is given twice holds codes and steps
 *            of either token, in any mixture.
 * 8-bit formats, for each head vector: m = max |x|, step = m / M, code =
 * x * M / m rounded to nearest, ties to even (M = 127 or 448; exact products
 * and correctly rounded quotients, so a code is the nearest one). m = 0 gives
 * step 0 and codes 0. A vector that holds an Inf or NaN gets a NaN step and
 * codes 0: it reads back as NaN.
 *   dev_status  device int32 or NULL; KVC_DEV_BAD_SLOT (that token is not written)
 * Errors: KVC_E_NULL, KVC_E_SHAPE, KVC_E_SIZE, KVC_E_ALIGN, KVC_E_ALIAS,
 * KVC_E_HIP. */
int kvpage_write(const kvc_pages* spec, void* pages, size_t pages_bytes, uint32_t n_tokens, const kvc_rows* k,
                 const kvc_rows* v, const int64_t* slots, int32_t* dev_status, hipStream_t stream);

/* Read tokens back: bf16(code * step), one rounding. Rows of negative slots,
 * and of slots outside the cache (KVC_DEV_BAD_SLOT), are left as they were.
 * Errors as kvpage_write. */
int kvpage_read(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_tokens,
                const int64_t* slots, const kvc_rows* k_out, const kvc_rows* v_out, int32_t* dev_status,
                hipStream_t stream);

/* --------------------------------------------------------------- attention */

/* Workspace bytes of kvpage_attend for at most n_seqs sequences of at most
 * max_tokens tokens (table_cols * page_tokens of the call): never less for more of
 * either, so one workspace of a program's largest call serves all of its calls. 0 if
 * an argument is invalid. */
size_t kvpage_attend_workspace_bytes(const kvc_pages* spec, uint32_t n_seqs, uint32_t q_heads, uint32_t max_tokens);

/* Attention of one new token for each of n_seqs sequences over its pages:
 *     out[b][h] = sum_t p_t v_t,  p = softmax_t(scale * q[b][h] . k_t)
 * over the lens[b] tokens of sequence b, token t in page
 * table[b][t / page_tokens]; head h reads kv head h / (q_heads / num_kv_heads).
 * Keys and values are code * step as real numbers. A sequence of length 0
 * gives zeros and lse = -inf. What lies behind a sequence's length is not
 * used, whatever it holds.
 *   q, out     rows of n_seqs x q_heads (out elsewhere than q); q_heads a
 *              multiple of num_kv_heads
 *   table      device int32, row b at table + b * table_stride, table_cols >= 1
 *              entries (all may be read; those that lens[b] does not reach may
 *              hold anything). Sequences may share pages.
 *   lens       device int32 [n_seqs]
 *   scale      finite, and so times log2(e)
 *   lse        device f32 [n_seqs][q_heads] or NULL: ln sum_t exp(scale * q . k_t)
 *   ws         device workspace, 256-byte aligned, of
 *              kvpage_attend_workspace_bytes(spec, n_seqs, q_heads, table_cols * page_tokens)
 *              bytes or more
 *   dev_status device int32 or NULL; KVC_DEV_BAD_PAGE, KVC_DEV_BAD_LENGTH: the
 *              sequence's output is then unspecified (lengths are clamped, a
 *              page that is none is taken as page 0)
 * n_seqs * q_heads < 2^23; table_cols * page_tokens < 2^31, and n_seqs times
 * (table_cols * page_tokens / 128 + 1) < 2^31. Long sequences are cut up among
 * workgroups and their parts joined by a second launch, in an order that the
 * arguments alone decide: the same call gives the same bits.
 * The 8-bit formats' weights p_t * step are rounded to binary16 after division
 * by a power of two (about the largest step) for the matrix cores, bf16's are
 * split into two bf16 terms; products and sums are binary32. Of a weight times its
 * step, what lies below 2^-36 of the largest step (or of 2^-100) is lost. So q . k (before
 * and after the scale), and the weighted sums before they are divided by the
 * weights' (at most 8 times the tokens times the largest value), have to stay in
 * binary32's range; queries and keys may lie anywhere in bf16's. Where all
 * logits of a row are -inf, the row is as that of an empty sequence; a NaN in a
 * query or in a key or value that its length reaches gives NaN.
 * Errors: KVC_E_NULL, KVC_E_SHAPE, KVC_E_RANGE, KVC_E_SIZE, KVC_E_ALIGN,
 * KVC_E_ALIAS, KVC_E_HIP. */
int kvpage_attend(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_seqs, uint32_t q_heads,
                  const kvc_rows* q, const int32_t* table, uint32_t table_cols, uint64_t table_stride,
                  const int32_t* lens, float scale, const kvc_rows* out, float* lse, void* ws, size_t ws_bytes,
                  int32_t* dev_status, hipStream_t stream);

/* The pages of the agents behind a shared pool (see kvpage_attend). */
typedef struct kvc_tail {
    const kvc_pages* spec; /* num_kv_heads and head_dim are the pool's */
    const void* pages;
    size_t pages_bytes;
    const int32_t* table; /* row a: agent a's pages */
    uint32_t table_cols;
    uint64_t table_stride;
    const int32_t* lens; /* [n_agents] */
} kvc_tail;

/* Workspace bytes of kvpool_attend for at most n_agents agents; tail_spec NULL:
 * without tails, else for tails of at most max_tail_tokens tokens. Never less for more
 * agents, pool or tail tokens, or for tails than for none. 0 if an argument is invalid. */
size_t kvpool_attend_workspace_bytes(const kvc_shape* shape, uint32_t n_agents, uint32_t q_heads,
                                     const kvc_pages* tail_spec, uint32_t max_tail_tokens);

/* Attention of one new token of each of n_agents agents over layer `layer` of
 * a pool (all num_tokens tokens of it), and over the agent's own tail:
 *     out[a][h] = sum_t p_t v_t,  p = softmax over the pool's tokens and the tail's
 * The pool's keys are code * step; its values are the inverse transform of
 * the levels times the vector's scale, as real numbers. (kvpool_decode gives
 * these rounded to bf16.) The transform is linear, so it is applied to the
 * weighted sums of levels, once for each query head and part of the tokens;
 * each level is taken within 2^-17 of itself.
 *   pool       as written by kvpool_encode, read only
 *   q, out     rows of n_agents x q_heads; q_heads a multiple of num_kv_heads
 *   tail       NULL: the pool alone
 *   dev_status device int32 or NULL; KVC_DEV_BAD_HEADER (nothing is written),
 *              KVC_DEV_BAD_PAGE, KVC_DEV_BAD_LENGTH
 * The other arguments, roundings and errors are those of kvpage_attend
 * (n_agents * q_heads < 2^23). */
int kvpool_attend(const kvc_shape* shape, const void* pool, size_t pool_bytes, uint32_t layer, uint32_t n_agents,
                  uint32_t q_heads, const kvc_rows* q, float scale, const kvc_tail* tail, const kvc_rows* out,
                  float* lse, void* ws, size_t ws_bytes, int32_t* dev_status, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVATTEND_H */
