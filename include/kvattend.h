/*
 * kvattend.h - operators that use a cache while an agent generates, AMD
 * Instinct MI355X (gfx950). Same library, conventions and error codes as
 * kvcodec.h (libkvcodec.so, C ABI):
 *
 *  - kvc_norm_rotate: norms of queries and keys for each head and the position
 *    rotation, in one pass over the projection's rows;
 *  - kvpage_write, kvpage_read: a paged cache of one layer, quantised as it is
 *    written, and read back;
 *  - kvpage_append: norms, rotation and the write of the new keys and values in one;
 *  - kvpage_attend: attention of one new token per sequence over its pages;
 *  - kvpage_attend_window: the same with a sliding window and sinks;
 *  - kvpage_attend_prompt: attention of many new tokens of each sequence;
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
#define KVC_PAGE_FP4 4u  /* e2m1 codes, one power of two for each 32 channels (OCP microscaling) */

/* Further bits of *dev_status. */
enum {
    KVC_DEV_BAD_SLOT = 16,  /* a slot is not below num_pages * page_tokens */
    KVC_DEV_BAD_PAGE = 32,  /* a page number of a table is not a page */
    KVC_DEV_BAD_LENGTH = 64, /* a length is negative or longer than its table's row */
    KVC_DEV_BAD_START = 128  /* first rows of sequences fall, or leave the rows given */
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
 * kv_heads may be 0 (then k_in, k_out, k_weight are not used), and so may q_heads.
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
 *          int8, e4m3, or e2m1: two to a byte, the even channel in its low half)
 *   steps  f32 [2][num_kv_heads][page_tokens]        (8-bit formats), or bytes
 *          [2][num_kv_heads][page_tokens][head_dim / 32] (e2m1): byte s stands for
 *          2^(s - 127), 255 for NaN */
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
 * KVC_PAGE_FP4, for each 32 channels: with m = max |x| and 2^a <= m < 2^(a+1), the
 * power is 2^(a-2), or 2^(a-1) if m > 1.75 * 2^a, held to 2^-125 .. 2^125; code =
 * x / power rounded to nearest, ties to even, and cut off at 6. m = 0 gives codes 0;
 * channels that hold an Inf or NaN get the power 255 and codes 0: all 32 read
 * back as NaN.
 *   dev_status  device int32 or NULL; KVC_DEV_BAD_SLOT (that token is not written)
 * Errors: KVC_E_NULL, KVC_E_SHAPE, KVC_E_SIZE, KVC_E_ALIGN, KVC_E_ALIAS,
 * KVC_E_HIP. */
int kvpage_write(const kvc_pages* spec, void* pages, size_t pages_bytes, uint32_t n_tokens, const kvc_rows* k,
                 const kvc_rows* v, const int64_t* slots, int32_t* dev_status, hipStream_t stream);

/* Read tokens back: bf16(code * step), one rounding (none for KVC_PAGE_FP4). Rows of negative slots,
 * and of slots outside the cache (KVC_DEV_BAD_SLOT), are left as they were.
 * Errors as kvpage_write. */
int kvpage_read(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_tokens,
                const int64_t* slots, const kvc_rows* k_out, const kvc_rows* v_out, int32_t* dev_status,
                hipStream_t stream);

/* Norms, rotation and the write in one pass over the projection's rows:
 * kvc_norm_rotate of q and k, and kvpage_write of the keys it gives (rounded to
 * bf16, but not kept) and of v. The bytes of q_out and of the pages are those of the
 * two calls.
 *   q_in, k_in, v_in  rows of n_tokens x q_heads and twice n_tokens x num_kv_heads;
 *                  n_tokens <= 2^26 - 4. q_heads may be 0 (q_in, q_out, q_weight are not used)
 *   q_out          rows; the same as q_in turns in place
 *   slots          as for kvpage_write; a token with a negative slot (padding) or one
 *                  outside the cache has its queries turned all the same
 * The other arguments, roundings and errors are those of the two calls. */
int kvpage_append(const kvc_pages* spec, void* pages, size_t pages_bytes, uint32_t n_tokens, uint32_t q_heads,
                  const kvc_rows* q_in, const kvc_rows* k_in, const kvc_rows* v_in, const void* q_weight,
                  const void* k_weight, float eps, const int64_t* positions, const float* inv_freq, uint32_t n_pairs,
                  uint32_t pairing, const int64_t* slots, const kvc_rows* q_out, int32_t* dev_status,
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
 * by a power of two (about the largest step) for the matrix cores, bf16's and
 * KVC_PAGE_FP4's are split into two bf16 terms; products and sums are binary32. Of a weight times its
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

/* Workspace bytes of kvpage_attend_window; never less for more sequences, tokens,
 * window or sinks. 0 if an argument is invalid. */
size_t kvpage_attend_window_workspace_bytes(const kvc_pages* spec, uint32_t n_seqs, uint32_t q_heads,
                                            uint32_t max_tokens, uint32_t window, uint32_t sinks);

/* kvpage_attend of a new token that sees the last `window` tokens of its sequence
 * (itself among them) and the first `sinks`: token t counts if t < sinks or
 * t >= lens[b] - window. window 0: every token counts, whatever sinks is.
 * Tokens in between are not used, whatever their pages hold, and table entries of
 * pages without a token that counts may hold anything.
 *   ws         kvpage_attend_window_workspace_bytes(spec, n_seqs, q_heads,
 *              table_cols * page_tokens, window, sinks) bytes or more
 * The other arguments, roundings and errors are those of kvpage_attend. */
int kvpage_attend_window(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_seqs,
                         uint32_t q_heads, const kvc_rows* q, const int32_t* table, uint32_t table_cols,
                         uint64_t table_stride, const int32_t* lens, uint32_t window, uint32_t sinks, float scale,
                         const kvc_rows* out, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                         hipStream_t stream);

/* Workspace bytes of kvpage_attend_prompt for at most n_seqs sequences with at most
 * n_tokens new tokens together, of at most max_tokens tokens each; never less for
 * more of any. 0 if an argument is invalid. */
size_t kvpage_attend_prompt_workspace_bytes(const kvc_pages* spec, uint32_t n_seqs, uint32_t n_tokens,
                                            uint32_t q_heads, uint32_t max_tokens, uint32_t window, uint32_t sinks);

/* Attention of the new tokens of each of n_seqs sequences over its pages, which
 * hold the new tokens' keys and values already (kvpage_append): a prompt, a part of one
 * behind a context, or drafted tokens. Sequence b has the rows starts[b] to
 * starts[b + 1] - 1, which are the last of its lens[b] tokens; row i of m stands at
 * position p = lens[b] - m + i and sees the tokens t <= p, with a window those
 * with t < sinks or t > p - window. window 0: all of them. A row that sees no token (m >
 * lens[b]) gives zeros and lse = -inf. Rows before starts[0] and from
 * starts[n_seqs] on are left as they were. Table entries of pages without a token that
 * a row sees may hold anything.
 *   q, out     rows of n_tokens x q_heads (out elsewhere than q)
 *   starts     device int32 [n_seqs + 1], rising, from 0 to n_tokens at most
 *   lse        device f32 [n_tokens][q_heads] or NULL
 *   ws         kvpage_attend_prompt_workspace_bytes(spec, n_seqs, n_tokens, q_heads,
 *              table_cols * page_tokens, window, sinks) bytes or more
 *   dev_status besides those of kvpage_attend KVC_DEV_BAD_START (outputs are then
 *              unspecified)
 * n_tokens * q_heads < 2^30 and, with g = q_heads / num_kv_heads, num_kv_heads *
 * (n_tokens * g / 64 + n_seqs) < 2^23; n_seqs < 2^20; table_cols * page_tokens < 2^31.
 * The same call gives the same bits. Weights are rounded once, to bf16 (2^-8; bf16 and
 * KVC_PAGE_FP4 pages) or, times the step, to binary16 (2^-11; 8-bit formats): a row sums
 * over many tokens, and the rounding errors do not add up as the weights do. (Calls with
 * few new tokens of each sequence in the mean run as kvpage_attend does, with its
 * roundings: a sequence's bits may differ with the others of its call.) The
 * softmax's sums are those of the weights before that. Products and sums are
 * binary32. Logits in powers of two (scale * q . k * log2 e) have to stay below 2^24 in
 * size, 8-bit key steps that are not 0 between 2^-90 and 2^90. A NaN in a key or value,
 * or an Inf in a value, makes rows that see its token NaN or Inf (of a value: in its
 * channel; in its whole vector or 32 channels where they share a step), and no others.
 * The other arguments and errors are those of kvpage_attend. */
int kvpage_attend_prompt(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_seqs,
                         uint32_t n_tokens, uint32_t q_heads, const kvc_rows* q, const int32_t* starts,
                         const int32_t* table, uint32_t table_cols, uint64_t table_stride, const int32_t* lens,
                         uint32_t window, uint32_t sinks, float scale, const kvc_rows* out, float* lse, void* ws,
                         size_t ws_bytes, int32_t* dev_status, hipStream_t stream);

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
