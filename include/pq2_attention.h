/*
 * pq2_attention.h -- C ABI of what a decoder needs between its QKV projection
 * and its output projection: the rotary embedding, a paged INT8 key-value
 * cache, attention of new tokens over its pages, and attention over packed
 * prompts.  Part of libpq2.so; the conventions, status codes and element
 * types are those of pq2.h (device pointers on the current device,
 * caller-owned buffers, everything checked on the host before any HIP call,
 * work enqueued on `stream`, nothing allocated, nothing kept after the call).
 *
 * Tensors of heads are [rows][heads][head_dim] with a row stride and a head
 * stride in elements, head_dim elements contiguous: columns of a projection's
 * output, or any other layout whose rows do not meet.  Their pointers are
 * 16-byte aligned and their strides multiples of 16 bytes.  Query head h reads
 * key-value head h / (heads / kv_heads).
 *
 * Index arrays (positions, slots, tables, lengths, starts) are int32 in
 * device memory; their values cannot be checked on the host.  The kernels
 * check every one that becomes an address: what each entry point does with a
 * value out of range is stated there, and none reads or writes outside the
 * buffers given.
 *
 * Attention takes finite queries, keys and values: a NaN or infinity among a
 * sequence's own tokens may reach other rows of that sequence, also rows whose mask
 * hides it; other sequences, and what lies behind a sequence's end, have no
 * influence.  Scores, and sums of weights (up to 2^8, of prompts in fp16 2^15) times
 * values, are FP32 before they are normalised: q . k, scale * q . k and 2^40 times
 * the largest value stay within its range; products of weights and values below 2^-100
 * lose bits.
 */
#ifndef PQ2_ATTENTION_H
#define PQ2_ATTENTION_H

#include "pq2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (inclusive) of the entry points below. */
#define PQ2_MAX_ATTN_ROWS (1 << 24)      /* rows (tokens) of a tensor of heads   */
#define PQ2_MAX_ATTN_HEADS 1024          /* query heads; kv_heads <= heads       */
#define PQ2_MAX_ATTN_SEQS 65535          /* sequences of one call                */

/* ---- The cache
 *
 * Pages of page_tokens = 16, 32, 64, 128 or 256 tokens; head_dim = 64, 128 or
 * 256.  Page p holds, for each key-value head h, the block at
 * (p * kv_heads + h) * page_tokens * (2 * head_dim + 8):
 *  - int8 key codes [page_tokens][head_dim], then int8 value codes of the same
 *    shape, then float key scales [page_tokens], float value scales
 *    [page_tokens].
 * A code c with scale s stands for c * s.  Slot i of the cache is token
 * i % page_tokens of page i / page_tokens.  Codes and scale of a row x of
 * head_dim elements are those of pq2_quantize_act_i8 with the row as its
 * group: s = max|x| / 127, c = clamp(rint(x / s), +-127).
 *
 * Bytes of one page; -1 if page_tokens or head_dim is none of the above, or
 * kv_heads < 1 or > PQ2_MAX_ATTN_HEADS. */
int64_t pq2_kv_page_bytes(int64_t page_tokens, int64_t kv_heads, int64_t head_dim);

/* Rotary embedding of q and k, and the codes of k and v into the cache, in one
 * launch.  Row t is rotated by row p = positions[t] of the tables, over the
 * first rot_dim elements of each head, pair (a, b) being elements i and
 * i + rot_dim/2 (interleaved 0) or 2i and 2i + 1 (interleaved 1):
 *
 *   a' = a cos[p][i] - b sin[p][i]      b' = b cos[p][i] + a sin[p][i]
 *
 * each product and sum one FP32 operation.  k's codes are those of the FP32
 * results, v's those of v; q_out, k_out and v_out are rounded once.
 *  - A position out of the tables takes the nearest row.
 *  - A slot outside the cache (a padded token's -1) is not written; the row's
 *    other outputs are.
 *  - Slots of one call are distinct: of rows with the same slot, the slot may
 *    hold parts of each. */
typedef struct pq2_kv_write_args {
    const void* q;            /* [m][heads][head_dim] of in_dtype; NULL: none (and q_out NULL)   */
    const void* k;            /* [m][kv_heads][head_dim]                                         */
    const void* v;
    int64_t q_stride, q_head, k_stride, k_head, v_stride, v_head;
    void* q_out;              /* rotated q, of out_dtype; may be q itself (pointer, strides, type) */
    void* k_out;              /* rotated k, of out_dtype; may be k itself; NULL: none            */
    void* v_out;              /* v in out_dtype; NULL: none                                      */
    int64_t qo_stride, qo_head, ko_stride, ko_head, vo_stride, vo_head;
    const float* cos;         /* [table_rows][rot_dim / 2], 16-byte aligned; read if rot_dim > 0 */
    const float* sin;
    const int32_t* positions; /* [m]; read if rot_dim > 0                                        */
    const int32_t* slots;     /* [m]; read if cache is given                                     */
    void* cache;              /* pages * pq2_kv_page_bytes bytes, 16-byte aligned; NULL: none    */
    int64_t m, heads, kv_heads, head_dim;
    int64_t rot_dim;          /* 0 (no rotation) or a multiple of 8 up to head_dim               */
    int64_t table_rows, pages, page_tokens;
    int in_dtype;             /* PQ2_BF16 / PQ2_F16 / PQ2_F32                                    */
    int out_dtype;            /* PQ2_BF16 / PQ2_F16 / PQ2_F32                                    */
    int interleaved;          /* 0 or 1                                                          */
} pq2_kv_write_args;

/* Errors: EINVAL (null args, k, v, or tables, positions or slots that are read; no output;
 *         q without q_out or q_out without q; dtype; interleaved; overlap), ESHAPE (m, heads, kv_heads, head_dim,
 *         page_tokens, rot_dim, a stride; pages < 1 or pages * page_tokens > 2^31; table_rows < 1 or > 2^31 - 1),
 *         EALIGN, ELAUNCH, EDEVICE. */
int pq2_kv_write(const pq2_kv_write_args* args, void* stream);

/* Tokens out of the cache again: row starts[s] + t of k_out and v_out is token t of
 * sequence s, code * scale rounded once to out_dtype.  Sequence s has
 * starts[s + 1] - starts[s] tokens; its token t is token t % page_tokens of page
 * table[s][t / page_tokens].
 *  - starts[0] is 0 and starts never falls.  Rows from starts[seqs] on are left as
 *    they were.
 *  - A row whose page is outside the cache, or beyond the table, is zero. */
typedef struct pq2_kv_read_args {
    const void* cache;
    const int32_t* table;     /* [seqs][table_stride], table_pages of each row used              */
    const int32_t* starts;    /* [seqs + 1]                                                      */
    void* k_out;              /* [rows][kv_heads][head_dim] of out_dtype                         */
    void* v_out;
    int64_t ko_stride, ko_head, vo_stride, vo_head;
    int64_t rows, seqs, table_stride, table_pages, kv_heads, head_dim, pages, page_tokens;
    int out_dtype;
} pq2_kv_read_args;

/* Errors: EINVAL (null, dtype, overlap), ESHAPE, EALIGN, ELAUNCH, EDEVICE. */
int pq2_kv_read(const pq2_kv_read_args* args, void* stream);

/* ---- Attention of new tokens over the cache
 *
 * Sequence s has lens[s] tokens in the cache, its new ones among them (written
 * by pq2_kv_write before), and n = starts[s + 1] - starts[s] <= max_new new
 * ones: row starts[s] + i of q is the token at position p = lens[s] - n + i, and
 *
 *   out = sum_j w_j v_j,  w = softmax_j(scale * q . k_j)  over the keys j <= p,
 *                                               and j > p - window if window > 0
 *
 * with k_j and v_j as their codes and scales give them.  Sums and the softmax
 * are FP32, weights meet values with 16 bits, elements of q below 2^-14 of their row's
 * largest are rounded to multiples of 2^-24 of it; out is rounded once.  A row's bits depend on its
 * sequence's length and the call's sizes, not on the other sequences.
 *  - A row that sees no key is zero.
 *  - Keys in pages outside the cache are not seen, nor those beyond the table.
 *  - What the pages hold behind a sequence's length has no influence.
 *  - Rows of q that belong to no sequence are left as they were in out.
 * The cache is split over its length where the sequences alone would leave
 * compute units idle; the last workgroup of a row joins the parts in order.
 *
 * Workspace: `partials` (floats) and `counters` (32-bit words, zero before the
 * first call, zero again after each call), of the sizes that
 * pq2_attention_paged_workspace gives for the same seqs, max_new, heads,
 * kv_heads, head_dim and max_len.  Calls (and captured graphs) that share a
 * workspace are ordered by the caller. */
typedef struct pq2_attention_paged_args {
    const void* q;            /* [rows][heads][head_dim] of dtype                                */
    void* out;                /* the same; not q itself                                          */
    int64_t q_stride, q_head, out_stride, out_head;
    const void* cache;
    const int32_t* table;     /* [seqs][table_stride], table_pages of each row used              */
    const int32_t* lens;      /* [seqs]                                                          */
    const int32_t* starts;    /* [seqs + 1]; NULL: one new token each, row s of q (rows = seqs)  */
    float* partials;          /* 16-byte aligned; NULL if the size is 0                          */
    uint32_t* counters;
    int64_t rows, seqs, table_stride, table_pages, heads, kv_heads, head_dim, pages, page_tokens;
    int64_t max_new;          /* most new tokens of a sequence: later ones are not computed      */
    int64_t max_len;          /* longest length expected; a longer one is computed, more slowly  */
    int64_t window;           /* keys that a token sees, itself among them; 0: all               */
    float scale;              /* > 0; finite, also times log2(e)                                   */
    int dtype;                /* PQ2_BF16 or PQ2_F16                                             */
} pq2_attention_paged_args;

/* Sizes of the workspace: floats of `partials` into *partials, words of
 * `counters` into *counters (both 0 where nothing is split).
 * Errors: EINVAL (null), ESHAPE. */
int pq2_attention_paged_workspace(int64_t seqs, int64_t max_new, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                  int64_t max_len, int64_t* partials, int64_t* counters);

/* Errors: EINVAL (null, dtype, scale, window < 0, overlap), ESHAPE (sizes; heads % kv_heads; rows != seqs without
 *         starts; more than 2^23 tiles of 16 query rows: seqs * kv_heads * ceil(max_new * heads / kv_heads / 16)), EALIGN, ELAUNCH, EDEVICE. */
int pq2_attention_paged(const pq2_attention_paged_args* args, void* stream);

/* ---- Attention over packed prompts
 *
 * Sequence s has queries at rows starts_q[s] .. starts_q[s + 1] - 1 of q and out
 * and keys and values at rows starts_k[s] .. starts_k[s + 1] - 1 of k and v, nq
 * and nk of them (nk > nq behind a prefix; either may be 0).  Query i is at
 * position p = nk - nq + i among the keys:
 *
 *   out = sum_j w_j v_j,  w = softmax_j(scale * q . k_j)  over all keys j of the sequence,
 *                  with causal over j <= p, with window > 0 (causal only) also j > p - window
 *
 * Scores, softmax and sums are FP32; the weights are rounded to dtype before
 * they meet the values, as matrix cores take them (an fp16 weight below 2^-21 of its
 * row's largest to a multiple of 2^-31 of that), and normalised by the sum
 * of the rounded ones; out is rounded once.
 *  - A row that sees no key is zero.  Rows of other sequences have no influence.
 *  - starts begin at 0 and never fall; rows of q behind the last sequence are left as
 *    they were in out. */
typedef struct pq2_attention_prompt_args {
    const void* q;            /* [rows_q][heads][head_dim] of dtype                              */
    const void* k;            /* [rows_k][kv_heads][head_dim]                                    */
    const void* v;
    void* out;                /* as q; not q itself                                              */
    int64_t q_stride, q_head, k_stride, k_head, v_stride, v_head, out_stride, out_head;
    const int32_t* starts_q;  /* [seqs + 1]                                                      */
    const int32_t* starts_k;  /* [seqs + 1]                                                      */
    int64_t rows_q, rows_k, seqs, heads, kv_heads, head_dim;
    int64_t window;
    float scale;              /* > 0; finite, also times log2(e)                                   */
    int dtype;                /* PQ2_BF16 or PQ2_F16                                             */
    int causal;               /* 0 or 1                                                          */
} pq2_attention_prompt_args;

/* Errors: EINVAL (null, dtype, causal, scale, window < 0 or without causal, overlap), ESHAPE (sizes; rows_q * heads /
 *         kv_heads > 2^30), EALIGN, ELAUNCH, EDEVICE. */
int pq2_attention_prompt(const pq2_attention_prompt_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PQ2_ATTENTION_H */
