/*
 * fvattn_cache.h -- a cache of keys and values in blocks ("pages"), and the
 * attention of one new token a sequence over it.
 *
 * A model that generates causally keeps the keys and values of the tokens so
 * far.  A page holds `page` consecutive tokens of one sequence for every key
 * head, and one head's part of it is a contiguous page x D tile, as a block of
 * the tiled layout of fvattn.h is.  A table row lists a sequence's pages in
 * order: token n is row n % page of page table[b][n / page].  Pages of a
 * sequence may lie anywhere in the pool, and several sequences may read the
 * same page (a shared prefix).
 *
 * Conventions are those of fvattn.h: device pointers owned by the caller, no
 * allocation, asynchronous on the stream, argument errors before any launch,
 * errors of a kernel in the status word that fvattn_get_status reads.
 */
#ifndef FVATTN_CACHE_H
#define FVATTN_CACHE_H

#include "fvattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int pages;        /* pages in the pool */
    int Hkv;          /* key heads */
    int D;            /* head dim, 64 or 128 */
    int page;         /* tokens a page: 16, 32, 64 or 128 */
    void *k, *v;      /* [pages, Hkv, page, D] bf16, 16-byte aligned */
} fvattn_cache;

/* Rotation by position, applied to keys and queries as they are written.
 * Pair i of a head (i < D/2) belongs to one of up to three position axes
 * (a text has one; a video has frame, row and column): the first pairs[0]
 * pairs to axis 0, the next pairs[1] to axis 1, and so on.  With
 * (c, s) = (table[n][i], table[n][D/2 + i]) and n the token's position on that
 * axis, (a, b) becomes (a c - b s, a s + b c) in fp32, rounded once to bf16.
 * Pair i is elements (2i, 2i + 1), or (i, D/2 + i) with halves = 1. */
typedef struct {
    const float *table;      /* [rows, D] fp32: D/2 cosines, then D/2 sines */
    int rows;                /* positions n in [0, rows) */
    int axes;                /* 1 to 3 */
    int pairs[3];            /* sum D/2 */
    const int32_t *pos;      /* [tokens, axes] positions of each token */
    int halves;
} fvattn_rotation;

/* Append new keys and values to the pages of B sequences.  Sequence b's new
 * tokens are rows cu[b] .. cu[b+1]-1 of k and v (cu NULL: row b alone), and
 * lens[b] is its length with them: its last new token is token lens[b] - 1.
 *   rows            rows of k, v, q; rows before cu[0] and from cu[B] on are
 *                   left alone (cu may be a slice of a larger batch's)
 *   k, v            [rows, Hkv, D] bf16, a row's heads contiguous, rows
 *                   k_stride and v_stride elements apart (multiples of 8)
 *   q, q_out        optional [rows, Hq, D] bf16 in and out, rows q_stride and
 *                   q_out_stride elements apart: the tokens' queries, rotated
 *                   likewise.  q_out may be q
 *   rot             NULL: keys (and queries) are copied as they are
 *   table, width    [B, width] int32 page numbers; entries past a sequence's
 *                   last page are not read
 * A position outside the table, a token outside [0, width * page) and a page
 * outside the pool set FVATTN_ERR_BOUNDS, and that token is not written,
 * neither to the pages nor to q_out.
 * Only the new tokens' rows of the pages change.  No two sequences may append
 * to one page.  Pointers 16-byte aligned (cu, lens, table and pos: 4). */
int fvattn_cache_append(const fvattn_cache *c, int B, long long rows, const int32_t *cu, const int32_t *lens,
                        const int32_t *table, int width,
                        const void *k, long long k_stride, const void *v, long long v_stride,
                        const void *q, long long q_stride, int Hq, void *q_out, long long q_out_stride,
                        const fvattn_rotation *rot, fvattn_stream_t stream);

/* fvattn_cache_append into a q_out that holds nothing yet: its rows that
 * fvattn_cache_append leaves alone (rows of no sequence, refused tokens) get
 * zero.  q is required, and q_out is not q. */
int fvattn_cache_append_fresh(const fvattn_cache *c, int B, long long rows, const int32_t *cu, const int32_t *lens,
                              const int32_t *table, int width,
                              const void *k, long long k_stride, const void *v, long long v_stride,
                              const void *q, long long q_stride, int Hq, void *q_out, long long q_out_stride,
                              const fvattn_rotation *rot, fvattn_stream_t stream);

/* Parts that fvattn_cache_attn splits a sequence's tokens into, for up to
 * `longest` tokens a sequence, and the tokens a part holds (a multiple of
 * 64).  They follow from the arguments and the number of SMs of the current
 * device (148 without one).  0 for bad arguments. */
int fvattn_cache_attn_parts(int B, int Hq, int Hkv, int D, long long longest, int *tokens);

/* Bytes of device workspace fvattn_cache_attn needs (0 when it does not
 * split): per query head and part D + 2 fp32.  Asked for with the call's
 * device current: another GPU may split otherwise, and a workspace sized for
 * it be refused. */
size_t fvattn_cache_attn_workspace_size(int B, int Hq, int Hkv, int D, long long longest);

/* Attention of one query a sequence over its cached tokens: for each head j
 *   O_bj = softmax_n(scale * q_bj . k_n) v_n,  lse_bj = ln sum_n exp(scale * q_bj . k_n)
 * over tokens n < lens[b] of key head j / (Hq / Hkv).  A sequence of length 0
 * gets O = 0, lse = -inf.  fp32 softmax and sums; P is rounded to bf16 for the
 * product.  Rows of a page at and after lens[b] may hold anything.  A table
 * that lists only some of a sequence's pages (lens[b] then counts the tokens
 * listed, and only the last page may be part filled) attends to those.
 *   q        [B, Hq, D] bf16, rows q_stride elements apart (a multiple of 8)
 *   longest  no sequence is longer (a host number: it sets the split)
 *   o        [B, Hq, D] bf16, contiguous; lse [B, Hq] fp32, may be NULL
 *   workspace  256-byte aligned; may be NULL when its size is 0
 * A length outside [0, min(longest, width * page)] or a page outside the pool
 * sets FVATTN_ERR_BOUNDS; the length is clamped, and page 0 is read in the
 * page's place.  The bits of a sequence's result follow from its own tokens
 * and the split, not from other sequences' lengths. */
int fvattn_cache_attn(const fvattn_cache *c, int B, int Hq, const void *q, long long q_stride,
                      const int32_t *table, int width, const int32_t *lens, long long longest, float scale,
                      void *o, float *lse, void *workspace, size_t ws_bytes, fvattn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FVATTN_CACHE_H */
