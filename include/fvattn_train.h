/*
 * fvattn_train.h -- gradients of the block-sparse attention of fvattn.h.
 *
 * Training through fvattn_sparse_attn needs two calls: a forward that keeps
 * each row's log-sum-exp, and a backward that computes the probabilities
 * again from it.  Layouts, ownership, streams, workspaces and errors are
 * those of fvattn.h.  The kv lists are constants of the call: no gradient
 * flows into routing.  The gradient of fvattn_reorder is
 * fvattn_inverse_reorder and the other way round.
 */
#ifndef FVATTN_TRAIN_H
#define FVATTN_TRAIN_H

#include "fvattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* fvattn_sparse_attn that also returns the log-sum-exp of each row's scores,
 *   lse_t = ln sum_u exp(scale * q_t . k_u)
 * over the real tokens u of the row's kept blocks.  O has the bits that
 * fvattn_sparse_attn writes.
 *   lse      [B, H, Npad] fp32 output (all rows written)
 *   kv_cnt   may be 0 here: such a row keeps no block, O = 0, lse = -inf
 * Other arguments, workspace size and errors as fvattn_sparse_attn. */
int fvattn_sparse_attn_lse(const fvattn_geom *g, const void *q_t, const void *k_t, const void *v_t,
                           const int32_t *kv_idx, const int32_t *kv_cnt, float scale,
                           void *o_t, float *lse, unsigned long long *sm_stats,
                           void *workspace, size_t ws_bytes, fvattn_stream_t stream);

/* Bytes of device workspace fvattn_sparse_attn_bwd needs: row statistics
 * (9 bytes a row), the block mask as bits, its lists by query tile and by
 * key tile (4 bytes per list slot: 2 x 70 MB for 40 heads at nb = 660) and
 * the work order.  0 for a null pointer. */
size_t fvattn_sparse_attn_bwd_workspace_size(const fvattn_geom *g);

/* Gradients of fvattn_sparse_attn_lse with respect to Q, K and V.  With
 * P_tu = exp(scale * q_t . k_u - lse_t) on the kept real keys (0 elsewhere):
 *   dV_u = sum_t P_tu dO_t
 *   dS_tu = P_tu (dO_t . v_u - sum_w P_tw dO_t . v_w)
 *   dQ_t = scale * sum_u dS_tu k_u,   dK_u = scale * sum_t dS_tu q_t
 * The products run on the tensor cores in bf16 with fp32 accumulation (P and
 * dS are rounded to bf16 as operands); statistics and sums are fp32.  The
 * sum in dS is dO_t . O_t in exact arithmetic; it is formed from P where the
 * bf16 O is too coarse for it.  No atomics touch a result: the output bits
 * depend only on the inputs, not on the schedule nor on how heads are split
 * across calls.  K and V of blocks that no list holds change no bit of them,
 * whatever they hold.  A NaN or infinity in a block reaches the rows and keys
 * paired with it and, with blocks below 128 tokens, those of the other blocks
 * in the same 128 rows (as in fvattn_sparse_attn).
 *   q_t, k_t, v_t, do_t  [B, H, Npad, D] bf16 from fvattn_reorder (padding
 *                        rows zero)
 *   o_t, lse             as fvattn_sparse_attn_lse wrote them for the same
 *                        q_t, k_t, v_t, lists and scale
 *   kv_idx, kv_cnt       the forward's lists (cnt in [0, nb], distinct
 *                        indices).  A count or index out of range, or an
 *                        index listed twice in a row, sets
 *                        FVATTN_ERR_BOUNDS in the status word; it is
 *                        clamped, skipped or taken once
 *   dq_t, dk_t, dv_t     [B, H, Npad, D] bf16 outputs (all rows written;
 *                        padding rows, rows that keep no block and keys
 *                        that no row keeps get zero)
 *   workspace            >= fvattn_sparse_attn_bwd_workspace_size bytes,
 *                        256-byte aligned; rewritten by every call
 * Outputs must not overlap inputs or one another.  scale finite and > 0.
 * Status: fvattn_get_status. */
int fvattn_sparse_attn_bwd(const fvattn_geom *g, const void *q_t, const void *k_t, const void *v_t,
                           const void *o_t, const void *do_t, const float *lse,
                           const int32_t *kv_idx, const int32_t *kv_cnt, float scale,
                           void *dq_t, void *dk_t, void *dv_t,
                           void *workspace, size_t ws_bytes, fvattn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FVATTN_TRAIN_H */
