/*
 * bakron_moe.h -- the expert layer for any number of tokens, forward and
 * backward, on the packed 4-bit experts of bakron_q4.h (MI355X, gfx950):
 *
 *   bakron_moe_route         chooses top_k experts per token and sorts the
 *                            choices by expert;
 *   bakron_moe_gather        brings tokens' rows into that order;
 *   bakron_q4_experts        multiplies each expert's rows by its layer;
 *   bakron_gated_act         act(a) b between the products, a and b kept in 8
 *                            bits where a backward pass will want them;
 *   bakron_moe_combine       brings rows back to their tokens, weighted;
 *   *_grad                   the gradients of all of these (bakron_moe_gather's
 *                            is bakron_moe_combine without weights).
 *
 * (bakron_q4_moe is the whole layer in one call for up to 64 tokens, without
 * gradients.)
 *
 * Conventions are those of bakron_q4.h: device pointers owned by the caller,
 * work enqueued on `stream` in order (no library streams, no allocation, no
 * synchronisation: every call can be captured into a HIP graph), workspaces
 * undefined after a call, return codes BAKRON_*, nothing enqueued on an error,
 * inputs and outputs do not overlap.  Values are BAKRON_Q4_BF16 or
 * BAKRON_Q4_FP16, row r starting at element r * ld, 2-byte aligned (16-byte
 * aligned rows are moved fastest); sums are float32, rounded once to that type;
 * the same call on the same inputs always gives the same bits.
 *
 * A choice is the pair (t, j): token t's j-th expert, number t top_k + j.
 * Choices are sorted by expert and, within an expert, by number; choice
 * (t, j) is sorted row place[t, j], and expert e has the sorted rows
 * offsets[e] .. offsets[e + 1] - 1.  A token may make fewer than top_k
 * choices (logits of -infinity or NaN are never chosen): the choices that it
 * does not make have place -1 and come to no row, so that offsets[experts],
 * the number of sorted rows in use, may be below tokens top_k.  How many
 * there are is known on the device only; buffers of sorted rows have room for
 * tokens top_k, and rows from offsets[experts] on are not written by any call.
 * Entries of place outside [0, rows) are no row.  Offsets are taken as lying in
 * [0, rows]; where they decrease (bakron_moe_route's never do) an expert has no
 * rows, and which of the others' rows are written is not specified.  Neither
 * causes an access out of bounds.  Two choices with one place are two tokens
 * writing one row, which ends as some mixture of both.
 */
#ifndef BAKRON_MOE_H
#define BAKRON_MOE_H

#include "bakron_q4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A third type, of logits and unpacked checkpoints (beside BAKRON_Q4_BF16 and
 * BAKRON_Q4_FP16). */
#define BAKRON_MOE_F32 2

/* Activations of bakron_gated_act. */
#define BAKRON_MOE_SILU 0  /* act(v) = v sigmoid(v) */
#define BAKRON_MOE_GELU 1  /* act(v) = v sigmoid(2 sqrt(2 / pi) (v + 0.044715 v^3)), the tanh form */
/* (a sigmoid below 2^-126, of arguments under -87.3, counts as 0) */

#define BAKRON_MOE_MAX_ROWS 16777216   /* tokens, and tokens top_k, of one call */
#define BAKRON_MOE_MAX_TOP_K 16        /* experts chosen per token */
#define BAKRON_MOE_MAX_PLACES 32       /* rows per token that bakron_moe_gather and _combine take */
#define BAKRON_MOE_MAX_EXPERTS 256

/* Workspace bytes of bakron_moe_route (0 when it needs none or an argument is
 * outside its limits).  Host only. */
size_t bakron_moe_route_workspace_bytes(int64_t tokens, int64_t experts, int32_t top_k);

/*
 * bakron_moe_route -- the choice of experts, their shares, and the sorted
 * order.
 *
 * logits     [in]  tokens x experts of BAKRON_MOE_F32, BAKRON_Q4_BF16 or
 *                  BAKRON_Q4_FP16 (row stride ld, aligned to the type).
 * experts, top_k [in] 1 <= top_k <= min(experts, BAKRON_MOE_MAX_TOP_K),
 *                  experts <= BAKRON_MOE_MAX_EXPERTS (BAKRON_ERR_BAD_ARG
 *                  otherwise); tokens and tokens top_k up to
 *                  BAKRON_MOE_MAX_ROWS (BAKRON_ERR_BAD_SIZE).
 * ids        [out] tokens x top_k int32: the experts of largest logit, largest
 *                  first, equal ones in the order of their index; -1 where
 *                  only -infinity and NaN are left.
 * weights    [out] tokens x top_k floats: the softmax of the chosen logits
 *                  (of logits of +infinity, equal shares); 0 where ids is -1.
 * place      [out] tokens x top_k int32: the sorted row, -1 where ids is -1.
 * order      [out] tokens top_k int32: the choice at each sorted row, -1 from
 *                  offsets[experts] on.
 * offsets    [out] experts + 1 int32.
 * tokens == 0 writes offsets (zeros) only.
 */
int bakron_moe_route(const void* logits, int64_t ld, int64_t tokens, int32_t type, int64_t experts, int32_t top_k,
                     int32_t* ids, float* weights, int32_t* place, int32_t* order, int32_t* offsets, void* workspace,
                     size_t workspace_bytes, hipStream_t stream);

/*
 * bakron_moe_route_grad -- the gradient of the shares with respect to the
 * logits: with w and g the weights and dweights of token t,
 *     dlogits[t, ids[t, j]] = w_j (g_j - sum_i w_i g_i),   0 for every other expert,
 * sums over the choices that were made (g is not looked at where ids is -1).
 *
 * dweights, weights, ids [in] tokens x top_k, as bakron_moe_route left them.
 * dlogits    [out] tokens x experts of `type`, row stride ld.
 */
int bakron_moe_route_grad(const float* dweights, const float* weights, const int32_t* ids, int64_t tokens,
                          int64_t experts, int32_t top_k, void* dlogits, int64_t ld, int32_t type, hipStream_t stream);

/*
 * bakron_moe_gather -- rows into the sorted order: xs[place[t, j]] = x[t].
 *
 * x          [in]  tokens x cols, row stride ldx.
 * place      [in]  tokens x top_k int32, 1 <= top_k <= BAKRON_MOE_MAX_PLACES.
 * xs         [out] rows x cols, row stride ldxs; rows that no place names
 *                  stay as they are.
 * cols up to BAKRON_MAX_DIM, tokens up to BAKRON_MOE_MAX_ROWS, rows up to twice
 * that (two sorted buffers, whose rows one token's places may name).
 */
int bakron_moe_gather(const void* x, int64_t ldx, int64_t tokens, int32_t type, int64_t cols, int32_t top_k,
                      const int32_t* place, void* xs, int64_t ldxs, int64_t rows, hipStream_t stream);

/*
 * bakron_moe_combine -- sorted rows back to their tokens:
 *     y[t] = sum_j weights[t, j] ys[place[t, j]],
 * over the choices that have a row, in the order of j (no choice: zeros).
 * weights may be null: every weight is 1.
 */
int bakron_moe_combine(const void* ys, int64_t ldys, int64_t rows, int32_t type, int64_t cols, int32_t top_k,
                       const int32_t* place, const float* weights, int64_t tokens, void* y, int64_t ldy,
                       hipStream_t stream);

/*
 * bakron_moe_combine_grad -- bakron_moe_combine's gradients:
 *     dys[place[t, j]] = weights[t, j] dy[t],   dweights[t, j] = sum_c dy[t, c] ys[place[t, j], c]
 * (0 where the choice has no row).  Rows of dys that no place names stay as
 * they are.  cols == 0 writes zeros to dweights.
 */
int bakron_moe_combine_grad(const void* dy, int64_t lddy, const void* ys, int64_t ldys, int64_t rows, int32_t type,
                            int64_t cols, int32_t top_k, const int32_t* place, const float* weights, int64_t tokens,
                            void* dys, int64_t lddys, float* dweights, hipStream_t stream);

/* Workspace bytes of bakron_q4_experts and of its gradient (0 when none is
 * needed or an argument is outside the limits).  Host only. */
size_t bakron_q4_experts_workspace_bytes(int64_t rows, int64_t experts, int64_t m, int64_t n, int64_t group_size);
size_t bakron_q4_experts_grad_workspace_bytes(int64_t rows, int64_t experts, int64_t m, int64_t n, int64_t group_size);

/*
 * bakron_q4_experts -- each expert's rows times its layer:
 *     y[p] = W_e x[p],   offsets[e] <= p < offsets[e + 1].
 * Precision and range are those of bakron_q4_linear.
 *
 * x          [in]  rows x n, row stride ldx; rows from offsets[experts] on
 *                  may hold anything.
 * rows       [in]  0 <= rows <= BAKRON_MOE_MAX_ROWS: the room that x and y
 *                  have.  The kernel and its tiles are chosen for rows / experts
 *                  rows per expert; any distribution is served, but at the
 *                  price of that form (few rows on average: an expert's
 *                  codes are read again for every 32 of its rows).
 * packed, experts, m, n, group_size [in] a stack packed by bakron_q4_pack,
 *                  1 <= experts <= BAKRON_MOE_MAX_EXPERTS.
 * offsets    [in]  experts + 1 int32 on the device.
 * y          [out] rows x m, row stride ldy; rows from offsets[experts] on
 *                  stay as they are.  n == 0 writes zeros.
 */
int bakron_q4_experts(const void* x, int64_t ldx, int64_t rows, int32_t type, const void* packed, int64_t experts,
                      int64_t m, int64_t n, int64_t group_size, const int32_t* offsets, void* y, int64_t ldy,
                      void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * bakron_q4_experts_grad -- the gradient of bakron_q4_experts with respect to
 * its rows, dx[p] = dy[p] W_e.  Experts with many rows: each weight is rounded
 * once to dy's type, as bakron_q4_linear_grad does it, so that a result is off by
 * two roundings of its type instead of one (1.41 times in the mean square).  With
 * few: dy times a step is rounded to 16 bits (2^-16 relative), and the codes are
 * exact.  Which of the two it is goes by rows, experts and the layer's size.
 *
 * dy         [in]  rows x m; dx [out] rows x n.  m == 0 writes zeros.
 *                  Everything else as in bakron_q4_experts.
 */
int bakron_q4_experts_grad(const void* dy, int64_t lddy, int64_t rows, int32_t type, const void* packed,
                           int64_t experts, int64_t m, int64_t n, int64_t group_size, const int32_t* offsets, void* dx,
                           int64_t lddx, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Checkpoints: rows x cols values in 8 bits.  Each row's blocks of 32 columns
 * (the last one cut) have a step of their own, a power of two: the smallest
 * 2^s, s >= -126, with which the block's largest |v| / 2^s rounds to 127 at
 * most.  A value is kept as round(v / 2^s), ties to even, and stands for that
 * times 2^s: off by half a step at most, 1 / 127 of the block's largest
 * value (2^-127 where that is more; a largest value within 1 / 256 of the
 * type's largest may stand for one beyond the type).  A block with an infinity
 * or NaN in it stands for NaN throughout.
 *
 * Layout: rows of 32 ceil(cols / 32) int8 codes (zeros beyond cols), and at the
 * next 256 bytes rows of ceil(cols / 32) bytes s + 127 (255: NaN).
 * bakron_ck8_bytes is 0 when rows or cols is 0 or outside its limits.
 */
size_t bakron_ck8_bytes(int64_t rows, int64_t cols);

/* A checkpoint (256-byte aligned) of rows x cols values of a 16-bit type. */
int bakron_ck8_pack(const void* x, int64_t ldx, int64_t rows, int32_t type, int64_t cols, void* ck, hipStream_t stream);

/* What it stands for, in BAKRON_Q4_BF16 (exact where the value is not below
 * 2^-126), BAKRON_Q4_FP16 (rounded, where it has to be) or BAKRON_MOE_F32 (exact). */
int bakron_ck8_unpack(const void* ck, int64_t rows, int64_t cols, int32_t type, void* x, int64_t ldx,
                      hipStream_t stream);

/*
 * bakron_gated_act -- h = act(a) * b, entry by entry.
 *
 * a, b       [in]  rows x cols, row strides lda, ldb (two halves of one buffer,
 *                  say).
 * act        [in]  BAKRON_MOE_SILU or BAKRON_MOE_GELU.
 * count      [in]  null, or one int32 on the device: only rows below it are
 *                  read or written (offsets + experts, for sorted rows).
 * h          [out] rows x cols, row stride ldh.
 * ck_a, ck_b [out] both null, or checkpoints of a and b (256-byte aligned).
 */
int bakron_gated_act(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int32_t type, int64_t cols,
                     int32_t act, const int32_t* count, void* h, int64_t ldh, void* ck_a, void* ck_b,
                     hipStream_t stream);

/*
 * bakron_gated_act_grad -- its gradients from the checkpoints: with a and b
 * the values that ck_a and ck_b stand for,
 *     da = dh b act'(a),   db = dh act(a).
 */
int bakron_gated_act_grad(const void* dh, int64_t lddh, const void* ck_a, const void* ck_b, int64_t rows, int32_t type,
                          int64_t cols, int32_t act, const int32_t* count, void* da, int64_t ldda, void* db,
                          int64_t lddb, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BAKRON_MOE_H */
