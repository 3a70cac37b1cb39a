/*
 * bakron_q4.h -- layers on the codes of libbakron.so (MI355X, gfx950): the
 * linear layer, its input gradient and a mixture-of-experts layer computed
 * directly on 4-bit codes, without writing the weights out.
 *
 * A layer rounded by bakron_solve, bakron_gptq or their grouped forms is
 * codes c (m x n, here 0 .. 15, i.e. maxq <= 15), a step s and a zero point
 * z per (output row i, group of group_size input columns); its weights are
 *     w_ij = s_i,q (c_ij - z_i,q),   q = j / group_size.
 * bakron_q4_pack lays codes and grids out once; every other call reads that
 * layout.
 *
 * The conventions are those of bakron.h: device pointers owned by the
 * caller, work enqueued on `stream` in order (no library streams, no
 * allocation, no synchronisation: every call can be captured into a HIP
 * graph), workspaces undefined after a call, return codes BAKRON_*, nothing
 * enqueued on an error, inputs and outputs do not overlap.  In addition:
 *   - Activations and gradients are BAKRON_Q4_BF16 or BAKRON_Q4_FP16, row t
 *     (token t) starting at element t * ld, ld >= the row's length; only
 *     2-byte alignment is asked for (16-byte aligned rows, i.e. a 16-byte
 *     aligned pointer and ld a multiple of 8, are read fastest).
 *   - Sums are float32; results are rounded once to the activations' type
 *     (beyond its largest value to infinity).  Each sum runs over (16 + c) x,
 *     with (16 + z) sum x taken off after every 1024 columns at most: a result's
 *     error is that of roundings of 2^-24 of such a partial sum, about 23 steps
 *     times |sum x| over those columns, however long the row is.
 *   - A non-finite value in a token's row makes that token's results
 *     non-finite (which of inf and NaN is not specified) and touches no
 *     other token.
 *   - Range: sums are held in units of a step, so sum_j 31 |x_j|, and in a row
 *     of several groups that sum times the ratio of any two of its steps, has
 *     to stay below 2^127; beyond it a result may be infinite or NaN.
 *   - A token's result does not depend on the other tokens of the call, but
 *     for its last bits: their number, the alignment of the rows and, in
 *     bakron_q4_moe, the experts that they chose decide on the order of its
 *     sums.  The same call on the same inputs always gives the same bits.
 */
#ifndef BAKRON_Q4_H
#define BAKRON_Q4_H

#include "bakron.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of activations, gradients and results. */
#define BAKRON_Q4_BF16 0
#define BAKRON_Q4_FP16 1

#define BAKRON_Q4_MAX_TOKENS 16777216  /* rows of x or dy in one call */
#define BAKRON_Q4_MAX_LAYERS 256       /* layers of one stack (experts) */
#define BAKRON_Q4_MOE_MAX_TOKENS 64    /* tokens of one bakron_q4_moe call */
#define BAKRON_Q4_MOE_MAX_TOP_K 16     /* experts chosen per token */

/*
 * Bytes of the packed form of `count` layers of m x n with grids per group of
 * group_size columns (0: one grid per row).  0 when an argument is outside
 * bakron_q4_pack's limits or m, n or count is 0.  Host only.
 */
size_t bakron_q4_packed_bytes(int64_t count, int64_t m, int64_t n, int64_t group_size);

/*
 * bakron_q4_pack -- codes and grids of `count` layers of one shape (1 for a
 * linear layer, the number of experts for a stack) in the layout that the
 * other calls read: half a byte per code, 8 bytes per grid entry; m is
 * padded to 16 and n to 128.
 *
 * codes      [in]  count x m x n uint8 in [0, 15] (the caller's to keep: only
 *                  the low four bits are used).
 * scale, zero [in] count x m x G floats, G = ceil(n / group_size), or
 *                  count x m when group_size is 0: the grids the layer was
 *                  rounded with, finite.  A scale is 0 (its weights are 0) or
 *                  of magnitude 2^-100 .. 2^100.  Neither is checked here.
 * count      [in]  0 <= count <= BAKRON_Q4_MAX_LAYERS.
 * m, n       [in]  0 <= m, n <= BAKRON_MAX_DIM.
 * group_size [in]  0 or a positive multiple of 64 (BAKRON_ERR_BAD_ARG
 *                  otherwise).
 * packed     [out] bakron_q4_packed_bytes bytes, 256-byte aligned.
 */
int bakron_q4_pack(const uint8_t* codes, const float* scale, const float* zero, int64_t count, int64_t m, int64_t n,
                   int64_t group_size, void* packed, hipStream_t stream);

/*
 * Workspace bytes of bakron_q4_linear (0 when it needs none or an argument is
 * outside its limits).  Host only.
 */
size_t bakron_q4_linear_workspace_bytes(int64_t tokens, int64_t m, int64_t n, int64_t group_size);

/*
 * bakron_q4_linear -- y = x W^T: y[t, i] = sum_j x[t, j] w_ij.
 *
 * x          [in]  tokens x n, row stride ldx.
 * tokens     [in]  0 <= tokens <= BAKRON_Q4_MAX_TOKENS; any number, from one
 *                  decoding token to a whole prompt.
 * type       [in]  BAKRON_Q4_BF16 or BAKRON_Q4_FP16, of x and y.
 * packed, m, n, group_size [in] one layer as packed by bakron_q4_pack.
 * y          [out] tokens x m, row stride ldy.  n == 0 writes zeros; m == 0
 *                  or tokens == 0 enqueues nothing.
 */
int bakron_q4_linear(const void* x, int64_t ldx, int64_t tokens, int32_t type, const void* packed, int64_t m, int64_t n,
                     int64_t group_size, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                     hipStream_t stream);

/* Workspace bytes of bakron_q4_linear_grad, as above.  Host only. */
size_t bakron_q4_linear_grad_workspace_bytes(int64_t tokens, int64_t m, int64_t n, int64_t group_size);

/*
 * bakron_q4_linear_grad -- the gradient of bakron_q4_linear with respect to
 * its input, dx = dy W: dx[t, j] = sum_i dy[t, i] w_ij.  Step and zero point
 * change with the row that is summed over, so each weight is rounded once to
 * dy's type (in units of about the largest weight of its group's columns, in
 * float16 down to 2^-29 of it without loss), as a layer kept in that type
 * would be; the sums are float32.
 *
 * dy         [in]  tokens x m, row stride lddy.
 * dx         [out] tokens x n, row stride lddx.  m == 0 writes zeros; n == 0
 *                  or tokens == 0 enqueues nothing.
 * Everything else: as in bakron_q4_linear.
 */
int bakron_q4_linear_grad(const void* dy, int64_t lddy, int64_t tokens, int32_t type, const void* packed, int64_t m,
                          int64_t n, int64_t group_size, void* dx, int64_t lddx, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of bakron_q4_moe, as above.  Host only. */
size_t bakron_q4_moe_workspace_bytes(int64_t tokens, int64_t hidden, int64_t ffn, int64_t experts, int32_t top_k,
                                     int64_t group_size);

/*
 * bakron_q4_moe -- a whole mixture-of-experts layer for a few tokens.  Per
 * token t:
 *     l_e = sum_j x[t, j] router[e, j]                       (float32)
 *     ids[t] = the top_k experts of largest l, largest first; equal logits go
 *              to the lower index, NaN counts as -infinity
 *     weights[t] = softmax of l over ids[t]
 *     y[t] = sum_k weights[t, k] down_e ( silu(gate_e x_t) * (up_e x_t) ),
 *            e = ids[t, k],  silu(v) = v / (1 + exp(-v)).
 * Only experts that a token chose are read.
 *
 * x          [in]  tokens x hidden, row stride ldx.
 * tokens     [in]  0 <= tokens <= BAKRON_Q4_MOE_MAX_TOKENS (BAKRON_ERR_BAD_SIZE
 *                  beyond: bakron_moe.h has the layer for any number; layer
 *                  e of a stack starts at e times
 *                  bakron_q4_packed_bytes(1, ...)).
 * router     [in]  experts x hidden, contiguous, of x's type.
 * gate, up   [in]  stacks of `experts` packed layers, ffn x hidden.
 * down       [in]  a stack of `experts` packed layers, hidden x ffn.
 * experts, top_k [in] 1 <= top_k <= min(experts, BAKRON_Q4_MOE_MAX_TOP_K),
 *                  experts <= BAKRON_Q4_MAX_LAYERS (BAKRON_ERR_BAD_ARG
 *                  otherwise).
 * group_size [in]  of all three stacks.
 * y          [out] tokens x hidden, row stride ldy.  ffn == 0 writes zeros;
 *                  hidden == 0 or tokens == 0 enqueues nothing.
 * ids        [out] tokens x top_k int32.
 * weights    [out] tokens x top_k floats.
 */
int bakron_q4_moe(const void* x, int64_t ldx, int64_t tokens, int32_t type, const void* router, const void* gate,
                  const void* up, const void* down, int64_t hidden, int64_t ffn, int64_t experts, int32_t top_k,
                  int64_t group_size, void* y, int64_t ldy, int32_t* ids, float* weights, void* workspace,
                  size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BAKRON_Q4_H */
