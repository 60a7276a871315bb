/* Products grouped by expert beside the MoE layer of moe.h, for AMD Instinct MI355X
 * (gfx950): C ABI.
 *
 * For experts whose matrices are the caller's own, in bf16 or microscaled (moe_mx.h):
 *   moe_group               sorts the (token, expert) pairs of a routing by expert
 *   moe_grouped_matmul      bf16 rows times their expert's bf16 weights
 *   moe_mx_grouped_matmul   the same of microscaled rows and weights
 *   moe_combine             the experts' rows back to their tokens, weighted
 * The conventions of moe.h hold: device pointers owned by the caller, work enqueued on
 * `stream`, arguments checked before anything is enqueued, moe_status return values.  Errors:
 * MOE_EINVAL (a size, stride or option out of range, a misaligned pointer), MOE_EDTYPE,
 * MOE_ENULL, MOE_EWORKSPACE, MOE_EHIP.  An output must not overlap an input.
 */
#ifndef INT4_ROUTED_EXPERT_MOE_GROUPED_H
#define INT4_ROUTED_EXPERT_MOE_GROUPED_H

#include "moe_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Pair p = s * k + j is choice j of token s: expert idx[s, j] (idx [S, k] as from moe_route;
 * any value outside [0, E) is a dropped pair).  Sorted by expert, pairs of one expert in
 * their own order, the dropped ones last:
 *   first [E + 1]  expert e has positions first[e] .. first[e + 1] - 1; first[E] is the
 *                  number of pairs that were not dropped
 *   order [S * k]  the pair at each position
 *   place [S, k]   each pair's position, -1 where it was dropped
 * E <= 1024, S * k <= 2^24.  ws: a device workspace of moe_group_workspace_bytes bytes (0 for
 * small batches; ws may then be NULL), 4-byte aligned, not initialised, used by one call at a
 * time.  S = 0 writes zeros to first. */
int64_t moe_group_workspace_bytes(int32_t S, int32_t k, int32_t E);
int moe_group(const int32_t *idx, int32_t S, int32_t k, int32_t E, int32_t *first, int32_t *order, int32_t *place,
              void *ws, size_t ws_bytes, void *stream);

/* Which rows belong to which expert.  Expert e's are rows first[e] .. first[e + 1] - 1 of the
 * output (first [n + 1], not decreasing, on the device; n <= 1024).  Row i's input is x's row i,
 * or row order[i] / top_k of it where order is not NULL (order and top_k as for moe_group:
 * the row of the pair's token). */
typedef struct moe_groups {
  const int32_t *first;
  const int32_t *order;
  int32_t n;
  int32_t top_k;
} moe_groups;

/* y[i, n] = t(sum_k x[r(i), k] w[e(i), n, k]), summed in fp32 (in an order that depends on the
 * sizes), for the rows i < T of y that belong to an expert.  Other rows of y, those from
 * first[n] on, are left as they were.  x: [x_rows, K] bf16, rows ldx elements apart; w: [n, N, K]
 * bf16, rows ldw and experts `expert` elements apart; y: [T, N] of y_dtype.  T <= 2^24, N <=
 * 2^24, K <= 2^24, x_rows >= 1 where T > 0.  first is taken within [0, T]; a row whose input
 * lies outside [0, x_rows) becomes NaN; nothing outside the operands is read or written
 * whatever first and order hold (where first decreases, the rows that belong to an expert are
 * unspecified, all of them).
 * Any alignment is taken; rows of a multiple of 16 bytes at multiples of 16 are fastest.
 * Others may first be copied: ws is a device workspace of moe_grouped_matmul_workspace_bytes
 * bytes (0 where nothing is copied; ws may then be NULL), 16-byte aligned, not initialised,
 * used by one call at a time.  T = 0 is a no-op.
 * Slow for many rows (ten to twenty times as long): with order, an x of 4 GiB or more from its first
 * row to its last; rows of x or w 16 MiB or more apart; ldy of 2^22 or more. */
int64_t moe_grouped_matmul_workspace_bytes(const void *x, int64_t ldx, int32_t x_rows, const void *w, int64_t ldw,
                                           int64_t expert, const moe_groups *g, int32_t T, int32_t N, int32_t K);
int moe_grouped_matmul(const void *x, int64_t ldx, int32_t x_rows, const void *w, int64_t ldw, int64_t expert,
                       const moe_groups *g, int32_t T, int32_t N, int32_t K, void *y, int32_t y_dtype, int64_t ldy,
                       void *ws, size_t ws_bytes, void *stream);

/* The same of microscaled rows x [x_rows] and weights w [n][N], B blocks each (moe_mx.h: their
 * layout, and what is copied to ws; slow for the same distances, of codes or of scales). */
int64_t moe_mx_grouped_matmul_workspace_bytes(const moe_mx_rows *x, int32_t x_rows, const moe_mx_rows *w,
                                              const moe_groups *g, int32_t T, int32_t N, int32_t B);
int moe_mx_grouped_matmul(const moe_mx_rows *x, int32_t x_rows, const moe_mx_rows *w, const moe_groups *g, int32_t T,
                          int32_t N, int32_t B, void *y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes,
                          void *stream);

/* y[s] = t(sum_j w[s, j] z[place[s, j]] + add[s]), in fp32 and in the order of j, add last.  z:
 * [T, H] of z_dtype; w: [S, k] fp32; place: [S, k] (moe_group's; a position outside [0, T)
 * contributes nothing, whatever its weight); add: [S, H] of z_dtype, or NULL; y: [S, H] of
 * y_dtype.  Rows of z, add and y are ldz, lda and ldy elements apart, at any alignment.  S *
 * k <= 2^24, H <= 2^30.  S = 0 is a no-op. */
int moe_combine(const void *z, int32_t z_dtype, int64_t ldz, int32_t T, const float *w, const int32_t *place, int32_t S,
                int32_t k, int32_t H, const void *add, int64_t lda, void *y, int32_t y_dtype, int64_t ldy,
                void *stream);

#ifdef __cplusplus
}
#endif
#endif
