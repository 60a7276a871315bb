/* Microscaled 4-bit floating point beside the MoE layer of moe.h, for AMD Instinct MI355X
 * (gfx950): C ABI.
 *
 *   moe_mx_quant       rows of fp32 or bf16 as microscaled rows
 *   moe_mx_silu_quant  silu(gate) * up as microscaled rows
 *   moe_mx_values      the numbers that microscaled rows stand for
 *   moe_mx_matmul      product of microscaled rows with microscaled weights
 * (moe_grouped.h has the product grouped by expert.)  The conventions of moe.h hold: device
 * pointers owned by the caller, work enqueued on `stream`, arguments checked before anything
 * is enqueued, moe_status return values.  Errors: MOE_EINVAL (a size, stride or option out of
 * range, a misaligned pointer), MOE_EDTYPE, MOE_ENULL, MOE_EHIP.  S = 0 is a no-op.  An output
 * must not overlap an input.
 */
#ifndef INT4_ROUTED_EXPERT_MOE_MX_H
#define INT4_ROUTED_EXPERT_MOE_MX_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Microscaled rows (MXFP4 of the "OCP Microscaling Formats (MX) Specification", 1.0).  A
 * row of H values is B = ceil(H / 32) blocks of 32.  Each block has 16 bytes of codes q and
 * one scale byte e:
 *   value of element i = e2m1(code i) * 2^(e - 127),
 * element 2j of the block in the low nibble of byte j, element 2j + 1 in the high one.  A
 * code is a sign, two bits of exponent (bias 1) and one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4,
 * 6 and their negatives.  e = 255: every value of the block is NaN.  Blocks lie one after
 * another: 16 B bytes of codes in a row of q, B bytes in a row of e.  Rows of q start at
 * multiples of 16 bytes and are ldq bytes apart, a multiple of 16; rows of e start at any byte
 * and are lde bytes apart.
 *
 * Quantised blocks:
 *   e = floor(log2(max|v|)) - 2 + 127          MOE_MX_FLOOR (6.3 of the specification), or
 *   e = the least with max|v| <= 6 * 2^(e-127)  MOE_MX_UP (no value is cut off),
 * at least 0; codes = v / 2^(e-127) rounded to the nearest, ties to the even code, magnitudes
 * over 6 to 6 (MOE_MX_FLOOR cuts off up to a quarter of a block's largest values).  A block
 * of zeros has e = 0; one that holds an infinity or a NaN has e = 255 and codes 0.  A row's
 * last block is filled up with zeros.  H <= 2^25. */
enum moe_mx_rounding { MOE_MX_FLOOR = 0, MOE_MX_UP = 1 };

/* q, e of the S rows x [S, H] (x_dtype, any alignment, rows ldx elements apart). */
int moe_mx_quant(const void *x, int32_t x_dtype, int64_t ldx, int32_t S, int32_t H, int32_t rounding, uint8_t *q,
                 int64_t ldq, uint8_t *e, int64_t lde, void *stream);

/* q, e of v = g / (1 + exp(-g)) * u, computed in fp32; g and u [S, I] as for moe_silu_quant. */
int moe_mx_silu_quant(const void *g, const void *u, int32_t x_dtype, int64_t ldx, int32_t S, int32_t I,
                      int32_t rounding, uint8_t *q, int64_t ldq, uint8_t *e, int64_t lde, void *stream);

/* y [S, H] = the first H values of each row (rounded to y_dtype only where the type cannot hold
 * them: bf16 holds all but the far ends of e, where values leave its range). */
int moe_mx_values(const uint8_t *q, int64_t ldq, const uint8_t *e, int64_t lde, int32_t S, int32_t H, void *y,
                  int32_t y_dtype, int64_t ldy, void *stream);

/* A matrix of microscaled rows. */
typedef struct moe_mx_rows {
  const uint8_t *q, *e;
  int64_t ldq, lde;           /* bytes from one row to the next */
  int64_t expert_q, expert_e; /* from one expert's matrix to the next (moe_mx_grouped_matmul's weights) */
} moe_mx_rows;

/* y[s, n] = t(sum_k x[s, k] w[n, k]) over the 32 B values of each row of x [S] and w [N].
 * Products are exact, blocks are scaled by both powers of two and summed in fp32 (in an order
 * that depends on the sizes); sums below 2^-126 may vanish.  A NaN of a row reaches that
 * row's outputs only.  B <= 2^20, S <= 2^24, N <= 2^24.  Large products first copy scales
 * that do not lie as their kernels need them (rows of a multiple of 16 bytes at multiples of
 * 16): ws is a device workspace of moe_mx_matmul_workspace_bytes bytes for the same operands
 * (0 where nothing is copied; ws may then be NULL), 16-byte aligned, not initialised, used by
 * one call at a time.  Also MOE_EWORKSPACE.  Slow for many rows (ten to twenty times as long): rows of x
 * or w 16 MiB or more apart, ldy of 2^22 or more. */
int64_t moe_mx_matmul_workspace_bytes(const moe_mx_rows *x, const moe_mx_rows *w, int32_t S, int32_t N, int32_t B);
int moe_mx_matmul(const moe_mx_rows *x, const moe_mx_rows *w, int32_t S, int32_t N, int32_t B, void *y,
                  int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif
