/* Dense operators beside the MoE layer of moe.h, for AMD Instinct MI355X (gfx950): C ABI.
 *
 * What a decoder layer computes around its experts, with activations and weights in int8:
 *   moe_norm_quant  residual sum, root-mean-square norm, the norm's rows in int8
 *   moe_qmatmul     int8 rows times int8 weights, a scale per token and output channel
 *   moe_silu_quant  silu(gate) * up, its rows in int8
 *   moe_rope        rotary positions of queries and keys (moe_rope_freqs: frequencies)
 * The conventions of moe.h hold: device pointers owned by the caller, work enqueued on
 * `stream`, arguments checked before anything is enqueued, moe_status return values.
 */
#ifndef INT4_ROUTED_EXPERT_MOE_DENSE_H
#define INT4_ROUTED_EXPERT_MOE_DENSE_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows in int8.  Where a call below writes int8 rows, row r of values v gets
 *   d[r] = fp32(max|v| / 127),  q[r, c] = rint(fp32(v[r, c] / d[r])) in [-127, 127]
 * (ties to even; moe_cfg.act_int8's rule), from the fp32 values before any rounding
 * to an output type; q[r, c] * d[r] is what the integer stands for.  A row of zeros has
 * d = 0 and q = 0; a row holding an infinity or a NaN has d = inf or NaN and q = 0, so
 * that everything computed from it is NaN.
 *
 * Conventions shared by these calls: they need no workspace unless they name one and
 * allocate nothing; rows may be any number of elements apart (the ld arguments and
 * strides count elements); any width and alignment is taken (pointers must be aligned to
 * their element), 16-byte aligned rows are fastest; S = 0 is a no-op.  Errors: MOE_EINVAL
 * (a size, stride or option out of range, a misaligned pointer), MOE_EDTYPE, MOE_ENULL,
 * MOE_EHIP.  An output must not overlap an input except where the call says so. */

/* Residual sum and root-mean-square norm of S rows of H elements, with the norm's rows
 * in int8:
 *   h = t(x + residual),  v = h / sqrt(mean(h^2) + eps) * gamma,  y = t_y(v),
 *   q, d = v in int8.
 * x, residual and h have x_dtype; the norm is that of the stored (rounded) h.  gamma:
 * [H] of g_dtype.  residual may be NULL (h = x); h, y and the pair q, d may each be NULL,
 * not all of them, and h needs a residual.  h may be residual or x, and y may be x, at
 * the same stride and in the same type (in place).  eps >= 0.  Squares are added up in fp32
 * over eight neighbouring elements and in fp64 beyond (in fp64 throughout where H > 16384,
 * or where they leave the range of fp32: a finite row of any magnitude has its norm), in an
 * order that depends on H alone: a row's bits do not depend on the batch or on where it
 * lies. */
int moe_norm_quant(const void *x, int32_t x_dtype, int64_t ldx, const void *residual, int64_t ldr, const void *gamma,
                   int32_t g_dtype, float eps, int32_t S, int32_t H, void *h, int64_t ldh, void *y, int32_t y_dtype,
                   int64_t ldy, int8_t *q, int64_t ldq, float *d, void *stream);

/* SwiGLU of S rows of I elements, v = g / (1 + exp(-g)) * u, as y = t_y(v) and as int8
 * rows.  g and u have x_dtype and the same stride; the halves of a joint gate/up product
 * are g and g + I with ldx >= 2 I.  y and the pair q, d may each be NULL, not both; y may
 * be g or u at the same dtype and stride. */
int moe_silu_quant(const void *g, const void *u, int32_t x_dtype, int64_t ldx, int32_t S, int32_t I, void *y,
                   int32_t y_dtype, int64_t ldy, int8_t *q, int64_t ldq, float *d, void *stream);

/* Product of int8 rows with int8 weights:
 *   y[s, n] = t(fp32(sum_k q[s, k] w[n, k]) * (d[s] * dw[n])),
 * the sum exact in int32 (K <= 131071).  q: [S, K] and d: [S] as written by the calls
 * above (any int8 values are taken); w: [N, K] two's complement bytes and dw: [N], the
 * interchange form of MOE_WF_Q8_ROW.  y: [S, N] of y_dtype.  Rows whose length and
 * distance are multiples of 16 and that start at a multiple of 16 bytes are used where
 * they lie.  Others may first be copied to such places, where that is faster: ws is a
 * device workspace of at least moe_qmatmul_workspace_bytes bytes for the same operands (0
 * where nothing is copied; ws may then be NULL), 16-byte aligned, not initialised, used
 * by one call at a time.  A result does not depend on the other rows of the call.  Also
 * MOE_EWORKSPACE. */
int64_t moe_qmatmul_workspace_bytes(const int8_t *q, int64_t ldq, const int8_t *w, int64_t ldw, int32_t S, int32_t N,
                                    int32_t K);
int moe_qmatmul(const int8_t *q, int64_t ldq, const float *d, const int8_t *w, int64_t ldw, const float *dw, int32_t S,
                int32_t N, int32_t K, void *y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes, void *stream);

/* Rotary positions.  rot (even) of a head's D dimensions, from `offset`, form rot / 2
 * pairs: (2i, 2i + 1) of that part (MOE_ROPE_INTERLEAVED) or (i, i + rot / 2)
 * (MOE_ROPE_HALF).  Pair i of token s turns by a = pos[s] * freqs[i]:
 *   (x1, x2) -> factor * (x1 cos a - x2 sin a, x2 cos a + x1 sin a).
 * a is the whole product, reduced in fp64 with what its rounding leaves off, so far
 * positions lose nothing (|a| < 2^62; beyond 2^53 a position counts as the nearest fp64).  q: [S, heads, D] and
 * k: [S, kheads, D] of x_dtype (k may be NULL with kheads = 0), both turned in the same
 * launch, each with its own token stride and head stride; q_out and k_out likewise.
 * Dimensions outside the part are copied, or left alone where an output is its input
 * (in place, same strides).  pos: [S] int32, or int64 with pos_i64 = 1; freqs: [rot / 2]
 * fp64, device.  Limits: D <= 1024, (heads + kheads) * D <= 2^20. */
enum moe_rope_layout { MOE_ROPE_HALF = 0, MOE_ROPE_INTERLEAVED = 1 };
typedef struct moe_rope_tensor {
  const void *x;
  void *out;
  int64_t x_token, x_head, out_token, out_head; /* strides in elements; the outputs' at least D */
  int32_t heads;
} moe_rope_tensor;
int moe_rope(const moe_rope_tensor *q, const moe_rope_tensor *k, int32_t x_dtype, int32_t S, int32_t D, int32_t rot,
             int32_t offset, int32_t layout, const void *pos, int32_t pos_i64, const double *freqs, double factor,
             void *stream);

/* Frequencies for moe_rope (host): freqs[i] = theta^(-2 i / rot), i < rot / 2, scaled for
 * contexts longer than the trained one by `scaling`:
 *   MOE_ROPE_PLAIN   as they are;
 *   MOE_ROPE_LINEAR  divided by scale (positions interpolated);
 *   MOE_ROPE_NTK     theta * scale^(rot / (rot - 2)) in theta's place: the fastest pair keeps
 *                    its frequency, the slowest is divided by scale (rot > 2);
 *   MOE_ROPE_YARN    each pair by how often it turns within the trained length L: f where it
 *                    turns at least beta_fast times, f / scale where at most beta_slow times,
 *                    between them a blend that is linear in the pair's index (its ends rounded
 *                    outwards to whole indices); *factor = 0.1 ln(scale) + 1 (YaRN, "YaRN:
 *                    Efficient Context Window Extension of Large Language Models", 3.1-3.4).
 * factor (1 otherwise) multiplies cosines and sines in moe_rope.  scale >= 1, theta > 1,
 * trained_length >= 1 and beta_fast > beta_slow > 0 (the last two for MOE_ROPE_YARN). */
enum moe_rope_scaling { MOE_ROPE_PLAIN = 0, MOE_ROPE_LINEAR = 1, MOE_ROPE_NTK = 2, MOE_ROPE_YARN = 3 };
int moe_rope_freqs(int32_t rot, double theta, int32_t scaling, double scale, int32_t trained_length, double beta_fast,
                   double beta_slow, double *freqs, double *factor);

#ifdef __cplusplus
}
#endif
#endif
