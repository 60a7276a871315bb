// C ABI of the dense operators: argument checks and host helpers.  Declarations
// and contracts: include/moe_dense.h.
#include <algorithm>
#include <cmath>

#include "dense.h"

namespace moe {
namespace {

bool known(int32_t dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }
int size_of(int32_t dtype) { return dtype == MOE_BF16 ? 2 : 4; }
bool aligned(const void *p, int n) { return (uintptr_t)p % (uintptr_t)n == 0; }

int status(hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  set_hip_error(e);
  return MOE_EHIP;
}

// An output of S rows at the address of an input: it has to be that input's type and stride.
bool in_place_ok(const void *out, int out_size, int64_t ldo, const void *in, int in_size, int64_t ldi, int32_t S) {
  return !out || out != in || (out_size == in_size && (S == 1 || ldo == ldi));
}

// The outputs that norm and SwiGLU share.
int check_rows(const RowArgs &a, int32_t y_dtype) {
  if ((a.q == nullptr) != (a.d == nullptr)) return MOE_ENULL;
  if (a.y && (a.ldy < a.H || !aligned(a.y, size_of(y_dtype)))) return MOE_EINVAL;
  if (a.q && (a.ldq < a.H || !aligned(a.d, 4))) return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm_quant(const void *x, int32_t x_dtype, int64_t ldx, const void *residual, int64_t ldr, const void *gamma,
                   int32_t g_dtype, float eps, int32_t S, int32_t H, void *h, int64_t ldh, void *y, int32_t y_dtype,
                   int64_t ldy, int8_t *q, int64_t ldq, float *d, void *stream) {
  if (S < 0 || H < 1 || !(eps >= 0.f) || !std::isfinite(eps)) return MOE_EINVAL;
  if (!known(x_dtype) || !known(g_dtype) || (y && !known(y_dtype))) return MOE_EDTYPE;
  if (S == 0) return MOE_OK;
  if (!x || !gamma || (!h && !y && !q && !d) || (h && !residual)) return MOE_ENULL;
  const int xs = size_of(x_dtype);
  if (ldx < 0 || !aligned(x, xs) || !aligned(gamma, size_of(g_dtype)) ||
      (residual && (ldr < 0 || !aligned(residual, xs))) || (h && (ldh < H || !aligned(h, xs))))
    return MOE_EINVAL;
  if (!in_place_ok(h, xs, ldh, x, xs, ldx, S) || !in_place_ok(h, xs, ldh, residual, xs, ldr, S) ||
      !in_place_ok(y, size_of(y_dtype), ldy, x, xs, ldx, S))
    return MOE_EINVAL;
  RowArgs a{};
  a.S = S; a.H = H; a.eps = eps;
  a.g_bf16 = g_dtype == MOE_BF16; a.y_bf16 = y_dtype == MOE_BF16;
  a.x = x; a.residual = residual; a.gamma = gamma; a.h = h; a.y = y; a.q = q; a.d = d;
  a.ldx = ldx; a.ldr = ldr; a.ldh = ldh; a.ldy = ldy; a.ldq = ldq;
  if (const int v = check_rows(a, y_dtype)) return v;
  return status(launch_norm_quant(a, x_dtype == MOE_BF16, (hipStream_t)stream));
}

int moe_silu_quant(const void *g, const void *u, int32_t x_dtype, int64_t ldx, int32_t S, int32_t I, void *y,
                   int32_t y_dtype, int64_t ldy, int8_t *q, int64_t ldq, float *d, void *stream) {
  if (S < 0 || I < 1) return MOE_EINVAL;
  if (!known(x_dtype) || (y && !known(y_dtype))) return MOE_EDTYPE;
  if (S == 0) return MOE_OK;
  if (!g || !u || (!y && !q && !d)) return MOE_ENULL;
  const int xs = size_of(x_dtype);
  if (ldx < 0 || !aligned(g, xs) || !aligned(u, xs)) return MOE_EINVAL;
  if (!in_place_ok(y, size_of(y_dtype), ldy, g, xs, ldx, S) || !in_place_ok(y, size_of(y_dtype), ldy, u, xs, ldx, S))
    return MOE_EINVAL;
  RowArgs a{};
  a.S = S; a.H = I; a.y_bf16 = y_dtype == MOE_BF16;
  a.x = g; a.residual = u; a.y = y; a.q = q; a.d = d;
  a.ldx = ldx; a.ldr = ldx; a.ldy = ldy; a.ldq = ldq;
  if (const int v = check_rows(a, y_dtype)) return v;
  return status(launch_silu_quant(a, x_dtype == MOE_BF16, (hipStream_t)stream));
}

int64_t moe_qmatmul_workspace_bytes(const int8_t *q, int64_t ldq, const int8_t *w, int64_t ldw, int32_t S, int32_t N,
                                    int32_t K) {
  if (S < 0 || N < 1 || K < 1 || K > 131071 || ldq < 0 || ldw < 0) return MOE_EINVAL;
  if (S == 0) return 0;
  QmmArgs a{};
  a.S = S; a.N = N; a.K = K; a.q = q; a.w = w; a.ldq = ldq; a.ldw = ldw;
  return qmatmul_workspace(a);
}

int moe_qmatmul(const int8_t *q, int64_t ldq, const float *d, const int8_t *w, int64_t ldw, const float *dw, int32_t S,
                int32_t N, int32_t K, void *y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes, void *stream) {
  const int64_t need = moe_qmatmul_workspace_bytes(q, ldq, w, ldw, S, N, K);
  if (need < 0) return (int)need;
  if (!known(y_dtype)) return MOE_EDTYPE;
  if (S == 0) return MOE_OK;
  if (!q || !d || !w || !dw || !y || (need > 0 && !ws)) return MOE_ENULL;
  if (ldy < N || !aligned(d, 4) || !aligned(dw, 4) || !aligned(y, size_of(y_dtype)) || (need > 0 && !aligned(ws, 16)))
    return MOE_EINVAL;
  if ((uint64_t)need > ws_bytes) return MOE_EWORKSPACE;
  QmmArgs a{};
  a.S = S; a.N = N; a.K = K; a.y_bf16 = y_dtype == MOE_BF16;
  a.q = q; a.w = w; a.d = d; a.dw = dw; a.y = y;
  a.ldq = ldq; a.ldw = ldw; a.ldy = ldy;
  a.ws = (int8_t *)ws;
  return status(launch_qmatmul(a, (hipStream_t)stream));
}

int moe_rope(const moe_rope_tensor *q, const moe_rope_tensor *k, int32_t x_dtype, int32_t S, int32_t D, int32_t rot,
             int32_t offset, int32_t layout, const void *pos, int32_t pos_i64, const double *freqs, double factor,
             void *stream) {
  if (S < 0 || D < 2 || D > 1024 || rot < 2 || rot % 2 || offset < 0 || offset > D - rot ||
      (layout != MOE_ROPE_HALF && layout != MOE_ROPE_INTERLEAVED) || (pos_i64 != 0 && pos_i64 != 1))
    return MOE_EINVAL;
  if (!known(x_dtype)) return MOE_EDTYPE;
  if (S == 0) return MOE_OK;
  if (!q || !pos || !freqs) return MOE_ENULL;
  if (!aligned(pos, pos_i64 ? 8 : 4) || !aligned(freqs, 8)) return MOE_EINVAL;
  RopeArgs a{};
  a.S = S; a.D = D; a.half = rot / 2; a.offset = offset; a.pos_i64 = pos_i64; a.factor = factor;
  a.pos = pos; a.freqs = freqs;
  int64_t heads = 0;
  for (int i = 0; i < 2; ++i) {
    const moe_rope_tensor *t = i ? k : q;
    if (!t) continue;
    if (t->heads < (i ? 0 : 1)) return MOE_EINVAL;
    if (t->heads == 0) continue;
    if (!t->x || !t->out) return MOE_ENULL;
    const int xs = size_of(x_dtype);
    if (t->x_token < 0 || t->x_head < 0 || (S > 1 && t->out_token < D) || (t->heads > 1 && t->out_head < D) ||
        t->out_token < 0 || t->out_head < 0 || !aligned(t->x, xs) || !aligned(t->out, xs))
      return MOE_EINVAL;
    if (t->x == t->out && ((S > 1 && t->x_token != t->out_token) || (t->heads > 1 && t->x_head != t->out_head)))
      return MOE_EINVAL;
    heads += t->heads;
    a.t[i] = *t;
  }
  if (heads * D > (1 << 20)) return MOE_EINVAL;
  return status(launch_rope(a, x_dtype == MOE_BF16, layout == MOE_ROPE_INTERLEAVED, (hipStream_t)stream));
}

int moe_rope_freqs(int32_t rot, double theta, int32_t scaling, double scale, int32_t trained_length, double beta_fast,
                   double beta_slow, double *freqs, double *factor) {
  if (rot < 2 || rot % 2 || !(theta > 1.0) || !std::isfinite(theta) || !(scale >= 1.0) || !std::isfinite(scale))
    return MOE_EINVAL;
  if (scaling < MOE_ROPE_PLAIN || scaling > MOE_ROPE_YARN || (scaling == MOE_ROPE_NTK && rot < 4)) return MOE_EINVAL;
  if (scaling == MOE_ROPE_YARN && (trained_length < 1 || !(beta_fast > beta_slow) || !(beta_slow > 0.0) ||
                                   !std::isfinite(beta_fast)))
    return MOE_EINVAL;
  if (!freqs || !factor) return MOE_ENULL;
  if (scaling == MOE_ROPE_NTK) theta *= std::pow(scale, (double)rot / (rot - 2));
  double low = 0.0, high = 0.0;
  if (scaling == MOE_ROPE_YARN) {
    // pair index at which a frequency turns n times in the trained length
    auto index = [&](double n) { return rot * std::log(trained_length / (n * 2.0 * M_PI)) / (2.0 * std::log(theta)); };
    low = std::max(std::floor(index(beta_fast)), 0.0);
    high = std::min(std::ceil(index(beta_slow)), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(theta, -2.0 * i / rot);
    if (scaling == MOE_ROPE_LINEAR) {
      freqs[i] = f / scale;
    } else if (scaling == MOE_ROPE_YARN) {
      // high <= low: the blend lies before the first pair (high <= 0: every pair is slow) or beyond the last
      const double slow = high > low ? std::min(std::max((i - low) / (high - low), 0.0), 1.0) : (high <= 0.0 ? 1.0 : 0.0);
      freqs[i] = f / scale * slow + f * (1.0 - slow);
    } else {
      freqs[i] = f;
    }
  }
  *factor = scaling == MOE_ROPE_YARN ? 0.1 * std::log(scale) + 1.0 : 1.0;
  return MOE_OK;
}

}  // extern "C"
