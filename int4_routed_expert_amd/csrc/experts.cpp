// C ABI of microscaled rows and products and of the work grouped by expert: argument checks.
// Declarations and contracts: include/moe_mx.h, include/moe_grouped.h.
#include "experts.h"

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

constexpr int32_t kMostBlocks = 1 << 20;

// q, e of S rows of B blocks.
int check_codes(const void *q, int64_t ldq, const void *e, int64_t lde, int64_t S, int64_t B, bool out) {
  if (!q || !e) return MOE_ENULL;
  if (!aligned(q, 16) || ldq % 16 || ldq < 0 || lde < 0) return MOE_EINVAL;
  if (out && S > 1 && (ldq < 16 * B || lde < B)) return MOE_EINVAL;
  return MOE_OK;
}

int quant(bool silu, const void *x, const void *u, int32_t x_dtype, int64_t ldx, int32_t S, int32_t H, int32_t rounding,
          uint8_t *q, int64_t ldq, uint8_t *e, int64_t lde, void *stream) {
  if (S < 0 || H < 1 || H > 32 * kMostBlocks || (rounding != MOE_MX_FLOOR && rounding != MOE_MX_UP)) return MOE_EINVAL;
  if (!known(x_dtype)) return MOE_EDTYPE;
  if (S == 0) return MOE_OK;
  if (!x || (silu && !u)) return MOE_ENULL;
  const int xs = size_of(x_dtype);
  if (ldx < 0 || !aligned(x, xs) || (silu && !aligned(u, xs))) return MOE_EINVAL;
  if (const int v = check_codes(q, ldq, e, lde, S, (H + 31) / 32, true)) return v;
  MxArgs a{};
  a.S = S; a.H = H; a.up = rounding == MOE_MX_UP;
  a.x = x; a.u = u; a.q = q; a.e = e;
  a.ldx = ldx; a.ldq = ldq; a.lde = lde;
  return status((silu ? launch_mx_silu_quant : launch_mx_quant)(a, x_dtype == MOE_BF16, (hipStream_t)stream));
}

// The sizes and tensors that every product has.
int check_product(ProdArgs &a, int32_t T, int32_t N, int32_t width, int32_t most, int32_t x_rows, const moe_groups *g) {
  if (T < 0 || T > kMaxRows || N < 1 || N > kMaxRows || width < 1 || width > most || x_rows < 0 || (T > 0 && x_rows < 1))
    return MOE_EINVAL;
  a.T = T; a.N = N; a.x_rows = x_rows; a.E = 1; a.top_k = 1;
  if (g) {
    if (g->n < 1 || g->n > kMaxE || (g->order && g->top_k < 1)) return MOE_EINVAL;
    if (!aligned(g->first, 4) || !aligned(g->order, 4)) return MOE_EINVAL;
    if (T > 0 && !g->first) return MOE_ENULL;
    a.E = g->n; a.first = g->first; a.order = g->order;
    if (g->order) a.top_k = g->top_k;
  }
  return MOE_OK;
}
int check_out(ProdArgs &a, void *y, int32_t y_dtype, int64_t ldy) {
  if (!known(y_dtype)) return MOE_EDTYPE;
  if (a.T == 0) return MOE_OK;
  if (!y) return MOE_ENULL;
  if (!aligned(y, size_of(y_dtype)) || ldy < 0 || (a.T > 1 && ldy < a.N)) return MOE_EINVAL;
  a.y = y; a.y_bf16 = y_dtype == MOE_BF16; a.ldy = ldy;
  return MOE_OK;
}

int bf16_product(ProdArgs &a, const void *x, int64_t ldx, int32_t x_rows, const void *w, int64_t ldw, int64_t expert,
                 const moe_groups *g, int32_t T, int32_t N, int32_t K) {
  if (!g) return MOE_ENULL;
  if (const int v = check_product(a, T, N, K, 16 * kMostBlocks, x_rows, g)) return v;
  if (ldx < 0 || ldw < 0 || expert < 0 || !aligned(x, 2) || !aligned(w, 2)) return MOE_EINVAL;
  a.row_bytes = 2 * K;
  a.x = (const uint8_t *)x; a.w = (const uint8_t *)w;
  a.ldx = 2 * ldx; a.ldw = 2 * ldw; a.expert = 2 * expert;
  return MOE_OK;
}

int mx_product(ProdArgs &a, const moe_mx_rows *x, int32_t x_rows, const moe_mx_rows *w, const moe_groups *g, int32_t T,
               int32_t N, int32_t B) {
  if (!x || !w) return MOE_ENULL;
  if (const int v = check_product(a, T, N, B, kMostBlocks, x_rows, g)) return v;
  if (T == 0) return MOE_OK;
  if (const int v = check_codes(x->q, x->ldq, x->e, x->lde, x_rows, B, false)) return v;
  if (const int v = check_codes(w->q, w->ldq, w->e, w->lde, N, B, false)) return v;
  if (g && (w->expert_q < 0 || w->expert_q % 16 || w->expert_e < 0)) return MOE_EINVAL;
  a.row_bytes = 16 * B;
  a.x = x->q; a.xe = x->e; a.w = w->q; a.we = w->e;
  a.ldx = x->ldq; a.ldxe = x->lde; a.ldw = w->ldq; a.ldwe = w->lde;
  if (g) a.expert = w->expert_q, a.expert_e = w->expert_e;
  return MOE_OK;
}

int run_product(ProdArgs &a, bool mx, void *y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes, void *stream) {
  if (const int v = check_out(a, y, y_dtype, ldy)) return v;
  if (a.T == 0) return MOE_OK;
  const int64_t need = product_workspace(a, mx);
  if (need > 0 && !ws) return MOE_ENULL;
  if (need > 0 && !aligned(ws, 16)) return MOE_EINVAL;
  if ((uint64_t)need > ws_bytes) return MOE_EWORKSPACE;
  a.ws = (uint8_t *)ws;
  return status(launch_product(a, mx, (hipStream_t)stream));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_mx_quant(const void *x, int32_t x_dtype, int64_t ldx, int32_t S, int32_t H, int32_t rounding, uint8_t *q,
                 int64_t ldq, uint8_t *e, int64_t lde, void *stream) {
  return quant(false, x, nullptr, x_dtype, ldx, S, H, rounding, q, ldq, e, lde, stream);
}

int moe_mx_silu_quant(const void *g, const void *u, int32_t x_dtype, int64_t ldx, int32_t S, int32_t I,
                      int32_t rounding, uint8_t *q, int64_t ldq, uint8_t *e, int64_t lde, void *stream) {
  return quant(true, g, u, x_dtype, ldx, S, I, rounding, q, ldq, e, lde, stream);
}

int moe_mx_values(const uint8_t *q, int64_t ldq, const uint8_t *e, int64_t lde, int32_t S, int32_t H, void *y,
                  int32_t y_dtype, int64_t ldy, void *stream) {
  if (S < 0 || H < 1 || H > 32 * kMostBlocks) return MOE_EINVAL;
  if (!known(y_dtype)) return MOE_EDTYPE;
  if (S == 0) return MOE_OK;
  if (!y) return MOE_ENULL;
  if (!aligned(y, size_of(y_dtype)) || ldy < 0 || (S > 1 && ldy < H)) return MOE_EINVAL;
  if (const int v = check_codes(q, ldq, e, lde, S, (H + 31) / 32, false)) return v;
  MxArgs a{};
  a.S = S; a.H = H;
  a.q = (uint8_t *)q; a.e = (uint8_t *)e; a.y = y;
  a.ldq = ldq; a.lde = lde; a.ldy = ldy;
  return status(launch_mx_values(a, y_dtype == MOE_BF16, (hipStream_t)stream));
}

int64_t moe_mx_matmul_workspace_bytes(const moe_mx_rows *x, const moe_mx_rows *w, int32_t S, int32_t N, int32_t B) {
  ProdArgs a{};
  if (const int v = mx_product(a, x, S, w, nullptr, S, N, B)) return v;
  return S == 0 ? 0 : product_workspace(a, true);
}
int moe_mx_matmul(const moe_mx_rows *x, const moe_mx_rows *w, int32_t S, int32_t N, int32_t B, void *y,
                  int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes, void *stream) {
  ProdArgs a{};
  if (const int v = mx_product(a, x, S, w, nullptr, S, N, B)) return v;
  return run_product(a, true, y, y_dtype, ldy, ws, ws_bytes, stream);
}

int64_t moe_group_workspace_bytes(int32_t S, int32_t k, int32_t E) {
  if (S < 0 || k < 1 || (int64_t)S * k > kMaxRows || E < 1 || E > kMaxE) return MOE_EINVAL;
  return group_workspace((int64_t)S * k, E);
}
int moe_group(const int32_t *idx, int32_t S, int32_t k, int32_t E, int32_t *first, int32_t *order, int32_t *place,
              void *ws, size_t ws_bytes, void *stream) {
  const int64_t need = moe_group_workspace_bytes(S, k, E);
  if (need < 0) return (int)need;
  if (!first || (S > 0 && (!idx || !order || !place)) || (need > 0 && !ws)) return MOE_ENULL;
  if (!aligned(idx, 4) || !aligned(first, 4) || !aligned(order, 4) || !aligned(place, 4) || (need > 0 && !aligned(ws, 4)))
    return MOE_EINVAL;
  if ((uint64_t)need > ws_bytes) return MOE_EWORKSPACE;
  GroupArgs a{};
  a.T = S * k; a.E = E;
  a.idx = idx; a.first = first; a.order = order; a.place = place;
  a.counts = (uint32_t *)ws;
  return status(launch_group(a, (hipStream_t)stream));
}

int64_t moe_grouped_matmul_workspace_bytes(const void *x, int64_t ldx, int32_t x_rows, const void *w, int64_t ldw,
                                           int64_t expert, const moe_groups *g, int32_t T, int32_t N, int32_t K) {
  ProdArgs a{};
  if (const int v = bf16_product(a, x, ldx, x_rows, w, ldw, expert, g, T, N, K)) return v;
  return T == 0 ? 0 : product_workspace(a, false);
}
int moe_grouped_matmul(const void *x, int64_t ldx, int32_t x_rows, const void *w, int64_t ldw, int64_t expert,
                       const moe_groups *g, int32_t T, int32_t N, int32_t K, void *y, int32_t y_dtype, int64_t ldy,
                       void *ws, size_t ws_bytes, void *stream) {
  ProdArgs a{};
  if (const int v = bf16_product(a, x, ldx, x_rows, w, ldw, expert, g, T, N, K)) return v;
  if (T > 0 && (!x || !w)) return MOE_ENULL;
  return run_product(a, false, y, y_dtype, ldy, ws, ws_bytes, stream);
}

int64_t moe_mx_grouped_matmul_workspace_bytes(const moe_mx_rows *x, int32_t x_rows, const moe_mx_rows *w,
                                              const moe_groups *g, int32_t T, int32_t N, int32_t B) {
  if (!g) return MOE_ENULL;
  ProdArgs a{};
  if (const int v = mx_product(a, x, x_rows, w, g, T, N, B)) return v;
  return T == 0 ? 0 : product_workspace(a, true);
}
int moe_mx_grouped_matmul(const moe_mx_rows *x, int32_t x_rows, const moe_mx_rows *w, const moe_groups *g, int32_t T,
                          int32_t N, int32_t B, void *y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes,
                          void *stream) {
  if (!g) return MOE_ENULL;
  ProdArgs a{};
  if (const int v = mx_product(a, x, x_rows, w, g, T, N, B)) return v;
  return run_product(a, true, y, y_dtype, ldy, ws, ws_bytes, stream);
}

int moe_combine(const void *z, int32_t z_dtype, int64_t ldz, int32_t T, const float *w, const int32_t *place, int32_t S,
                int32_t k, int32_t H, const void *add, int64_t lda, void *y, int32_t y_dtype, int64_t ldy,
                void *stream) {
  if (S < 0 || k < 1 || H < 1 || H > 1 << 30 || T < 0 || (int64_t)S * k > kMaxRows) return MOE_EINVAL;
  if (!known(z_dtype) || !known(y_dtype)) return MOE_EDTYPE;
  if (S == 0) return MOE_OK;
  if ((T > 0 && !z) || !w || !place || !y) return MOE_ENULL;
  const int zs = size_of(z_dtype);
  if (ldz < 0 || lda < 0 || ldy < 0 || (S > 1 && ldy < H) || !aligned(z, zs) || !aligned(add, zs) ||
      !aligned(y, size_of(y_dtype)) || !aligned(w, 4) || !aligned(place, 4))
    return MOE_EINVAL;
  CombineArgs a{};
  a.S = S; a.k = k; a.H = H; a.T = T; a.y_bf16 = y_dtype == MOE_BF16;
  a.z = z; a.add = add; a.w = w; a.place = place; a.y = y;
  a.ldz = ldz; a.lda = lda; a.ldy = ldy;
  return status(launch_combine(a, z_dtype == MOE_BF16, (hipStream_t)stream));
}

}  // extern "C"
