// Kernel arguments and launchers of the dense operators (rows in int8, the int8
// product, rotary positions).
#pragma once

#include "../../include/moe_dense.h"
#include "dot.h"

namespace moe {

// Outputs of more than this go past the caches (non-temporal stores), int8 rows aside: the
// next call reads those, and reads them several times.  Norm of 512 rows of 6144 bf16: 8.9
// us in place of 10.2, of 2048 24.7 in place of 29.5; norm, product and SwiGLU of 8192
// tokens, one after another, 657 in place of 680 (675 with the int8 rows past the caches
// too).  Of 256 rows (8 MB) the calls after the norm would be 2 us slower.
constexpr int64_t kStreamBytes = 12 << 20;

// A store of v at p (ALIGN: what p is surely aligned to), past the caches where `stream`.
template <int ALIGN = 0, class T>
__device__ inline void put(void *p, const T &v, bool stream) {
  typedef T any __attribute__((aligned(ALIGN ? ALIGN : (int)alignof(T))));
  auto *q = (__attribute__((address_space(1))) any *)p;
  if (stream) {
    asm volatile("");  // kept apart: the two stores would be merged into a plain one
    __builtin_nontemporal_store(v, q);
    asm volatile("");
  } else {
    *q = v;
  }
}

// norm: x, residual, gamma, h; SwiGLU: x is the gate, residual the up rows.
struct RowArgs {
  int S, H;
  bool stream;
  float eps;
  int g_bf16, y_bf16;
  const void *x, *residual, *gamma;
  void *h, *y;
  int8_t *q;
  float *d;
  int64_t ldx, ldr, ldh, ldy, ldq;
};

struct QmmArgs {
  int S, N, K, y_bf16;
  bool stream;
  int y_vec;  // four neighbouring outputs may be stored at once
  const int8_t *q, *w;
  const float *d, *dw;
  void *y;
  int64_t ldq, ldw, ldy;
  int8_t *ws;
};

struct RopeArgs {
  bool stream;
  int S, D, half, offset, pos_i64;
  double factor;
  const void *pos;
  const double *freqs;
  moe_rope_tensor t[2];
};

// ---- elements of fp32 and bf16 rows ---------------------------------------------
__device__ inline float bf16_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// fp32 to bf16, round to nearest even.
__device__ inline uint16_t f_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Two fp32 values as bf16, lo in the low half (one conversion instruction).
__device__ inline uint32_t pack2_bf16(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

template <bool BF16>
__device__ inline float load_el(const void *p, int64_t i) {
  if constexpr (BF16) return bf16_f(ldg<uint16_t>((const uint16_t *)p + i));
  else return ldg<float>((const float *)p + i);
}
template <bool BF16>
__device__ inline void store_el(void *p, int64_t i, float v) {
  if constexpr (BF16) stg<uint16_t>((uint16_t *)p + i, f_bf16(v));
  else stg<float>((float *)p + i, v);
}

hipError_t launch_norm_quant(const RowArgs &a, int x_bf16, hipStream_t st);
hipError_t launch_silu_quant(const RowArgs &a, int x_bf16, hipStream_t st);
hipError_t launch_qmatmul(const QmmArgs &a, hipStream_t st);
int64_t qmatmul_workspace(const QmmArgs &a);
hipError_t launch_rope(const RopeArgs &a, int x_bf16, int interleaved, hipStream_t st);

}  // namespace moe
