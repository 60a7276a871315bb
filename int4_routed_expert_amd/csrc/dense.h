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

// Of a wave-uniform address, through the scalar cache: for memory that the kernel does not write.
template <class T>
__device__ inline T ldk(const T *p) {
  return *(const __attribute__((address_space(4))) T *)p;
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

// ---- eight neighbours of a row ---------------------------------------------------
typedef u32x4_t u32x4_w __attribute__((aligned(4)));
typedef u32x4_t u32x4_h __attribute__((aligned(2)));
typedef f32x4_t f32x4_w __attribute__((aligned(4)));
typedef uint64_t u64_b __attribute__((aligned(1)));

// Eight neighbours.  A bf16 row that starts in the middle of a word is read as the words
// that hold the eight (each holds at least one of them), shifted together: loads from
// odd places take the hardware several times as long.
template <bool BF16, bool ON16>
__device__ inline void load8(const void *p, int64_t i, float *v) {
  if constexpr (BF16) {
    const uint16_t *q = (const uint16_t *)p + i;
    uint32_t d[4];
    if constexpr (ON16) {
      const uint4 r = ldg<uint4>(q);
      d[0] = r.x; d[1] = r.y; d[2] = r.z; d[3] = r.w;
    } else {
      const uint32_t sh = (uint32_t)(uintptr_t)q & 2;
      const u32x4_t r = *(const __attribute__((address_space(1))) u32x4_w *)((uintptr_t)q & ~(uintptr_t)3);
      const uint32_t e = ldg<uint32_t>((const void *)((uintptr_t)(q + 7) & ~(uintptr_t)3));
      d[0] = __builtin_amdgcn_alignbyte(r.y, r.x, sh);
      d[1] = __builtin_amdgcn_alignbyte(r.z, r.y, sh);
      d[2] = __builtin_amdgcn_alignbyte(r.w, r.z, sh);
      d[3] = __builtin_amdgcn_alignbyte(e, r.w, sh);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(d[j] << 16);
      v[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
    }
  } else {
    const float *q = (const float *)p + i;
    const f32x4_t r0 = *(const __attribute__((address_space(1))) f32x4_w *)q;
    const f32x4_t r1 = *(const __attribute__((address_space(1))) f32x4_w *)(q + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = r0[j];
      v[4 + j] = r1[j];
    }
  }
}

hipError_t launch_norm_quant(const RowArgs &a, int x_bf16, hipStream_t st);
hipError_t launch_silu_quant(const RowArgs &a, int x_bf16, hipStream_t st);
hipError_t launch_qmatmul(const QmmArgs &a, hipStream_t st);
int64_t qmatmul_workspace(const QmmArgs &a);
hipError_t launch_rope(const RopeArgs &a, int x_bf16, int interleaved, hipStream_t st);

}  // namespace moe
