// Rows in int8 from a norm or a SwiGLU, one scale per row.
//   norm:   h = t(x + residual), v = h / sqrt(mean(h^2) + eps) * gamma
//   SwiGLU: v = g / (1 + exp(-g)) * u
//   then d = max|v| / 127 and q = rint(v / d).
// Bound by memory: the row stays in registers between the statistics and the outputs, so
// each input is read and each output written once (counters: 1.00 times the unique bytes).
// Measured: norm 8192 x 6144 bf16 with residual, norm and int8 rows 97 us, 4.7 TB/s (fp32
// in: 132 us, 5.7); SwiGLU 4096 x 12288 bf16 63 us, 4.0 TB/s (fp32: 85 us, 5.3; a copy of 1
// GiB runs at 5.1): in bf16 the exponential and the divisions take about as long as the
// memory.  One row of 6144: 4.6 us, two barriers and a trip to memory.  Rows away from
// 16-byte boundaries: norm 4096 x 5001 bf16 69 us (5000 wide: 49), bound by its stores at odd
// places; SwiGLU 32 (31).
#include <algorithm>

#include "dense.h"

namespace moe {
namespace {

enum RowOp { kNorm, kSilu };

// silu(g) u in the order and with the functions of the experts' SwiGLU: int8 codes come
// out next to a rounding border the same wherever the same values are computed.  (With the
// exponential and the quotient from the hardware's approximations SwiGLU 4096 x 12288
// takes 57 us.)
__device__ inline float silu_times(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Division of many numbers by one: the product with its reciprocal and one correction
// step, which rounds as the division does except next to a midpoint of two fp32 values
// (three operations in place of about ten), where that neither overflows nor underflows.
struct Divisor {
  float d, r;
  bool near;
  __device__ explicit Divisor(float by) : d(by) {
    near = d >= 0x1p-100f && d <= 0x1p100f;
    r = __fdiv_rn(1.0f, d);
  }
  __device__ float fast(float v) const {  // near only
    const float p = v * r;
    return fmaf(fmaf(-p, d, v), r, p);
  }
};

// v as an int8 code.  The division is IEEE fp32; a denormal scale has too few bits to
// hold |v / d| at 127, hence the clamp.
__device__ inline int code_of(float v, float d) {
  return (int)fminf(fmaxf(rintf(__fdiv_rn(v, d)), -127.0f), 127.0f);
}

constexpr int kRowThreads = 256;

__device__ inline double block_sum(double v, double *s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.;
  for (int i = 0; i < (int)blockDim.x / 64; ++i) t += s[i];
  return t;
}

// |v| as bits: they order like the values, with infinity and then the NaNs on top, so
// one integer maximum finds the row's largest magnitude and whether it is finite.
__device__ inline uint32_t block_max(uint32_t v, uint32_t *s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t t = 0;
  for (int i = 0; i < (int)blockDim.x / 64; ++i) t = max(t, s[i]);
  return t;
}

// sqrt(mean + eps) from the sum of a row's squares.  Sums over lanes and waves are fp64, so
// that the fp32 mean is nearly always the rounded one.
__device__ inline float root_of(double sum, const RowArgs &a) { return sqrtf((float)(sum / a.H) + a.eps); }

// Where the root is so far from 1 that squares may leave the range of fp32 (values beyond
// 2^48, or below 2^-48 with as small an eps), the sum and the root are fp64, and the row is
// brought near 1 by a power of two, so that its division is an ordinary one.
__device__ inline bool far_root(float root) { return !(root >= 0x1p-48f && root <= 0x1p48f); }
__device__ inline float far_root_of(double sum, const RowArgs &a, float &scale) {
  const double r = sqrt(sum / a.H + (double)a.eps);
  scale = r > 1. ? 0x1p-100f : 0x1p100f;
  return (float)(r * scale);
}

// Rows of any length: the row is read once for the statistics and again for each
// output; a thread meets the same elements in every pass, so outputs may be inputs.  One
// element at a time by one workgroup a row, bound by that: norm 2000 x 20000 bf16 with
// residual 365 us, 1.0 TB/s (2 x 20000: 74 us), SwiGLU 121 us, 1.7 TB/s.
template <RowOp OP, bool BF16>
__global__ __launch_bounds__(kRowThreads) void k_rows_long(RowArgs a) {
  __shared__ double s_sum[kRowThreads / 64];
  __shared__ uint32_t s_max[kRowThreads / 64];
  for (int64_t r = blockIdx.x; r < a.S; r += gridDim.x) {
    const int64_t xr = r * a.ldx, rr = r * a.ldr, hr = r * a.ldh, yr = r * a.ldy, qr = r * a.ldq;
    float root = 1.f, scale = 1.f;
    auto input = [&](int64_t c) {
      float v = load_el<BF16>(a.x, xr + c);
      if (a.residual) {
        v += load_el<BF16>(a.residual, rr + c);
        if constexpr (BF16) v = bf16_f(f_bf16(v));
      }
      return v;
    };
    auto value = [&](int64_t c) {
      if constexpr (OP == kSilu) {
        return silu_times(load_el<BF16>(a.x, xr + c), load_el<BF16>(a.residual, rr + c));
      } else {
        const float g = a.g_bf16 ? load_el<true>(a.gamma, c) : load_el<false>(a.gamma, c);
        return __fdiv_rn((a.h ? load_el<BF16>(a.h, hr + c) : input(c)) * scale, root) * g;
      }
    };
    if constexpr (OP == kNorm) {
      double sum = 0.;
      for (int64_t c = threadIdx.x; c < a.H; c += kRowThreads) {
        const float v = input(c);
        if (a.h) store_el<BF16>(a.h, hr + c, v);
        sum = fma((double)v, (double)v, sum);
      }
      sum = block_sum(sum, s_sum);
      root = root_of(sum, a);
      if (far_root(root)) root = far_root_of(sum, a, scale);
    }
    float d = 0.f;
    if (a.q) {
      uint32_t m = 0;
      for (int64_t c = threadIdx.x; c < a.H; c += kRowThreads) m = max(m, __float_as_uint(value(c)) & 0x7FFFFFFFu);
      d = __fdiv_rn(__uint_as_float(block_max(m, s_max)), 127.0f);
      if (threadIdx.x == 0) stg<float>(a.d + r, d);
    }
    const bool usable = d > 0.f && d < __builtin_inff();
    for (int64_t c = threadIdx.x; c < a.H; c += kRowThreads) {
      const float v = value(c);
      if (a.q) stg<int8_t>(a.q + qr + c, usable ? (int8_t)code_of(v, d) : (int8_t)0);
      if (a.y) {
        if (a.y_bf16) store_el<true>(a.y, yr + c, v);
        else store_el<false>(a.y, yr + c, v);
      }
    }
  }
}

// ---- rows held in registers ----------------------------------------------------------
// A row belongs to W waves and stays in their registers between the passes.  Iteration it
// of wave w holds the row's block it W + w of 512 elements, 8 neighbours a lane, moved in
// 16-byte pieces.  ON16: every row starts at a multiple of 16 bytes (8 for the int8 rows).
template <int W>
__device__ inline int col_of(int tid, int it) {
  return (it * W + (tid >> 6)) * 512 + (tid & 63) * 8;
}

template <bool BF16, bool ON16>
__device__ inline void store8(void *p, int64_t i, const float *v, bool stream) {
  if constexpr (BF16) {
    const u32x4_t d = {pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7])};
    uint16_t *q = (uint16_t *)p + i;
    if constexpr (ON16) put(q, d, stream);
    else *(__attribute__((address_space(1))) u32x4_h *)q = d;
  } else {
    float *q = (float *)p + i;
    const f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    // both halves of a piece of 32 bytes together: past the caches, half lines cost a write each
    auto *to = (__attribute__((address_space(1))) f32x4_w *)q;
    if (stream) {
      asm volatile("");
      __builtin_nontemporal_store(a, to);
      __builtin_nontemporal_store(b, (__attribute__((address_space(1))) f32x4_w *)(q + 4));
      asm volatile("");
    } else {
      *to = a;
      *(__attribute__((address_space(1))) f32x4_w *)(q + 4) = b;
    }
  }
}

// The 8 elements of iteration it, those below H (others are left alone).
template <int W, bool ON16, bool BF16>
__device__ inline void load_it(const void *p, int64_t row, int H, int tid, int it, float *v) {
  const int c = col_of<W>(tid, it);
  if (c + 8 <= H) {
    load8<BF16, ON16>(p, row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < H) v[j] = load_el<BF16>(p, row + c + j);
  }
}
template <int W, bool ON16, bool BF16>
__device__ inline void store_it(void *p, int64_t row, int H, int tid, int it, const float *v, bool stream) {
  const int c = col_of<W>(tid, it);
  if (c + 8 <= H) {
    store8<BF16, ON16>(p, row + c, v, stream);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < H) store_el<BF16>(p, row + c + j, v[j]);
  }
}

// The wave's sum and maximum, in every lane (the row operations leave them in lane 63).
template <int CTRL, int ROW_MASK = 0xF>
__device__ inline double dpp_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROW_MASK, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROW_MASK, 0xF, false);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ inline double wave_sum(double v) {
  v = dpp_add<0xB1>(v);        // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);        // quad_perm [2,3,0,1]
  v = dpp_add<0x141>(v);       // row_half_mirror
  v = dpp_add<0x140>(v);       // row_mirror
  v = dpp_add<0x142, 0xA>(v);  // row_bcast:15
  v = dpp_add<0x143, 0xC>(v);  // row_bcast:31
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ inline uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false));
}
__device__ inline uint32_t wave_max(uint32_t v) {
  v = dpp_max<0xB1>(v);        // quad_perm [1,0,3,2]
  v = dpp_max<0x4E>(v);        // quad_perm [2,3,0,1]
  v = dpp_max<0x141>(v);       // row_half_mirror
  v = dpp_max<0x140>(v);       // row_mirror
  v = dpp_max<0x142, 0xA>(v);  // row_bcast:15
  v = dpp_max<0x143, 0xC>(v);  // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Four values as int8 codes: adding 1.5 2^23 to v / d rounds to the nearest integer, ties
// to even, and leaves it in the low bits.
struct Codes : Divisor {
  bool usable;
  __device__ explicit Codes(float scale) : Divisor(scale) { usable = d > 0.f && d < __builtin_inff(); }
  __device__ uint32_t one(float v) const { return __float_as_uint(fast(v) + 12582912.0f); }
  __device__ uint32_t four(const float *v) const {
    if (near) {
      const uint32_t lo = __builtin_amdgcn_perm(one(v[1]), one(v[0]), 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(one(v[3]), one(v[2]), 0x04000C0Cu);
      return lo | hi;
    }
    uint32_t w = 0;
    if (usable) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w |= ((uint32_t)code_of(v[j], d) & 0xFFu) << (8 * j);
    }
    return w;
  }
};

// (8 x 2: registers for three workgroups on a compute unit, 65 us against 72 for norm 4096
// x 8192.  Norm with one block a wave: for eight waves a SIMD, 23.0 us against 23.9 for
// 16384 rows of 333 bf16.)
template <RowOp OP, int W, int IT>
constexpr int kRowWaves = W == 8 && IT == 2 ? 6 : OP == kNorm && W <= 4 && IT == 1 ? 8 : 1;
template <RowOp OP, bool BF16, int W, int IT, bool ON16>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W, (kRowWaves<OP, W, IT>)) void k_rows(RowArgs a) {
  // each row of a workgroup's turn uses the other half, so one barrier orders both uses
  __shared__ __align__(16) double s_sum[2][W * IT];
  __shared__ __align__(16) uint32_t s_max[2][W];
  constexpr int kRowsAtOnce = W == 1 ? 4 : 1;
  const int tid = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * kRowsAtOnce + (W == 1 ? threadIdx.x >> 6 : 0); r < a.S;
       r += (int64_t)gridDim.x * kRowsAtOnce, turn ^= 1) {
    float v[IT][8] = {}, o[IT][8] = {};
#pragma unroll
    for (int it = 0; it < IT; ++it) load_it<W, ON16, BF16>(a.x, r * a.ldx, a.H, tid, it, v[it]);
    if (OP == kSilu || a.residual) {
#pragma unroll
      for (int it = 0; it < IT; ++it) load_it<W, ON16, BF16>(a.residual, r * a.ldr, a.H, tid, it, o[it]);
    }
    if constexpr (OP == kNorm) {
      // gamma is requested with the row where the registers allow it, else after the sum
      constexpr bool kEarly = IT == 1;
      float g[IT][8] = {};
      auto load_gamma = [&] {
        if (a.g_bf16) {
#pragma unroll
          for (int it = 0; it < IT; ++it) load_it<W, ON16, true>(a.gamma, 0, a.H, tid, it, g[it]);
        } else {
#pragma unroll
          for (int it = 0; it < IT; ++it) load_it<W, ON16, false>(a.gamma, 0, a.H, tid, it, g[it]);
        }
      };
      if constexpr (kEarly) load_gamma();
      // A lane's eight squares are added in fp32, a block's 64 such sums by its wave and the
      // blocks in their order in fp64: the same additions for every W and IT, so a row's
      // bits do not depend on the batch.
      double part[IT];
      auto add_up = [&] {
        double sum = 0.;
        if constexpr (W > 1) {
          if ((tid & 63) == 0) {
#pragma unroll
            for (int it = 0; it < IT; ++it) s_sum[turn][it * W + (tid >> 6)] = part[it];
          }
          __syncthreads();
#pragma unroll
          for (int i = 0; i < W * IT; ++i) sum += s_sum[turn][i];
        } else {
#pragma unroll
          for (int it = 0; it < IT; ++it) sum += part[it];
        }
        return sum;
      };
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        float eight = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[it][j] += o[it][j];
          if constexpr (BF16) v[it][j] = bf16_f(f_bf16(v[it][j]));
          eight = fmaf(v[it][j], v[it][j], eight);
        }
        part[it] = wave_sum((double)eight);
        if (a.h) store_it<W, ON16, BF16>(a.h, r * a.ldh, a.H, tid, it, v[it], a.stream);
      }
      const Divisor root(root_of(add_up(), a));
      if constexpr (!kEarly) load_gamma();
      if (__builtin_expect(!far_root(root.d), 1)) {
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[it][j] = root.fast(v[it][j]) * g[it][j];
      } else {  // all of a row's threads: they have the same sum
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          double eight = 0.;
#pragma unroll
          for (int j = 0; j < 8; ++j) eight = fma((double)v[it][j], (double)v[it][j], eight);
          part[it] = wave_sum(eight);
        }
        if constexpr (W > 1) __syncthreads();  // the first sums have been read
        float scale;
        const float far = far_root_of(add_up(), a, scale);
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[it][j] = __fdiv_rn(v[it][j] * scale, far) * g[it][j];
      }
    } else {
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[it][j] = silu_times(v[it][j], o[it][j]);
    }
    if (a.y) {
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        if (a.y_bf16) store_it<W, ON16, true>(a.y, r * a.ldy, a.H, tid, it, v[it], a.stream);
        else store_it<W, ON16, false>(a.y, r * a.ldy, a.H, tid, it, v[it], a.stream);
      }
    }
    if (a.q) {
      uint32_t m = 0;
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // elements beyond H are 0 (or NaN in a row whose root is not finite, itself NaN)
          m = max(m, __float_as_uint(v[it][j]) & 0x7FFFFFFFu);
        }
      m = wave_max(m);
      if constexpr (W > 1) {
        if ((tid & 63) == 0) s_max[turn][tid >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) m = max(m, s_max[turn][i]);
      }
      const Codes c(__fdiv_rn(__uint_as_float(m), 127.0f));
      if (tid == 0) stg<float>(a.d + r, c.d);
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const uint32_t w[2] = {c.four(v[it]), c.four(v[it] + 4)};
        const int k = col_of<W>(tid, it);
        int8_t *to = a.q + r * a.ldq + k;
        if (k + 8 <= a.H) {
          const uint64_t both = ((uint64_t)w[1] << 32) | w[0];
          if constexpr (ON16) *(__attribute__((address_space(1))) uint64_t *)to = both;
          else *(__attribute__((address_space(1))) u64_b *)to = both;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (k + j < a.H) stg<int8_t>(to + j, (int8_t)(w[j >> 2] >> (8 * (j & 3))));
        }
      }
    }
  }
}

template <RowOp OP, bool BF16, int W, int IT>
void launch_one(const RowArgs &a, bool vec, hipStream_t st) {
  constexpr int kRowsAtOnce = W == 1 ? 4 : 1;
  const dim3 g((unsigned)std::min<int64_t>(((int64_t)a.S + kRowsAtOnce - 1) / kRowsAtOnce, 1 << 20));
  const dim3 b(W == 1 ? 256 : 64 * W);
  if (vec) MOE_LAUNCH((k_rows<OP, BF16, W, IT, true>), g, b, 0, st, a);
  else MOE_LAUNCH((k_rows<OP, BF16, W, IT, false>), g, b, 0, st, a);
}

bool on16(const void *p, int64_t ld, int size) { return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0; }

template <RowOp OP, bool BF16>
void launch_held(const RowArgs &a0, hipStream_t st) {
  RowArgs a = a0;
  const int64_t each = (a.h ? (BF16 ? 2 : 4) : 0) + (a.y ? (a.y_bf16 ? 2 : 4) : 0) + (a.q ? 1 : 0);
  a.stream = each * a.S * a.H > kStreamBytes;
  const int xs = BF16 ? 2 : 4;
  const bool vec = on16(a.x, a.ldx, xs) && on16(a.residual, a.ldr, xs) && on16(a.h, a.ldh, xs) &&
                   on16(a.y, a.ldy, a.y_bf16 ? 2 : 4) && on16(a.gamma, 0, 1) && (uintptr_t)a.q % 8 == 0 && a.ldq % 8 == 0;
  // The fewest registers that hold the row keep the most rows in flight; among the ways to
  // split it the measured order (bf16, 25 million elements, us): 1024 wide: norm 47 at 1 x
  // 2 (W x IT), SwiGLU 28, 47 and 32 at 2 x 1; 2048: norm 46 at 4 x 1, 47 at 2 x 2, SwiGLU 32
  // and 28; 4096: 49 and 28 at 4 x 2, 50 and 33 at 8 x 1; 6144: 51 and 36 at 12 x 1, 57 and
  // 31 at 4 x 3; 8192: 53 and 28 at 8 x 2, 59 and 35 at 16 x 1.  Of few rows the latency
  // counts: one of 6144 takes 4.5 us at 12 x 1, 4.9 at 8 x 2, 5.3 at 4 x 3, 5.5 at 16 x 1
  // (before the sums over lanes became fp64, which adds 0.2).
  constexpr bool norm = OP == kNorm;
  const bool few = a.S <= 64;
  if (a.H <= 512) launch_one<OP, BF16, 1, 1>(a, vec, st);
  else if (a.H <= 1024) few ? launch_one<OP, BF16, 2, 1>(a, vec, st) : launch_one<OP, BF16, 1, 2>(a, vec, st);
  else if (a.H <= 2048) few || norm ? launch_one<OP, BF16, 4, 1>(a, vec, st) : launch_one<OP, BF16, 2, 2>(a, vec, st);
  else if (a.H <= 4096) few ? launch_one<OP, BF16, 8, 1>(a, vec, st) : launch_one<OP, BF16, 4, 2>(a, vec, st);
  else if (a.H <= 6144) few || norm ? launch_one<OP, BF16, 12, 1>(a, vec, st) : launch_one<OP, BF16, 4, 3>(a, vec, st);
  else if (a.H <= 8192) launch_one<OP, BF16, 8, 2>(a, vec, st);
  else if (a.H <= 12288) launch_one<OP, BF16, 12, 2>(a, vec, st);
  else if (a.H <= 16384) few || norm ? launch_one<OP, BF16, 16, 2>(a, vec, st) : launch_one<OP, BF16, 8, 4>(a, vec, st);
  else MOE_LAUNCH((k_rows_long<OP, BF16>), dim3((unsigned)std::min(a.S, 1 << 20)), dim3(kRowThreads), 0, st, a);
}

template <RowOp OP>
hipError_t launch_rows(const RowArgs &a, int x_bf16, hipStream_t st) {
  ProfScope ps(OP == kNorm ? "norm_quant" : "silu_quant", st);
  if (x_bf16) launch_held<OP, true>(a, st);
  else launch_held<OP, false>(a, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_quant(const RowArgs &a, int x_bf16, hipStream_t st) { return launch_rows<kNorm>(a, x_bf16, st); }
hipError_t launch_silu_quant(const RowArgs &a, int x_bf16, hipStream_t st) { return launch_rows<kSilu>(a, x_bf16, st); }

}  // namespace moe
