// Microscaled rows (blocks of 32 e2m1 codes and one e8m0 scale) from rows or from a SwiGLU, and
// back.
#include <algorithm>
#include <type_traits>

#include "experts.h"

namespace moe {
namespace {

constexpr int kMxThreads = 256;
constexpr uint32_t kInfBits = 0x7F800000u;

// The order and the functions of the experts' SwiGLU (rows.hip).
__device__ inline float silu_times(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Lane l of quad l / 4 takes eight neighbours, a quad a block: a wave reads and writes runs.
// Units of eight are counted through all rows; a workgroup finds its first one's row, a lane
// goes on from there in 32 bits (without a division where a row has as many units as the
// workgroup).
struct Unit {
  int64_t row;
  int c;  // first element
};
template <int MOST>
__device__ inline Unit unit_of(int64_t first_row, uint32_t first_unit, uint32_t i, uint32_t per_row) {
  const uint32_t n = first_unit + i;
  uint32_t r;
  if (per_row >= MOST) r = n >= per_row;
  else r = n / per_row;
  return {first_row + r, (int)(n - r * per_row) * 8};
}

template <bool BF16, bool ON16>
__device__ inline void load_unit(const void *p, int64_t row, int c, int H, float *v) {
  if (c + 8 <= H) {
    load8<BF16, ON16>(p, row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < H ? load_el<BF16>(p, row + c + j) : 0.f;
  }
}

template <int CTRL>
__device__ inline uint32_t quad_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}

// A block's scale from m, the bits of its largest magnitude in fp32: m = 2^(field - 127) (1 +
// fraction), so e = field - 2; over 1.5 times that it exceeds 6 2^(e-127).
__device__ inline int scale_of(uint32_t m, int up) {
  const int field = (int)(m >> 23);
  return m >= kInfBits ? 255 : max(field - 2, 0) + (up && field >= 2 && (m & 0x7FFFFFu) > 0x400000u);
}

// A lane has eight neighbours of a block of 32, a quad the block: its largest magnitude takes two
// exchanges within the quad, and no value leaves its registers.  U units of eight a thread, all of them
// loaded ahead of the first's arithmetic.  Bound by memory: 8192 x 6144 30.3 us from bf16 (4.2 TB/s), 45.7
// from fp32 (5.0), where a copy of 1 GiB reaches 5.1; the SwiGLU 67 us (3.4 TB/s): vector instructions take
// 72% of the SIMDs' cycles (50% without it), those of expf and the division among them, which are the
// other SwiGLUs' so that their codes agree.  Rows that start at odd places: 4096 x 5001 16.6 us (3.1 TB/s).
// Four rows of 2048: 3.2 us, of which a launch 2.3.
// The conversion divides by its scale operand, a power of two, and rounds once, to the even code at
// ties, magnitudes over 6 to 6.  With e = 0 that power is no normal number: values and scale are raised by
// 2^126 first, which is exact.
template <bool BF16, bool SILU, bool ON16, int U>
__global__ __launch_bounds__(kMxThreads) void k_mx_quant(MxArgs a) {
  const uint32_t per_row = (uint32_t)(a.H + 31) / 32 * 4;
  const int64_t n0 = (int64_t)blockIdx.x * kMxThreads * U;
  const int64_t r0 = n0 / per_row;
  const uint32_t u0 = (uint32_t)(n0 - r0 * per_row);
  float v[U][8], o[U][8];
  Unit at[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    at[i] = unit_of<kMxThreads * U>(r0, u0, i * kMxThreads + threadIdx.x, per_row);
    if (at[i].row < a.S) {
      load_unit<BF16, ON16>(a.x, at[i].row * a.ldx, at[i].c, a.H, v[i]);
      if constexpr (SILU) load_unit<BF16, ON16>(a.u, at[i].row * a.ldx, at[i].c, a.H, o[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (at[i].row >= a.S) continue;  // whole quads: a row has a multiple of four units
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (SILU) v[i][j] = silu_times(v[i][j], o[i][j]);
      m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);  // magnitudes order as their bits, NaN on top
    }
    m = quad_max<0xB1>(m);  // quad_perm [1,0,3,2]
    m = quad_max<0x4E>(m);  // quad_perm [2,3,0,1]
    const int e = scale_of(m, a.up);
    float s = __uint_as_float((uint32_t)e << 23);
    if (__builtin_expect(e == 0, 0)) {
      s = 0x1p-1f;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= 0x1p126f;
    }
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[i][0], v[i][1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[i][2], v[i][3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[i][4], v[i][5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[i][6], v[i][7], s, 3);
    if (e == 255) w = 0;
    stg<uint32_t>(a.q + at[i].row * a.ldq + at[i].c / 2, w);
    if ((threadIdx.x & 3) == 0) stg<uint8_t>(a.e + at[i].row * a.lde + at[i].c / 32, (uint8_t)e);
  }
}

// The value of code c (0..15) times 2^(e - 127): the code's three low bits as the top of a
// float's exponent and mantissa are its magnitude times 2^-126, the denormal 0.5 among them.
__device__ inline float mx_value(uint32_t c, float scale) {
  return __uint_as_float(((c & 8) << 28) | ((c & 7) << 22)) * 0x1p126f * scale;
}

// A lane takes eight codes.  Bound by its writes: 8192 x 6144 to bf16 24.8 us (5.1 TB/s), 4096 x 5001, whose
// rows start at odd places, 15.0 us (3.5 TB/s) with 16-byte stores at any element, 33.6 one by one.
template <bool BF16, bool ON16, int U>
__global__ __launch_bounds__(kMxThreads) void k_mx_values(MxArgs a) {
  const uint32_t per_row = (uint32_t)(a.H + 7) / 8;
  const int64_t n0 = (int64_t)blockIdx.x * kMxThreads * U;
  const int64_t r0 = n0 / per_row;
  const uint32_t u0 = (uint32_t)(n0 - r0 * per_row);
  uint32_t w[U], e[U];
  Unit at[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    at[i] = unit_of<kMxThreads * U>(r0, u0, i * kMxThreads + threadIdx.x, per_row);
    if (at[i].row < a.S) {
      w[i] = ldg<uint32_t>(a.q + at[i].row * a.ldq + at[i].c / 2);
      e[i] = ldg<uint8_t>(a.e + at[i].row * a.lde + at[i].c / 32);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (at[i].row >= a.S) continue;
    const float scale = __uint_as_float(e[i] == 255 ? 0x7FC00000u : e[i] == 0 ? 0x00400000u : e[i] << 23);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = mx_value(w[i] >> (4 * j), scale);
    const int64_t to = at[i].row * a.ldy + at[i].c;
    if (at[i].c + 8 <= a.H) {
      if constexpr (BF16) {
        typedef std::conditional_t<ON16, u32x4_t, u32x4_h> any;
        const u32x4_t d = {pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7])};
        *(__attribute__((address_space(1))) any *)((uint16_t *)a.y + to) = d;
      } else {
        typedef std::conditional_t<ON16, f32x4_t, f32x4_w> any;
        *(__attribute__((address_space(1))) any *)((float *)a.y + to) = f32x4_t{v[0], v[1], v[2], v[3]};
        *(__attribute__((address_space(1))) any *)((float *)a.y + to + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at[i].c + j < a.H) store_el<BF16>(a.y, to + j, v[j]);
    }
  }
}

bool on16(const void *p, int64_t ld, int size) { return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0; }

// A launch holds fewer than 2^32 threads and counts its units in 32 bits past the first row:
// long inputs go in pieces of rows.
int64_t rows_at_once(int64_t per_row) { return std::max<int64_t>(1, ((int64_t)1 << 31) / per_row); }

// Few units: one a thread, so that they spread over the chip.
constexpr int64_t kFewUnits = 256 * kMxThreads * 4;

// Units a thread of many (8192 x 6144 bf16: 31.7 us with four, 34.0 with eight; SwiGLU 69.6 us with two,
// 70.2 with four).
template <bool SILU>
constexpr int kMany = SILU ? 2 : 4;
template <bool BF16, bool SILU, bool ON16>
void launch_quant_one(const MxArgs &a, hipStream_t st) {
  const int64_t units = (int64_t)a.S * ((a.H + 31) / 32 * 4);
  if (units <= kFewUnits)
    MOE_LAUNCH((k_mx_quant<BF16, SILU, ON16, 1>), dim3((unsigned)((units + kMxThreads - 1) / kMxThreads)), dim3(kMxThreads), 0, st, a);
  else
    MOE_LAUNCH((k_mx_quant<BF16, SILU, ON16, kMany<SILU>>), dim3((unsigned)((units + kMany<SILU> * kMxThreads - 1) / (kMany<SILU> * kMxThreads))),
               dim3(kMxThreads), 0, st, a);
}

template <bool SILU>
hipError_t launch_quant(const MxArgs &a, int x_bf16, hipStream_t st) {
  const int xs = x_bf16 ? 2 : 4;
  const bool vec = on16(a.x, a.ldx, xs) && (!SILU || on16(a.u, a.ldx, xs));
  const int64_t step = rows_at_once((a.H + 31) / 32 * 4);
  for (int64_t s = 0; s < a.S; s += step) {
    MxArgs c = a;
    c.S = (int)std::min<int64_t>(step, a.S - s);
    c.x = (const char *)a.x + s * a.ldx * xs;
    if (SILU) c.u = (const char *)a.u + s * a.ldx * xs;
    c.q += s * a.ldq;
    c.e += s * a.lde;
    ProfScope ps(SILU ? "mx_silu_quant" : "mx_quant", st);
    if (x_bf16) vec ? launch_quant_one<true, SILU, true>(c, st) : launch_quant_one<true, SILU, false>(c, st);
    else vec ? launch_quant_one<false, SILU, true>(c, st) : launch_quant_one<false, SILU, false>(c, st);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <bool BF16, bool ON16>
void launch_values_one(const MxArgs &a, hipStream_t st) {
  const int64_t units = (int64_t)a.S * ((a.H + 7) / 8);
  if (units <= kFewUnits)
    MOE_LAUNCH((k_mx_values<BF16, ON16, 1>), dim3((unsigned)((units + kMxThreads - 1) / kMxThreads)), dim3(kMxThreads), 0, st, a);
  else
    MOE_LAUNCH((k_mx_values<BF16, ON16, 4>), dim3((unsigned)((units + 4 * kMxThreads - 1) / (4 * kMxThreads))), dim3(kMxThreads), 0, st, a);
}

}  // namespace

hipError_t launch_mx_quant(const MxArgs &a, int x_bf16, hipStream_t st) { return launch_quant<false>(a, x_bf16, st); }
hipError_t launch_mx_silu_quant(const MxArgs &a, int x_bf16, hipStream_t st) { return launch_quant<true>(a, x_bf16, st); }

hipError_t launch_mx_values(const MxArgs &a, int y_bf16, hipStream_t st) {
  const int ys = y_bf16 ? 2 : 4;
  const bool vec = on16(a.y, a.ldy, ys);
  const int64_t step = rows_at_once((a.H + 7) / 8);
  for (int64_t s = 0; s < a.S; s += step) {
    MxArgs c = a;
    c.S = (int)std::min<int64_t>(step, a.S - s);
    c.y = (char *)a.y + s * a.ldy * ys;
    c.q += s * a.ldq;
    c.e += s * a.lde;
    ProfScope ps("mx_values", st);
    if (y_bf16) vec ? launch_values_one<true, true>(c, st) : launch_values_one<true, false>(c, st);
    else vec ? launch_values_one<false, true>(c, st) : launch_values_one<false, false>(c, st);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
