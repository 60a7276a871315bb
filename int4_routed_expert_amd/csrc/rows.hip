// Rows in int8 from a norm or a SwiGLU: one pass of arithmetic per element, one scale
// per row.  norm: v = h / sqrt(mean(h^2) + eps) * gamma with h = t(x + residual);
// SwiGLU: v = g / (1 + exp(-g)) * u.  Then d = max|v| / 127 and q = rint(v / d).
#include "dense.h"

namespace moe {
namespace {

enum RowOp { kNorm, kSilu };

__device__ inline float silu_gate(float g) { return g / (1.0f + expf(-g)); }

// v as an int8 code.  The division is IEEE fp32; a denormal scale has too few bits to
// hold |v / d| at 127, hence the clamp.
__device__ inline int code_of(float v, float d) {
  return (int)fminf(fmaxf(rintf(__fdiv_rn(v, d)), -127.0f), 127.0f);
}

constexpr int kRowThreads = 256;

__device__ inline float block_sum(float v, float *s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
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

// Rows of any length: the row is read once for the statistics and again for each
// output; a thread meets the same elements in every pass, so outputs may be inputs.
template <RowOp OP, bool BF16>
__global__ __launch_bounds__(kRowThreads) void k_rows_long(RowArgs a) {
  __shared__ float s_sum[kRowThreads / 64];
  __shared__ uint32_t s_max[kRowThreads / 64];
  for (int64_t r = blockIdx.x; r < a.S; r += gridDim.x) {
    const int64_t xr = r * a.ldx, rr = r * a.ldr, hr = r * a.ldh, yr = r * a.ldy, qr = r * a.ldq;
    float rstd = 1.f;
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
        return silu_gate(load_el<BF16>(a.x, xr + c)) * load_el<BF16>(a.residual, rr + c);
      } else {
        const float g = a.g_bf16 ? load_el<true>(a.gamma, c) : load_el<false>(a.gamma, c);
        return (a.h ? load_el<BF16>(a.h, hr + c) : input(c)) * rstd * g;
      }
    };
    if constexpr (OP == kNorm) {
      float sum = 0.f;
      for (int64_t c = threadIdx.x; c < a.H; c += kRowThreads) {
        const float v = input(c);
        if (a.h) store_el<BF16>(a.h, hr + c, v);
        sum = fmaf(v, v, sum);
      }
      rstd = 1.0f / sqrtf(block_sum(sum, s_sum) / (float)a.H + a.eps);
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

template <RowOp OP>
hipError_t launch_rows(const RowArgs &a, int x_bf16, hipStream_t st) {
  ProfScope ps(OP == kNorm ? "norm_quant" : "silu_quant", st);
  const dim3 g((unsigned)std::min<int64_t>(a.S, 1 << 20)), b(kRowThreads);
  if (x_bf16) MOE_LAUNCH((k_rows_long<OP, true>), g, b, 0, st, a);
  else MOE_LAUNCH((k_rows_long<OP, false>), g, b, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_quant(const RowArgs &a, int x_bf16, hipStream_t st) { return launch_rows<kNorm>(a, x_bf16, st); }
hipError_t launch_silu_quant(const RowArgs &a, int x_bf16, hipStream_t st) { return launch_rows<kSilu>(a, x_bf16, st); }

}  // namespace moe
