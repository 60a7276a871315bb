// Rotary positions: pair i of a head turns by a = pos * freqs[i].
//   (x1, x2) -> factor * (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
//
// Bound by memory: every element is read and written once.  A workgroup takes a few
// tokens (a part of one token's heads where there are few tokens), forms their sines and
// cosines once in LDS, a pair a thread, and streams the heads in units of 16 bytes (two
// elements or one where the sizes ask for it).  8192 tokens, 72 heads of 128, bf16: 54 us,
// 5.6 TB/s (interleaved 56; a copy of 1 GiB runs at 5.1).  Units of one element cost a load
// and a store each: 4096 tokens, 34 heads of 129, 40 us, of 128 16 us.
#include <algorithm>

#include "dense.h"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeAngles = 1024;  // angles a workgroup may hold (8 KB of LDS)

// factor times cosine and sine of pos * f, rounded to fp32 once (within 2^-35 of the true
// value before that) for |pos * f| < 2^62: quarter turns are taken off in fp64, from the
// product and its rounding error and by pi / 2 in two parts, a second time for those that the
// first estimate of their number missed (from 2^49 on), and the rest, |r| <= pi / 4, goes
// through the Taylor series to r^11 and r^12 in fp64, whose next terms are below 2^-36.
__device__ inline float2 cos_sin(double pos, double f, double factor) {
  const double a = pos * f;
  const double n = rint(a * 0.63661977236758134308);  // 2 / pi
  const double r0 = fma(-n, 6.12323399573676603587e-17, fma(-n, 1.57079632679489661923, a)) + fma(pos, f, -a);
  const double m = rint(r0 * 0.63661977236758134308);
  const double r = fma(-m, 1.57079632679489661923, r0);
  const int quarter = ((int)(int64_t)n + (int)m) & 3;
  const double r2 = r * r;
  double s = fma(r2, -1. / 39916800, 1. / 362880), c = fma(r2, 1. / 479001600, -1. / 3628800);
  s = fma(r2, s, -1. / 5040);
  c = fma(r2, c, 1. / 40320);
  s = fma(r2, s, 1. / 120);
  c = fma(r2, c, -1. / 720);
  s = fma(r2, s, -1. / 6);
  c = fma(r2, c, 1. / 24);
  s = fma(r * r2, s, r);
  c = fma(r2, fma(r2, c, -0.5), 1.);
  const double cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
  return make_float2((float)(factor * (quarter == 1 || quarter == 2 ? -cc : cc)), (float)(factor * (quarter >= 2 ? -ss : ss)));
}

typedef f32x4_t f32x4_w __attribute__((aligned(4)));
typedef float f32x2_w __attribute__((ext_vector_type(2), aligned(4)));

// V neighbouring elements as floats: 16 bytes' worth (bf16 on a multiple of 16 bytes, fp32
// on any word), two (on a word) or one.
template <bool BF16, int V>
__device__ inline void load_v(const void *p, int64_t i, float *v) {
  if constexpr (V == 1) {
    v[0] = load_el<BF16>(p, i);
  } else if constexpr (BF16) {
    uint32_t d[V / 2];
    if constexpr (V == 2) {
      d[0] = ldg<uint32_t>((const uint16_t *)p + i);
    } else {
      const uint4 r = ldg<uint4>((const uint16_t *)p + i);
      d[0] = r.x; d[1] = r.y; d[2] = r.z; d[3] = r.w;
    }
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      v[2 * j] = __uint_as_float(d[j] << 16);
      v[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
    }
  } else if constexpr (V == 2) {
    const f32x2_w r = *(const __attribute__((address_space(1))) f32x2_w *)((const float *)p + i);
    v[0] = r.x; v[1] = r.y;
  } else {
    const f32x4_w r = *(const __attribute__((address_space(1))) f32x4_w *)((const float *)p + i);
    v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
  }
}
template <bool BF16, int V>
__device__ inline void store_v(void *p, int64_t i, const float *v, bool stream) {
  if constexpr (V == 1) {
    store_el<BF16>(p, i, v[0]);
  } else if constexpr (BF16 && V == 2) {
    stg<uint32_t>((uint16_t *)p + i, pack2_bf16(v[0], v[1]));
  } else if constexpr (BF16) {
    const u32x4_t d = {pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7])};
    put((uint16_t *)p + i, d, stream);
  } else if constexpr (V == 2) {
    *(__attribute__((address_space(1))) f32x2_w *)((float *)p + i) = f32x2_w{v[0], v[1]};
  } else {
    const f32x4_t d = {v[0], v[1], v[2], v[3]};
    put<4>((float *)p + i, d, stream);
  }
}

// n / d for n < 2^20, d < 2^11 as a product: m = ceil(2^32 / d) is less than 1 too large a
// factor per n, so floor(n m / 2^32) is the quotient while n d < 2^32.
__device__ inline int quot(int n, uint32_t m, int d) { return d == 1 ? n : (int)__umulhi((uint32_t)n, m); }

struct RopePlan {
  int tokens;     // tokens of a workgroup
  int parts;      // workgroups that share a token's heads (1 where tokens > 1)
  int units;      // units of one head: turning ones first, then those that are only copied
  int turning;
  uint32_t m_units, m_token;
};

// A turning unit: V elements that form V / 2 neighbouring pairs (interleaved), or V pairs of
// V elements of each half; one pair where V = 1.  A copied unit: V elements.
template <bool BF16, int V, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void k_rope(RopeArgs a, RopePlan p) {
  __shared__ float2 s_cs[kRopeAngles];
  const int64_t s0 = (int64_t)(blockIdx.x / p.parts) * p.tokens;
  const int part = blockIdx.x % p.parts;
  const int tokens = (int)min((int64_t)p.tokens, a.S - s0);
  for (int i = threadIdx.x; i < tokens * a.half; i += kRopeThreads) {
    const int t = i / a.half, k = i - t * a.half;
    const double pos = a.pos_i64 ? (double)ldg<int64_t>((const int64_t *)a.pos + s0 + t)
                                 : (double)ldg<int32_t>((const int32_t *)a.pos + s0 + t);
    s_cs[i] = cos_sin(pos, ldg<double>(a.freqs + k), a.factor);
  }
  __syncthreads();
  const int heads = a.t[0].heads + a.t[1].heads;
  const int per_token = heads * p.units, total = tokens * per_token;
  for (int u = threadIdx.x + part * kRopeThreads; u < total; u += p.parts * kRopeThreads) {
    const int t = p.tokens == 1 ? 0 : quot(u, p.m_token, per_token);
    const int w = u - t * per_token, hd = quot(w, p.m_units, p.units), e = w - hd * p.units;
    const bool second = hd >= a.t[0].heads;
    const int h = second ? hd - a.t[0].heads : hd;
    const int64_t s = s0 + t;
    const void *x = second ? a.t[1].x : a.t[0].x;
    void *out = second ? a.t[1].out : a.t[0].out;
    const int64_t in = s * (second ? a.t[1].x_token : a.t[0].x_token) + h * (second ? a.t[1].x_head : a.t[0].x_head);
    const int64_t to = s * (second ? a.t[1].out_token : a.t[0].out_token) + h * (second ? a.t[1].out_head : a.t[0].out_head);
    if (e >= p.turning) {
      if (x == out) continue;
      int c = (e - p.turning) * V;
      if (c >= a.offset) c += 2 * a.half;
      float v[V];
      load_v<BF16, V>(x, in + c, v);
      store_v<BF16, V>(out, to + c, v, a.stream);
      continue;
    }
    // the fused operations are written out, so that every unit size gives the same bits
    auto turn = [](float2 k, float x1, float x2, float &y1, float &y2) {
      y1 = fmaf(x1, k.x, -(x2 * k.y));
      y2 = fmaf(x2, k.x, x1 * k.y);
    };
    if constexpr (INTER && V > 1) {
      float v[V], w[V];
      load_v<BF16, V>(x, in + a.offset + e * V, v);
      const float2 *cs = s_cs + t * a.half + e * (V / 2);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) turn(cs[j], v[2 * j], v[2 * j + 1], w[2 * j], w[2 * j + 1]);
      store_v<BF16, V>(out, to + a.offset + e * V, w, a.stream);
    } else {
      const int c1 = a.offset + (INTER ? 2 * e : e * V), c2 = INTER ? c1 + 1 : c1 + a.half;
      float v1[V], v2[V], w1[V], w2[V];
      load_v<BF16, V>(x, in + c1, v1);
      load_v<BF16, V>(x, in + c2, v2);
      const float2 *cs = s_cs + t * a.half + e * V;
#pragma unroll
      for (int j = 0; j < V; ++j) turn(cs[j], v1[j], v2[j], w1[j], w2[j]);
      store_v<BF16, V>(out, to + c1, w1, a.stream);
      store_v<BF16, V>(out, to + c2, w2, a.stream);
    }
  }
}

template <bool BF16, bool INTER>
void launch(const RopeArgs &a, hipStream_t st) {
  // The widest unit that divides the part, its place and the rest of a head; bf16 also
  // needs every row at a multiple of it.
  constexpr int kV = BF16 ? 8 : 4;
  auto fits = [&](int v) {
    bool ok = a.D % v == 0 && a.offset % v == 0 && (INTER && v > 1 ? 2 * a.half : a.half) % v == 0;
    if (BF16)
      for (const auto &t : a.t)
        if (t.heads)
          ok = ok && (uintptr_t)t.x % (2 * v) == 0 && (uintptr_t)t.out % (2 * v) == 0 && t.x_token % v == 0 &&
               t.x_head % v == 0 && t.out_token % v == 0 && t.out_head % v == 0;
    return ok;
  };
  const int V = fits(kV) ? kV : fits(2) ? 2 : 1;
  RopePlan p{};
  p.turning = INTER && V > 1 ? 2 * a.half / V : a.half / V;
  p.units = p.turning + (a.D - 2 * a.half) / V;
  const int per_token = (a.t[0].heads + a.t[1].heads) * p.units;
  // Tokens until a workgroup's threads all have a unit, while the angles fit and every
  // compute unit still has a few workgroups; a token shared between workgroups where
  // there are fewer tokens than that.
  p.tokens = std::max(1, std::min({kRopeThreads / per_token, kRopeAngles / a.half, a.S / 1024}));
  p.parts = std::max(1, std::min((per_token + kRopeThreads - 1) / kRopeThreads, 1024 / a.S));
  if (p.tokens > 1) p.parts = 1;
  auto magic = [](int d) { return d > 1 ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0u; };
  p.m_units = magic(p.units);
  p.m_token = magic(per_token);
  const int64_t blocks = ((int64_t)a.S + p.tokens - 1) / p.tokens * p.parts;
  const dim3 b(kRopeThreads);
  // a launch holds fewer than 2^32 threads: longer inputs go in pieces
  const int64_t most = (int64_t)(1 << 20);
  for (int64_t at = 0; at < blocks; at += most) {
    RopeArgs c = a;
    c.stream = (int64_t)a.S * (a.t[0].heads + a.t[1].heads) * a.D * (BF16 ? 2 : 4) > kStreamBytes;
    const int64_t s = at / p.parts * p.tokens;
    c.S = (int)(a.S - s);
    c.pos = (const char *)a.pos + s * (a.pos_i64 ? 8 : 4);
    for (auto &t : c.t)
      if (t.heads) {
        t.x = (const char *)t.x + s * t.x_token * (BF16 ? 2 : 4);
        t.out = (char *)t.out + s * t.out_token * (BF16 ? 2 : 4);
      }
    const dim3 g((unsigned)std::min(blocks - at, most));
    if (V == kV) MOE_LAUNCH((k_rope<BF16, kV, INTER>), g, b, 0, st, c, p);
    else if (V == 2) MOE_LAUNCH((k_rope<BF16, 2, INTER>), g, b, 0, st, c, p);
    else MOE_LAUNCH((k_rope<BF16, 1, INTER>), g, b, 0, st, c, p);
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, int x_bf16, int interleaved, hipStream_t st) {
  ProfScope ps("rope", st);
  if (x_bf16) interleaved ? launch<true, true>(a, st) : launch<true, false>(a, st);
  else interleaved ? launch<false, true>(a, st) : launch<false, false>(a, st);
  return hipGetLastError();
}

}  // namespace moe
