// Rotary positions: pair i of a head turns by a = pos * freqs[i].
//   (x1, x2) -> factor * (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
#include "dense.h"

namespace moe {
namespace {

// One thread per (token, head, pair); its threads also copy what lies outside the part.
template <bool BF16>
__global__ __launch_bounds__(256) void k_rope_pairs(RopeArgs a, int interleaved) {
  for (int64_t s = blockIdx.x; s < a.S; s += gridDim.x) {
    const double pos = a.pos_i64 ? (double)((const int64_t *)a.pos)[s] : (double)((const int32_t *)a.pos)[s];
    for (int ti = 0; ti < 2; ++ti) {
      const moe_rope_tensor &t = a.t[ti];
      for (int u = threadIdx.x; u < t.heads * a.half; u += blockDim.x) {
        const int hd = u / a.half, i = u - hd * a.half;
        const int c1 = a.offset + (interleaved ? 2 * i : i), c2 = interleaved ? c1 + 1 : c1 + a.half;
        const int64_t in = s * t.x_token + hd * t.x_head, out = s * t.out_token + hd * t.out_head;
        const double w = pos * a.freqs[i];
        const float c = a.factor * (float)cos(w), sn = a.factor * (float)sin(w);
        const float x1 = load_el<BF16>(t.x, in + c1), x2 = load_el<BF16>(t.x, in + c2);
        store_el<BF16>(t.out, out + c1, x1 * c - x2 * sn);
        store_el<BF16>(t.out, out + c2, x2 * c + x1 * sn);
      }
      const int rest = a.D - 2 * a.half;
      if (t.x != t.out)
        for (int u = threadIdx.x; u < t.heads * rest; u += blockDim.x) {
          const int hd = u / rest, i = u - hd * rest;
          const int c = i < a.offset ? i : i + 2 * a.half;
          store_el<BF16>(t.out, s * t.out_token + hd * t.out_head + c,
                         load_el<BF16>(t.x, s * t.x_token + hd * t.x_head + c));
        }
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, int x_bf16, int interleaved, hipStream_t st) {
  ProfScope ps("rope", st);
  const dim3 g((unsigned)std::min(a.S, 1 << 20)), b(256);
  if (x_bf16) MOE_LAUNCH(k_rope_pairs<true>, g, b, 0, st, a, interleaved);
  else MOE_LAUNCH(k_rope_pairs<false>, g, b, 0, st, a, interleaved);
  return hipGetLastError();
}

}  // namespace moe
