// Product of int8 rows with int8 weights: y[s, n] = (sum_k q[s, k] w[n, k]) * (d[s] * dw[n]),
// the sum exact in int32.
#include "dense.h"

namespace moe {
namespace {

// One wave per output.
__global__ __launch_bounds__(256) void k_qmm_plain(QmmArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t n_out = (int64_t)a.S * a.N;
  for (int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); o < n_out; o += (int64_t)gridDim.x * 4) {
    const int64_t s = o / a.N, n = o - s * a.N;
    const int8_t *q = a.q + s * a.ldq, *w = a.w + n * a.ldw;
    int sum = 0;
    for (int k = lane; k < a.K; k += 64) sum += (int)ldg<int8_t>(q + k) * (int)ldg<int8_t>(w + k);
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
    if (lane == 0) {
      const float v = (float)sum * (a.d[s] * a.dw[n]);
      if (a.y_bf16) stg<uint16_t>((uint16_t *)a.y + s * a.ldy + n, f_bf16(v));
      else stg<float>((float *)a.y + s * a.ldy + n, v);
    }
  }
}

}  // namespace

int64_t qmatmul_workspace(int, int, int) { return 0; }

hipError_t launch_qmatmul(const QmmArgs &a, hipStream_t st) {
  ProfScope ps("qmatmul", st);
  const int64_t blocks = ((int64_t)a.S * a.N + 3) / 4;
  MOE_LAUNCH(k_qmm_plain, dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace moe
