// Products of rows with weights, dense or grouped by expert, both operands bf16 or microscaled:
// y[i, n] = sum_k x[r(i), k] w[e(i), n, k], summed in fp32.
#include <algorithm>

#include "experts.h"
#include "tiles.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Both kinds of row meet the matrix instructions in the same bytes: a lane brings 16 of a row,
// eight bf16 or one block of 32 codes, and a block's scale.
enum Kind { kBf16, kMx };

// D (16 x 16) += A B over 64 bytes of the 16 rows of each: lane l holds bytes 16 (l / 16) .. of
// row l % 16, with the block's scale.  Sums: lane l holds rows 4 (l / 16) .. + 3 of A by row l %
// 16 of B.
template <Kind KIND>
__device__ inline f32x4 mfma16(i32x4 a, i32x4 b, int sa, int sb, f32x4 c) {
  if constexpr (KIND == kMx) {
    // of the eight registers that e2m1 operands share with wider types the first four count
    const i32x8 A = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 B = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, sa, 0, sb);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
}

// Bytes [k, k + 16) of a row, zeros beyond its end.
template <Kind KIND>
__device__ inline i32x4 chunk_at(const uint8_t *row, int k, int row_bytes) {
  if constexpr (KIND == kMx) {
    if (k >= row_bytes) return i32x4{0, 0, 0, 0};
    return load16<true>((const int8_t *)row + k);
  } else {
    return load16_tail((const int8_t *)row, k, row_bytes);
  }
}
// The scale of the block at byte k of a row.
__device__ inline int scale_at(const uint8_t *row, int k, int row_bytes) {
  return k < row_bytes ? ldg<uint8_t>(row + (k >> 4)) : 0;
}

// ---- where a tile lies --------------------------------------------------------------------
// Tiles of `rows` rows never cross experts.  They are counted on the GPU, by each wave for
// itself: a lane adds up the tiles of its share of the experts, a scan over the lanes finds the
// expert of tile `t` (of `cols` column tiles for each row tile; an expert's tiles are neighbours).
struct Where {
  int expert, lo, hi;  // its rows
  int tile, tiles;     // the row tile within the expert, of how many
  int col;
};

__device__ inline int tiles_in(const ProdArgs &a, int e, int rows, int &lo, int &hi) {
  lo = min(max(ldg<int32_t>(a.first + e), 0), a.T);
  hi = min(max(ldg<int32_t>(a.first + e + 1), 0), a.T);
  return hi > lo ? (hi - lo + rows - 1) / rows : 0;
}

// False where there is no tile t.
__device__ inline bool locate(const ProdArgs &a, int t, int rows, int cols, Where &w) {
  int before = 0;  // row tiles of the experts ahead
  if (!a.first) {
    w.expert = 0; w.lo = 0; w.hi = a.T;
    w.tiles = (a.T + rows - 1) / rows;
    if (t >= w.tiles * cols) return false;
  } else {
    const int lane = threadIdx.x & 63, share = (a.E + 63) / 64;
    int n = 0, lo, hi;
    for (int i = 0; i < share; ++i) {
      const int e = lane * share + i;
      if (e < a.E) n += tiles_in(a, e, rows, lo, hi);
    }
    int scan = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(scan, o);
      if (lane >= o) scan += up;
    }
    const int total = __builtin_amdgcn_readlane(scan, 63), want = t / cols;
    if (want >= total) return false;
    const int at = 63 - __builtin_clzll(__ballot(scan - n <= want));  // the last lane that starts at or ahead of it
    before = __builtin_amdgcn_readlane(scan - n, at);
    int e = at * share;
    for (;; ++e) {  // ends: the lane's experts hold the tile
      w.tiles = __builtin_amdgcn_readfirstlane(tiles_in(a, e, rows, lo, hi));
      if (want < before + w.tiles || e + 1 >= a.E) break;
      before += w.tiles;
    }
    w.expert = e;
    w.lo = __builtin_amdgcn_readfirstlane(lo);
    w.hi = __builtin_amdgcn_readfirstlane(hi);
  }
  const int in = t - before * cols;
  w.col = in / w.tiles;
  w.tile = in % w.tiles;
  return true;
}

// The row of x that row i of y is computed from, -1 where there is none.
__device__ inline int source_of(const ProdArgs &a, int i) {
  int r = i;
  if (a.order) {
    const int p = ldg<int32_t>(a.order + i);
    r = p < 0 ? -1 : p / a.top_k;
  }
  return (uint32_t)r < (uint32_t)a.x_rows ? r : -1;
}

// Four neighbouring outputs y[i, n .. n + 3], those below N, past the caches where STREAM.
template <bool STREAM>
__device__ inline void store4(const ProdArgs &a, int64_t i, int n, f32x4 v) {
  if (a.y_vec && n + 4 <= a.N) {
    if (a.y_bf16) {
      auto *to = (__attribute__((address_space(1))) uint64_t *)((uint16_t *)a.y + i * a.ldy + n);
      const uint64_t both = ((uint64_t)pack2_bf16(v[2], v[3]) << 32) | pack2_bf16(v[0], v[1]);
      if constexpr (STREAM) __builtin_nontemporal_store(both, to);
      else *to = both;
    } else {
      auto *to = (__attribute__((address_space(1))) f32x4_t *)((float *)a.y + i * a.ldy + n);
      if constexpr (STREAM) __builtin_nontemporal_store((f32x4_t)v, to);
      else *to = (f32x4_t)v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < a.N) {
        if (a.y_bf16) store_el<true>(a.y, i * a.ldy + n + j, v[j]);
        else store_el<false>(a.y, i * a.ldy + n + j, v[j]);
      }
  }
}

// ---- straight from memory -----------------------------------------------------------------
// A workgroup takes 16 weight rows and 16 NT rows of one expert; its W waves share out the row's
// steps of 64 bytes and add their sums in LDS in a fixed order.
template <Kind KIND, int NT, int W>
__global__ __launch_bounds__(64 * W) void k_product_few(ProdArgs a, int cols) {
  __shared__ f32x4 s_acc[W][NT][64];
  Where at;
  if (!locate(a, blockIdx.x, 16 * NT, cols, at)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = at.col * 16, i0 = at.lo + at.tile * 16 * NT;
  const int row = lane & 15, kq = (lane >> 4) * 16;
  const int n = min(n0 + row, a.N - 1);
  const uint8_t *w = a.w + at.expert * a.expert + n * a.ldw, *we = nullptr;
  if constexpr (KIND == kMx) we = a.we + at.expert * a.expert_e + n * a.ldwe;
  const uint8_t *x[NT], *xe[NT];
  int src[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    src[t] = source_of(a, min(i0 + 16 * t + row, at.hi - 1));
    x[t] = a.x + max(src[t], 0) * a.ldx;
    if constexpr (KIND == kMx) xe[t] = a.xe + max(src[t], 0) * a.ldxe;
  }
  f32x4 acc[NT] = {};
  const int steps = (a.row_bytes + 63) / 64;
  const int lo = (int)((int64_t)steps * wave / W), hi = (int)((int64_t)steps * (wave + 1) / W);
#pragma unroll 2
  for (int s = lo; s < hi; ++s) {
    const int k = s * 64 + kq;
    const i32x4 A = chunk_at<KIND>(w, k, a.row_bytes);
    int sa = 0;
    if constexpr (KIND == kMx) sa = scale_at(we, k, a.row_bytes);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const i32x4 B = chunk_at<KIND>(x[t], k, a.row_bytes);
      int sb = 0;
      if constexpr (KIND == kMx) sb = scale_at(xe[t], k, a.row_bytes);
      acc[t] = mfma16<KIND>(A, B, sa, sb, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) s_acc[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < NT; t += W) {
    f32x4 sum = s_acc[0][t][lane];
#pragma unroll
    for (int v = 1; v < W; ++v) sum += s_acc[v][t][lane];
    const int i = i0 + 16 * t + row, to = n0 + (lane >> 4) * 4;
    if (src[t] < 0) sum = f32x4{__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
    if (i < at.hi && to < a.N) store4<false>(a, i, to, sum);
  }
}

// Row tiles of `rows` rows that T rows of E experts can make.
int64_t most_tiles(const ProdArgs &a, int rows) {
  const int64_t whole = (a.T + rows - 1) / rows;
  return a.first ? a.T / rows + std::min(a.E, a.T) : whole;
}

template <Kind KIND, int NT>
void launch_few(const ProdArgs &a, hipStream_t st) {
  constexpr int W = 8;
  const int cols = (a.N + 15) / 16;
  MOE_LAUNCH((k_product_few<KIND, NT, W>), dim3((unsigned)(most_tiles(a, 16 * NT) * cols)), dim3(64 * W), 0, st, a, cols);
}

}  // namespace

int64_t product_workspace(const ProdArgs &a, bool mx) { return 0; }

hipError_t launch_product(const ProdArgs &a0, bool mx, hipStream_t st) {
  ProdArgs a = a0;
  const int ys = a.y_bf16 ? 2 : 4;
  a.y_vec = (uintptr_t)a.y % (a.y_bf16 ? 8 : 16) == 0 && a.ldy % 4 == 0;
  a.stream = (int64_t)a.T * a.N * ys > kStreamBytes;
  // a launch holds fewer than 2^32 threads: many weight rows go in pieces
  const int64_t step = std::max<int64_t>(1, ((int64_t)1 << 22) / most_tiles(a, 16)) * 16;
  for (int64_t n = 0; n < a.N; n += step) {
    ProdArgs c = a;
    c.N = (int)std::min<int64_t>(step, a.N - n);
    c.w += n * a.ldw;
    if (mx) c.we += n * a.ldwe;
    c.y = (char *)a.y + n * ys;
    ProfScope ps(mx ? "mx_product_few" : "product_few", st);
    if (mx) launch_few<kMx, 1>(c, st);
    else launch_few<kBf16, 1>(c, st);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
