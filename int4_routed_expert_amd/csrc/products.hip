// Products of rows with weights, dense or grouped by expert, both operands bf16 or microscaled:
// y[i, n] = sum_k x[r(i), k] w[e(i), n, k], summed in fp32.
#include <algorithm>
#include <type_traits>

#include "experts.h"
#include "tiles.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
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

// The same of 32 rows each over 32 bytes: lane l holds 16 bytes of row l % 32, lanes 32 .. 63 the
// other 16; sums as v_mfma_i32_32x32x32_i8's (qmatmul.hip).  Each lane's scale is byte `step` of sa
// or sb.
template <Kind KIND>
__device__ inline f32x16 mfma32(i32x4 a, i32x4 b, int sa, int sb, int step, f32x16 c) {
  if constexpr (KIND == kMx) {
    const i32x8 A = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 B = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    switch (step) {
      case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, 0, sa, 0, sb);
      case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, 1, sa, 1, sb);
      case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, 2, sa, 2, sb);
      default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, 3, sa, 3, sb);
    }
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
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
// block's expert (there are `cols` column tiles for each row tile).
struct Where {
  int expert, lo, hi;  // its rows
  int tile, tiles;     // the row tile within the expert, of how many (> 0)
  int col;
};

struct Range {
  int lo, hi;
  __device__ int tiles(int rows) const { return hi > lo ? (hi - lo + rows - 1) / rows : 0; }
};
__device__ inline Range range_of(const ProdArgs &a, int e) {
  return {min(max(ldg<int32_t>(a.first + e), 0), a.T), min(max(ldg<int32_t>(a.first + e + 1), 0), a.T)};
}

// Blocks go to the XCDs round-robin; each XCD gets a contiguous run of tiles, so that those in
// flight on it share weights, and within an expert rows, in its L2.  An expert's tiles go in strips of
// kStrip row tiles, column by column.  False where there is no tile for the block.
constexpr int kStrip = 4;
__device__ inline bool locate(const ProdArgs &a, int block, int rows, int cols, Where &w) {
  const int lane = threadIdx.x & 63, share = (a.E + 63) / 64;
  int total = (a.T + rows - 1) / rows, n = 0, scan = 0;
  if (a.first) {
    for (int i = 0; i < share; ++i) {
      const int e = lane * share + i;
      if (e < a.E) n += range_of(a, e).tiles(rows);
    }
    scan = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(scan, o);
      if (lane >= o) scan += up;
    }
    total = __builtin_amdgcn_readlane(scan, 63);
  }
  const int per = (total * cols + kXcds - 1) / kXcds;
  const int t = block % kXcds * per + block / kXcds;
  if (block / kXcds >= per || t >= total * cols) return false;
  int before = 0;  // row tiles of the experts ahead
  if (a.first) {
    const int want = t / cols;
    const int at = 63 - __builtin_clzll(__ballot(scan - n <= want));  // the last lane that starts at or ahead of it
    before = __builtin_amdgcn_readlane(scan - n, at);
    int e = at * share;
    Range r = range_of(a, e);
    while (want >= before + r.tiles(rows) && e + 1 < a.E) {  // ends: the lane's experts hold the tile
      before += r.tiles(rows);
      r = range_of(a, ++e);
    }
    w.expert = e;
    w.lo = __builtin_amdgcn_readfirstlane(r.lo);
    w.hi = __builtin_amdgcn_readfirstlane(r.hi);
    w.tiles = r.tiles(rows);
  } else {
    w.expert = 0; w.lo = 0; w.hi = a.T; w.tiles = total;
  }
  const int in = t - before * cols, strip = in / (kStrip * cols), left = in - strip * kStrip * cols;
  const int g = min(kStrip, w.tiles - strip * kStrip);
  w.tile = strip * kStrip + left % g;
  w.col = left / g;
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

__device__ inline f32x4 nan4() {
  const float n = __builtin_nanf("");
  return f32x4{n, n, n, n};
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
    if (src[t] < 0) sum = nan4();
    if (i < at.hi && to < a.N) store4<false>(a, i, to, sum);
  }
}

// ---- through LDS ----------------------------------------------------------------------------
// A workgroup takes BN weight rows x BS rows of one expert, its WN x WS waves each their part in
// blocks of 32 x 32; both operands go through LDS in stages of kBK bytes of K, NBUF of them, as in
// the int8 product (qmatmul.hip, where the pipeline is described: 16 bytes a lane and 32 cycles an
// instruction are the same).  Microscaled rows add a byte a block: 16 of a row, two stages'
// worth, are one load into LDS, and a lane reads the four of its blocks of a stage as one word, of
// which each instruction takes one byte.  For that a lane's blocks are neighbours: lanes 0 .. 31
// take blocks 0 .. 3 of a stage's eight, lanes 32 .. 63 blocks 4 .. 7, in both operands.
constexpr int kScBlocks = 16;  // scales of a row that are loaded at once

template <Kind KIND, int BN, int BS, int WN, int WS, int NBUF>
__global__ __launch_bounds__(64 * WN * WS) void k_product_tile(ProdArgs a, int cols) {
  constexpr int kThr = 64 * WN * WS;
  constexpr int TN = BN / WN / 32, TS = BS / WS / 32;  // 32x32 blocks of a wave
  constexpr int kRows = BN + BS, kStage = kRows * kBK;
  constexpr int kPer = kStage / 16 / kThr;  // chunks a thread moves per stage
  static_assert(kStage % (16 * kThr) == 0 && NBUF % 2 == 0, "stage split");
  constexpr bool kMicro = KIND == kMx;
  constexpr int kSc = kMicro ? (kRows + kThr - 1) / kThr : 0;  // scale loads of a thread per two stages
  constexpr int kScSize = kSc * kThr * kScBlocks;
  constexpr int kWide = BN / WN, kLd = kWide + 4;  // a wave's weights, and what a row's sums of them take in LDS
  constexpr int kTurn = WN * WS * 32 * kLd * 4, kEnd = kTurn + BS * 4;
  constexpr int kLds = std::max(NBUF * kStage + NBUF * kScSize, kEnd);
  __shared__ __align__(128) uint8_t s_buf[kLds];
  Where at;
  if (!locate(a, blockIdx.x, BS, cols, at)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave / WS, wsv = wave % WS;
  const int n0 = at.col * BN, i0 = at.lo + at.tile * BS;

  // row r of the tile: of the weights, or of x
  auto row_of = [&](int r) __attribute__((always_inline)) {
    return r < BN ? min(n0 + r, a.N - 1) : max(source_of(a, min(i0 + r - BN, at.hi - 1)), 0);
  };
  // this thread's chunks of a stage: LDS position tid + i kThr, which holds chunk c of row r
  const uint8_t *src[kPer], *sc[kSc + 1];
  int kc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    constexpr int kC = kBK / 16;
    const int p = tid + i * kThr, r = p / kC;
    kc[i] = ((p % kC) ^ mix_of(r)) << 4;
    src[i] = (r < BN ? a.w + at.expert * a.expert + row_of(r) * a.ldw : a.x + row_of(r) * a.ldx) + kc[i];
  }
#pragma unroll
  for (int i = 0; i < kSc; ++i) {
    const int r = min(tid + i * kThr, kRows - 1);
    sc[i] = r < BN ? a.we + at.expert * a.expert_e + row_of(r) * a.ldwe : a.xe + row_of(r) * a.ldxe;
  }
  const int stages = (a.row_bytes + kBK - 1) / kBK, whole = a.row_bytes / kBK;
  const int sc_bytes = a.row_bytes / 16;

  f32x16 acc[TN][TS];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TS; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  const int row = lane & 31, ck = lane >> 5;
  constexpr int kSteps = kBK / 32;
  int at_w[kSteps], at_x[kSteps];
#pragma unroll
  for (int kk = 0; kk < kSteps; ++kk) {
    at_w[kk] = chunk_of(wn * kWide + row, ck * kSteps + kk);
    at_x[kk] = chunk_of(BN + wsv * (BS / WS) + row, ck * kSteps + kk);
  }
  constexpr int kF = TN + TS, kM = TN * TS;
  auto frag = [&](const uint8_t *buf, int f, int kk) __attribute__((always_inline)) {
    return *(const i32x4 *)(buf + (f < TN ? at_w[kk] + f * 32 * kBK : at_x[kk] + (f - TN) * 32 * kBK));
  };
  const uint8_t *s_sc = s_buf + NBUF * kStage;
  const int sc_w = (wn * kWide + row) * kScBlocks + ck * 4, sc_x = (BN + wsv * (BS / WS) + row) * kScBlocks + ck * 4;
  // the scales of fragment f in the stage whose scales lie at `from`
  auto scale = [&](int f, int from) __attribute__((always_inline)) {
    return *(const int *)(s_sc + from + (f < TN ? sc_w + f * 32 * kScBlocks : sc_x + (f - TN) * 32 * kScBlocks));
  };

  const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)s_buf + wave * 1024);
  auto clip = [&](int s) __attribute__((always_inline)) {  // before stage s is requested
    if (s >= whole) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if ((int64_t)s * kBK + kc[i] >= a.row_bytes) src[i] = g_zeros;
    }
    if constexpr (kMicro) {
      if (s % 2 == 0 && s * 8 >= sc_bytes) {
#pragma unroll
        for (int i = 0; i < kSc; ++i) sc[i] = g_zeros;
      }
    }
  };
  auto request = [&](int i, int buffer) __attribute__((always_inline)) {
    load_to_lds((const int8_t *)src[i], lds, buffer * kStage + i * kThr * 16);
    src[i] += kBK;
  };
  // The scales of stages s and s + 1 (s even), with the requests of stage s.  A buffer of scales is
  // written again NBUF pairs of stages later, when its last readers have met twice.
  auto request_scales = [&](int s) __attribute__((always_inline)) {
    if constexpr (kMicro) {
#pragma unroll
      for (int i = 0; i < kSc; ++i) {
        load_to_lds((const int8_t *)sc[i], lds + (s / 2 % NBUF) * kScSize, NBUF * kStage + i * kThr * 16);
        sc[i] += kScBlocks;
      }
    }
  };
  constexpr int kG = kM >= 8 ? 1 : kM >= 4 ? 2 : 4, kGroups = kSteps / kG;
  constexpr int kSpread = kGroups > 1 ? 2 : 1;
  // Requests in flight behind the stage that is waited for: the NBUF - 2 stages after it, half of which
  // are even and bring scales.
  constexpr int kBehind = (NBUF - 2) * kPer + (NBUF - 2) / 2 * kSc;
#pragma unroll
  for (int s = 0; s < NBUF; ++s) {
    clip(s);
    if (s % 2 == 0) request_scales(s);
#pragma unroll
    for (int i = 0; i < (s < NBUF - 1 ? kPer : kPer / kSpread); ++i) request(i, s);
  }
  wait_and_meet<kBehind + kPer / kSpread>();
  i32x4 F[2][kG][kF];
  int S[2][kF] = {};
#pragma unroll
  for (int f = 0; f < kG * kF; ++f) F[0][f / kF][f % kF] = frag(s_buf, f % kF, f / kF);
  if constexpr (kMicro) {
#pragma unroll
    for (int f = 0; f < kF; ++f) S[0][f] = scale(f, 0);
  }
  // Multiply group `now` of a stage (its fragments F[cur], its scales S[sn]) while the fragments of
  // group g in `buffer` are read, and with g = 0 the next stage's scales, which lie at sc_from; buffer
  // `again` is requested meanwhile.
  auto multiply = [&](int cur, int sn, int now, int buffer, int g, int sc_from, int again, int r0, int r1)
      __attribute__((always_inline)) {
    constexpr int kAll = kG * kM;
#pragma unroll
    for (int m = 0; m < kAll; ++m) {
#pragma unroll
      for (int f = 0; f < kG * kF; ++f)
        if (f * kAll / (kG * kF) == m) F[cur ^ 1][f / kF][f % kF] = frag(s_buf + buffer * kStage, f % kF, g * kG + f / kF);
      if constexpr (kMicro) {
#pragma unroll
        for (int f = 0; f < kF; ++f)
          if (g == 0 && f * kAll / kF == m) S[sn ^ 1][f] = scale(f, sc_from);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i >= r0 && i < r1 && (i - r0) * kAll / (r1 - r0) == m) request(i, again);
      const int k = m / kM, i = m % kM / TS, j = m % TS;
      acc[i][j] = mfma32<KIND>(F[cur][k][i], F[cur][k][TN + j], S[sn][i], S[sn][TN + j], now * kG + k, acc[i][j]);
      // the compiler moves scaled products together, past the barrier below: 256 x 256 tiles spill then
      if constexpr (kMicro) asm volatile("" : "+a"(acc[i][j]));
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto stage = [&](int s, int b) __attribute__((always_inline)) {  // stage s, in buffer b
    const int cur = b * kGroups & 1, sn = b & 1;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
      multiply((cur + g - 1) & 1, sn, g - 1, b, g, 0, (b + NBUF - 1) % NBUF, g < kSpread ? kPer * g / kSpread : 0,
               g < kSpread ? kPer * (g + 1) / kSpread : 0);
    }
    wait_and_meet<kBehind>();
    clip(s + NBUF);
    if (b % 2 == 0) request_scales(s + NBUF);
    multiply((cur + kGroups - 1) & 1, sn, kGroups - 1, (b + 1) % NBUF, 0, ((s + 1) / 2 % NBUF) * kScSize + (b + 1) % 2 * 8, b, 0,
             kPer / kSpread);
  };
  int s = 0;
  for (; s + NBUF <= stages; s += NBUF) {
#pragma unroll
    for (int b = 0; b < NBUF; ++b) stage(s + b, b);
  }
#pragma unroll
  for (int b = 0; b < NBUF - 1; ++b)
    if (s + b < stages) stage(s + b, b);
  wait_and_meet<0>();  // the last requests, beyond K, have arrived too
  // Each wave turns its sums round in its own part of the buffers, 32 rows at a time, so that they
  // leave as runs of a row's neighbouring outputs.
  int *s_src = (int *)(s_buf + kTurn);
  if (a.order) {
    for (int i = tid; i < BS; i += kThr) s_src[i] = source_of(a, min(i0 + i, at.hi - 1));
    __syncthreads();
  }
  float *out = (float *)s_buf + wave * 32 * kLd;
  constexpr int kRun = kWide / 4, kTok = 64 / kRun;  // lanes of a row's run, rows at a time
#pragma unroll
  for (int j = 0; j < TS; ++j) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(f32x4 *)(out + row * kLd + i * 32 + 8 * e + 4 * ck) =
            f32x4{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
    own_lds_done();
    const int n = n0 + wn * kWide + (lane % kRun) * 4;
    auto leave = [&](auto stream) __attribute__((always_inline)) {
#pragma unroll 4
      for (int r = lane / kRun; r < 32; r += kTok) {
        const int sl = wsv * (BS / WS) + j * 32 + r;
        f32x4 v = *(const f32x4 *)(out + r * kLd + (lane % kRun) * 4);
        if (i0 + sl < at.hi && n < a.N) {
          if (a.order && s_src[sl] < 0) v = nan4();
          store4<decltype(stream)::value>(a, i0 + sl, n, v);
        }
      }
    };
    if (a.stream) leave(std::true_type());
    else leave(std::false_type());
    own_lds_done();
  }
}

// ---- rows on 16-byte boundaries -------------------------------------------------------------
// Copies rows to the workspace, each at a multiple of 16 bytes and filled up with zeros to one: the
// loads into LDS need that.  A lane moves 16 bytes.  Rows of experts that have none to compute are
// left out.
struct Copy {
  const uint8_t *from;
  uint8_t *to;
  int64_t ld, expert;  // bytes between the source's rows and experts
  int64_t begin, end;  // 16-byte pieces of this launch
  int N, row_bytes, chunks;
};
constexpr int kCopyThreads = 256;
__global__ __launch_bounds__(kCopyThreads) void k_product_align(ProdArgs a, Copy c) {
  const int64_t block0 = c.begin + (int64_t)blockIdx.x * kCopyThreads;
  const int64_t r0 = block0 / c.chunks;
  const uint32_t u = (uint32_t)(block0 - r0 * c.chunks) + threadIdx.x;
  if (block0 + threadIdx.x >= c.end) return;
  const int64_t r = r0 + u / c.chunks;
  const int k = (int)(u % c.chunks) * 16;
  const int64_t e = r / c.N;
  if (a.first && c.expert && ldg<int32_t>(a.first + e) >= ldg<int32_t>(a.first + e + 1)) return;
  const i32x4 v = load16_tail((const int8_t *)c.from + e * c.expert + (r - e * c.N) * c.ld, k, c.row_bytes);
  stg<uint4>(c.to + (block0 + threadIdx.x) * 16, make_uint4((uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]));
}

// ---- which kernel ---------------------------------------------------------------------------
enum ProdKernel { kFew16, kFew32, kTile64, kTile128, kTile256 };
constexpr int kRowsOf[] = {16, 32, 64, 128, 256};

struct ProdPlan {
  ProdKernel kernel;
  bool copy_x, copy_w;  // the operand that the tiles cannot read as it lies: bf16 rows, or scales
  int64_t ld, bytes_x, bytes;  // of the copies: a row, the rows of x, all
};

bool on16(const void *p, int64_t ld, int64_t rows, int64_t expert, int E) {
  return (uintptr_t)p % 16 == 0 && (rows == 1 || ld % 16 == 0) && (E == 1 || expert % 16 == 0);
}

ProdPlan plan_of(const ProdArgs &a, bool mx) {
  ProdPlan p{};
  const int busy = a.first ? std::min(a.E, a.T) : 1;
  const double rows = (double)a.T / busy;
  p.kernel = rows < 16 ? kFew16 : rows < 40 ? kFew32 : rows < 100 ? kTile64 : rows < 400 ? kTile128 : kTile256;
  if (p.kernel >= kTile64) {
    const int64_t row = mx ? a.row_bytes / 16 : a.row_bytes;
    const bool even = row % 16 == 0;
    p.copy_x = !even || !(mx ? on16(a.xe, a.ldxe, a.x_rows, 0, 1) : on16(a.x, a.ldx, a.x_rows, 0, 1));
    p.copy_w = !even || !(mx ? on16(a.we, a.ldwe, a.N, a.expert_e, a.E) : on16(a.w, a.ldw, a.N, a.expert, a.E));
    p.ld = (row + 15) / 16 * 16;
    p.bytes_x = p.copy_x ? a.x_rows * p.ld : 0;
    p.bytes = p.bytes_x + (p.copy_w ? (int64_t)a.E * a.N * p.ld : 0);
  }
  return p;
}

// Row tiles of `rows` rows that T rows of E experts can make.
int64_t most_tiles(const ProdArgs &a, int rows) {
  const int64_t whole = ((int64_t)a.T + rows - 1) / rows;
  return a.first ? a.T / rows + std::min(a.E, a.T) : whole;
}
unsigned blocks_of(const ProdArgs &a, int rows, int cols) {
  return (unsigned)((most_tiles(a, rows) * cols + kXcds - 1) / kXcds * kXcds);
}

template <Kind KIND, int NT>
void launch_few(const ProdArgs &a, hipStream_t st) {
  constexpr int W = 8;
  const int cols = (a.N + 15) / 16;
  MOE_LAUNCH((k_product_few<KIND, NT, W>), dim3(blocks_of(a, 16 * NT, cols)), dim3(64 * W), 0, st, a, cols);
}
template <Kind KIND, int BN, int BS, int WN, int WS, int NBUF>
void launch_tile(const ProdArgs &a, hipStream_t st) {
  const int cols = (a.N + BN - 1) / BN;
  MOE_LAUNCH((k_product_tile<KIND, BN, BS, WN, WS, NBUF>), dim3(blocks_of(a, BS, cols)), dim3(64 * WN * WS), 0, st, a, cols);
}

template <Kind KIND>
void launch_piece(const ProdArgs &a, ProdKernel k, hipStream_t st) {
  switch (k) {
    case kFew16: launch_few<KIND, 1>(a, st); break;
    case kFew32: launch_few<KIND, 2>(a, st); break;
    case kTile64: launch_tile<KIND, 128, 64, 2, 2, 4>(a, st); break;
    case kTile128: launch_tile<KIND, 128, 128, 2, 2, 2>(a, st); break;
    case kTile256: launch_tile<KIND, 256, 256, 2, 2, 2>(a, st); break;
  }
}

hipError_t launch_copy(const ProdArgs &a, const uint8_t *from, uint8_t *to, int64_t ld, int64_t expert, int64_t rows, int N,
                       int row_bytes, hipStream_t st) {
  Copy c{from, to, ld, expert, 0, 0, N, row_bytes, (row_bytes + 15) / 16};
  const int64_t units = rows * c.chunks;
  constexpr int64_t kMost = (int64_t)1 << 30;  // a launch holds fewer than 2^32 threads
  for (c.begin = 0; c.begin < units; c.begin += kMost) {
    c.end = std::min(units, c.begin + kMost);
    ProfScope ps("product_align", st);
    MOE_LAUNCH(k_product_align, dim3((unsigned)((c.end - c.begin + kCopyThreads - 1) / kCopyThreads)), dim3(kCopyThreads), 0, st, a, c);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace

int64_t product_workspace(const ProdArgs &a, bool mx) { return plan_of(a, mx).bytes; }

hipError_t launch_product(const ProdArgs &a0, bool mx, hipStream_t st) {
  ProdArgs a = a0;
  const int ys = a.y_bf16 ? 2 : 4;
  a.y_vec = (uintptr_t)a.y % (a.y_bf16 ? 8 : 16) == 0 && a.ldy % 4 == 0;
  a.stream = (int64_t)a.T * a.N * ys > kStreamBytes;
  const ProdPlan p = plan_of(a, mx);
  const int row = mx ? a.row_bytes / 16 : a.row_bytes;
  if (p.copy_x) {
    const hipError_t err = launch_copy(a, mx ? a.xe : a.x, a.ws, mx ? a.ldxe : a.ldx, 0, a.x_rows, a.x_rows, row, st);
    if (err != hipSuccess) return err;
    (mx ? a.xe : a.x) = a.ws;
    (mx ? a.ldxe : a.ldx) = p.ld;
  }
  if (p.copy_w) {
    uint8_t *to = a.ws + p.bytes_x;
    const hipError_t err = launch_copy(a, mx ? a.we : a.w, to, mx ? a.ldwe : a.ldw, mx ? a.expert_e : a.expert,
                                       (int64_t)a.E * a.N, a.N, row, st);
    if (err != hipSuccess) return err;
    (mx ? a.we : a.w) = to;
    (mx ? a.ldwe : a.ldw) = p.ld;
    (mx ? a.expert_e : a.expert) = (int64_t)a.N * p.ld;
  }
  if (!mx && (p.copy_x || p.copy_w)) a.row_bytes = (int)p.ld;
  // A launch holds fewer than 2^32 threads: many weight rows go in pieces.  (Tiles of 16 rows, of 16
  // weight rows and 512 threads each, are for up to 16 rows an expert, so that the quotient is at least 1.)
  const int64_t step = std::max<int64_t>(1, ((int64_t)1 << 18) / most_tiles(a, kRowsOf[p.kernel])) * 256;
  for (int64_t n = 0; n < a.N; n += step) {
    ProdArgs c = a;
    c.N = (int)std::min<int64_t>(step, a.N - n);
    c.w += n * a.ldw;
    if (mx) c.we += n * a.ldwe;
    c.y = (char *)a.y + n * ys;
    static constexpr const char *kNames[] = {"product_few16", "product_few32", "product_tile64", "product_tile128", "product_tile256"};
    ProfScope ps(kNames[p.kernel], st);
    if (mx) launch_piece<kMx>(c, p.kernel, st);
    else launch_piece<kBf16>(c, p.kernel, st);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
