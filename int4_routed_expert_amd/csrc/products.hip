// Products of rows with weights, dense or grouped by expert, both operands bf16 or microscaled:
// y[i, n] = sum_k x[r(i), k] w[e(i), n, k], summed in fp32.
#include <algorithm>
#include <cmath>
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

// The scale of the block at byte k of a row.
__device__ inline int scale_at(const uint8_t *row, int k, int row_bytes) {
  return k < row_bytes ? ldg<uint8_t>(row + (k >> 4)) : 0;
}

// ---- where a tile lies --------------------------------------------------------------------
// Tiles of `rows` rows that never cross experts, `cols` of them side by side for each.  They are
// counted on the GPU, by each wave for itself: a lane adds up the row tiles of its share of the
// experts, and a scan over the lanes says where that share begins.
struct Where {
  int expert, lo, hi;  // its rows
  int tile, col;       // the row tile within the expert, the column tile
};

struct Range {
  int lo, hi;
  __device__ int tiles(int rows) const { return hi > lo ? (hi - lo + rows - 1) / rows : 0; }
};
// Blocks go to the XCDs round-robin; each XCD gets a contiguous run of tiles, so that those in
// flight on it share weights, and within an expert rows, in its L2.  An expert's tiles go in strips of
// kStrip row tiles, column by column.
constexpr int kStrip = 4;
struct Tiles {
  int rows, cols, share;
  int n, from;  // this lane's row tiles, and those ahead of them
  int per;      // tiles of an XCD
  int total;
  __device__ inline __attribute__((always_inline)) Tiles(const ProdArgs &a, int rows, int cols) : rows(rows), cols(cols), share((a.E + 63) / 64), n(0), from(0) {
    if (a.first) {
      const int lane = threadIdx.x & 63;
      for (int i = 0; i < share; ++i) {
        const int e = lane * share + i;
        if (e < a.E) n += Range{bound(a, ldg<int32_t>(a.first + e)), bound(a, ldg<int32_t>(a.first + e + 1))}.tiles(rows);
      }
      from = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(from, o);
        if (lane >= o) from += up;
      }
      // (a `first` that decreases can describe rows many times over)
      total = (int)min((int64_t)__builtin_amdgcn_readlane(from, 63) * cols, (int64_t)1 << 30);
      from -= n;
    } else {
      total = (a.T + rows - 1) / rows * cols;
    }
    per = (total + kXcds - 1) / kXcds;
  }
  __device__ static int bound(const ProdArgs &a, int i) { return min(max(i, 0), a.T); }

  // Tile i of XCD x; false where there is none.
  __device__ inline __attribute__((always_inline)) bool find(const ProdArgs &a, int x, int i, Where &w) const {
    const int t = x * per + i;
    if (i >= per || t >= total) return false;
    int before = 0, tiles;  // row tiles of the experts ahead, of this one
    if (a.first) {
      const int want = t / cols;
      const int at = 63 - __builtin_clzll(__ballot(from <= want));  // the last lane that starts at or ahead of it
      before = __builtin_amdgcn_readlane(from, at);
      int e = at * share, lo = bound(a, ldk(a.first + e)), hi = bound(a, ldk(a.first + e + 1));
      while (want >= before + Range{lo, hi}.tiles(rows) && e + 1 < a.E) {  // ends: the lane's experts hold the tile
        before += Range{lo, hi}.tiles(rows);
        ++e;
        lo = hi;
        hi = bound(a, ldk(a.first + e + 1));
      }
      w.expert = e; w.lo = lo; w.hi = hi;
      tiles = Range{lo, hi}.tiles(rows);
    } else {
      w.expert = 0; w.lo = 0; w.hi = a.T;
      tiles = total / cols;
    }
    const int in = t - before * cols, strip = in / (kStrip * cols), left = in - strip * kStrip * cols;
    const int g = min(kStrip, tiles - strip * kStrip);
    w.tile = strip * kStrip + left % g;
    w.col = left / g;
    return true;
  }
};

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

// Four neighbouring outputs y[i, n .. n + 3], those below N.
__device__ inline void store4(const ProdArgs &a, int64_t i, int n, f32x4 v) {
  if (a.y_vec && n + 4 <= a.N) {
    if (a.y_bf16) {
      auto *to = (__attribute__((address_space(1))) uint64_t *)((uint16_t *)a.y + i * a.ldy + n);
      const uint64_t both = ((uint64_t)pack2_bf16(v[2], v[3]) << 32) | pack2_bf16(v[0], v[1]);
      *to = both;
    } else {
      auto *to = (__attribute__((address_space(1))) f32x4_t *)((float *)a.y + i * a.ldy + n);
      *to = (f32x4_t)v;
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

// 16 bytes of outputs y[i, n ..] from LDS, those below N: eight bf16 or four fp32.
template <bool BF16>
__device__ inline void store16(const ProdArgs &a, int64_t i, int n, const uint8_t *from) {
  constexpr int kEach = BF16 ? 8 : 4, kSize = BF16 ? 2 : 4;
  typedef std::conditional_t<BF16, u32x4_h, u32x4_w> any;  // at any element
  char *to = (char *)a.y + (i * a.ldy + n) * kSize;
  if (n + kEach <= a.N) {
    const u32x4_t v = *(const u32x4_t *)from;
    if (a.stream) put(to, v, true);
    else *(__attribute__((address_space(1))) any *)to = v;
  } else {
#pragma unroll 1
    for (int j = 0; n + j < a.N; ++j) {
      if constexpr (BF16) stg<uint16_t>(to + 2 * j, *(const uint16_t *)(from + 2 * j));
      else stg<uint32_t>(to + 4 * j, *(const uint32_t *)(from + 4 * j));
    }
  }
}

// ---- a row of an expert -------------------------------------------------------------------------
// Bound by the weights, each read once for a row of x.  A wave takes R weight rows and meets them and
// the row of x in runs of 1 KB, 16 bytes a lane: whole cache lines, several runs on their way at once.
// The matrix instruction wants 16 rows of 64 bytes; it is given 16 pieces of 64 bytes of one row
// instead, on both sides, and the 16 sums on the diagonal add up to the product (what lies beside it is
// not used: the matrix cores have time to spare here).  R = 2 spreads a small matrix over the chip, R = 8
// reads x less often: microscaled, a token's eight experts of 4096 x 6144 19.9 us (107 MB, 5.4 TB/s) with
// R = 8, and one row by 4096 x 6144 3.5 us from the caches, 5.0 from memory, with R = 2.
constexpr int kRun = 1024;

// Bytes [k, k + 16) of a row, zeros beyond its end.  ON16: the row and its length are multiples of 16 bytes.
template <bool ON16>
__device__ inline i32x4 run_at(const uint8_t *row, int k, int row_bytes) {
  if constexpr (ON16) return k < row_bytes ? load16<true>((const int8_t *)row + k) : i32x4{0, 0, 0, 0};
  else return load16_tail((const int8_t *)row, k, row_bytes);
}

template <Kind KIND, int R, bool ON16>
__global__ __launch_bounds__(256) void k_product_vec(ProdArgs a, int cols) {
  constexpr int kU = 12 / (R + 1) > 1 ? 12 / (R + 1) : 1;  // runs in flight
  const Tiles tiles(a, 1, cols);
  Where at;
  if (!tiles.find(a, blockIdx.x % kXcds, blockIdx.x / kXcds, at)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (at.col * 4 + wave) * R, i0 = at.lo + at.tile;
  const uint8_t *w[R], *we[R], *xe = nullptr;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int n = min(n0 + r, a.N - 1);
    w[r] = a.w + at.expert * a.expert + n * a.ldw;
    if constexpr (KIND == kMx) we[r] = a.we + at.expert * a.expert_e + n * a.ldwe;
  }
  const int src = source_of(a, i0);
  const uint8_t *x = a.x + max(src, 0) * a.ldx;
  if constexpr (KIND == kMx) xe = a.xe + max(src, 0) * a.ldxe;
  f32x4 acc[R] = {};
  for (int k0 = 0; k0 < a.row_bytes; k0 += kU * kRun) {
    i32x4 W[kU][R], X[kU];
    int sw[kU][R] = {}, sx[kU] = {};
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = k0 + u * kRun + lane * 16;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        W[u][r] = run_at<ON16>(w[r], k, a.row_bytes);
        if constexpr (KIND == kMx) sw[u][r] = scale_at(we[r], k, a.row_bytes);
      }
      X[u] = run_at<ON16>(x, k, a.row_bytes);
      if constexpr (KIND == kMx) sx[u] = scale_at(xe, k, a.row_bytes);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = mfma16<KIND>(W[u][r], X[u], sw[u][r], sx[u], acc[r]);
  }
  // the diagonal: lane l has rows 4 (l / 16) .. + 3 of column l % 16
  const int d = lane & 15, e = d & 3;
  const bool mine = d >> 2 == lane >> 4;
  float out = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const f32x4 v = acc[r];
    const float sum = wave_sum_to63(mine ? (e == 0 ? v[0] : e == 1 ? v[1] : e == 2 ? v[2] : v[3]) : 0.f);
    const float all = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum), 63));
    out = lane == r ? all : out;
  }
  if (src < 0) out = __builtin_nanf("");
  const int n = n0 + lane;
  if (lane < R && n < a.N) {
    if (a.y_bf16) store_el<true>(a.y, i0 * a.ldy + n, out);
    else store_el<false>(a.y, i0 * a.ldy + n, out);
  }
}

// ---- straight from memory -----------------------------------------------------------------
// A workgroup takes 16 weight rows and 16 rows of one expert; its waves share out the row's steps of 64
// bytes, four of them on their way at once, and add their sums in LDS in a fixed order.  Nothing is
// staged, so a small product ends after little more than two trips to memory: microscaled 77 x 577 x 1120
// 3.6 us, of which a launch 2.3.  Bound by the weights where rows are few: 32 bf16 rows of 256 experts of
// 4096 x 6144 240 us (1.41 GB, 5.9 TB/s); by its reads from L2 beyond, where tiles are faster.
template <Kind KIND, bool ON16>
__global__ __launch_bounds__(512) void k_product_few(ProdArgs a, int cols) {
  constexpr int kU = 4, kW = 8;
  __shared__ f32x4 s_acc[kW][64];
  const Tiles tiles(a, 16, cols);
  Where at;
  if (!tiles.find(a, blockIdx.x % kXcds, blockIdx.x / kXcds, at)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = at.col * 16, i0 = at.lo + at.tile * 16;
  const int row = lane & 15, kq = (lane >> 4) * 16;
  const int n = min(n0 + row, a.N - 1), src = source_of(a, min(i0 + row, at.hi - 1));
  const uint8_t *w = a.w + at.expert * a.expert + n * a.ldw, *x = a.x + max(src, 0) * a.ldx, *we = nullptr, *xe = nullptr;
  if constexpr (KIND == kMx) {
    we = a.we + at.expert * a.expert_e + n * a.ldwe;
    xe = a.xe + max(src, 0) * a.ldxe;
  }
  f32x4 acc = {};
  const int steps = (a.row_bytes + 63) / 64;
  const int lo = (int)((int64_t)steps * wave / kW), hi = (int)((int64_t)steps * (wave + 1) / kW);
  for (int s = lo; s < hi; s += kU) {
    i32x4 A[kU], B[kU];
    int sa[kU] = {}, sb[kU] = {};
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = s + u < hi ? (s + u) * 64 + kq : a.row_bytes;
      A[u] = run_at<ON16>(w, k, a.row_bytes);
      B[u] = run_at<ON16>(x, k, a.row_bytes);
      if constexpr (KIND == kMx) {
        sa[u] = scale_at(we, k, a.row_bytes);
        sb[u] = scale_at(xe, k, a.row_bytes);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) acc = mfma16<KIND>(A[u], B[u], sa[u], sb[u], acc);
  }
  s_acc[wave][lane] = acc;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int v = 1; v < kW; ++v) acc += s_acc[v][lane];
  const int i = i0 + row, to = n0 + (lane >> 4) * 4;
  if (src < 0) acc = nan4();
  if (i < at.hi && to < a.N) store4(a, i, to, acc);
}

// ---- through LDS ----------------------------------------------------------------------------
// A workgroup takes tiles of BN weight rows x BS rows of one expert, one after another; its WN x WS
// waves have blocks of 32 x 32 of it, both operands go through LDS in stages of kBK bytes of K, NBUF
// of them, and a stage's buffer is requested anew as soon as it has been read (as in the int8 product
// of qmatmul.hip: 16 bytes a lane and 32 cycles an instruction are the same).  Small tiles for few rows,
// where starts and padding count; large ones for many, as an operand is read once a tile.
//
// Microscaled 8192 x 12288 x 6144: 296 us in a graph of such calls (4.2 PFLOP/s; the instructions alone reach 6.4
// on such data, by power), 281 to 376 in single ones, 317 on average; 42 us of it are starts and ends of tiles,
// mostly their outputs.  16384 rows of 256 experts, 4096 x 6144: 750 us, 4.6 TB/s of weights.  Bf16, 65536 rows of
// 256 experts, 6144 x 2048: 1.99 ms in a graph, 2.13 to 2.37 in single calls, 2.20 on average, 4.1 to 4.6 TB/s with
// the matrix cores busy for 44 to 52% of it: experts of few rows wait for weights, others for products.
//
// The stages of a workgroup's tiles are one stream: while a tile's last stages are multiplied, the
// first ones of the next tile are on their way, and its outputs leave while they arrive.  (A tile's
// start and end by themselves took 12 us of 8192 x 12288 x 6144's 54 a tile.)
//
// An expert's last tile has fewer rows: a wave multiplies only the blocks that have some, which lie in
// turn with the waves beside it (NS of them, 1 .. TS).
//
// Microscaled rows add a byte a block: 16 of a row, two stages' worth, are one load into LDS, and a
// lane reads the four of its blocks of a stage as one word, of which each instruction takes one byte.
// For that a lane's blocks are neighbours: lanes 0 .. 31 take blocks 0 .. 3 of a stage's eight, lanes 32
// .. 63 blocks 4 .. 7, in both operands.  Rows r and r + 16 of them meet in a bank: conflicts take 26% (dense)
// to 29% (grouped) of the cycles in which LDS is read, 4.5% with bf16.
// One 16-byte load from base + at straight into LDS, to lds + off + 16 lane (base and lds wave-uniform,
// off a constant), by the lanes of `lanes`; it is issued, and counted, whichever they are.  All of the
// wave's lanes are active where it stands.  A load may read a scalar register that a vector instruction wrote
// (v_readlane, v_readfirstlane) five instructions later at the earliest, which the compiler does not see to
// inside assembly; scalar instructions wait for such a write by themselves, so base is copied by one.
__device__ inline __attribute__((always_inline)) void load_to_lds(uint64_t lanes, const uint8_t *base, uint32_t at, uint32_t lds, int off) {
  uint64_t from;
  asm volatile("s_mov_b64 %0, %3\n\ts_add_u32 m0, %1, %4\n\ts_mov_b64 exec, %5\n\tglobal_load_lds_dwordx4 %2, %0\n\ts_mov_b64 exec, -1"
               : "=&s"(from) : "s"(lds), "v"(at), "s"(base), "i"(off), "s"(lanes) : "memory", "m0", "scc", "exec");
}

// v, of which the compiler no longer knows what it was: what is derived from it is derived here, and
// takes no registers elsewhere.
__device__ inline int anew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The kernel's arguments, loaded again: those that only a tile's start and end need take no registers
// between them.
__device__ inline __attribute__((always_inline)) ProdArgs args_anew() {
  auto p = (const __attribute__((address_space(4))) ProdArgs *)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const ProdArgs *)p;
}

constexpr int kScBlocks = 16;  // scales of a row that are loaded at once

template <Kind KIND, int BN, int BS, int WN, int WS, int NBUF, int TOGETHER>
__global__ __launch_bounds__(64 * WN * WS) void k_product_tile(ProdArgs a, int cols) {
  constexpr int kWaves = WN * WS, kThr = 64 * kWaves;
  constexpr int TN = BN / WN / 32, TS = BS / WS / 32;  // 32x32 blocks of a wave
  constexpr int kRows = BN + BS, kStage = kRows * kBK;
  constexpr int kPer = kStage / 16 / kThr;  // chunks a thread moves per stage
  static_assert(kStage % (16 * kThr) == 0, "stage split");
  constexpr bool kMicro = KIND == kMx;
  constexpr int kSc = kMicro ? (kRows + kThr - 1) / kThr : 0;  // scale loads of a thread per two stages
  constexpr int kScSize = kMicro ? kRows * kScBlocks : 0;
  // Buffers of scales: one in use and those on their way.  Of four stages the readers of a pair's second
  // scales have not met again when the pair two further on is requested.
  constexpr int kScBufs = NBUF <= 3 ? 2 : 4;
  constexpr int kScAt = NBUF * kStage, kOutAt = kScAt + kScBufs * kScSize;
  // A wave turns 32 rows of kLine bytes of outputs round at once: whole cache lines, or parts of them
  // where LDS has no room for more.
  constexpr int kRoom = 160 * 1024 / TOGETHER - kOutAt;
  constexpr int kLine = kRoom >= kWaves * 32 * 128 ? 128 : kRoom >= kWaves * 32 * 64 ? 64 : 32;
  constexpr int kOut = 32 * kLine;
  static_assert(kRoom >= kWaves * kOut, "LDS");
  __shared__ __align__(128) uint8_t s_buf[kOutAt + kWaves * kOut];
  const Tiles tiles(a, BS, cols);
  const int xcd = blockIdx.x % kXcds, apart = gridDim.x / kXcds;
  int turn = blockIdx.x / kXcds;
  Where at, next;
  if (!tiles.find(a, xcd, turn, at)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / WS, wsv = wave % WS;
  const int row = lane & 31, ck = lane >> 5;

  // This thread's chunks of a stage: LDS position tid + i kThr, which holds chunk c of row r of the
  // tile, the weights' rows first.  (kThr / 8 rows further on chunks are mixed alike.)
  constexpr int kC = kBK / 16;
  static_assert(kThr / kC % 16 == 0, "chunks are mixed over 16 rows");
  const int kc = ((tid % kC) ^ mix_of(tid / kC)) << 4;
  static_assert(BN % 64 == 0, "a wave's scales are of one operand");
  constexpr int kApart = kThr / kC;  // rows from one chunk of a thread to the next
  static_assert(BN % kApart == 0, "a load has rows of one operand");
  // A tile's operands by a base each (that of x its first row, or with order the whole of it) and a
  // 32-bit offset a chunk; the base goes on through K.
  const uint8_t *w_at, *x_at, *we_at, *xe_at;
  uint32_t src[kPer], sc[kSc + 1];
  uint32_t bad = 0, bad_next = 0;  // bit j: this lane's row of block j has no input
  auto set_up = [&](const Where &w, uint32_t &lost) __attribute__((always_inline)) {
    const ProdArgs a = args_anew();
    const int n0 = w.col * BN, i0 = w.lo + w.tile * BS, tid = anew(threadIdx.x), row = tid & 31;
    const int x0 = a.order ? 0 : min(i0, a.x_rows - 1);
    w_at = a.w + w.expert * a.expert + n0 * a.ldw;
    x_at = a.x + x0 * a.ldx;
    auto x_row = [&](int r) __attribute__((always_inline)) { return source_of(a, min(i0 + r, w.hi - 1)); };
    auto x_off = [&](int r) __attribute__((always_inline)) { return (uint32_t)max(x_row(r) - x0, 0); };
    auto w_off = [&](int r) __attribute__((always_inline)) { return (uint32_t)min(r, a.N - 1 - n0); };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = tid / kC + i * kApart;
      src[i] = kc + (i * kApart < BN ? w_off(r) * (uint32_t)a.ldw : x_off(r - BN) * (uint32_t)a.ldx);
    }
    if constexpr (kMicro) {
      we_at = a.we + w.expert * a.expert_e + n0 * a.ldwe;
      xe_at = a.xe + x0 * a.ldxe;
#pragma unroll
      for (int i = 0; i < kSc; ++i) {
        const int r = min(tid + i * kThr, kRows - 1);
        sc[i] = r < BN ? w_off(r) * (uint32_t)a.ldwe : x_off(r - BN) * (uint32_t)a.ldxe;
      }
    }
    lost = 0;
    if (a.order || a.x_rows < a.T) {
#pragma unroll
      for (int j = 0; j < TS; ++j) lost |= (x_row((wsv + WS * j) * 32 + row) < 0 ? 1u : 0u) << j;
    }
  };
  set_up(at, bad);
  const int sc_bytes = a.row_bytes / 16;
  // stages of a tile: an even number, so that scales come in pairs (beyond K they are zeros)
  const int stages = max(((a.row_bytes + kBK - 1) / kBK + 1) & ~1, (NBUF + 1) & ~1);

  constexpr int kSteps = kBK / 32;
  // this lane's bytes of k step 0 in the wave's first blocks; those of step kk differ in bits 4 and 5
  const int at_w = chunk_of(wn * (BN / WN) + row, ck * kSteps), at_x = chunk_of(BN + wsv * 32 + row, ck * kSteps);
  // fragment f of a k step of the stage at `buf`: the wave's TN weight blocks, then its blocks of rows
  auto frag = [&](int buf, int f, int kk) __attribute__((always_inline)) {
    return *(const i32x4 *)(s_buf + (f < TN ? (at_w ^ kk << 4) + buf + f * 32 * kBK : (at_x ^ kk << 4) + buf + (f - TN) * 32 * WS * kBK));
  };
  const int sc_w = kScAt + (wn * (BN / WN) + row) * kScBlocks + ck * 4, sc_x = kScAt + (BN + wsv * 32 + row) * kScBlocks + ck * 4;
  // its scales; those of the stage's pair lie at `pair`
  auto scale = [&](int pair, int f) __attribute__((always_inline)) {
    return *(const int *)(s_buf + pair + (f < TN ? sc_w + f * 32 * kScBlocks : sc_x + (f - TN) * 32 * WS * kScBlocks));
  };

  const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)s_buf + wave * 1024);
  // Stage s of the tile that was set up last is requested next, into `buf`: `lanes` have bytes of its rows,
  // the others write zeros themselves.
  uint64_t lanes;
  const uint8_t *w_k, *x_k;
  auto aim = [&](int s, int buf) __attribute__((always_inline)) {
    w_k = w_at + s * kBK;
    x_k = x_at + s * kBK;
    const bool in = s * kBK + kc < a.row_bytes;
    lanes = __ballot(in);
    if (!in) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) *(u32x4_t *)(s_buf + buf + (tid + i * kThr) * 16) = u32x4_t{0, 0, 0, 0};
    }
  };
  auto request = [&](int i, int buf) __attribute__((always_inline)) {
    load_to_lds(lanes, i * kApart < BN ? w_k : x_k, src[i], lds + buf, i * kThr * 16);
  };
  int sc_put = 0, sc_get = 0;  // the pair of scales to be requested next, and that in use
  auto following = [](int at, int size, int n) __attribute__((always_inline)) { return at + size == n * size ? 0 : at + size; };
  auto request_scales = [&](int s) __attribute__((always_inline)) {  // of stages s and s + 1 of a tile
    if constexpr (kMicro) {
      const bool in = s * 8 < sc_bytes;
#pragma unroll
      for (int i = 0; i < kSc; ++i) {
        const bool mine = tid + i * kThr < kRows;  // the others would write into the next buffer
        load_to_lds(__ballot(in && mine), (wave * 64 + i * kThr < BN ? we_at : xe_at) + s * 8, sc[i], lds + sc_put, kScAt + i * kThr * 16);
        if (!in && mine) *(u32x4_t *)(s_buf + kScAt + sc_put + (tid + i * kThr) * 16) = u32x4_t{0, 0, 0, 0};
      }
      sc_put = following(sc_put, kScSize, kScBufs);
    }
  };
  // Requests in flight behind stage s + 1 when a stage s with s % 2 == U waits for it: stages s + 2 .. s +
  // NBUF - 1, the even ones with scales.
  constexpr auto kBehind = [](int u) {
    int n = 0;
    for (int k = 2; k < NBUF; ++k) n += kPer + ((u + k) % 2 == 0 ? kSc : 0);
    return n;
  };
  constexpr int kFull = TN * TS;
  constexpr int kG = kFull >= 8 ? 1 : kFull >= 4 ? 2 : 4, kGroups = kSteps / kG;  // k steps whose fragments are read at once
  constexpr int kSpread = kGroups > 1 ? 2 : 1;
  constexpr int kF = TN + TS;
#pragma unroll
  for (int s = 0; s < NBUF; ++s) {
    aim(s, s * kStage);
    if (s % 2 == 0) request_scales(s);
#pragma unroll
    for (int i = 0; i < (s < NBUF - 1 ? kPer : kPer / kSpread); ++i) request(i, s * kStage);
  }
  wait_and_meet<kBehind(1) + ((NBUF - 1) % 2 == 0 ? kSc : 0) + kPer / kSpread>();
  i32x4 F[2][kG][kF];
  int S[2][kF] = {};
  int buf = 0, last = (NBUF - 1) * kStage;  // buffers of the current stage and of the one before it
  int ask = NBUF - 1;                       // the stage requested last, of the tile that was set up last
  auto read_first = [&](int f0) __attribute__((always_inline)) {  // of a tile's first group, fragments f0 ..
#pragma unroll
    for (int k = 0; k < kG; ++k)
#pragma unroll
      for (int f = 0; f < kF; ++f)
        if (f >= f0) F[0][k][f] = frag(buf, f, k);
    if constexpr (kMicro) {
#pragma unroll
      for (int f = 0; f < kF; ++f)
        if (f >= f0) S[0][f] = scale(sc_get, f);
    }
  };
  read_first(0);

  bool more = true;
  auto tile = [&](auto blocks) __attribute__((always_inline)) {
    constexpr int NS = decltype(blocks)::value, kM = TN * NS, kUse = TN + NS;
    f32x16 acc[TN][NS];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    // Multiply group `now` of a stage (its fragments F[cur], its scales S[sn]) while the fragments of
    // group g of the stage at `from` are read, with g = 0 the next stage's scales too, and buffer
    // `again` is requested.
    auto multiply = [&](int cur, int sn, int now, int from, int g, int pair, int again, int r0, int r1)
        __attribute__((always_inline)) {
      constexpr int kAll = kG * kM;
#pragma unroll
      for (int m = 0; m < kAll; ++m) {
#pragma unroll
        for (int f = 0; f < kG * kUse; ++f)
          if (f * kAll / (kG * kUse) == m) F[cur ^ 1][f / kUse][f % kUse] = frag(from, f % kUse, g * kG + f / kUse);
        if constexpr (kMicro) {
#pragma unroll
          for (int f = 0; f < kUse; ++f)
            if (g == 0 && f * kAll / kUse == m) S[sn ^ 1][f] = scale(pair, f);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i >= r0 && i < r1 && (i - r0) * kAll / (r1 - r0) == m) request(i, again);
        const int k = m / kM, i = m % kM / NS, j = m % NS;
        acc[i][j] = mfma32<KIND>(F[cur][k][i], F[cur][k][TN + j], S[sn][i], S[sn][TN + j], now * kG + k, acc[i][j]);
        // the compiler moves scaled products together, past the barrier below: 256 x 256 tiles spill then
        if constexpr (kMicro) asm volatile("" : "+a"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto stage = [&](auto odd) __attribute__((always_inline)) {  // a stage of the tile, an even or an odd one
      constexpr int u = decltype(odd)::value, cur = u * kGroups & 1;
#pragma unroll
      for (int g = 1; g < kGroups; ++g)
        multiply((cur + g - 1) & 1, u, g - 1, buf, g, 0, last, g < kSpread ? kPer * g / kSpread : 0,
                 g < kSpread ? kPer * (g + 1) / kSpread : 0);
      wait_and_meet<kBehind(u)>();
      if (++ask == stages) ask = 0;
      if constexpr (u == NBUF % 2) {  // of these two stages the one that can ask for stage 0
        if (ask == 0) {  // of the next tile (after the last one its own are loaded again, and not used)
          turn += apart;
          more = tiles.find(args_anew(), xcd, turn, next);
          if (more) set_up(next, bad_next);
        }
      }
      aim(ask, buf);
      if ((u + NBUF) % 2 == 0) request_scales(ask);
      const int then = following(buf, kStage, NBUF);
      const int pair = u ? following(sc_get, kScSize, kScBufs) : sc_get + 8;
      multiply((cur + kGroups - 1) & 1, u, kGroups - 1, then, 0, pair, buf, 0, kPer / kSpread);
      if (u) sc_get = pair;
      last = buf;
      buf = then;
    };
#pragma unroll 1
    for (int s = 0; s < stages; s += 2) {
      stage(std::integral_constant<int, 0>());
      stage(std::integral_constant<int, 1>());
    }
    // Each wave turns its sums round in LDS, kLine bytes of 32 rows at a time, so that they leave as whole
    // cache lines.  A wave's accesses to LDS are carried out in order, so none waits for another.
    const ProdArgs b = args_anew();
    auto leave = [&](auto bf16) __attribute__((always_inline)) {
      constexpr bool BF16 = decltype(bf16)::value;
      constexpr int kI = BF16 && TN > 1 && kLine == 128 ? 2 : 1;  // blocks of weights at once
      constexpr int kE = std::min(4, kLine / (BF16 ? 16 : 32));    // quarters of a block at once
      constexpr int kSize = BF16 ? 2 : 4, kEach = 16 / kSize;      // outputs of a 16-byte piece
      constexpr int kCh = kI * kE * 8 / kEach;                     // pieces of a row
      constexpr int kQ = kCh / 2;                                  // rows, and pieces, of a lane
      const int lane = anew(tid) & 63, row = lane & 31, ck = lane >> 5;
      uint8_t *out = s_buf + kOutAt + wave * kOut;
      auto piece = [&](int r, int c) __attribute__((always_inline)) { return out + r * kLine + ((c ^ (mix_of(r) & (kLine / 16 - 1))) << 4); };
      const int i0 = at.lo + at.tile * BS, n0 = at.col * BN + wn * (BN / WN);
      uint8_t *y = (uint8_t *)b.y + (i0 * b.ldy + n0) * kSize;
      const int rows = at.hi - i0;
      const bool whole = n0 + BN / WN <= b.N;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const bool lost = bad >> j & 1;
        const float none = __builtin_nanf("");
        const int r0 = (wsv + WS * j) * 32;
#pragma unroll
        for (int i = 0; i < TN; i += kI)
#pragma unroll
          for (int e0 = 0; e0 < 4; e0 += kE) {
#pragma unroll
            for (int h = 0; h < kI; ++h)
#pragma unroll
              for (int e = e0; e < e0 + kE; ++e) {
                f32x4 v = {acc[i + h][j][4 * e], acc[i + h][j][4 * e + 1], acc[i + h][j][4 * e + 2], acc[i + h][j][4 * e + 3]};
                if (lost) v = f32x4{none, none, none, none};
                if constexpr (BF16)
                  *(uint64_t *)(piece(row, h * 4 + e - e0) + ck * 8) = ((uint64_t)pack2_bf16(v[2], v[3]) << 32) | pack2_bf16(v[0], v[1]);
                else
                  *(f32x4 *)piece(row, 2 * (e - e0) + ck) = v;
              }
            asm volatile("" ::: "memory");
            const int n = i * 32 + e0 * 8;  // of the wave's outputs
            if (whole) {
              u32x4_t v[kQ];
#pragma unroll
              for (int q = 0; q < kQ; ++q) v[q] = *(const u32x4_t *)piece(lane / kCh + q * (64 / kCh), lane % kCh);
#pragma unroll
              for (int q = 0; q < kQ; ++q) {
                typedef std::conditional_t<BF16, u32x4_h, u32x4_w> any;  // at any element
                const int r = r0 + lane / kCh + q * (64 / kCh);
                auto *to = (__attribute__((address_space(1))) any *)(y + n * kSize + (uint32_t)(r * (int)b.ldy + lane % kCh * kEach) * kSize);
                if (r < rows) {
                  if (kLine == 128 && b.stream) put<16>((void *)to, v[q], true);
                  else *to = v[q];
                }
              }
            } else {
#pragma unroll 1
              for (int r = lane / kCh; r < 32; r += 64 / kCh)
                if (r0 + r < rows) store16<BF16>(b, i0 + r0 + r, n0 + n + lane % kCh * kEach, piece(r, lane % kCh));
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
          }
      }
    };
    if (b.y_bf16) leave(std::true_type());
    else leave(std::false_type());
    if (NS < TS) read_first(kUse);
  };
  do {
    const int blocks = (min(at.hi - at.lo - at.tile * BS, BS) + 32 * WS - 1) / (32 * WS);
    if constexpr (TS == 1) {
      tile(std::integral_constant<int, 1>());
    } else if constexpr (TS == 2) {
      if (blocks > 1) tile(std::integral_constant<int, 2>());
      else tile(std::integral_constant<int, 1>());
    } else {
      static_assert(TS == 4, "blocks of a wave");
      if (blocks > 3) tile(std::integral_constant<int, 4>());
      else if (blocks > 2) tile(std::integral_constant<int, 3>());
      else if (blocks > 1) tile(std::integral_constant<int, 2>());
      else tile(std::integral_constant<int, 1>());
    }
    at = next;
    bad = bad_next;
  } while (more);
  wait_and_meet<0>();  // the last requests, the last tile's first stages once more, have arrived
}

// ---- rows on 16-byte boundaries -------------------------------------------------------------
// Copies the rows of x, of the weights or of both to the workspace, each at a multiple of 16 bytes and
// filled up with zeros to one: the loads into LDS need that.  A lane moves 16 bytes.  Rows of experts that
// have none to compute are left out.
struct Copy {
  const uint8_t *from;
  uint8_t *to;
  int64_t ld, expert;  // bytes between the source's rows and experts
  int64_t pieces;      // of 16 bytes
  int N;               // rows of an expert
};
struct Copies {
  Copy x, w;
  int64_t begin;  // the pieces of this launch, x's first
  int row_bytes, chunks;
};
constexpr int kCopyThreads = 256;
__global__ __launch_bounds__(kCopyThreads) void k_product_align(ProdArgs a, Copies c) {
  int64_t block0 = c.begin + (int64_t)blockIdx.x * kCopyThreads;
  const int64_t x_blocks = (c.x.pieces + kCopyThreads - 1) / kCopyThreads * kCopyThreads;
  const bool w = block0 >= x_blocks;
  const Copy &p = w ? c.w : c.x;
  if (w) block0 -= x_blocks;
  if (block0 + threadIdx.x >= p.pieces) return;
  const int64_t r0 = block0 / c.chunks;
  const uint32_t u = (uint32_t)(block0 - r0 * c.chunks) + threadIdx.x;
  const int64_t r = r0 + u / c.chunks;
  const int k = (int)(u % c.chunks) * 16;
  const int64_t e = r / p.N;
  if (w && a.first && ldg<int32_t>(a.first + e) >= ldg<int32_t>(a.first + e + 1)) return;
  const i32x4 v = load16_tail((const int8_t *)p.from + e * p.expert + (r - e * p.N) * p.ld, k, c.row_bytes);
  stg<uint4>(p.to + (block0 + threadIdx.x) * 16, make_uint4((uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]));
}

// ---- which kernel ---------------------------------------------------------------------------
enum ProdKernel { kVec2, kVec8, kFew16, kTile32, kTile64, kTile128, kTile256x128, kTile256, kKernels };
struct Shape {
  const char *name;
  int rows, cols, threads;  // of a workgroup: rows of x, of weights
  int together;             // tiles: workgroups on a compute unit
};
constexpr Shape kShapes[kKernels] = {{"product_vec2", 1, 8, 256, 0},      {"product_vec8", 1, 32, 256, 0},
                                     {"product_few16", 16, 16, 512, 0},   {"product_tile32", 32, 64, 128, 2},
                                     {"product_tile64", 64, 128, 256, 1}, {"product_tile128", 128, 128, 256, 2},
                                     {"product_tile256x128", 128, 256, 256, 1}, {"product_tile256", 256, 256, 256, 1}};
constexpr int kUnits = 256;  // compute units

struct ProdPlan {
  ProdKernel kernel;
  bool copy_x, copy_w;  // the operand that the tiles cannot read as it lies: bf16 rows, or scales
  int64_t ld, bytes_x, bytes;  // of the copies: a row, the rows of x, all
};

// Row tiles of `rows` rows that T rows of E experts can make.
int64_t most_tiles(const ProdArgs &a, int rows) {
  const int64_t whole = ((int64_t)a.T + rows - 1) / rows;
  return a.first ? a.T / rows + std::min(a.E, a.T) : whole;
}
// Column tiles of a launch, 0 where the kernel's row tiles alone are too many.  Tiles are counted in 31 bits,
// and a direct kernel has a workgroup for each (blocks_of rounds them up): fewer than 2^32 threads.
int64_t cols_at_once(const ProdArgs &a, const Shape &s) {
  const int64_t most = s.together ? (int64_t)1 << 30 : (((int64_t)1 << 32) - 1) / s.threads - kXcds;
  // row tiles are added up in 31 bits even if every expert has all rows
  return (int64_t)a.E * ((a.T + s.rows - 1) / s.rows) >> 31 ? 0 : most / most_tiles(a, s.rows);
}

bool on16(const void *p, int64_t ld, int64_t rows, int64_t expert, int E) {
  return (uintptr_t)p % 16 == 0 && (rows == 1 || ld % 16 == 0) && (E == 1 || expert % 16 == 0);
}

// The kernel with the least estimated time, fitted to some 150 measured shapes (us, with the launch; of
// 151 it takes the best kernel or one within 8% of it but for eleven, where it loses up to 24%, and
// 1.5% on average).  Every kernel waits for the weights of the experts that have rows, at 4.4 to 5.6
// TB/s.  The direct kernels: a start, a trip to memory per step of K, and each further workgroup of a
// compute unit.  Tiles: for each round of them a start and end and a time per stage, `alone` where there
// is one tile for a compute unit; this and the weights' time add up as squares.  Grouped rows are thought
// to be spread evenly over the experts, which they are not: some more tiles.  Measured (vec2, vec8, few16,
// tile32, tile64, tile128, tile256x128, tile256):
//   microscaled, 1 x 4096 x 2048                 3.5   4.5   4.3  5.4  6.4  8.7  10   12
//   microscaled, 64 x 4096 x 6144                64    54    25   11   19   26   32   39
//   microscaled, 1024 x 12288 x 2048             2570  1311  340  52   35   26   22   21
//   bf16, 64 rows of 256 experts, 4096 x 2048    186   160   175  169  170  186  201  208
//   bf16, 16384 of 256, 4096 x 2048              20409 12817 4447 1148 919  872  775  943
//   bf16, 32768 of 32, 2048 x 2048               15200 11625 3638 668  445  324  284  279
ProdPlan plan_of(const ProdArgs &a, bool mx) {
  struct Direct { double start, step, more, each, grouped, rate; int bytes; };
  static constexpr Direct kDirect[2][3] = {
      {{0, 0.734, 0.094, 0.262, 0, 4.4e6, 1024}, {0.264, 1.811, 0.441, 0, 0, 4.9e6, 1024}, {0.835, 0.052, 0.048, 0.438, 0, 5.2e6, 64}},
      {{0.491, 0.082, 0.09, 0.25, 0.4, 4.4e6, 1024}, {1.1, 1.05, 0.9, 0.6, 0.6, 5.2e6, 1024}, {0.471, 0.101, 0.095, 0.274, 0.093, 5.2e6, 64}}};
  struct Tile { double once, stage, alone; };
  static constexpr Tile kTile[kKernels - kTile32] = {{1.03, 0.33, 0.25}, {1.62, 0.33, 0.40}, {2.22, 0.93, 0.72}, {4.42, 0.68, 0.78}, {5.67, 1.05, 1.25}};
  ProdPlan p{};
  const int64_t row = mx ? a.row_bytes / 16 : a.row_bytes;  // what may have to be copied
  const bool even = row % 16 == 0;
  const bool x_lies = even && (mx ? on16(a.xe, a.ldxe, a.x_rows, 0, 1) : on16(a.x, a.ldx, a.x_rows, 0, 1));
  const bool w_lies = even && (mx ? on16(a.we, a.ldwe, a.N, a.expert_e, a.E) : on16(a.w, a.ldw, a.N, a.expert, a.E));
  const double busy = a.first ? std::min<double>(a.T, a.E * (1 - std::exp(-(double)a.T / a.E))) : 1.0, each = a.T / busy;
  const double weights = busy * a.N * a.row_bytes * (mx ? 17.0 / 16 : 1.0);
  double best = 1e30;
  for (int k = 0; k < kTile32; ++k) {
    const Direct &d = kDirect[mx][k];
    const Shape &s = kShapes[k];
    if (cols_at_once(a, s) == 0) continue;
    const double steps = std::ceil((double)a.row_bytes / d.bytes), cols = std::ceil((double)a.N / s.cols);
    const double tiles = s.rows == 1 ? a.T : a.first ? busy * std::max(1.0, each / s.rows + 0.5) : std::ceil((double)a.T / s.rows);
    const double n = std::ceil(tiles * cols / kUnits) - 1;
    double us = 2.4 + std::max(d.start + d.step * steps + n * (d.more * steps + d.each + (a.first ? d.grouped : 0.0)), weights / d.rate);
    if (!mx && !(x_lies && w_lies)) us *= 1.5;
    if (us < best) {
      best = us;
      p.kernel = (ProdKernel)k;
    }
  }
  // the tiles' offsets within an operand have 32 bits
  p.ld = (row + 15) / 16 * 16;
  const int64_t x_far = a.order ? (int64_t)a.x_rows : 256, ldx = x_lies ? 0 : p.ld, ldw = w_lies ? 0 : p.ld;
  const bool near = !(std::max({256 * std::max({a.ldw, a.ldwe, ldw}), x_far * std::max({a.ldx, a.ldxe, ldx}), 1024 * a.ldy}) >> 32);
  const double copied = (x_lies ? 0.0 : (double)a.x_rows * row) + (w_lies ? 0.0 : busy * a.N * row);
  const double copy = x_lies && w_lies ? 0.0 : 3.0 + copied / 2e6;
  for (int k = kTile32; near && k < kKernels; ++k) {
    const Tile &t = kTile[k - kTile32];
    const Shape &s = kShapes[k];
    const double stages = std::ceil(a.row_bytes / 256.0) * 2, cols = std::ceil((double)a.N / s.cols);
    const double tiles = cols * (a.first ? 1.15 * busy * std::max(1.0, each / s.rows + 0.5) : std::ceil((double)a.T / s.rows));
    const double n = std::ceil(tiles / kUnits);
    const double us = copy + 2.5 + std::hypot(n == 1 ? t.once + t.alone * stages : std::ceil(n / s.together) * (t.once + t.stage * stages),
                                              weights / 5.6e6);
    if (us < best) {
      best = us;
      p.kernel = (ProdKernel)k;
    }
  }
  if (!a.first && a.T == 1) p.kernel = kVec2;
  if (p.kernel >= kTile32) {
    p.copy_x = !x_lies;
    p.copy_w = !w_lies;
    p.bytes_x = p.copy_x ? a.x_rows * p.ld : 0;
    p.bytes = p.bytes_x + (p.copy_w ? (int64_t)a.E * a.N * p.ld : 0);
  }
  return p;
}

unsigned blocks_of(const ProdArgs &a, int rows, int cols) {
  return (unsigned)((most_tiles(a, rows) * cols + kXcds - 1) / kXcds * kXcds);
}

template <Kind KIND, int R, bool ON16>
void launch_vec(const ProdArgs &a, hipStream_t st) {
  const int cols = (a.N + 4 * R - 1) / (4 * R);
  MOE_LAUNCH((k_product_vec<KIND, R, ON16>), dim3(blocks_of(a, 1, cols)), dim3(256), 0, st, a, cols);
}
template <Kind KIND, bool ON16>
void launch_few(const ProdArgs &a, hipStream_t st) {
  const int cols = (a.N + 15) / 16;
  MOE_LAUNCH((k_product_few<KIND, ON16>), dim3(blocks_of(a, 16, cols)), dim3(512), 0, st, a, cols);
}
template <Kind KIND, int BN, int BS, int WN, int WS, int NBUF, int TOGETHER>
void launch_tile(const ProdArgs &a, hipStream_t st) {
  const int cols = (a.N + BN - 1) / BN;
  const unsigned most = kUnits * TOGETHER;  // on the chip at once
  MOE_LAUNCH((k_product_tile<KIND, BN, BS, WN, WS, NBUF, TOGETHER>), dim3(std::min(blocks_of(a, BS, cols), most)), dim3(64 * WN * WS), 0, st, a, cols);
}

template <Kind KIND, bool ON16>
void launch_direct(const ProdArgs &a, ProdKernel k, hipStream_t st) {
  switch (k) {
    case kVec2: launch_vec<KIND, 2, ON16>(a, st); break;
    case kVec8: launch_vec<KIND, 8, ON16>(a, st); break;
    default: launch_few<KIND, ON16>(a, st); break;
  }
}
template <Kind KIND>
void launch_piece(const ProdArgs &a, ProdKernel k, hipStream_t st) {
  switch (k) {
    case kTile32: launch_tile<KIND, 64, 32, 2, 1, 4, 2>(a, st); break;
    case kTile64: launch_tile<KIND, 128, 64, 2, 2, 4, 1>(a, st); break;
    case kTile128: launch_tile<KIND, 128, 128, 2, 2, 2, 2>(a, st); break;
    case kTile256x128: launch_tile<KIND, 256, 128, 2, 2, 3, 1>(a, st); break;
    case kTile256: launch_tile<KIND, 256, 256, 2, 2, 2, 1>(a, st); break;
    default: {
      // rows at multiples of 16 bytes (microscaled ones are), or of any bytes
      const bool even = KIND == kMx || (a.row_bytes % 16 == 0 && on16(a.x, a.ldx, a.x_rows, 0, 1) && on16(a.w, a.ldw, a.N, a.expert, a.E));
      if (even) launch_direct<KIND, true>(a, k, st);
      else if constexpr (KIND == kBf16) launch_direct<KIND, false>(a, k, st);
      break;
    }
  }
}

// Copies what the plan says, and points the arguments at it.
hipError_t launch_copies(ProdArgs &a, const ProdPlan &p, bool mx, hipStream_t st) {
  Copies c{};
  c.row_bytes = mx ? a.row_bytes / 16 : a.row_bytes;
  c.chunks = (int)(p.ld / 16);
  const uint8_t *&x = mx ? a.xe : a.x, *&w = mx ? a.we : a.w;
  int64_t &ldx = mx ? a.ldxe : a.ldx, &ldw = mx ? a.ldwe : a.ldw, &expert = mx ? a.expert_e : a.expert;
  c.x = {x, a.ws, ldx, 0, p.copy_x ? (int64_t)a.x_rows * c.chunks : 0, a.x_rows};
  c.w = {w, a.ws + p.bytes_x, ldw, expert, p.copy_w ? (int64_t)a.E * a.N * c.chunks : 0, a.N};
  auto blocks = [](int64_t pieces) { return (pieces + kCopyThreads - 1) / kCopyThreads; };
  const int64_t all = blocks(c.x.pieces) + blocks(c.w.pieces);
  constexpr int64_t kMost = 1 << 22;  // a launch holds fewer than 2^32 threads
  for (int64_t b = 0; b < all; b += kMost) {
    c.begin = b * kCopyThreads;
    ProfScope ps("product_align", st);
    MOE_LAUNCH(k_product_align, dim3((unsigned)std::min(kMost, all - b)), dim3(kCopyThreads), 0, st, a, c);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (p.copy_x) x = a.ws, ldx = p.ld;
  if (p.copy_w) w = a.ws + p.bytes_x, ldw = p.ld, expert = (int64_t)a.N * p.ld;
  if (!mx) a.row_bytes = (int)p.ld;
  return hipSuccess;
}

}  // namespace

int64_t product_workspace(const ProdArgs &a, bool mx) { return plan_of(a, mx).bytes; }

hipError_t launch_product(const ProdArgs &a0, bool mx, hipStream_t st) {
  ProdArgs a = a0;
  const int ys = a.y_bf16 ? 2 : 4;
  a.y_vec = (uintptr_t)a.y % (a.y_bf16 ? 8 : 16) == 0 && a.ldy % 4 == 0;
  // past the caches only whole 16-byte pieces
  a.stream = (int64_t)a.T * a.N * ys > kStreamBytes && (uintptr_t)a.y % 16 == 0 && a.ldy * ys % 16 == 0;
  const ProdPlan p = plan_of(a, mx);
  if (p.copy_x || p.copy_w) {
    const hipError_t err = launch_copies(a, p, mx, st);
    if (err != hipSuccess) return err;
  }
  const Shape &s = kShapes[p.kernel];
  const int64_t step = cols_at_once(a, s) * s.cols;  // many weight rows go in pieces
  for (int64_t n = 0; n < a.N; n += step) {
    ProdArgs c = a;
    c.N = (int)std::min<int64_t>(step, a.N - n);
    c.w += n * a.ldw;
    if (mx) c.we += n * a.ldwe;
    c.y = (char *)a.y + n * ys;
    ProfScope ps(s.name, st);
    if (mx) launch_piece<kMx>(c, p.kernel, st);
    else launch_piece<kBf16>(c, p.kernel, st);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
