// Product of int8 rows with int8 weights: y[s, n] = (sum_k q[s, k] w[n, k]) * (d[s] * dw[n]),
// the sum exact in int32, scaled once in fp32.  Three kernels, chosen by estimated time
// (plan_of): a dot-product kernel for up to four tokens (eight where weight rows are few and
// long), a direct matrix-core kernel for few tokens or small operands, LDS tiles for the
// others.  Measured (bf16 outputs):
//   1 x 4096 x 6144 (S x N x K)   5.9 us, 4.3 TB/s; 1 x 12288 x 6144 12.4 us, 6.1 TB/s (a
//                                 copy of 1 GiB runs at 5.1): bound by the weights' bytes
//   256 x 6144 x 6144             18 us, 1.07 POP/s: 192 tiles leave a quarter of the 256
//                                 compute units idle, and the others take in 1.2 MB each at
//                                 76 KB/us (77% of it hits in its XCD's L2, which alone
//                                 would give 120)
//   8192 x 12288 x 6144           510 to 550 us on different cards, 2.25 to 2.43 POP/s (a
//                                 library int8 product: 2.04): the matrix cores are busy
//                                 62% of the cycles; a SIMD has one wave, which waits at a
//                                 barrier every 128 bytes of K, and the chip clocks down to
//                                 1.8 GHz to stay within its power (all operands zero: 484)
// Outputs of a width that is no multiple of 4 are stored element by element and not past the
// caches: 8192 x 12287 x 6144 586 us, 256 x 6143 x 6144 18.5.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "dense.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef u32x4_t u32x4_w __attribute__((aligned(4)));

__device__ const uint8_t g_zeros[16] __attribute__((aligned(16))) = {};

// 16 bytes at p.  W4: p lies on a whole word; else the words that hold them (every one
// holds at least one of them) are read and shifted together: a load from an odd address
// takes the hardware several times as long (one token, 4096 x 6143: 13.8 us against 7.1).
template <bool W4>
__device__ inline i32x4 load16(const int8_t *p) {
  if constexpr (W4) {
    return __builtin_bit_cast(i32x4, *(const __attribute__((address_space(1))) u32x4_w *)p);
  } else {
    const int8_t *base = (const int8_t *)((uintptr_t)p & ~(uintptr_t)3);
    const u32x4_t d = *(const __attribute__((address_space(1))) u32x4_w *)base;
    const uint32_t e = ldg<uint32_t>((const int8_t *)((uintptr_t)(p + 15) & ~(uintptr_t)3));
    const uint32_t sh = (uint32_t)(uintptr_t)p & 3;
    return i32x4{(int)__builtin_amdgcn_alignbyte(d.y, d.x, sh), (int)__builtin_amdgcn_alignbyte(d.z, d.y, sh),
                 (int)__builtin_amdgcn_alignbyte(d.w, d.z, sh), (int)__builtin_amdgcn_alignbyte(e, d.w, sh)};
  }
}

// Bytes [k, k + 16) of a row of K bytes, zeros beyond its end.  The row's last, partial
// chunk is read as the 16 bytes that end with it and shifted down, so nothing beyond the
// row is touched.
__device__ inline i32x4 load16_tail(const int8_t *row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (k >= K) return v;
  if (k + 16 <= K) return load16<false>(row + k);
  if (K >= 16) {
    const u32x4_t r = __builtin_bit_cast(u32x4_t, load16<false>(row + K - 16));
    const int drop = k + 16 - K;  // 1..15 bytes of the previous chunk in front
    unsigned __int128 x = ((unsigned __int128)(((uint64_t)r.w << 32) | r.z) << 64) | (((uint64_t)r.y << 32) | r.x);
    x >>= 8 * drop;
    return i32x4{(int)(uint32_t)x, (int)(uint32_t)(x >> 32), (int)(uint32_t)(x >> 64), (int)(uint32_t)(x >> 96)};
  }
  uint32_t w[4] = {0, 0, 0, 0};
  for (int j = k; j < K; ++j) w[(j - k) >> 2] |= (uint32_t)(uint8_t)ldg<int8_t>(row + j) << (8 * ((j - k) & 3));
  return i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// Four neighbouring outputs y[s, n .. n + 3], those below N, past the caches where STREAM.
template <bool STREAM>
__device__ inline void store4(const QmmArgs &a, int64_t s, int n, float v0, float v1, float v2, float v3) {
  const float v[4] = {v0, v1, v2, v3};
  if (a.y_vec && n + 4 <= a.N) {
    if (a.y_bf16) {
      const uint2 p = make_uint2((uint32_t)f_bf16(v0) | ((uint32_t)f_bf16(v1) << 16),
                                 (uint32_t)f_bf16(v2) | ((uint32_t)f_bf16(v3) << 16));
      auto *to = (__attribute__((address_space(1))) uint64_t *)((uint16_t *)a.y + s * a.ldy + n);
      const uint64_t both = ((uint64_t)p.y << 32) | p.x;
      if constexpr (STREAM) __builtin_nontemporal_store(both, to);
      else *to = both;
    } else {
      auto *to = (__attribute__((address_space(1))) f32x4_t *)((float *)a.y + s * a.ldy + n);
      const f32x4_t p = {v0, v1, v2, v3};
      if constexpr (STREAM) __builtin_nontemporal_store(p, to);
      else *to = p;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < a.N) {
        if (a.y_bf16) store_el<true>(a.y, s * a.ldy + n + j, v[j]);
        else store_el<false>(a.y, s * a.ldy + n + j, v[j]);
      }
  }
}

// ---- up to eight tokens -----------------------------------------------------------
// Bound by the weights, each read once.  A wave takes R weight rows and meets them and
// the NS tokens in runs of 1 KB, 16 bytes a lane (whole rows of cache lines: 16 rows of 64
// bytes a load, as the matrix instruction wants them, reach half the rate), multiplies
// with v_dot4 and adds up over its lanes.  KS waves share a row where rows are few.
__device__ inline int dot16(i32x4 a, i32x4 b, int c) {
  c = __builtin_amdgcn_sdot4(a[0], b[0], c, false);
  c = __builtin_amdgcn_sdot4(a[1], b[1], c, false);
  c = __builtin_amdgcn_sdot4(a[2], b[2], c, false);
  return __builtin_amdgcn_sdot4(a[3], b[3], c, false);
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ inline int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROW_MASK, 0xF, false);
}
__device__ inline int wave_total(int v) {  // the sum over the lanes, in every lane
  v = dpp_add<0xB1>(v);        // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);        // quad_perm [2,3,0,1]
  v = dpp_add<0x141>(v);       // row_half_mirror
  v = dpp_add<0x140>(v);       // row_mirror
  v = dpp_add<0x142, 0xA>(v);  // row_bcast:15
  v = dpp_add<0x143, 0xC>(v);  // row_bcast:31
  return __builtin_amdgcn_readlane(v, 63);
}

template <int NS, int R, int KS, bool W4>
__global__ __launch_bounds__(256) void k_qmm_vec(QmmArgs a) {
  constexpr int kU = R + NS <= 2 ? 6 : R + NS <= 5 ? 4 : 2;  // runs in flight
  static_assert(R * NS <= 64, "an output a lane");
  __shared__ int s_sum[4][R * NS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int part = wave % KS;
  const int64_t n0 = ((int64_t)blockIdx.x * (4 / KS) + wave / KS) * R;
  const int8_t *wr[R], *qr[NS];
#pragma unroll
  for (int r = 0; r < R; ++r) wr[r] = a.w + min(n0 + r, (int64_t)a.N - 1) * a.ldw;
#pragma unroll
  for (int s = 0; s < NS; ++s) qr[s] = a.q + (int64_t)min(s, a.S - 1) * a.ldq;
  int acc[R][NS] = {};
  const int whole = a.K & ~15;
  int k = (part * 64 + lane) * 16;
  auto meet = [&](auto load) __attribute__((always_inline)) {
    i32x4 W[R], Q[NS];
#pragma unroll
    for (int r = 0; r < R; ++r) W[r] = load(wr[r]);
#pragma unroll
    for (int s = 0; s < NS; ++s) Q[s] = load(qr[s]);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int s = 0; s < NS; ++s) acc[r][s] = dot16(W[r], Q[s], acc[r][s]);
  };
  for (; k + (kU - 1) * KS * 1024 < whole; k += kU * KS * 1024) {
    i32x4 W[kU][R], Q[kU][NS];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
#pragma unroll
      for (int r = 0; r < R; ++r) W[u][r] = load16<W4>(wr[r] + k + u * KS * 1024);
#pragma unroll
      for (int s = 0; s < NS; ++s) Q[u][s] = load16<W4>(qr[s] + k + u * KS * 1024);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int s = 0; s < NS; ++s) acc[r][s] = dot16(W[u][r], Q[u][s], acc[r][s]);
  }
  for (; k < whole; k += KS * 1024) meet([&](const int8_t *row) { return load16<W4>(row + k); });
  if (k < a.K) meet([&](const int8_t *row) { return load16_tail(row, k, a.K); });
  int mine = 0;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int t = wave_total(acc[r][s]);
      mine = lane == s * R + r ? t : mine;
    }
  if constexpr (KS > 1) {
    if (lane < R * NS) s_sum[wave][lane] = mine;
    __syncthreads();
    if (part) return;
    if (lane < R * NS) {
#pragma unroll
      for (int i = 1; i < KS; ++i) mine += s_sum[wave + i][lane];
    }
  }
  const int s = lane / R;
  const int64_t n = n0 + lane % R;
  if (lane < R * NS && s < a.S && n < a.N) {
    const float v = (float)mine * (ldg<float>(a.d + s) * ldg<float>(a.dw + n));
    if (a.y_bf16) store_el<true>(a.y, s * a.ldy + n, v);
    else store_el<false>(a.y, s * a.ldy + n, v);
  }
}

// ---- few tokens or small operands -----------------------------------------------------
// A workgroup takes 16 MT weight rows and 16 NT tokens; its W waves split K and add their
// int32 sums in LDS.  v_mfma_i32_16x16x64_i8 with the weights as rows and the tokens as
// columns, both operands straight from memory: lane l holds 16 bytes of row (or token) l %
// 16 at k + 16 (l / 16).  Nothing is staged, so a small product ends after little more
// than one trip to memory (77 x 577 x 1111: 4.2 us; tiles 6.5 and the copies before them).
template <int MT, int NT, int W, bool W4>
__global__ __launch_bounds__(64 * W) void k_qmm_few(QmmArgs a) {
  constexpr int kU = MT * NT >= 4 ? 2 : 4;  // k steps in flight
  __shared__ i32x4 s_acc[W][MT * NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nb = (a.N + 16 * MT - 1) / (16 * MT);
  const int n0 = (int)(blockIdx.x % nb) * 16 * MT, s0 = (int)(blockIdx.x / nb) * 16 * NT;
  const int col = lane & 15, kq = (lane >> 4) * 16;
  const int8_t *wr[MT], *qr[NT];
#pragma unroll
  for (int m = 0; m < MT; ++m) wr[m] = a.w + (int64_t)min(n0 + 16 * m + col, a.N - 1) * a.ldw + kq;
#pragma unroll
  for (int t = 0; t < NT; ++t) qr[t] = a.q + (int64_t)min(s0 + 16 * t + col, a.S - 1) * a.ldq + kq;
  i32x4 acc[MT][NT] = {};
  // whole steps of 64 bytes shared out evenly; the last wave takes the partial one
  const int steps = a.K / 64;
  const int lo = (int)((int64_t)steps * wave / W), hi = (int)((int64_t)steps * (wave + 1) / W);
  int st = lo;
  for (; st + kU <= hi; st += kU) {
    i32x4 A[kU][MT], B[kU][NT];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
#pragma unroll
      for (int m = 0; m < MT; ++m) A[u][m] = load16<W4>(wr[m] + (st + u) * 64);
#pragma unroll
      for (int t = 0; t < NT; ++t) B[u][t] = load16<W4>(qr[t] + (st + u) * 64);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[m][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[u][m], B[u][t], acc[m][t], 0, 0, 0);
  }
  for (; st < hi; ++st) {
    i32x4 A[MT], B[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) A[m] = load16<W4>(wr[m] + st * 64);
#pragma unroll
    for (int t = 0; t < NT; ++t) B[t] = load16<W4>(qr[t] + st * 64);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[m][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[m], B[t], acc[m][t], 0, 0, 0);
  }
  if (wave == W - 1 && steps * 64 < a.K) {
    i32x4 A[MT], B[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) A[m] = load16_tail(wr[m] - kq, steps * 64 + kq, a.K);
#pragma unroll
    for (int t = 0; t < NT; ++t) B[t] = load16_tail(qr[t] - kq, steps * 64 + kq, a.K);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[m][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[m], B[t], acc[m][t], 0, 0, 0);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) s_acc[wave][m * NT + t][lane] = acc[m][t];
  __syncthreads();
  for (int b = wave; b < MT * NT; b += W) {
    i32x4 sum = s_acc[0][b][lane];
#pragma unroll
    for (int v = 1; v < W; ++v) sum += s_acc[v][b][lane];
    const int s = s0 + 16 * (b % NT) + col, n = n0 + 16 * (b / NT) + (lane >> 4) * 4;
    if (s < a.S && n < a.N) {
      const float ds = ldg<float>(a.d + s);
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = (float)sum[j] * (ds * ldg<float>(a.dw + min(n + j, a.N - 1)));
      store4<false>(a, s, n, v[0], v[1], v[2], v[3]);
    }
  }
}

// ---- many tokens -----------------------------------------------------------------
// A workgroup takes BN weight rows x BS tokens; WN x WS waves each their (BN / WN) x (BS /
// WS) part in blocks of v_mfma_i32_32x32x32_i8 (weights as rows, tokens as columns).  Both
// operands go through LDS in stages of kBK bytes of K, NBUF of them: a stage's buffer is
// requested anew as soon as the stage has been read.  KS teams of such waves may share a
// tile, each with every KS-th stage, and add up at the end.  Stages of 128 bytes of K: a
// row of a stage is a whole cache line (rows of 64 bytes reach 64 KB/us a compute unit out
// of L2, rows of 128 120).  The 256 x 256 tile gives a wave 128 x 128 outputs, 256
// accumulators a lane, so that reading LDS takes half the matrix cores' time; smaller
// tiles spread smaller products over the chip.
constexpr int kXcds = 8;

// Where the 16-byte chunk c of a stage's row r lies: the rows' chunks are permuted so that
// lanes reading one chunk of 16 neighbouring rows spread over all banks (no conflicts are
// counted; permuted over 8 rows, 8192 x 12288 x 6144 took 611 us where this took 597).
constexpr int kBK = 128;
__device__ inline int mix_of(int r) { return (r >> 1) & 7; }
__device__ inline int chunk_of(int r, int c) { return r * kBK + ((c ^ mix_of(r)) << 4); }

// One 16-byte load per lane from p straight into LDS, to lds + off + 16 lane (lds
// wave-uniform, off a constant).
__device__ inline __attribute__((always_inline)) void load_to_lds(const int8_t *p, uint32_t lds, int off) {
  asm volatile("s_add_u32 m0, %0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p), "i"(off) : "memory", "m0", "scc");
}

// Waits until at most N of this wave's loads are in flight and its reads of LDS are done,
// then for the workgroup's other waves.  One piece of assembly, so that no access to LDS
// moves between the two.
template <int N>
__device__ inline void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// This wave's writes to LDS are done and seen by its reads.
__device__ inline void own_lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int BN, int BS, int WN, int WS, int NBUF, int KS>
__global__ __launch_bounds__(64 * WN * WS * KS) void k_qmm_tile(QmmArgs a, int tiles_n, int tiles_s, int group) {
  constexpr int kThr = 64 * WN * WS;  // of one of the KS teams
  constexpr int TN = BN / WN / 32, TS = BS / WS / 32;  // 32x32 blocks of a wave
  constexpr int kRows = BN + BS, kStage = kRows * kBK;
  constexpr int kPer = kStage / 16 / kThr;  // chunks a thread moves per stage
  static_assert(kStage % (16 * kThr) == 0, "stage split");
  constexpr int kWide = BN / WN, kLd = kWide + 4;  // a wave's weights, and what a token's sums of them take in LDS
  constexpr int kTurn = WN * WS * 32 * kLd * 4, kEnd = kTurn + kRows * 4;
  constexpr int kSums = KS > 1 ? (KS - 1) * BN * BS * 4 : 0;  // the other teams' sums
  constexpr int kLds = std::max({KS * NBUF * kStage, kEnd, kSums});
  __shared__ __align__(128) uint8_t s_all[kLds];
  const int lane = threadIdx.x & 63;
  const int team = KS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / kThr) : 0;
  const int tid = threadIdx.x - team * kThr, wave = tid >> 6;
  uint8_t *s_buf = s_all + team * NBUF * kStage;
  float *s_sc = (float *)(s_all + kTurn);  // after the last stage: the weights' scales, then the tokens'
  const int wn = wave / WS, wsv = wave % WS;

  // Blocks go to the XCDs round-robin; each XCD gets a contiguous run of tiles, ordered in
  // strips of `group` token tiles so that the tiles in flight on it share operands in its L2.
  const int total = tiles_n * tiles_s;
  const int per = (total + kXcds - 1) / kXcds;
  const int t = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
  if ((int)(blockIdx.x / kXcds) >= per || t >= total) return;
  const int strip = t / (group * tiles_n), in = t - strip * group * tiles_n;
  const int g = min(group, tiles_s - strip * group);
  const int ts = strip * group + in % g, tn = in / g;
  const int n0 = tn * BN, s0 = ts * BS;

  // this thread's chunks of a stage: LDS position tid + i kThr, which holds chunk c of row r
  const int8_t *src[kPer];
  int kc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    constexpr int kC = kBK / 16;  // chunks of a row
    const int p = tid + i * kThr, r = p / kC;
    kc[i] = ((p % kC) ^ mix_of(r)) << 4;
    src[i] = r < BN ? a.w + (int64_t)min(n0 + r, a.N - 1) * a.ldw : a.q + (int64_t)min(s0 + r - BN, a.S - 1) * a.ldq;
  }
  // a team takes every KS-th stage of K; beyond K its stages are zeros
  const int stages = (a.K + KS * kBK - 1) / (KS * kBK);
  const int whole = a.K / kBK;

  i32x16 acc[TN][TS];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TS; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  const int row = lane & 31, ck = lane >> 5;
  // where this lane finds its 16 bytes of k step kk in the wave's first weight and token
  // blocks (32 rows further on they lie 32 kBK bytes further: chunks are mixed over 16 rows)
  constexpr int kSteps = kBK / 32;
  int at_w[kSteps], at_t[kSteps];
#pragma unroll
  for (int kk = 0; kk < kSteps; ++kk) {
    at_w[kk] = chunk_of(wn * (BN / WN) + row, kk * 2 + ck);
    at_t[kk] = chunk_of(BN + wsv * (BS / WS) + row, kk * 2 + ck);
  }
  // fragment f of a k step: the wave's TN weight blocks, then its TS token blocks
  auto frag = [&](const uint8_t *buf, int f, int kk) __attribute__((always_inline)) {
    return *(const i32x4 *)(buf + (f < TN ? at_w[kk] + f * 32 * kBK : at_t[kk] + (f - TN) * 32 * kBK));
  };

  // The wait for a stage leaves the requests of the stages after it in flight, so the
  // requests are written in assembly: a load into LDS known to the compiler makes it
  // wait for all of them before the next read of LDS.  A wave issues one instruction in
  // about four cycles, so what surrounds the MFMAs is kept short: the sources advance by
  // a stage, and only near the end of K are chunks beyond it pointed at zeros.
  constexpr int kF = TN + TS, kM = TN * TS;
  const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)s_buf + wave * 1024);
#pragma unroll
  for (int i = 0; i < kPer; ++i) src[i] += kc[i] + team * kBK;
  auto clip = [&](int s) __attribute__((always_inline)) {  // before stage s is requested
    const int at = s * KS + team;
    if (at >= whole) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if ((int64_t)at * kBK + kc[i] >= a.K) src[i] = (const int8_t *)g_zeros;
    }
  };
  auto request = [&](int i, int buffer) __attribute__((always_inline)) {
    load_to_lds(src[i], lds, buffer * kStage + i * kThr * 16);
    src[i] += KS * kBK;
  };
  // Fragments are read a group of kG k steps ahead, at least 4 MFMAs: they take longer to
  // arrive than one MFMA takes.
  constexpr int kG = kM >= 8 ? 1 : kM >= 4 ? 2 : 4, kGroups = kSteps / kG;
  static_assert(kSteps % kG == 0 && NBUF % 2 == 0, "groups of k steps");
  // A stage's new requests go out over its own last group and the first of the next stage:
  // all in one group they wait for each other (8192x12288x6144: 582 us, 558 over two, 571
  // over four, where the last arrive late).
  constexpr int kSpread = kGroups > 1 ? 2 : 1;
#pragma unroll
  for (int s = 0; s < NBUF; ++s) {
    clip(s);
#pragma unroll
    for (int i = 0; i < (s < NBUF - 1 ? kPer : kPer / kSpread); ++i) request(i, s);
  }
  wait_and_meet<(NBUF - 2) * kPer + kPer / kSpread>();
  i32x4 F[2][kG][kF];
#pragma unroll
  for (int f = 0; f < kG * kF; ++f) F[0][f / kF][f % kF] = frag(s_buf, f % kF, f / kF);
  // Multiply one group's fragments while the next group's are read and, in a stage's last
  // group, the stage just read is requested anew, spread between the MFMAs.
  auto multiply = [&](int cur, int buffer, int g, int again, int r0, int r1) __attribute__((always_inline)) {
    constexpr int kAll = kG * kM;
#pragma unroll
    for (int m = 0; m < kAll; ++m) {
#pragma unroll
      for (int f = 0; f < kG * kF; ++f)
        if (f * kAll / (kG * kF) == m) F[cur ^ 1][f / kF][f % kF] = frag(s_buf + buffer * kStage, f % kF, g * kG + f / kF);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i >= r0 && i < r1 && (i - r0) * kAll / (r1 - r0) == m) request(i, again);
      const int k = m / kM, i = m % kM / TS, j = m % TS;
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(F[cur][k][i], F[cur][k][TN + j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto stage = [&](int s, int b) __attribute__((always_inline)) {  // stage s, in buffer b
    const int cur = b * kGroups & 1;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
      multiply((cur + g - 1) & 1, b, g, (b + NBUF - 1) % NBUF, g < kSpread ? kPer * g / kSpread : 0, g < kSpread ? kPer * (g + 1) / kSpread : 0);
    }
    wait_and_meet<(NBUF - 2) * kPer>();
    clip(s + NBUF);
    multiply((cur + kGroups - 1) & 1, (b + 1) % NBUF, 0, b, 0, kPer / kSpread);
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
  if constexpr (KS > 1) {  // the first team adds the others' sums to its own
    i32x4 *sums = (i32x4 *)s_all;
    constexpr int kAcc = TN * TS * 4;  // pieces of four of a lane
    auto piece = [&](int t, int c) { return ((t - 1) * kAcc + c) * kThr + tid; };
    if (team) {
#pragma unroll
      for (int c = 0; c < kAcc; ++c) {
        const i32x16 &v = acc[c / 4 / TS][c / 4 % TS];
        sums[piece(team, c)] = i32x4{v[c % 4 * 4], v[c % 4 * 4 + 1], v[c % 4 * 4 + 2], v[c % 4 * 4 + 3]};
      }
    }
    __syncthreads();
    if (!team) {
#pragma unroll
      for (int t = 1; t < KS; ++t)
#pragma unroll
        for (int c = 0; c < kAcc; ++c) {
          const i32x4 v = sums[piece(t, c)];
          i32x16 &to = acc[c / 4 / TS][c / 4 % TS];
#pragma unroll
          for (int e = 0; e < 4; ++e) to[c % 4 * 4 + e] += v[e];
        }
    }
    __syncthreads();
  }
  // Each wave turns its sums round in its own part of the buffers, 32 tokens at a time, so
  // that they leave as runs of a token's neighbouring outputs.
  for (int i = threadIdx.x; i < kRows; i += KS * kThr)
    s_sc[i] = i < BN ? ldg<float>(a.dw + min(n0 + i, a.N - 1)) : ldg<float>(a.d + min(s0 + i - BN, a.S - 1));
  __syncthreads();
  if (team) return;
  int *out = (int *)s_buf + wave * 32 * kLd;
  constexpr int kRun = kWide / 4, kTok = 64 / kRun;  // lanes of a token's run, tokens at a time
#pragma unroll
  for (int j = 0; j < TS; ++j) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(i32x4 *)(out + row * kLd + i * 32 + 8 * e + 4 * ck) =
            i32x4{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
    own_lds_done();
    const int nl = wn * kWide + (lane % kRun) * 4;
    const float4 dw = *(const float4 *)(s_sc + nl);
    auto leave = [&](auto stream) __attribute__((always_inline)) {
#pragma unroll 4
      for (int r = lane / kRun; r < 32; r += kTok) {
        const int sl = wsv * (BS / WS) + j * 32 + r;
        const i32x4 v = *(const i32x4 *)(out + r * kLd + (lane % kRun) * 4);
        const float ds = s_sc[BN + sl];
        if (s0 + sl < a.S && n0 + nl < a.N)
          store4<decltype(stream)::value>(a, s0 + sl, n0 + nl, (float)v[0] * (ds * dw.x), (float)v[1] * (ds * dw.y),
                                          (float)v[2] * (ds * dw.z), (float)v[3] * (ds * dw.w));
      }
    };
    if (a.stream) leave(std::true_type());
    else leave(std::false_type());
    own_lds_done();
  }
}

// ---- rows on 16-byte boundaries ------------------------------------------------------
// Copies the token rows, the weight rows or both to the workspace, each at a multiple of
// 16 bytes and with zeros up to one: the loads into LDS need that.  One wave a row.
__global__ __launch_bounds__(256) void k_qmm_align(QmmArgs a, int8_t *q, int8_t *w, int ld) {
  const int64_t rows_q = q ? a.S : 0, rows = rows_q + (w ? a.N : 0);
  for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.x * 4) {
    const int8_t *from = r < rows_q ? a.q + r * a.ldq : a.w + (r - rows_q) * a.ldw;
    int8_t *to = r < rows_q ? q + r * ld : w + (r - rows_q) * ld;
#pragma unroll 2
    for (int k = (threadIdx.x & 63) * 16; k < ld; k += 1024) {
      const i32x4 v = load16_tail(from, k, a.K);
      stg<uint4>(to + k, make_uint4((uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]));
    }
  }
}

// ---- which kernel --------------------------------------------------------------------
enum QmmKernel { kVec, kFew1, kFew2, kTile32, kTile32x64, kTile64, kTile64x128, kTile128, kTile128Two, kTile256 };

bool on16(const int8_t *p, int64_t ld, int rows, int K) {
  return (uintptr_t)p % 16 == 0 && (rows == 1 || ld % 16 == 0) && K % 16 == 0;
}

constexpr int kVecFew = 1024;

struct QmmPlan {
  QmmKernel kernel;
  bool copy_q, copy_w;  // rows that the tiles need on 16-byte boundaries first
  int64_t bytes_q, bytes;  // workspace: of the token rows, of all
};

// The kernel with the least estimated time, fitted to measured ones (us).  A tile kernel:
// 2.5, and for each round of 256 tiles (one a compute unit) a part for its start and end and
// a part for every 128 of K (both with `together` tiles on a unit), or the time in which one
// tile alone gets through K.  The direct kernel: 2.3, and each workgroup moves 39 KB/us.  Of
// 62 shapes measured with every kernel the rule takes the best or one within 7% of it, but
// for a short K with many outputs, whose stores the estimates do not know: 256 x 6144 x 2048
// 11.1 us against 9.2, 512 x 6144 x 2048 14.9 against 13.5, 2048 x 6144 x 2048 37 to 46
// against 37, 4096 x 512 x 144 11.4 against 5.2; and 4 x 4096 x 512, below.
QmmPlan plan_of(const QmmArgs &a) {
  QmmPlan p{};
  const bool q16 = on16(a.q, a.ldq, a.S, a.K), w16 = on16(a.w, a.ldw, a.N, a.K);
  // Up to four tokens by dot products, the direct matrix kernel's time in brackets: 1 x 576 x
  // 6144 2.4 us (5.3), 1 x 4096 x 6144 5.8 (7.1), 4 x 4096 x 6144 6.4 (7.4), 4 x 12288 x 6144
  // 13.2 (14.5); behind it only at four tokens of a short K (4 x 4096 x 512 2.9 (2.6)) or of
  // very many rows (4 x 32768 x 6144 43 (41)).  Up to eight where rows are few and long:
  // 8 x 576 x 6144 3.9 (6.2, by 36 workgroups), 8 x 1024 x 2048 3.5 (3.5), 8 x 1024 x 16384
  // 8.4 (13.2).
  if (a.S <= 4 || (a.S <= 8 && a.N <= kVecFew && a.K >= 2048)) {
    p.kernel = kVec;
    return p;
  }
  struct Tile { QmmKernel kernel; int n, s, together; double once, stage, alone; };
  static constexpr Tile kTiles[] = {
      {kTile32, 32, 32, 1, 1.1, 0.083, 0.095},
      {kTile32x64, 32, 64, 1, 0.6, 0.13, 0.17}, {kTile64, 64, 64, 1, 1.2, 0.195, 0.18},
      {kTile64x128, 64, 128, 1, 3.0, 0.33, 0.22},  {kTile128, 128, 128, 1, 4.6, 0.56, 0},
      {kTile128Two, 128, 128, 2, 3.25, 0.55, 0}, {kTile256, 256, 256, 1, 18.0, 1.45, 0}};
  const double stages = (a.K + 127) / 128;
  const int64_t ld = ((int64_t)a.K + 15) / 16 * 16;
  const double moved = 2.0 * ((q16 ? 0 : a.S * ld) + (w16 ? 0 : a.N * ld));
  const double copy = moved > 0 ? 3.0 + moved / 4e6 : 0.0;
  double best = 1e30;
  for (int nt = 1; nt <= 2; ++nt) {
    const double groups = (double)((a.N + 15) / 16) * ((a.S + 16 * nt - 1) / (16 * nt));
    const double t = 2.3 + std::max(1.0, groups / 256) * 16 * (1 + nt) * a.K / 39e3;
    if (t < best && groups <= 1 << 18) {
      best = t;
      p.kernel = nt == 1 ? kFew1 : kFew2;
    }
  }
  for (const Tile &t : kTiles) {
    const double tiles = (double)((a.N + t.n - 1) / t.n) * ((a.S + t.s - 1) / t.s);
    const double rounds = std::ceil(tiles / (256 * t.together)) * t.together;
    const double us = copy + 2.5 + std::max(rounds * (t.once + t.stage * stages), t.alone * stages);
    if (us < best) {
      best = us;
      p.kernel = t.kernel;
    }
  }
  if (p.kernel >= kTile32) {
    p.copy_q = !q16;
    p.copy_w = !w16;
    p.bytes_q = q16 ? 0 : a.S * ld;
    p.bytes = p.bytes_q + (w16 ? 0 : a.N * ld);
  }
  return p;
}

template <int NS, int R, int KS, bool W4>
void launch_vec(const QmmArgs &a, hipStream_t st) {
  const int rows = R * 4 / KS;
  MOE_LAUNCH((k_qmm_vec<NS, R, KS, W4>), dim3((unsigned)((a.N + rows - 1) / rows)), dim3(256), 0, st, a);
}

// Few rows of a long K: four waves share one (1 x 576 x 16384 2.8 us, 3.3 by one wave).  Two
// rows a wave meet the same tokens where there are tokens to share and rows enough (4 x 4096
// x 6144 6.4 us, 7.1 by one row; 1 x 2048 x 6144 4.1 and 3.7).
template <int NS, bool W4>
void launch_vec_for(const QmmArgs &a, hipStream_t st) {
  if constexpr (NS > 4) {
    launch_vec<NS, 1, 4, W4>(a, st);
  } else if (a.N <= kVecFew && a.K > 8192) {
    launch_vec<NS, 1, 4, W4>(a, st);
  } else {
    if constexpr (NS > 1) {
      if (a.N > 2048) return launch_vec<NS, 2, 1, W4>(a, st);
    }
    launch_vec<NS, 1, 1, W4>(a, st);
  }
}

template <int NT, bool W4>
void launch_few(const QmmArgs &a, hipStream_t st) {
  const unsigned groups = (unsigned)((a.N + 15) / 16) * (unsigned)((a.S + 16 * NT - 1) / (16 * NT));
  MOE_LAUNCH((k_qmm_few<1, NT, 8, W4>), dim3(groups), dim3(512), 0, st, a);
}

template <bool W4>
void launch_direct(const QmmArgs &a, QmmKernel k, hipStream_t st) {
  if (k == kFew1) launch_few<1, W4>(a, st);
  else if (k == kFew2) launch_few<2, W4>(a, st);
  else if (a.S == 1) launch_vec_for<1, W4>(a, st);
  else if (a.S == 2) launch_vec_for<2, W4>(a, st);
  else if (a.S <= 4) launch_vec_for<4, W4>(a, st);
  else launch_vec_for<8, W4>(a, st);
}

template <int BN, int BS, int WN, int WS, int NBUF, int KS>
void launch_tile(const QmmArgs &a, hipStream_t st) {
  const int tn = (a.N + BN - 1) / BN, ts = (a.S + BS - 1) / BS;
  const int64_t total = (int64_t)tn * ts;
  const dim3 g((unsigned)((total + kXcds - 1) / kXcds * kXcds));
  const int group = 4;
  MOE_LAUNCH((k_qmm_tile<BN, BS, WN, WS, NBUF, KS>), g, dim3(64 * WN * WS * KS), 0, st, a, tn, ts, group);
}

}  // namespace

int64_t qmatmul_workspace(const QmmArgs &a) { return plan_of(a).bytes; }

namespace {

void launch_piece(const QmmArgs &a, QmmKernel kernel, hipStream_t st) {
  switch (kernel) {
    case kVec: case kFew1: case kFew2: {
      const bool w4 = (uintptr_t)a.q % 4 == 0 && (uintptr_t)a.w % 4 == 0 && (a.S == 1 || a.ldq % 4 == 0) &&
                      (a.N == 1 || a.ldw % 4 == 0);
      if (w4) launch_direct<true>(a, kernel, st);
      else launch_direct<false>(a, kernel, st);
      break;
    }
    case kTile32: launch_tile<32, 32, 1, 1, 4, 2>(a, st); break;
    case kTile32x64: launch_tile<32, 64, 1, 2, 4, 1>(a, st); break;
    case kTile64: launch_tile<64, 64, 2, 2, 4, 1>(a, st); break;
    case kTile64x128: launch_tile<64, 128, 2, 4, 4, 1>(a, st); break;
    case kTile128: launch_tile<128, 128, 2, 4, 4, 1>(a, st); break;
    case kTile128Two: launch_tile<128, 128, 2, 2, 2, 1>(a, st); break;
    case kTile256: launch_tile<256, 256, 2, 2, 2, 1>(a, st); break;
  }
}

}  // namespace

hipError_t launch_qmatmul(const QmmArgs &a0, hipStream_t st) {
  QmmArgs a = a0;
  a.y_vec = (uintptr_t)a.y % (a.y_bf16 ? 8 : 16) == 0 && a.ldy % 4 == 0;
  a.stream = (int64_t)a.S * a.N * (a.y_bf16 ? 2 : 4) > kStreamBytes;
  const QmmPlan p = plan_of(a);
  if (p.copy_q || p.copy_w) {
    ProfScope ps("qmatmul_align", st);
    int8_t *q = p.copy_q ? a.ws : nullptr, *w = p.copy_w ? a.ws + p.bytes_q : nullptr;
    const int ld = (a.K + 15) / 16 * 16;
    const int64_t rows = (q ? (int64_t)a.S : 0) + (w ? (int64_t)a.N : 0);
    MOE_LAUNCH(k_qmm_align, dim3((unsigned)std::min<int64_t>((rows + 3) / 4, 1 << 18)), dim3(256), 0, st, a, q, w, ld);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (q) a.q = q, a.ldq = ld;
    if (w) a.w = w, a.ldw = ld;
    a.K = ld;
  }
  // a launch holds fewer than 2^32 threads: very long operands go in pieces
  constexpr int kMost = 1 << 18;
  for (int64_t s = 0; s < a.S; s += kMost)
    for (int64_t n = 0; n < a.N; n += kMost) {
      QmmArgs c = a;
      c.S = (int)std::min<int64_t>(kMost, a.S - s);
      c.N = (int)std::min<int64_t>(kMost, a.N - n);
      c.q += s * a.ldq;
      c.w += n * a.ldw;
      c.d += s;
      c.dw += n;
      c.y = (char *)a.y + (s * a.ldy + n) * (a.y_bf16 ? 2 : 4);
      static constexpr const char *kNames[] = {"qmatmul_vec", "qmatmul_few", "qmatmul_few32", "qmatmul_tile32", "qmatmul_tile32x64",
                                               "qmatmul_tile64", "qmatmul_tile64x128", "qmatmul_tile128", "qmatmul_tile128x2", "qmatmul_tile256"};
      ProfScope ps(kNames[p.kernel], st);
      launch_piece(c, p.kernel, st);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace moe
