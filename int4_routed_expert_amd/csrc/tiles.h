// Device helpers of the matrix products: 16 bytes of a row at any address, and tiles that
// go through LDS.
#pragma once

#include "dense.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

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

constexpr int kXcds = 8;

// Where the 16-byte chunk c of a stage's row r lies: the rows' chunks are permuted so that
// lanes reading one chunk of 16 neighbouring rows spread over all banks (the int8 product
// counts no conflicts; permuted over 8 rows, its 8192 x 12288 x 6144 took 611 us where this
// took 597).
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

}  // namespace
}  // namespace moe
