// The (token, expert) pairs of a routing sorted by expert, and the experts' rows returned to
// their tokens.
#include <algorithm>

#include "experts.h"

namespace moe {
namespace {

// ---- grouping ------------------------------------------------------------------------
// A stable counting sort without atomics in the ranks: a wave takes 64 neighbouring pairs
// at a time, finds the lanes that hold the same expert by one ballot a bit, and keeps its own
// counter per expert in LDS.  Up to kOnePairs pairs one workgroup counts and places all of
// them; beyond, chunks are counted by one launch and placed by a second, each workgroup of
// which adds up the counters of the chunks before its own.  Bound by latency: with 256 experts 8 pairs
// take 5.4 us, 8192 9.5 (18 in one workgroup), 65536 12.3, 2^21 44 us (0.6 TB/s of the pairs' lists).
constexpr int kGroupWaves = 16, kGroupThreads = 64 * kGroupWaves;
constexpr int kOnePairs = 2048;
constexpr int kMostChunks = 256;

__device__ inline int key_of(const GroupArgs &a, int p) {
  const int e = ldg<int32_t>(a.idx + p);
  return (uint32_t)e < (uint32_t)a.E ? e : a.E;
}

// The wave's lanes that hold the same key (bits: how many its values have).
__device__ inline uint64_t same_key(int key, int bits, uint64_t live) {
  uint64_t m = live;
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    m &= (key >> b) & 1 ? set : ~set;
  }
  return m;
}
// Orders the wave's accesses to its own counters: those of all lanes ahead of it first.
__device__ inline void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
__device__ inline int below(uint64_t m) { return __popcll(m & ((1ull << (threadIdx.x & 63)) - 1)); }

// This wave's part [lo, hi) of pairs [begin, end), in whole runs of 64.
__device__ inline void wave_part(int begin, int end, int &lo, int &hi) {
  const int runs = (end - begin + 63) / 64, per = (runs + kGroupWaves - 1) / kGroupWaves, w = threadIdx.x >> 6;
  lo = min(begin + w * per * 64, end);
  hi = min(begin + (w + 1) * per * 64, end);
}

__device__ inline void count_part(const GroupArgs &a, int lo, int hi, int bits, uint32_t *mine) {
  for (int p = lo + (threadIdx.x & 63); p - (int)(threadIdx.x & 63) < hi; p += 64) {
    const bool live = p < hi;
    const int key = live ? key_of(a, p) : 0;
    const uint64_t m = same_key(key, bits, __ballot(live));
    if (live && below(m) == 0) mine[key] += __popcll(m);
    wave_order();
  }
}

__global__ __launch_bounds__(kGroupThreads) void k_group_count(GroupArgs a, int chunk, int bits) {
  __shared__ uint32_t s_count[kGroupWaves * (kMaxE + 1)];  // [waves][E + 1]
  const int keys = a.E + 1;
  for (int i = threadIdx.x; i < kGroupWaves * keys; i += kGroupThreads) s_count[i] = 0;
  __syncthreads();
  const int begin = blockIdx.x * chunk, end = min(begin + chunk, a.T);
  int lo, hi;
  wave_part(begin, end, lo, hi);
  count_part(a, lo, hi, bits, s_count + (threadIdx.x >> 6) * keys);
  __syncthreads();
  for (int k = threadIdx.x; k < keys; k += kGroupThreads) {
    uint32_t n = 0;
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w) n += s_count[w * keys + k];
    stg<uint32_t>(a.counts + (int64_t)blockIdx.x * keys + k, n);
  }
}

__global__ __launch_bounds__(kGroupThreads) void k_group_place(GroupArgs a, int chunk, int chunks, int bits) {
  __shared__ uint32_t s_count[kGroupWaves * (kMaxE + 1)];  // [waves][E + 1]
  __shared__ uint32_t s_all[kGroupWaves], s_before[kGroupWaves];
  const int keys = a.E + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t *mine = s_count + wave * keys;
  for (int i = threadIdx.x; i < kGroupWaves * keys; i += kGroupThreads) s_count[i] = 0;
  __syncthreads();
  const int begin = blockIdx.x * chunk, end = min(begin + chunk, a.T);
  int lo, hi;
  wave_part(begin, end, lo, hi);
  count_part(a, lo, hi, bits, mine);
  __syncthreads();
  static_assert(kMaxE <= kGroupThreads, "thread e takes expert e");
  uint32_t before = 0, all = 0;  // of the chunks before this one, of all
  if ((int)threadIdx.x < a.E) {
    if (chunks > 1) {
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const uint32_t n = ldg<uint32_t>(a.counts + (int64_t)c * keys + threadIdx.x);
        before += c < (int)blockIdx.x ? n : 0;
        all += n;
      }
    } else {
#pragma unroll
      for (int w = 0; w < kGroupWaves; ++w) all += s_count[w * keys + threadIdx.x];
    }
  }
  uint32_t scan = all, sum = before;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t n = (uint32_t)__shfl_up((int)scan, o);
    if (lane >= o) scan += n;
    sum += (uint32_t)__shfl_xor((int)sum, o);
  }
  if (lane == 63) {
    s_all[wave] = scan;
    s_before[wave] = sum;
  }
  __syncthreads();
  uint32_t base = scan - all, valid = 0, kept = 0;  // pairs not dropped: of all, of the chunks before this one
  for (int w = 0; w < kGroupWaves; ++w) {
    if (w < wave) base += s_all[w];
    valid += s_all[w];
    kept += s_before[w];
  }
  if (blockIdx.x == 0) {
    if ((int)threadIdx.x < a.E) stg<int32_t>(a.first + threadIdx.x, (int32_t)base);
    if (threadIdx.x == 0) stg<int32_t>(a.first + a.E, (int32_t)valid);
  }
  if ((int)threadIdx.x < a.E) {
    uint32_t at = base + before;
    for (int w = 0; w < kGroupWaves; ++w) {
      const uint32_t n = s_count[w * keys + threadIdx.x];
      s_count[w * keys + threadIdx.x] = at;
      at += n;
    }
  }
  if (threadIdx.x == 0) {  // the dropped pairs come last
    uint32_t at = valid + (uint32_t)begin - kept;
    for (int w = 0; w < kGroupWaves; ++w) {
      const uint32_t n = s_count[w * keys + a.E];
      s_count[w * keys + a.E] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int p = lo + lane; p - lane < hi; p += 64) {
    const bool live = p < hi;
    const int key = live ? key_of(a, p) : 0;
    const uint64_t m = same_key(key, bits, __ballot(live));
    const int rank = below(m);
    if (live) {
      const int at = (int)mine[key] + rank;
      stg<int32_t>(a.order + at, p);
      stg<int32_t>(a.place + p, key < a.E ? at : -1);
    }
    wave_order();
    if (live && rank == 0) mine[key] += __popcll(m);
    wave_order();
  }
}

__global__ void k_group_none(int32_t *first, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) stg<int32_t>(first + i, 0);
}

int bits_of(int E) {  // of the keys 0 .. E
  int b = 1;
  while (E >> b) ++b;
  return b;
}

int64_t chunks_of(int64_t T) { return T <= kOnePairs ? 1 : std::min<int64_t>(kMostChunks, (T + 1023) / 1024); }

// ---- return --------------------------------------------------------------------------
// A workgroup takes 2048 columns of a token, eight a lane: it reads its k rows in pieces of 16
// bytes, eight rows on their way at once, and adds them up in the order of j (no atomics: a token's
// sum does not depend on the others).  Bound by memory: 8192 tokens of 8 rows of 6144 bf16 193 us, 5.2 TB/s,
// 4096 of 8 fp32 rows of 4096 137 us, 4.9 TB/s; rows off 16 bytes, whose outputs leave one by one: 4096 of 8 rows
// of 5001 97 us (4.2 TB/s), in fp32 176 (4.7).  One token 7.9 us in a graph (launch, places, rows: two trips to
// memory one after the other).
constexpr int kCombineThreads = 256, kCombineCols = 8 * kCombineThreads;

// Eight columns of a row as they lie (bf16 two to a word), those below H; they are made numbers when they
// are added up, so that few registers hold many rows on their way.
template <bool BF16>
struct Cols {
  static constexpr int kWords = BF16 ? 4 : 8;
  uint32_t d[kWords];

  template <bool ON16>
  __device__ inline void load(const void *p, int64_t row, int c, int H) {
    if (c + 8 <= H) {
      if constexpr (BF16 && ON16) {
        const uint4 r = ldg<uint4>((const uint16_t *)p + row + c);
        d[0] = r.x; d[1] = r.y; d[2] = r.z; d[3] = r.w;
      } else {
        float v[8];
        load8<BF16, ON16>(p, row + c, v);
#pragma unroll
        for (int i = 0; i < kWords; ++i) d[i] = BF16 ? __float_as_uint(v[2 * i]) >> 16 | __float_as_uint(v[2 * i + 1]) : __float_as_uint(v[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) d[i] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < H) d[BF16 ? i / 2 : i] |= __float_as_uint(load_el<BF16>(p, row + c + i)) >> (BF16 && i % 2 == 0 ? 16 : 0);
    }
  }
  __device__ inline float at(int i) const {
    if constexpr (BF16) return __uint_as_float(i % 2 ? d[i / 2] & 0xFFFF0000u : d[i / 2] << 16);
    else return __uint_as_float(d[i]);
  }
};

template <bool BF16, bool ON16>
__global__ __launch_bounds__(kCombineThreads) void k_combine(CombineArgs a, int parts) {
  constexpr int kAhead = 8;  // rows on their way at once
  const int64_t s = blockIdx.x / parts;
  const int32_t *place = a.place + s * a.k;
  const float *weight = a.w + s * a.k;
  const int c = (int)(blockIdx.x % parts) * kCombineCols + threadIdx.x * 8;
  if (c >= a.H) return;
  float y[8] = {};
  Cols<BF16> last;
  for (int j0 = 0; j0 < a.k; j0 += kAhead) {
    Cols<BF16> v[kAhead];
    float w[kAhead];
    int p[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int at = min(j0 + j, a.k - 1);
      p[j] = ldk(place + at);
      w[j] = ldk(weight + at);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j0 + j < a.k && (uint32_t)p[j] < (uint32_t)a.T) v[j].template load<ON16>(a.z, p[j] * a.ldz, c, a.H);
    if (a.add && j0 + kAhead >= a.k) last.template load<ON16>(a.add, s * a.lda, c, a.H);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j0 + j < a.k && (uint32_t)p[j] < (uint32_t)a.T) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(w[j], v[j].at(i), y[i]);
      }
  }
  if (a.add) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += last.at(i);
  }
  const int64_t to = s * a.ldy + c;
  if (ON16 && c + 8 <= a.H) {
    if (a.y_bf16) {
      const u32x4_t d = {pack2_bf16(y[0], y[1]), pack2_bf16(y[2], y[3]), pack2_bf16(y[4], y[5]), pack2_bf16(y[6], y[7])};
      put((uint16_t *)a.y + to, d, a.stream);
    } else {
      put((float *)a.y + to, f32x4_t{y[0], y[1], y[2], y[3]}, a.stream);
      put((float *)a.y + to + 4, f32x4_t{y[4], y[5], y[6], y[7]}, a.stream);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.H) {
        if (a.y_bf16) store_el<true>(a.y, to + i, y[i]);
        else store_el<false>(a.y, to + i, y[i]);
      }
  }
}

bool on16(const void *p, int64_t ld, int size) { return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0; }

}  // namespace

int64_t group_workspace(int64_t T, int E) {
  const int64_t n = chunks_of(T);
  return n == 1 ? 0 : n * (E + 1) * 4;
}

hipError_t launch_group(const GroupArgs &a, hipStream_t st) {
  if (a.T == 0) {
    ProfScope ps("group_none", st);
    MOE_LAUNCH(k_group_none, dim3(1), dim3(256), 0, st, a.first, a.E + 1);
    return hipGetLastError();
  }
  const int chunks = (int)chunks_of(a.T), chunk = (int)(((int64_t)a.T + chunks - 1) / chunks), bits = bits_of(a.E);
  if (chunks > 1) {
    ProfScope ps("group_count", st);
    MOE_LAUNCH(k_group_count, dim3(chunks), dim3(kGroupThreads), 0, st, a, chunk, bits);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  ProfScope ps("group_place", st);
  MOE_LAUNCH(k_group_place, dim3(chunks), dim3(kGroupThreads), 0, st, a, chunk, chunks, bits);
  return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs &a0, int z_bf16, hipStream_t st) {
  CombineArgs a = a0;
  const int zs = z_bf16 ? 2 : 4, ys = a.y_bf16 ? 2 : 4;
  const bool vec = on16(a.z, a.ldz, zs) && on16(a.y, a.ldy, ys) && (!a.add || on16(a.add, a.lda, zs));
  a.stream = (int64_t)a.S * a.H * ys > kStreamBytes;
  const int parts = (a.H + kCombineCols - 1) / kCombineCols;
  // a launch holds fewer than 2^32 threads
  const int64_t step = std::max<int64_t>(1, ((int64_t)1 << 23) / parts);
  for (int64_t s = 0; s < a.S; s += step) {
    CombineArgs c = a;
    c.S = (int)std::min<int64_t>(step, a.S - s);
    c.w += s * a.k;
    c.place += s * a.k;
    if (a.add) c.add = (const char *)a.add + s * a.lda * zs;
    c.y = (char *)a.y + s * a.ldy * ys;
    const dim3 g((unsigned)((int64_t)c.S * parts)), b(kCombineThreads);
    ProfScope ps("combine", st);
    if (z_bf16) {
      if (vec) MOE_LAUNCH((k_combine<true, true>), g, b, 0, st, c, parts);
      else MOE_LAUNCH((k_combine<true, false>), g, b, 0, st, c, parts);
    } else {
      if (vec) MOE_LAUNCH((k_combine<false, true>), g, b, 0, st, c, parts);
      else MOE_LAUNCH((k_combine<false, false>), g, b, 0, st, c, parts);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
