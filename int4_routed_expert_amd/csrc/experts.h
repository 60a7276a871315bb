// Kernel arguments and launchers of microscaled rows, of products grouped by expert and of
// the grouping and return of tokens.
#pragma once

#include "../../include/moe_grouped.h"
#include "dense.h"

namespace moe {

// mx_quant: x; mx_silu_quant: x is the gate, u the up rows; mx_values: y out, q and e in.
struct MxArgs {
  int S, H, up;
  const void *x, *u;
  uint8_t *q, *e;
  void *y;
  int64_t ldx, ldq, lde, ldy;
};

// Products of rows with weights, both operands in bytes: bf16 elements, or codes of 16 bytes a
// block with a scale byte each.  first == nullptr: one group of T rows.
struct ProdArgs {
  int T, N;
  int row_bytes;  // of a row of x or w: 2 K (bf16), 16 B (microscaled)
  int E, top_k, x_rows, y_bf16;
  bool y_vec;  // four neighbouring outputs may be stored at once
  bool stream;
  const uint8_t *x, *w, *xe, *we;
  int64_t ldx, ldw, ldxe, ldwe, expert, expert_e;  // bytes
  const int32_t *first, *order;
  void *y;
  int64_t ldy;  // elements
  uint8_t *ws;
};

struct GroupArgs {
  int T, E;  // pairs, experts
  const int32_t *idx;
  int32_t *first, *order, *place;
  uint32_t *counts;  // [chunks, E + 1]
};

struct CombineArgs {
  int S, k, H, T, y_bf16;
  bool stream;
  const void *z, *add;
  const float *w;
  const int32_t *place;
  void *y;
  int64_t ldz, lda, ldy;
};

constexpr int kMaxRows = 1 << 24;  // rows of a product, pairs of a grouping

hipError_t launch_mx_quant(const MxArgs &a, int x_bf16, hipStream_t st);
hipError_t launch_mx_silu_quant(const MxArgs &a, int x_bf16, hipStream_t st);
hipError_t launch_mx_values(const MxArgs &a, int y_bf16, hipStream_t st);
int64_t product_workspace(const ProdArgs &a, bool mx);
hipError_t launch_product(const ProdArgs &a, bool mx, hipStream_t st);
int64_t group_workspace(int64_t T, int E);
hipError_t launch_group(const GroupArgs &a, hipStream_t st);
hipError_t launch_combine(const CombineArgs &a, int z_bf16, hipStream_t st);

}  // namespace moe
