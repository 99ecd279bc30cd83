// What the kernels of the experts' products share: their argument blocks and the tile
// list of the rows.
#pragma once

#include "device_common.h"
#include "host_internal.h"

namespace moe {

// y[r, o] = sum_d x[r, d] W[e][o, d] for the rows r of expert e; W[e] lies as [O, D], or
// as [D, O] (the input's gradient, which contracts over the rows of W), its rows `ws`
// elements apart in both cases.
struct ExpertArgs {
  const uint16_t* x;     // [P, D]
  const uint16_t* w;     // [E] matrices of N C elements
  const int32_t* off;    // [E + 1]
  void* y;               // [P, O] bf16 or fp32
  const int4* list;      // the tiled kernel's
  int64_t w_expert;      // elements of one expert's matrix
  int P, E, D, O, ws;
  int splits;            // of the contraction; with more than one, y is [splits, P, O] fp32 parts
};

// dW[e][n, c] = sum over the rows r of expert e of dy[r, n] x[r, c]
struct ExpertGradArgs {
  const uint16_t* dy;    // [P, N]
  const uint16_t* x;     // [P, C]
  const int32_t* off;
  void* dw;              // [E, N, C] bf16 or fp32
  const int32_t* order;  // [E] experts, those with the most rows first
  int P, E, N, C;
  int splits;            // of every expert's rows; with more than one, dw is [splits, E, N, C] fp32 parts
};

// Rows [lo, hi) of expert e, inside the buffers whatever the offsets hold.
struct RowRange {
  int lo, hi;
};
__device__ __forceinline__ RowRange rows_of(int at, int next, int P) {
  const int lo = min(max(at, 0), P);
  return RowRange{lo, min(max(next, lo), P)};
}

constexpr int kTileRows = 256;   // most rows of a tile
int tile_fragments(int cols);    // the tiles are 32 times as many columns (rows) wide
inline int64_t expert_tiles_bound(int64_t P, int64_t E) { return P / kTileRows + (P < E ? P : E); }

void launch_expert_tiles(const ExpertArgs& a, bool w_trans, bool f32, hipStream_t s);
void launch_expert_wgrad(const ExpertGradArgs& a, bool f32, hipStream_t s);

}  // namespace moe
