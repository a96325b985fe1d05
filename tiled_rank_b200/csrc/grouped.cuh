// Arguments and launch entry point of the experts' grouped products (grouped.cu).
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace tileq {

constexpr int kGroupedMaxE = 256;

// What the product reduces over and writes:
//   GG_FWD  y[p][o]     = sum_i W[e][o][i]  x[p][i]
//   GG_DX   dx[p][i]    = sum_o W[e][o][i] dy[p][o]
//   GG_DW   dW[e][o][i] = sum over the rows p of e of dy[p][o] x[p][i]
enum GroupedMode { GG_FWD = 0, GG_DX = 1, GG_DW = 2 };

struct GroupedArgs {
  // a: the operand of the output's contiguous dimension (128 TMEM lanes per
  // CTA), b: that of the output's rows (TMEM columns); wide fp8: exchanged
  alignas(64) CUtensorMap amap;
  alignas(64) CUtensorMap bmap;
  const int32_t *offsets;  // device [E + 1], or null: one expert with all P rows
  int E, P;
  int L;                   // contiguous output dimension (wide fp8: not used)
  int C;                   // GG_DW: output rows per expert; wide fp8: the contiguous output dimension
  int R;                   // GG_FWD, GG_DX: reduction length
  int splits;              // narrow kernel: CTAs that share a tile's reduction, 1, 2, 4 or 8
  int bf16;                // 16-bit operands: 1 bf16, 0 fp16
  void *out;
  int out_dtype;           // TILEQ_DT_*
  int store_words;         // 16-bit results that one store may take: 1, 2, 8 or 16 neighbours
                           // (fp32: 8 or 16 allow 32-byte stores)
  long long ldo, out_stride;
  const float *xs;         // fp8: scales of the rows [nKb][ld_xs], of the weights [E][nOb][nKb]
  const float *ws;
  long long ld_xs;
  int nOb, nKb;
  int *status;
};

enum GroupedKernel { GG_NARROW = 0, GG_WIDE = 1 };
// Tile of a kernel: TMEM lanes (of the pair, where CTAs work in pairs) and columns, rows of a box of the b operand
// where the reduction is its inner dimension, and whether the experts' rows are on the lanes.
struct GroupedTile {
  int lanes, cols, box_b;
  bool rows_on_lanes;
};
GroupedTile grouped_tile(GroupedKernel k, bool fp8);
// Clusters of `splits` CTAs of the narrow kernel that the current device runs at the same time.
int grouped_clusters(GroupedMode mode, bool fp8, int splits);
// fp8: e4m3 operands with block scales (GG_FWD only).
cudaError_t launch_grouped(const GroupedArgs &a, GroupedKernel k, GroupedMode mode, bool fp8, int grid,
                           cudaStream_t stream);

}  // namespace tileq
