// Arguments and launch entry points of the fp8 quantisers (fp8.cu).
#pragma once
#include "common.cuh"

namespace tileq {

struct QuantRowsArgs {
  const void *x;           // [T][ld_x], C columns (SwiGLU: C of the gate, then C of the up projection)
  const int32_t *rows;     // [R] row of x of each output row, or null
  const float *row_scale;  // [R] factor of each output row, or null
  uint8_t *q;              // [R][ld_q]
  float *scales;           // [ceil(C / 128)][ld_s]
  long long ld_x, ld_q, ld_s;
  long long R, T;
  int C, dtype, swiglu;
  int vec;                 // the width is a multiple of 8, rows allow 16-byte loads and 8-byte stores
};

struct QuantWeightsArgs {
  const void *w;           // [E][d_out][d_in]
  uint8_t *q;
  float *scales;           // [E][nO][nI]
  long long ld_w, stride_w, ld_q, stride_q;
  int d_out, d_in, nO, nI, dtype, vec;
};

cudaError_t launch_quant_rows(const QuantRowsArgs &a, cudaStream_t stream);
cudaError_t launch_quant_weights(const QuantWeightsArgs &a, int blocks, cudaStream_t stream);

}  // namespace tileq
