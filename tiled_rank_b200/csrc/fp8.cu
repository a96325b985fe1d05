// Quantisers of the fp8 products: rows to e4m3 with one power-of-two scale for
// every 128 columns (optionally gathered, optionally SwiGLU first), and weights
// with one scale for every 128 x 128 block.
//
//   scale = the smallest power of two s with max|v| / s <= 448, at least 2^-126
//           (1 for a block of zeros);  q = v / s rounded to e4m3, ties to even
// A power of two, because the division is then exact and the only rounding is
// the one to e4m3; a floating format loses no precision by it, only up to one
// bit of its range below 2^-6.  Both kernels are one pass over the data: a block
// stays in registers between its maximum and its rounding, and what bounds them
// is memory (2 or 4 bytes in, 1 byte out per value).
#include <cuda_fp8.h>

#include "fp8.cuh"
#include "kernels.cuh"

namespace tileq {
namespace {

// Eight consecutive values, widened; past `n` of them (or unaligned) one by one, zeros behind the end.
__device__ __forceinline__ void load8(const void *base, long long at, int n, int dtype, bool vec, float (&v)[8]) {
  if (vec && n >= 8) {
    if (dtype == TILEQ_DT_F32) {
      const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + at);
      const float4 a = __ldg(p), b = __ldg(p + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 u = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + at));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f;
        if (dtype == TILEQ_DT_BF16) {
          f.x = __uint_as_float(w[i] << 16);
          f.y = __uint_as_float(w[i] & 0xffff0000u);
        } else {
          f = __half22float2(u32_as_h2(w[i]));
        }
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f = 0.f;
    if (i < n) {
      if (dtype == TILEQ_DT_F32)
        f = reinterpret_cast<const float *>(base)[at + i];
      else if (dtype == TILEQ_DT_BF16)
        f = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[at + i]);
      else
        f = __half2float(reinterpret_cast<const __half *>(base)[at + i]);
    }
    v[i] = f;
  }
}

// Bits of max |v|: as integers, so that a NaN or an infinity wins.
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// Scale of a block from the bits of its maximum, and the factor 1 / scale.  With amax = 1.m * 2^k and
// 448 = 1.75 * 2^8 the scale's exponent is k - 8, one more if 1.m > 1.75.  A block with a NaN or an
// infinity becomes NaN as a whole.
__device__ __forceinline__ float scale_of(uint32_t amax, float &inv) {
  if (amax == 0) return inv = 1.f;
  if (amax >= 0x7f800000u) return inv = __uint_as_float(0x7fffffffu);
  const int e = max((int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), 1);
  inv = __uint_as_float((uint32_t)(254 - e) << 23);
  return __uint_as_float((uint32_t)e << 23);
}

__device__ __forceinline__ uint2 round8(const float (&v)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

__device__ __forceinline__ void store8(uint8_t *q, int n, bool vec, uint2 w) {
  if (vec && n >= 8) {
    *reinterpret_cast<uint2 *>(q) = w;
    return;
  }
  const unsigned long long b = (unsigned long long)w.y << 32 | w.x;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) q[i] = (uint8_t)(b >> 8 * i);
}

constexpr int kQRows = 8;    // rows of a CTA, a warp each
constexpr int kQCols = 1024; // columns of a CTA: four loads of 16 bytes in flight per lane

// A warp reads 256 columns at a time, 16 lanes a block of 128.  The scales of
// eight rows leave together: neighbouring rows are neighbours in a scale row, and
// single 4-byte stores would each cost a 32-byte sector.
template <bool SWIGLU>
__global__ void __launch_bounds__(kQRows * 32) quant_rows_kernel(const QuantRowsArgs P) {
  __shared__ float sc[kQCols / 128][kQRows];
  pdl_wait_and_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long r0 = (long long)blockIdx.x * kQRows, r = r0 + warp;
  const int c0 = blockIdx.y * kQCols;
  if (r < P.R) {
    const long long src = P.rows ? P.rows[r] : r;
    const bool live = src >= 0 && src < P.T;  // a row number outside x is padding: a row of zeros
    const float w = P.row_scale ? P.row_scale[r] : 1.f;
    float v[kQCols / 256][8];
#pragma unroll
    for (int u = 0; u < kQCols / 256; ++u) {
      const int c = c0 + u * 256 + lane * 8;
      load8(P.x, src * P.ld_x + c, live ? P.C - c : 0, P.dtype, P.vec_x, v[u]);
    }
    if constexpr (SWIGLU) {
#pragma unroll
      for (int u = 0; u < kQCols / 256; ++u) {
        const int c = c0 + u * 256 + lane * 8;
        float up[8];
        load8(P.x, src * P.ld_x + P.C + c, live ? P.C - c : 0, P.dtype, P.vec_x, up);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] / (1.f + expf(-v[u][i])) * up[i];
      }
    }
    if (P.row_scale && live) {
#pragma unroll
      for (int u = 0; u < kQCols / 256; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] *= w;
    }
#pragma unroll
    for (int u = 0; u < kQCols / 256; ++u) {
      const int c = c0 + u * 256 + lane * 8;
      uint32_t m = amax8(v[u]);
#pragma unroll
      for (int d = 8; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      float inv;
      const float s = scale_of(m, inv);
      store8(P.q + r * P.ld_q + c, P.C - c, P.vec_q, round8(v[u], inv));
      if ((lane & 15) == 0) sc[u * 2 + (lane >> 4)][warp] = s;
    }
  }
  __syncthreads();
  if (threadIdx.x < kQCols / 128 * kQRows) {
    const int b = threadIdx.x / kQRows, i = threadIdx.x % kQRows;
    if (c0 + b * 128 < P.C && r0 + i < P.R) P.scales[(c0 / 128 + b) * P.ld_s + r0 + i] = sc[b][i];
  }
}

// One CTA per 128 x 128 block, 64 values a thread.
__global__ void __launch_bounds__(256) quant_weights_kernel(const QuantWeightsArgs P) {
  __shared__ uint32_t top[8];
  pdl_wait_and_release();
  const long long per = (long long)P.nO * P.nI;
  const int e = (int)(blockIdx.x / per), b = (int)(blockIdx.x % per);
  const int o0 = b / P.nI * 128 + (int)(threadIdx.x >> 4), c = b % P.nI * 128 + (int)(threadIdx.x & 15) * 8;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int o = o0 + 16 * i;
    load8(P.w, e * P.stride_w + o * P.ld_w + c, o < P.d_out ? P.d_in - c : 0, P.dtype, P.vec_w, v[i]);
    m = max(m, amax8(v[i]));
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, top[i]);
  float inv;
  const float s = scale_of(m, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int o = o0 + 16 * i;
    if (o < P.d_out) store8(P.q + e * P.stride_q + o * P.ld_q + c, P.d_in - c, P.vec_q, round8(v[i], inv));
  }
  if (threadIdx.x == 0) P.scales[blockIdx.x] = s;
}

}  // namespace

cudaError_t launch_quant_rows(const QuantRowsArgs &a, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.R + kQRows - 1) / kQRows), (unsigned)((a.C + kQCols - 1) / kQCols));
  const cudaError_t e = launch_pdl(a.swiglu ? quant_rows_kernel<true> : quant_rows_kernel<false>, grid,
                                   dim3(kQRows * 32), 0, stream, a);
  if (e != cudaSuccess) return e;
  count_launches();
  return cudaGetLastError();
}

cudaError_t launch_quant_weights(const QuantWeightsArgs &a, int blocks, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(quant_weights_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  count_launches();
  return cudaGetLastError();
}

}  // namespace tileq
