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

// Eight consecutive values as loaded (two 16-byte words of fp32, one of 16 bits), and widened.
template <int DT>
struct Raw8 {
  uint4 w[DT == TILEQ_DT_F32 ? 2 : 1];
};
// VEC: one or two 16-byte loads where `live`; else value by value, `n` of them.  Zeros behind the end.
template <int DT, bool VEC>
__device__ __forceinline__ Raw8<DT> load8(const void *base, long long at, int n) {
  Raw8<DT> r;
  if constexpr (VEC) {
    const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(base) + at * (DT == TILEQ_DT_F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (DT == TILEQ_DT_F32 ? 2 : 1); ++i) r.w[i] = n > 0 ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
  } else {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0;
      if (i < n)
        v[i] = DT == TILEQ_DT_F32 ? reinterpret_cast<const uint32_t *>(base)[at + i]
                                  : reinterpret_cast<const uint16_t *>(base)[at + i];
    }
    if constexpr (DT == TILEQ_DT_F32) {
      r.w[0] = make_uint4(v[0], v[1], v[2], v[3]);
      r.w[1] = make_uint4(v[4], v[5], v[6], v[7]);
    } else {
      r.w[0] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void widen(const Raw8<DT> &r, float (&v)[8]) {
  if constexpr (DT == TILEQ_DT_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __uint_as_float(r.w[i].x);
      v[4 * i + 1] = __uint_as_float(r.w[i].y);
      v[4 * i + 2] = __uint_as_float(r.w[i].z);
      v[4 * i + 3] = __uint_as_float(r.w[i].w);
    }
  } else {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == TILEQ_DT_BF16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(u32_as_h2(w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
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

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t *q, int n, uint2 w) {
  if constexpr (VEC) {
    if (n > 0) *reinterpret_cast<uint2 *>(q) = w;
  } else {
    const unsigned long long b = (unsigned long long)w.y << 32 | w.x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint8_t)(b >> 8 * i);
  }
}

constexpr int kQRows = 8;    // rows of a CTA, a warp each
constexpr int kQCols = 1024; // columns of a CTA: four 16-byte loads a lane, issued before the first is used
constexpr int kQU = kQCols / 256;

// A warp reads 256 columns at a time, 16 lanes a block of 128.  The scales of
// eight rows leave together: neighbouring rows are neighbours in a scale row, and
// single 4-byte stores would each cost a 32-byte sector.
// VEC: the width is a multiple of 8 and rows start at 16 (8, of q) bytes.
// What a value goes through is what the gathered case pays for: x comes from L2
// for all but the first of a token's rows, so it is bound by instructions, not by
// HBM.  16-bit values without a factor therefore stay in pairs: the maxima of two
// blocks travel through the shuffles in the halves of one register, and bf16 is
// scaled before it is widened (exact: a power of two; below bf16's normal range
// the result is zero in e4m3 either way).
enum QuantKind { Q_PLAIN = 0, Q_FACTOR = 1, Q_SWIGLU = 2 };

// Maxima of the magnitudes of two loads (16-bit bit patterns, NaN on top): low half a's, high half b's.
template <int DT>
__device__ __forceinline__ uint32_t amax_pair(const Raw8<DT> &a, const Raw8<DT> &b) {
  const auto top = [](const uint4 &w) {
    const uint32_t k = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
  };
  const uint32_t x = top(a.w[0]), y = top(b.w[0]);
  return __vmaxu2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
}

template <int DT>
__device__ __forceinline__ uint2 round8_pairs(const Raw8<DT> &r, float inv) {
  if constexpr (DT == TILEQ_DT_BF16) {
    const __nv_bfloat162 f = __float2bfloat162_rn(inv);
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), f);
      const uint32_t u = *reinterpret_cast<const uint32_t *>(&p);
      h[i] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)),
                                      __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  } else {
    float v[8];
    widen<DT>(r, v);
    return round8(v, inv);
  }
}

template <int DT, QuantKind KIND, bool VEC>
__global__ void __launch_bounds__(kQRows * 32) quant_rows_kernel(const QuantRowsArgs P) {
  constexpr bool SWIGLU = KIND == Q_SWIGLU, PAIRS = KIND == Q_PLAIN && DT != TILEQ_DT_F32;
  __shared__ float sc[kQCols / 128][kQRows];
  pdl_wait_and_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long r0 = (long long)blockIdx.x * kQRows, r = r0 + warp;
  const int c0 = blockIdx.y * kQCols;
  if (r < P.R) {
    const long long src = P.rows ? P.rows[r] : r;
    const bool live = src >= 0 && src < P.T;  // a row number outside x is padding: a row of zeros
    Raw8<DT> raw[kQU], up[SWIGLU ? kQU : 1];
#pragma unroll
    for (int u = 0; u < kQU; ++u) {
      const int c = c0 + u * 256 + lane * 8;
      raw[u] = load8<DT, VEC>(P.x, src * P.ld_x + c, live ? P.C - c : 0);
      if constexpr (SWIGLU) up[u] = load8<DT, VEC>(P.x, src * P.ld_x + P.C + c, live ? P.C - c : 0);
    }
    uint8_t *q = P.q + r * P.ld_q + c0 + lane * 8;
    const int n = P.C - c0 - lane * 8;
    if constexpr (PAIRS) {
#pragma unroll
      for (int u = 0; u < kQU; u += 2) {
        uint32_t m = amax_pair<DT>(raw[u], raw[u + 1]);
#pragma unroll
        for (int d = 8; d; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t top = h ? m >> 16 : m & 0xffffu;
          float inv;
          const float s = scale_of(DT == TILEQ_DT_BF16 ? top << 16 : __float_as_uint(__half2float(__ushort_as_half((uint16_t)top))), inv);
          store8<VEC>(q + (u + h) * 256, n - (u + h) * 256, round8_pairs<DT>(raw[u + h], inv));
          if ((lane & 15) == 0) sc[(u + h) * 2 + (lane >> 4)][warp] = s;
        }
      }
    } else {
      const float w = P.row_scale ? P.row_scale[r] : 1.f;
#pragma unroll
      for (int u = 0; u < kQU; ++u) {
        float v[8];
        widen<DT>(raw[u], v);
        if constexpr (SWIGLU) {
          float b[8];
          widen<DT>(up[u], b);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.f + expf(-v[i])) * b[i];
        }
        if (KIND != Q_PLAIN && live) {  // rows of zeros stay zeros, whatever their factor
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= w;
        }
        uint32_t m = amax8(v);
#pragma unroll
        for (int d = 8; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        float inv;
        const float s = scale_of(m, inv);
        store8<VEC>(q + u * 256, n - u * 256, round8(v, inv));
        if ((lane & 15) == 0) sc[u * 2 + (lane >> 4)][warp] = s;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < kQCols / 128 * kQRows) {
    const int b = threadIdx.x / kQRows, i = threadIdx.x % kQRows;
    if (c0 + b * 128 < P.C && r0 + i < P.R) P.scales[(c0 / 128 + b) * P.ld_s + r0 + i] = sc[b][i];
  }
}

// One CTA per 128 x 128 block, 64 values a thread.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) quant_weights_kernel(const QuantWeightsArgs P) {
  __shared__ uint32_t top[8];
  pdl_wait_and_release();
  const long long per = (long long)P.nO * P.nI;
  const int e = (int)(blockIdx.x / per), b = (int)(blockIdx.x % per);
  const int o0 = b / P.nI * 128 + (int)(threadIdx.x >> 4), c = b % P.nI * 128 + (int)(threadIdx.x & 15) * 8;
  Raw8<DT> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int o = o0 + 16 * i;
    raw[i] = load8<DT, VEC>(P.w, e * P.stride_w + o * P.ld_w + c, o < P.d_out ? P.d_in - c : 0);
  }
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    widen<DT>(raw[i], v[i]);
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
    if (o < P.d_out) store8<VEC>(P.q + e * P.stride_q + o * P.ld_q + c, P.d_in - c, round8(v[i], inv));
  }
  if (threadIdx.x == 0) P.scales[blockIdx.x] = s;
}

template <int DT, QuantKind KIND>
void (*rows_kernel(bool vec))(const QuantRowsArgs) {
  return vec ? quant_rows_kernel<DT, KIND, true> : quant_rows_kernel<DT, KIND, false>;
}
template <int DT>
void (*rows_kernel(const QuantRowsArgs &a))(const QuantRowsArgs) {
  return a.swiglu ? rows_kernel<DT, Q_SWIGLU>(a.vec) : a.row_scale ? rows_kernel<DT, Q_FACTOR>(a.vec) : rows_kernel<DT, Q_PLAIN>(a.vec);
}
template <int DT>
void (*weights_kernel(bool vec))(const QuantWeightsArgs) {
  return vec ? quant_weights_kernel<DT, true> : quant_weights_kernel<DT, false>;
}

}  // namespace

cudaError_t launch_quant_rows(const QuantRowsArgs &a, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.R + kQRows - 1) / kQRows), (unsigned)((a.C + kQCols - 1) / kQCols));
  const auto kern = a.dtype == TILEQ_DT_F32    ? rows_kernel<TILEQ_DT_F32>(a)
                    : a.dtype == TILEQ_DT_BF16 ? rows_kernel<TILEQ_DT_BF16>(a)
                                               : rows_kernel<TILEQ_DT_F16>(a);
  const cudaError_t e = launch_pdl(kern, grid, dim3(kQRows * 32), 0, stream, a);
  if (e != cudaSuccess) return e;
  count_launches();
  return cudaGetLastError();
}

cudaError_t launch_quant_weights(const QuantWeightsArgs &a, int blocks, cudaStream_t stream) {
  const auto kern = a.dtype == TILEQ_DT_F32    ? weights_kernel<TILEQ_DT_F32>(a.vec)
                    : a.dtype == TILEQ_DT_BF16 ? weights_kernel<TILEQ_DT_BF16>(a.vec)
                                               : weights_kernel<TILEQ_DT_F16>(a.vec);
  const cudaError_t e = launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  count_launches();
  return cudaGetLastError();
}

}  // namespace tileq
