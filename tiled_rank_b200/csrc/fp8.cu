// Quantisers of the fp8 products: rows to e4m3 with one power-of-two scale for
// every 128 columns (optionally gathered, optionally SwiGLU first), and weights
// with one scale for every 128 x 128 block.
//
//   scale = the smallest power of two s with max|v| / s <= 448, at least 2^-126
//           (1 for a block of zeros);  q = v / s rounded to e4m3, ties to even
// A power of two, because the division is then exact and the only rounding is
// the one to e4m3; a floating format loses no precision by it, only up to one
// bit of its range below 2^-6.  Both kernels are one pass over the data: a block
// stays in registers between its maximum and its rounding.  Plain rows and weights
// are bounded by memory (2 or 4 bytes in, 1 byte out per value), gathered rows by
// L2's traffic to the SMs and the ALUs, SwiGLU by the instructions issued.
#include "fp8.cuh"
#include "kernels.cuh"

namespace tileq {
namespace {

// Eight consecutive values as loaded (two 16-byte words of fp32, one of 16 bits), and widened.
template <int DT>
struct Raw8 {
  static constexpr int W = DT == TILEQ_DT_F32 ? 2 : 1;
  uint4 w[W];
};
template <int DT>
__device__ __forceinline__ const char *address(const void *base, long long at) {
  return reinterpret_cast<const char *>(base) + at * (DT == TILEQ_DT_F32 ? 4 : 2);
}
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const char *p) {
  Raw8<DT> r;
#pragma unroll
  for (int i = 0; i < Raw8<DT>::W; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
  return r;
}
// n of the eight values, one by one; zeros behind them.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_some(const char *p, int n) {
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0;
    if (i < n)
      v[i] = DT == TILEQ_DT_F32 ? reinterpret_cast<const uint32_t *>(p)[i] : reinterpret_cast<const uint16_t *>(p)[i];
  }
  Raw8<DT> r;
  if constexpr (DT == TILEQ_DT_F32) {
    r.w[0] = make_uint4(v[0], v[1], v[2], v[3]);
    r.w[1] = make_uint4(v[4], v[5], v[6], v[7]);
  } else {
    r.w[0] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
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

// A maximum travels as 16 bits: the upper half of its fp32 pattern with a lowest bit that says whether anything
// was below it.  That keeps the order and all that the scale depends on (the exponent, and whether the significand
// is above 1.75), and two blocks' maxima fit one register on their way through the shuffles.
__device__ __forceinline__ uint32_t top16(uint32_t bits) { return (bits | ((bits & 0xffffu) + 0xffffu)) >> 16; }

// Bits of max |v|, a NaN above all.
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;\n" : "+f"(m) : "f"(fabsf(v[i])));
  return __float_as_uint(m) & 0x7fffffffu;
}
// Two loads of 16-bit values: low half the pattern of a's largest magnitude, high half b's.
template <int DT>
__device__ __forceinline__ uint32_t amax_pair(const Raw8<DT> &a, const Raw8<DT> &b) {
  const auto top = [](const uint4 &w) {
    const uint32_t k = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
  };
  const uint32_t x = top(a.w[0]), y = top(b.w[0]);
  return __vmaxu2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
}

// Scale of a block from its maximum (top16).  With amax = 1.m * 2^k and 448 = 1.75 * 2^8 the scale's exponent is k - 8,
// one more if 1.m > 1.75: 0x1f carries into the exponent just then.  1 for a block of zeros; a block with an infinity
// or a NaN becomes NaN as a whole.
__device__ __forceinline__ float scale_of(uint32_t top) {
  const int e = max((int)((top + 0x1fu) >> 7) - 8, 1);
  return __uint_as_float(top == 0 ? 0x3f800000u : top >= 0x7f80u ? 0x7fffffffu : (uint32_t)e << 23);
}
// The factors 1 / scale of two blocks from their maxima in the halves of m, as bf16 in the halves of the result.
__device__ __forceinline__ uint32_t inverse_pair(uint32_t m) {
  uint32_t e = ((m + 0x001f001fu) >> 7) & 0x01ff01ffu;
  uint32_t inv = (0x01060106u - __vmaxu2(e, 0x00090009u)) << 7;  // biased exponent 254 - max(e - 8, 1)
  if ((e + 0x00010001u) & 0x01000100u) {                         // e >= 255: near the top of the range, or beyond it
    if ((m & 0xffffu) >= 0x7f80u) inv |= 0x7fffu;
    if (m >> 16 >= 0x7f80u) inv |= 0x7fff0000u;
  }
  return inv;
}

// Four fp32 values to e4m3 (nearest even, cut to +-448), in the order of memory.
__device__ __forceinline__ uint32_t round4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint2 round8(const float (&v)[8], float inv) {
  return make_uint2(round4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    round4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}
// Eight values as loaded; inv2: the factor as bf16 in both halves.  bf16 is scaled before it is widened (exact: a
// power of two; below bf16's normal range the result is zero in e4m3 either way).
template <int DT>
__device__ __forceinline__ uint2 round8(const Raw8<DT> &r, uint32_t inv2) {
  float v[8];
  if constexpr (DT == TILEQ_DT_BF16) {
    const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162 *>(&inv2);
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), f);
      const uint32_t u = *reinterpret_cast<const uint32_t *>(&p);
      v[2 * i] = __uint_as_float(u << 16);
      v[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
    }
    return make_uint2(round4(v[0], v[1], v[2], v[3]), round4(v[4], v[5], v[6], v[7]));
  } else {
    widen<DT>(r, v);
    return round8(v, __uint_as_float(inv2 & 0xffff0000u));
  }
}
__device__ __forceinline__ void store_some(uint8_t *q, int n, uint2 w) {
  const unsigned long long b = (unsigned long long)w.y << 32 | w.x;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) q[i] = (uint8_t)(b >> 8 * i);
}

// g / (1 + exp(-g)) as num / d with e = exp(-|g|), d = 1 + e and num = g or g e: no g overflows the exponential, and d
// in [1, 2] is in the range where __fdividef is within 2 units of the last place.  With expf's 2 units the result is
// within 5 * 2^-23 of silu(g), far below e4m3's half step of 2^-4.  (A division rounded to nearest took 133 us instead
// of 119 for 8192 bf16 rows of 14336.)  An infinity gives an infinity or NaN, and its block becomes NaN.
__device__ __forceinline__ float silu(float g) {
  const float e = expf(-fabsf(g));
  return __fdividef(g < 0.f ? g * e : g, 1.f + e);
}

enum QuantKind { Q_PLAIN = 0, Q_FACTOR = 1, Q_SWIGLU = 2 };

constexpr int kQRows = 8;    // rows of a CTA, a warp each
constexpr int kQCols = 1024; // columns of a CTA: four 16-byte loads a lane, issued before the first is used
constexpr int kQU = kQCols / 256;
static_assert(TILEQ_FP8_MAX_C == 65535 * kQCols, "the grid's second extent");

// A warp's 1024 columns of a row, 16 lanes a block of 128.  x, up: this lane's first value of the gate (or the row)
// and of the up projection; n: values from this lane's first column to the end of the row.
// FULL: all 1024 are there and aligned.
template <int DT, QuantKind KIND, bool VEC, bool FULL>
__device__ __forceinline__ void quant_part(const char *x, const char *up, uint8_t *q, int n, bool live, float factor,
                                           uint32_t *tops, int lane) {
  constexpr bool SWIGLU = KIND == Q_SWIGLU, PAIRS = KIND == Q_PLAIN && DT != TILEQ_DT_F32;
  constexpr int ES = DT == TILEQ_DT_F32 ? 4 : 2;
  Raw8<DT> raw[kQU], ups[SWIGLU ? kQU : 1];
  auto load = [&](const char *p, int u) {
    if constexpr (FULL) return load8<DT>(p + u * 256 * ES);
    // past the end the row's last eight values once more: they are in the block already, or the block is not there
    if constexpr (VEC) return load8<DT>(p + min(u * 256, n - 8) * ES);
    return load_some<DT>(p + u * 256 * ES, n - u * 256);
  };
  if (live) {
#pragma unroll
    for (int u = 0; u < kQU; ++u) {
      raw[u] = load(x, u);
      if constexpr (SWIGLU) ups[u] = load(up, u);
    }
  } else {  // padding: a row of zeros, whatever its factor
#pragma unroll
    for (int u = 0; u < kQU; ++u)
#pragma unroll
      for (int i = 0; i < Raw8<DT>::W; ++i) {
        raw[u].w[i] = make_uint4(0, 0, 0, 0);
        if constexpr (SWIGLU) ups[u].w[i] = make_uint4(0, 0, 0, 0);
      }
    if constexpr (KIND != Q_PLAIN) factor = 1.f;
  }
#pragma unroll
  for (int u = 0; u < kQU; u += 2) {
    float v[2][8];
    uint32_t m;
    if constexpr (PAIRS) {
      m = amax_pair<DT>(raw[u], raw[u + 1]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        widen<DT>(raw[u + h], v[h]);
        if constexpr (SWIGLU) {
          float b[8];
          widen<DT>(ups[u + h], b);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[h][i] = silu(v[h][i]) * b[i];
        }
        if constexpr (KIND != Q_PLAIN) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[h][i] *= factor;
        }
      }
      m = top16(amax8(v[0])) | top16(amax8(v[1])) << 16;
    }
#pragma unroll
    for (int d = 8; d; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
    if constexpr (PAIRS && DT == TILEQ_DT_F16)
      m = top16(__float_as_uint(__half2float(__ushort_as_half((uint16_t)m)))) |
          top16(__float_as_uint(__half2float(__ushort_as_half((uint16_t)(m >> 16))))) << 16;
    if ((lane & 15) == 0) tops[(u + (lane >> 4)) * kQRows] = m;  // blocks 2 u and 2 u + 2, or those behind them
    const uint32_t inv = inverse_pair(m);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t inv2 = __byte_perm(inv, 0, h ? 0x3232 : 0x1010);
      uint2 w;
      if constexpr (PAIRS)
        w = round8<DT>(raw[u + h], inv2);
      else
        w = round8(v[h], __uint_as_float(inv2 & 0xffff0000u));
      uint8_t *to = q + (u + h) * 256;
      if constexpr (FULL) {
        *reinterpret_cast<uint2 *>(to) = w;
      } else if constexpr (VEC) {
        if (n > (u + h) * 256) *reinterpret_cast<uint2 *>(to) = w;
      } else {
        store_some(to, n - (u + h) * 256, w);
      }
    }
  }
}

// One CTA per eight rows x 1024 columns, columns in the outer order: a slice of x that many rows are gathered from
// stays in L2.  131072 gathered bf16 rows of 4096: 168 us in a captured run of calls (181 with inputs that change),
// 0.69 GB through HBM (63 % of measured) and 1.6 GB between L2 and the SMs, the ALUs at 78 %; hence the 16-bit maxima
// and the path for whole parts without any check.  8192 rows of 28672 without a gather: 113 us, 6.3 TB/s.  SwiGLU of
// 8192 bf16 rows of 14336: 119 us for 0.59 GB (91 us at the measured rate), 76 % of the issue slots busy with half of
// the warps that would fit (64 registers).  (Persistent CTAs with the next item's loads in flight: 276 us against 195
// for one item a CTA at the time, as their registers leave a third of the warps; a warp for eight rows: 175 against
// 168.)
// The scales of eight rows leave together: neighbouring rows are neighbours in a scale row, and single 4-byte
// stores would each cost a 32-byte sector.
// VEC: the width is a multiple of 8 and rows start at 16 (8, of q) bytes.
// CTAs per SM: how many warps are there to cover the loads counts for more than a register or two.
template <int DT, QuantKind KIND>
constexpr int quant_ctas() {
  return DT == TILEQ_DT_F32 ? (KIND == Q_SWIGLU ? 2 : 5) : KIND == Q_PLAIN ? 8 : KIND == Q_FACTOR ? 5 : 4;
}

template <int DT, QuantKind KIND, bool VEC>
__global__ void __launch_bounds__(kQRows * 32, quant_ctas<DT, KIND>()) quant_rows_kernel(const QuantRowsArgs P) {
  __shared__ uint32_t tops[kQCols / 256][kQRows];  // two blocks' maxima each: blocks 4 i and 4 i + 2, or 4 i + 1 and 4 i + 3
  pdl_wait_and_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long r0 = (long long)blockIdx.x * kQRows, r = r0 + warp;
  const int c0 = blockIdx.y * kQCols;
  if (r < P.R) {
    const long long src = P.rows ? P.rows[r] : r;
    const bool live = src >= 0 && src < P.T;  // a row number outside x is padding
    const int n = P.C - c0 - lane * 8;
    const char *x = address<DT>(P.x, (live ? src : 0) * P.ld_x + c0 + lane * 8);
    const char *up = address<DT>(x, P.C);
    uint8_t *q = P.q + r * P.ld_q + c0 + lane * 8;
    const float factor = KIND != Q_PLAIN && P.row_scale ? P.row_scale[r] : 1.f;
    if constexpr (VEC) {
      if (c0 + kQCols <= P.C)
        quant_part<DT, KIND, true, true>(x, up, q, n, live, factor, &tops[0][warp], lane);
      else
        quant_part<DT, KIND, true, false>(x, up, q, n, live, factor, &tops[0][warp], lane);
    } else {
      quant_part<DT, KIND, false, false>(x, up, q, n, live, factor, &tops[0][warp], lane);
    }
  }
  __syncthreads();
  if (threadIdx.x < kQCols / 128 * kQRows) {
    const int b = threadIdx.x / kQRows, i = threadIdx.x % kQRows;
    const uint32_t m = tops[(b >> 2) * 2 + (b & 1)][i];
    if (c0 + b * 128 < P.C && r0 + i < P.R) P.scales[(c0 / 128 + b) * P.ld_s + r0 + i] = scale_of(b & 2 ? m >> 16 : m & 0xffffu);
  }
}

// One CTA per 128 x 128 block, 64 values a thread (fp32 ones spill 4 bytes of them).  8 x 14336 x 4096 in bf16: 217 us,
// 6.5 TB/s.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) quant_weights_kernel(const QuantWeightsArgs P) {
  __shared__ uint32_t top[8];
  pdl_wait_and_release();
  const long long per = (long long)P.nO * P.nI;
  const int e = (int)(blockIdx.x / per), b = (int)(blockIdx.x % per);
  const int o0 = b / P.nI * 128 + (int)(threadIdx.x >> 4), c = b % P.nI * 128 + (int)(threadIdx.x & 15) * 8;
  const int n = P.d_in - c;  // values from this thread's first column to the end of the row
  Raw8<DT> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int o = o0 + 16 * i;
    const char *p = address<DT>(P.w, e * P.stride_w + o * P.ld_w + c);
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < Raw8<DT>::W; ++j) raw[i].w[j] = make_uint4(0, 0, 0, 0);
      if (o < P.d_out && n > 0) raw[i] = load8<DT>(p);
    } else {
      raw[i] = load_some<DT>(p, o < P.d_out ? n : 0);
    }
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
  const uint32_t t = top16(m);
  const float inv = __uint_as_float(inverse_pair(t) << 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int o = o0 + 16 * i;
    uint8_t *to = P.q + e * P.stride_q + o * P.ld_q + c;
    if (o < P.d_out) {
      if constexpr (VEC) {
        if (n > 0) *reinterpret_cast<uint2 *>(to) = round8(v[i], inv);
      } else {
        store_some(to, n, round8(v[i], inv));
      }
    }
  }
  if (threadIdx.x == 0) P.scales[blockIdx.x] = scale_of(t);
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
