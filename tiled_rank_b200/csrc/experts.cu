// C ABI of the experts' products (include/tileq.h): argument checks, tensor maps
// and the choice of kernel.  The kernels are in grouped.cu and fp8.cu.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "fp8.cuh"
#include "grouped.cuh"
#include "kernels.cuh"
#include "share.cuh"

namespace tileq {
namespace {

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
long long round_up(long long v, long long m) { return (v + m - 1) / m * m; }
long long div_up(long long v, long long m) { return (v + m - 1) / m; }

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// Rows and widths are rounded up to whole tiles in 32-bit integers.
constexpr int kMostRows = 0x7fff0000;

struct Operand {
  const void *base;
  int dtype;
  long long cols, rows, mats;  // extents, innermost first; mats == 0: a matrix
  long long ld, stride;        // elements
};

// Tensor map with a box of 128 bytes x box_rows, 128-byte swizzle, zeros outside.
bool encode(CUtensorMap *m, const Operand &o, int box_rows) {
  const auto fn = encoder();
  if (!fn) return false;
  const int es = o.dtype == TILEQ_DT_E4M3 ? 1 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)std::max(o.rows, 1ll), (cuuint64_t)std::max(o.mats, 1ll)};
  const cuuint64_t strides[2] = {(cuuint64_t)(o.ld * es), (cuuint64_t)((o.mats ? o.stride : o.ld) * es)};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType type = o.dtype == TILEQ_DT_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : o.dtype == TILEQ_DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return fn(m, type, 3, const_cast<void *>(o.base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int element_size(int dtype) { return dtype == TILEQ_DT_F32 ? 4 : dtype == TILEQ_DT_E4M3 ? 1 : 2; }
// The offsets and the status word, which no result may overwrite.
bool share_control(const tileq_grouped *g, const void *ws, const Memory &out) {
  return share(out, {g->expert_offsets, 4ll * (g->E + 1)}) || share(out, {ws, TILEQ_GROUPED_WS_BYTES});
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// Strides of the call, contiguous where 0; those of one row or one expert are not used and made valid.
struct Strides {
  long long x, y, w, we;
};
tileq_status strides_of(const tileq_grouped *g, int es, bool w_is_result, Strides *s) {
  const long long q = 16 / es;  // elements of 16 bytes
  s->x = g->ld_x ? g->ld_x : g->d_in;
  s->y = g->ld_y ? g->ld_y : g->d_out;
  s->w = g->ld_w ? g->ld_w : g->d_in;
  if (g->P <= 1) s->x = round_up(std::max<long long>(s->x, g->d_in), q), s->y = round_up(std::max<long long>(s->y, g->d_out), q);
  if (s->x < g->d_in || s->y < g->d_out || s->w < g->d_in) return TILEQ_ERR_INVALID_ARG;
  s->we = g->stride_w ? g->stride_w : s->w * g->d_out;
  const long long matrix = (long long)(g->d_out - 1) * s->w + g->d_in;
  if (g->d_out == 1) s->w = round_up(s->w, q);
  if (g->E == 1) s->we = round_up(std::max(s->we, matrix), q);
  if (s->we < matrix) return TILEQ_ERR_INVALID_ARG;
  // what a tensor map can express
  const long long most = (1ll << 40) - 16;
  if (s->x * es > most || s->y * es > most || (!w_is_result && (s->w * es > most || s->we * es > most)))
    return TILEQ_ERR_UNSUPPORTED;
  return TILEQ_OK;
}

tileq_status check(const tileq_grouped *g, const void *a, const void *b, const void *out, const void *ws,
                   size_t ws_bytes, bool fp8) {
  if (!g || g->E < 1 || g->E > TILEQ_GROUPED_MAX_E || g->P < 0 || g->d_in < 1 || g->d_out < 1) return TILEQ_ERR_INVALID_ARG;
  if (fp8 ? g->dtype != TILEQ_DT_E4M3 : g->dtype != TILEQ_DT_BF16 && g->dtype != TILEQ_DT_F16) return TILEQ_ERR_INVALID_ARG;
  if (g->out_dtype != TILEQ_DT_BF16 && g->out_dtype != TILEQ_DT_F16 && g->out_dtype != TILEQ_DT_F32)
    return TILEQ_ERR_INVALID_ARG;
  if (g->ld_x < 0 || g->ld_y < 0 || g->ld_w < 0 || g->stride_w < 0) return TILEQ_ERR_INVALID_ARG;
  if (!g->expert_offsets && g->E != 1) return TILEQ_ERR_INVALID_ARG;
  if (!aligned4(g->expert_offsets)) return TILEQ_ERR_INVALID_ARG;
  if (!a || !b || !out || !aligned16(a) || !aligned16(b) || !aligned16(out)) return TILEQ_ERR_INVALID_ARG;
  if (!ws) return TILEQ_ERR_INVALID_ARG;
  if (ws_bytes < TILEQ_GROUPED_WS_BYTES) return TILEQ_ERR_WORKSPACE;
  if (g->P > kMostRows || g->d_in > kMostRows || g->d_out > kMostRows) return TILEQ_ERR_UNSUPPORTED;
  return TILEQ_OK;
}

// Rows of the experts that have any, at least: the routing is on the device, so the host goes by P and E.
long long rows_per_expert(const tileq_grouped *g) { return g->P / std::min(g->E, std::max(g->P, 1)); }

// Most tiles of a kernel that the call can have.
long long tile_count(const GroupedTile &t, GroupedMode mode, const tileq_grouped *g, int contig) {
  const long long row_tiles = g->P / (t.rows_on_lanes ? t.lanes : t.cols) + std::min(g->E, g->P);
  const long long other = mode == GG_DW ? g->E * div_up(g->d_out, t.cols) : row_tiles;
  return div_up(contig, t.rows_on_lanes ? t.cols : t.lanes) * other;
}

// The wide kernel (256 x 256 tiles of a pair of CTAs; fp8: 128 x 256 of one) needs experts with rows to fill its
// columns and tiles to fill the GPU; else the narrow one (128 x 64 tiles).  Measured, us narrow / wide:
//   fwd 8 x 4096 -> 14336:   16 rows an expert 154 / 158, 64 rows 175 / 165;   60 x 2048 -> 1408, 68 rows: 70 / 62
//   dx  8 x 14336 -> 4096:   4 rows 138 / 134, 16 rows 145 / 140
//   dx  60 x 1408 -> 2048:   3 rows 52.9 / 55.4, 5 rows 55.6 / 55.7, 7 rows 57.1 / 55.7, 17 rows 58.9 / 57.8
//   fwd 1 x 4096 -> 1536:    256 rows (6 wide tiles) 15.1 / 16.6;   1 x 2048 -> 2048, 1024 rows (32) 19.0 / 11.7
//   fp8 8 x 4096 -> 14336:   12 rows 85 / 90, 16 rows 88 / 91, 24 rows 99 / 93, 64 rows 153 / 96
//   fp8 64 x 4096 -> 1536:   12 rows 80.1 / 77.9, 16 rows 79.7 / 79.1, 18 rows 83.0 / 78.8
//   fp8 1 x 8192 -> 1024:    512 rows (16 wide tiles) 21.1 / 27.6, 1024 rows (32) 32.3 / 27.9
//   fp8 1 x 4096 -> 1536:    256 rows (12 wide tiles) 14.8 / 16.2, 512 rows (24) 18.5 / 16.5
//   dW  512 x 512, 256 rows: 1 expert (4 wide tiles) 5.7 / 6.9, 6 experts (24) 6.7 / 6.9, 60 experts (240) 25.8 / 16.7
GroupedKernel pick(GroupedMode mode, const tileq_grouped *g, int contig, bool fp8) {
  const bool rows = mode == GG_DW || rows_per_expert(g) > (mode == GG_DX ? 6 : 16);
  return rows && tile_count(grouped_tile(GG_WIDE, fp8), mode, g, contig) >= 24 ? GG_WIDE : GG_NARROW;
}

// Where the narrow kernel has too few tiles for the GPU, clusters of CTAs share a tile's reduction, if it is long
// enough: a step takes a CTA about 0.28 us, the sums' meeting 2 us and 0.02 more for every column.  No more clusters
// than run at the same time (clusters of eight leave SMs idle: 16 of them took two rounds).  Measured, us without /
// with:  fwd 1 x 4096 -> 1536, 4 rows: 18.9 / 7.9;  1 x 2048 -> 2048, 64 rows: 12.5 / 10.0;  1 x 512 -> 512, 64 rows
// (8 steps, not taken): 6.9 / 8.2;  dW 512 x 512, 4096 rows: 24.4 / 13.8.
int pick_splits(GroupedMode mode, const tileq_grouped *g, long long tiles, int reduction, bool fp8) {
  const long long rows = rows_per_expert(g), steps = div_up(mode == GG_DW ? rows : reduction, fp8 ? 128 : 64);
  const long long columns = mode == GG_DW ? 64 : std::min(rows, 64ll);
  int best = 1;
  for (int s = 2; s <= 8; s *= 2)
    if (steps >= 2 * s && tiles <= grouped_clusters(mode, fp8, s) && 28 * (steps / best - steps / s) > (best == 1 ? 200 + 2 * columns : 0))
      best = s;
  return best;
}

// contig: the contiguous output dimension; weights and rows: the operands.  The rows' operand lies on the TMEM
// columns, but for the wide fp8 kernel; GG_DW has no weights among its operands, `weights` is x.
tileq_status run(GroupedArgs &a, GroupedMode mode, const tileq_grouped *g, const Operand &weights, const Operand &rows,
                 int contig, bool fp8, cudaStream_t stream) {
  const GroupedKernel k = pick(mode, g, contig, fp8);
  const GroupedTile t = grouped_tile(k, fp8);
  const bool on_lanes = t.rows_on_lanes;
  const int cg = t.lanes / 128;
  a.offsets = g->expert_offsets;
  a.E = g->E;
  a.P = g->P;
  a.L = contig;
  a.C = mode == GG_DW ? g->d_out : contig;
  a.bf16 = g->dtype == TILEQ_DT_BF16;
  a.out_dtype = g->out_dtype;
  const auto all = [&](long long n) { return contig % n == 0 && a.ldo % n == 0 && a.out_stride % n == 0; };
  // out is 16-byte aligned; the 32-byte stores of 16 bf16 or 8 fp32 want more
  const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  a.store_words = wide && all(16) ? 16 : all(8) && (wide || g->out_dtype != TILEQ_DT_F32) ? 8 : all(2) ? 2 : 1;
  const long long tiles = tile_count(t, mode, g, contig);
  if (tiles > (1ll << 30)) return TILEQ_ERR_UNSUPPORTED;
  if (!encode(&a.amap, on_lanes ? rows : weights, mode == GG_FWD ? 128 : 64) ||
      !encode(&a.bmap, on_lanes ? weights : rows, mode == GG_DW ? 64 : t.box_b))
    return TILEQ_ERR_CUDA;
  const int sms = sm_count();
  if (sms < 8) return TILEQ_ERR_CUDA;
  a.splits = k == GG_NARROW ? pick_splits(mode, g, tiles, a.R, fp8) : 1;
  const int group = cg * a.splits;
  const int grid = (int)std::min<long long>(sms / group, k == GG_WIDE ? 2 * tiles : tiles) * group;  // (wide: of half tiles)
  return launch_grouped(a, k, mode, fp8, grid, stream) == cudaSuccess ? TILEQ_OK : TILEQ_ERR_CUDA;
}

}  // namespace
}  // namespace tileq

using namespace tileq;

extern "C" {

tileq_status tileq_grouped_gemm(const tileq_grouped *g, const void *x, const void *w, void *y, void *ws,
                                size_t ws_bytes, tileq_stream_t stream) {
  const bool none = g && g->P == 0;  // nothing is read or written
  tileq_status st = check(g, none ? w : x, w, none ? w : y, ws, ws_bytes, false);
  if (st != TILEQ_OK) return st;
  Strides s;
  if ((st = strides_of(g, 2, false, &s)) != TILEQ_OK) return st;
  if (s.x % 8 || s.w % 8 || s.we % 8) return TILEQ_ERR_UNSUPPORTED;
  if (g->P == 0) return TILEQ_OK;
  const long long eo = element_size(g->out_dtype);
  const Memory out = {y, g->d_out * eo, g->P, s.y * eo};
  if (share(out, {x, g->d_in * 2ll, g->P, s.x * 2}) || share(out, {w, g->d_in * 2ll, g->d_out, s.w * 2, g->E, s.we * 2}) ||
      share_control(g, ws, out))
    return TILEQ_ERR_INVALID_ARG;
  GroupedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.R = g->d_in;
  a.out = y;
  a.ldo = s.y;
  a.status = static_cast<int *>(ws);
  return run(a, GG_FWD, g, {w, g->dtype, g->d_in, g->d_out, g->E, s.w, s.we}, {x, g->dtype, g->d_in, g->P, 0, s.x, 0},
             g->d_out, false, reinterpret_cast<cudaStream_t>(stream));
}

tileq_status tileq_grouped_gemm_dx(const tileq_grouped *g, const void *dy, const void *w, void *dx, void *ws,
                                   size_t ws_bytes, tileq_stream_t stream) {
  const bool none = g && g->P == 0;
  tileq_status st = check(g, none ? w : dy, w, none ? w : dx, ws, ws_bytes, false);
  if (st != TILEQ_OK) return st;
  Strides s;
  if ((st = strides_of(g, 2, false, &s)) != TILEQ_OK) return st;
  if (s.y % 8 || s.w % 8 || s.we % 8) return TILEQ_ERR_UNSUPPORTED;
  if (g->P == 0) return TILEQ_OK;
  const long long eo = element_size(g->out_dtype);
  const Memory out = {dx, g->d_in * eo, g->P, s.x * eo};
  if (share(out, {dy, g->d_out * 2ll, g->P, s.y * 2}) || share(out, {w, g->d_in * 2ll, g->d_out, s.w * 2, g->E, s.we * 2}) ||
      share_control(g, ws, out))
    return TILEQ_ERR_INVALID_ARG;
  GroupedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.R = g->d_out;
  a.out = dx;
  a.ldo = s.x;
  a.status = static_cast<int *>(ws);
  return run(a, GG_DX, g, {w, g->dtype, g->d_in, g->d_out, g->E, s.w, s.we}, {dy, g->dtype, g->d_out, g->P, 0, s.y, 0},
             g->d_in, false, reinterpret_cast<cudaStream_t>(stream));
}

tileq_status tileq_grouped_gemm_dw(const tileq_grouped *g, const void *x, const void *dy, void *dw, void *ws,
                                   size_t ws_bytes, tileq_stream_t stream) {
  if (g && g->P == 0) x = dy = dw;  // zeros are written; the maps' base is never read
  tileq_status st = check(g, x, dy, dw, ws, ws_bytes, false);
  if (st != TILEQ_OK) return st;
  Strides s;
  if ((st = strides_of(g, 2, true, &s)) != TILEQ_OK) return st;
  if (s.x % 8 || s.y % 8) return TILEQ_ERR_UNSUPPORTED;
  const long long eo = element_size(g->out_dtype);
  const Memory out = {dw, g->d_in * eo, g->d_out, s.w * eo, g->E, s.we * eo};
  if (share(out, {x, g->d_in * 2ll, g->P, s.x * 2}) || share(out, {dy, g->d_out * 2ll, g->P, s.y * 2}) ||
      share_control(g, ws, out))
    return TILEQ_ERR_INVALID_ARG;
  GroupedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.out = dw;
  a.ldo = s.w;
  a.out_stride = s.we;
  a.status = static_cast<int *>(ws);
  return run(a, GG_DW, g, {x, g->dtype, g->d_in, g->P, 0, s.x, 0}, {dy, g->dtype, g->d_out, g->P, 0, s.y, 0},
             g->d_in, false, reinterpret_cast<cudaStream_t>(stream));
}

tileq_status tileq_fp8_gemm(const tileq_grouped *g, const void *xq, const float *xs, int64_t ld_xs, const void *wq,
                            const float *w_scales, void *y, void *ws, size_t ws_bytes, tileq_stream_t stream) {
  const bool none = g && g->P == 0;
  tileq_status st = check(g, none ? wq : xq, wq, none ? wq : y, ws, ws_bytes, true);
  if (st != TILEQ_OK) return st;
  if ((!xs && !none) || !w_scales || !aligned4(xs) || !aligned4(w_scales) || ld_xs < 0 || (ld_xs && ld_xs < g->P))
    return TILEQ_ERR_INVALID_ARG;
  Strides s;
  if ((st = strides_of(g, 1, false, &s)) != TILEQ_OK) return st;
  if (s.x % 16 || s.w % 16 || s.we % 16) return TILEQ_ERR_UNSUPPORTED;
  if (g->P == 0) return TILEQ_OK;
  GroupedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.R = g->d_in;
  a.out = y;
  a.ldo = s.y;
  a.xs = xs;
  a.ws = w_scales;
  a.ld_xs = ld_xs ? ld_xs : g->P;
  a.nOb = (int)div_up(g->d_out, 128);
  a.nKb = (int)div_up(g->d_in, 128);
  const long long eo = element_size(g->out_dtype);
  const Memory out = {y, g->d_out * eo, g->P, s.y * eo};
  if (share(out, {xq, g->d_in, g->P, s.x}) || share(out, {wq, g->d_in, g->d_out, s.w, g->E, s.we}) ||
      share(out, {xs, 4ll * g->P, a.nKb, 4 * a.ld_xs}) || share(out, {w_scales, 4ll * g->E * a.nOb * a.nKb}) ||
      share_control(g, ws, out))
    return TILEQ_ERR_INVALID_ARG;
  a.status = static_cast<int *>(ws);
  return run(a, GG_FWD, g, {wq, TILEQ_DT_E4M3, g->d_in, g->d_out, g->E, s.w, s.we},
             {xq, TILEQ_DT_E4M3, g->d_in, g->P, 0, s.x, 0}, g->d_out, true, reinterpret_cast<cudaStream_t>(stream));
}

tileq_status tileq_fp8_quantize(const tileq_fp8_rows *p, const void *x, void *q, float *scales,
                                tileq_stream_t stream) {
  if (!p || p->R < 0 || p->T < 0 || p->C < 1 || (p->swiglu & ~1)) return TILEQ_ERR_INVALID_ARG;
  if (p->dtype != TILEQ_DT_BF16 && p->dtype != TILEQ_DT_F16 && p->dtype != TILEQ_DT_F32) return TILEQ_ERR_INVALID_ARG;
  if (p->ld_x < 0 || p->ld_q < 0 || p->ld_s < 0 || (!p->rows && p->T < p->R)) return TILEQ_ERR_INVALID_ARG;
  if (!aligned4(p->rows) || !aligned4(p->row_scale)) return TILEQ_ERR_INVALID_ARG;
  const long long width = (long long)p->C * (p->swiglu ? 2 : 1);
  const long long ld_x = p->ld_x ? p->ld_x : width, ld_q = p->ld_q ? p->ld_q : p->C, ld_s = p->ld_s ? p->ld_s : p->R;
  if ((p->T > 1 && ld_x < width) || (p->R > 1 && ld_q < p->C) || ld_s < p->R) return TILEQ_ERR_INVALID_ARG;
  if (p->R == 0) return TILEQ_OK;
  if (!q || !scales || !aligned16(q) || !aligned4(scales) || (!x && p->T > 0) || !aligned16(x)) return TILEQ_ERR_INVALID_ARG;
  if (p->C > TILEQ_FP8_MAX_C) return TILEQ_ERR_UNSUPPORTED;
  const int es = element_size(p->dtype);
  const Memory to = {q, p->C, p->R, p->R > 1 ? ld_q : 0}, to_scales = {scales, 4ll * p->R, div_up(p->C, 128), 4 * ld_s};
  const Memory from = {x, width * es, p->T, p->T > 1 ? ld_x * es : 0};
  const Memory of_rows[2] = {{p->rows, 4ll * p->R}, {p->row_scale, 4ll * p->R}};
  if (share(to, to_scales) || share(to, from) || share(to_scales, from)) return TILEQ_ERR_INVALID_ARG;
  for (const Memory &m : of_rows)
    if (share(to, m) || share(to_scales, m)) return TILEQ_ERR_INVALID_ARG;
  QuantRowsArgs a;
  a.x = x;
  a.rows = p->rows;
  a.row_scale = p->row_scale;
  a.q = static_cast<uint8_t *>(q);
  a.scales = scales;
  a.ld_x = ld_x;
  a.ld_q = ld_q;
  a.ld_s = ld_s;
  a.R = p->R;
  a.T = p->T;
  a.C = p->C;
  a.dtype = p->dtype;
  a.swiglu = p->swiglu;
  a.vec = p->C % 8 == 0 && (p->T <= 1 || ld_x * es % 16 == 0) && (!p->swiglu || (long long)p->C * es % 16 == 0) &&
          (p->R <= 1 || ld_q % 8 == 0);
  return launch_quant_rows(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? TILEQ_OK : TILEQ_ERR_CUDA;
}

tileq_status tileq_fp8_quantize_weights(const tileq_grouped *g, const void *w, void *q, int64_t ld_q,
                                        int64_t stride_q, float *scales, tileq_stream_t stream) {
  if (!g || g->E < 1 || g->E > TILEQ_GROUPED_MAX_E || g->d_in < 1 || g->d_out < 1) return TILEQ_ERR_INVALID_ARG;
  if (g->dtype != TILEQ_DT_BF16 && g->dtype != TILEQ_DT_F16 && g->dtype != TILEQ_DT_F32) return TILEQ_ERR_INVALID_ARG;
  if (g->ld_w < 0 || g->stride_w < 0 || ld_q < 0 || stride_q < 0) return TILEQ_ERR_INVALID_ARG;
  QuantWeightsArgs a;
  a.ld_w = g->ld_w ? g->ld_w : g->d_in;
  a.ld_q = ld_q ? ld_q : g->d_in;
  a.stride_w = g->stride_w ? g->stride_w : a.ld_w * g->d_out;
  a.stride_q = stride_q ? stride_q : a.ld_q * g->d_out;
  const auto short_of = [&](long long ld, long long stride) {
    return ld < g->d_in || (g->E > 1 && stride < (long long)(g->d_out - 1) * ld + g->d_in);
  };
  if (short_of(a.ld_w, a.stride_w) || short_of(a.ld_q, a.stride_q)) return TILEQ_ERR_INVALID_ARG;
  if (!w || !q || !scales || !aligned16(w) || !aligned16(q) || !aligned4(scales)) return TILEQ_ERR_INVALID_ARG;
  if (g->d_in > kMostRows || g->d_out > kMostRows) return TILEQ_ERR_UNSUPPORTED;
  const int es = element_size(g->dtype);
  a.w = w;
  a.q = static_cast<uint8_t *>(q);
  a.scales = scales;
  a.d_out = g->d_out;
  a.d_in = g->d_in;
  a.nO = (int)div_up(g->d_out, 128);
  a.nI = (int)div_up(g->d_in, 128);
  a.dtype = g->dtype;
  a.vec = a.d_in % 8 == 0 && a.ld_w * es % 16 == 0 && a.ld_q % 8 == 0 &&
          (g->E == 1 || (a.stride_w * es % 16 == 0 && a.stride_q % 8 == 0));
  const long long blocks = (long long)g->E * a.nO * a.nI;
  if (blocks > 0x7fffffff) return TILEQ_ERR_UNSUPPORTED;
  const Memory to = {q, g->d_in, g->d_out, a.ld_q, g->E, a.stride_q}, to_scales = {scales, 4 * blocks};
  const Memory from = {w, (long long)g->d_in * es, g->d_out, a.ld_w * es, g->E, a.stride_w * es};
  if (share(to, to_scales) || share(to, from) || share(to_scales, from)) return TILEQ_ERR_INVALID_ARG;
  return launch_quant_weights(a, (int)blocks, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? TILEQ_OK
                                                                                                    : TILEQ_ERR_CUDA;
}

}  // extern "C"
