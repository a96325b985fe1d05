// The experts' grouped products on the 5th-generation tensor cores: forward,
// gradient of the rows, gradient of the weights (GroupedMode), and the forward
// of e4m3 operands with a scale for every 128 of the reduction.  Rows are sorted
// by expert; expert e owns rows offsets[e] .. offsets[e + 1], read on the device.
//
// All three are one tile product with the roles of the operands exchanged:
//   out[c][l] = sum_r A[l][r] B[c][r]
// l, the output's contiguous dimension, lies on the 128 TMEM lanes of a CTA and
// c, its rows, on the TMEM columns:
//   GG_FWD  A = W[e]   (r contiguous)   B = x rows  (r contiguous)   r: d_in
//   GG_DX   A = W[e]^T (l contiguous)   B = dy rows (r contiguous)   r: d_out
//   GG_DW   A = x^T    (l contiguous)   B = dy^T    (c contiguous)   r: rows of e
// Weights on the lanes, so that the ragged dimension (the rows of an expert) is
// the MMA's N, which takes any multiple of 16 or 32 at run time: a short last
// tile costs its own columns only.  The epilogue stores a column's 32 lanes as
// one 64- or 128-byte run of an output row in every mode.
//
// One persistent CTA per SM (CG = 1) or a pair of CTAs on neighbouring SMs that
// share one MMA of 256 lanes (CG = 2: each CTA loads its own 128 rows of A and
// half of B's, so an SM reads 32 KB per 64-element step of a 256 x 256 tile
// instead of 48 KB).  Warps of a CTA:
//   0      producer: TMA tiles (128-byte swizzle) of one 128-byte reduction step
//          per stage into a ring;
//   1      MMA issuer (first CTA of a pair): four MMAs per stage into an fp32
//          TMEM accumulator, two or four accumulators in turn;
//   2      the table of the experts' rows and tiles, before the others start;
//   3      in GG_DW zeroes the rows of the next expert in the last stage of a
//          tile (of both operands: 0 * NaN would be NaN);
//   4..    epilogue: TMEM to registers, one rounding, stores.
// fp8: one 128-byte stage is one scale block.  Every block gets an accumulator
// of its own, which the epilogue warps fold into fp32 registers with
// xs[block][row] * ws[e][l / 128][block]: one FMA per product of sums, as the
// scales are no powers of two in general and cannot be left to the exponent.
// Every wait is bounded and reports TILEQ_ERR_TIMEOUT.
#include "grouped.cuh"

#include <atomic>

#include "kernels.cuh"
#include "tc_pair.cuh"

namespace tileq {
namespace {

constexpr int kScaleGroup = 4;      // fp8: blocks whose scales the fold's warps stage at a time
constexpr int kFirstEpw = 4;        // first epilogue warp
constexpr int kRegsControl = 56, kRegsEpilogue = 224;  // registers a thread where the warps split them
constexpr int kRowTileGroup = 8;    // column tiles that share a pass over the lane tiles

template <int CG_, int BN_, bool F8_>
struct GCfg {
  static constexpr int CG = CG_, BN = BN_;
  static constexpr bool F8 = F8_;
  static constexpr int LANES = 128 * CG;
  static constexpr int KE = F8 ? 128 : 64;  // reduction elements per stage (128 bytes)
  static constexpr int BOX_ROWS = BN == 256 ? 64 : 32;  // rows of one box of a row operand (B of GG_FWD, GG_DX)
  static constexpr int EPW = BN == 256 ? 8 : 4;
  static constexpr int COLS = BN / (EPW / 4);  // columns of one epilogue warp
  static constexpr int THREADS = (kFirstEpw + EPW) * 32;
  static constexpr bool SPLIT_REGS = F8 && BN == 256;
  static constexpr int CHUNK = 16;  // fp8: columns of one TMEM load of the fold
  static constexpr int SCALES = F8 ? 2 * kScaleGroup * BN * 4 : 0;
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = BN / CG * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int TAB = (2 * kGroupedMaxE + 2) * 4;
  static constexpr int SQ = (227 * 1024 - TAB - SCALES - 512) / STAGE;
  // fp8: the columns of a wide tile are two MMAs with accumulators of their own, each folded by its own four
  // epilogue warps: the fold of a part has the other part's MMA time on top of its next one's
  static constexpr int PARTS = F8 && BN == 256 ? 2 : 1;
  static constexpr int PC = BN / PARTS;  // columns of a part
  static constexpr int NACC = BN == 256 ? 2 : 4;
  static constexpr int TMEM_COLS = NACC * BN;
  static constexpr int BAR_OFF = SQ * STAGE;
  static constexpr int SCALE_OFF = BAR_OFF + ((3 * SQ + 2 * NACC * PARTS + 1) * 8 + 31) / 16 * 16;
  static constexpr int TAB_OFF = SCALE_OFF + SCALES;
  static constexpr int SMEM = TAB_OFF + TAB;
  static_assert(TMEM_COLS == 256 || TMEM_COLS == 512, "a power of two of tensor memory columns");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct Tile {
  int e, row0, rows;  // expert and its rows
  int l0, c0, ncols;  // first lane of the tile, first column, columns
};

// The tiles of the call, experts in order; first[e] = tiles before expert e.
// Within an expert the column tiles go in groups that share a pass over the lane
// tiles, so that the CTAs at work read few distinct rows of either operand.
template <class G, GroupedMode MODE>
struct Tiles {
  const int *first, *beg;
  int E, L, nL, C, e = 0;
  __device__ bool get(int w, Tile &t) {
    if (w >= first[E]) return false;
    while (w >= first[e + 1]) ++e;
    const int i = w - first[e], rows = beg[e + 1] - beg[e], total = MODE == GG_DW ? C : rows;
    const int nc = (total + G::BN - 1) / G::BN;
    const int grp = i / (kRowTileGroup * nL), rem = i - grp * kRowTileGroup * nL;
    const int gsz = min(kRowTileGroup, nc - grp * kRowTileGroup);
    const int l = rem / gsz, c = grp * kRowTileGroup + rem % gsz;
    // equal tiles, rounded to the MMA's step: one short tile would leave its CTAs idle
    const int step = 16 * G::CG, tc = ((total + nc - 1) / nc + step - 1) / step * step;
    t.e = e;
    t.row0 = beg[e];
    t.rows = rows;
    t.l0 = l * G::LANES;
    t.c0 = c * tc;
    t.ncols = min(tc, total - t.c0);
    return true;
  }
};

// TMEM to registers in the layout of 8 x 8 blocks (16x256b): of 32 lanes x 32
// columns at taddr, r[h][4 j + 2 g + i] is lane 16 h + 8 g + id / 4, column
// 8 j + 2 (id % 4) + i for thread id.  A thread so holds two neighbouring columns
// of four lanes: a column's scale, wanted by every lane, is read from shared
// memory once for four of them (one lane per thread would be bound by those
// reads), and the block transposes with one instruction for the stores.
// The values are there after wait_block of the same r.
__device__ __forceinline__ void ld_half(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void ld_half(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
template <int N>
__device__ __forceinline__ void ld_block(uint32_t taddr, uint32_t (&r)[2][N]) {
  ld_half(taddr, r[0]);
  ld_half(taddr + (16u << 16), r[1]);
}
// (the registers pass through the asm, so that no use of them moves in front of the wait)
__device__ __forceinline__ void tie(uint32_t (&r)[8]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}
__device__ __forceinline__ void tie(uint32_t (&r)[16]) {
  tie(*reinterpret_cast<uint32_t(*)[8]>(&r[0]));
  tie(*reinterpret_cast<uint32_t(*)[8]>(&r[8]));
}
template <int N>
__device__ __forceinline__ void wait_block(uint32_t (&r)[2][N]) {
  tc::wait_ld();
  tie(r[0]);
  tie(r[1]);
}
// acc += v * s, two fp32 FMAs in one instruction
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t v, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;\n" : "+l"(acc) : "l"(v), "l"(s));
}
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// mbar_wait by a whole warp with one answer: no lane leaves a loop in which the others still meet.
// (`remote`: the pair's other CTA has written memory before it arrived.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *status, bool remote = false) {
  return __all_sync(0xffffffffu, remote ? tc::mbar_wait_cluster(bar, parity, status) : mbar_wait(bar, parity, status));
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == TILEQ_DT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    return h2_as_u32(__floats2half2_rn(lo, hi));
  }
}

// Stores 8 columns (n of them exist) x 32 lanes (nl exist) to out + column * ldo + lane;
// v[g]: this thread's two columns of lane 8 g + id / 4.  16-bit results are
// transposed as 8 x 8 blocks, which leaves thread id the lanes 8 g + 2 (id % 4) + 0, 1
// of column id / 4; WORDS is how much of them one store may take: 1 a value, 2 the
// pair, 8 a run of eight lanes after a transposition among the four threads of a column.
template <int DT, int WORDS>
__device__ __forceinline__ void store_b16(uint16_t *out, long long ldo, int n, int nl, int id, const uint64_t (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int g = 0; g < 4; ++g)
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(w[g]) : "r"(pack2<DT>(low(v[g]), high(v[g]))));
  const int q = id & 3;
  out += (id >> 2) * ldo;
  const bool in = (id >> 2) < n;
  if constexpr (WORDS == 8) {
    const bool b0 = q & 1, b1 = q & 2;
    const uint32_t x = __shfl_xor_sync(0xffffffffu, b0 ? w[0] : w[1], 1);
    const uint32_t y = __shfl_xor_sync(0xffffffffu, b0 ? w[2] : w[3], 1);
    const uint32_t a0 = b0 ? x : w[0], a1 = b0 ? w[1] : x, a2 = b0 ? y : w[2], a3 = b0 ? w[3] : y;
    const uint32_t u = __shfl_xor_sync(0xffffffffu, b1 ? a0 : a2, 2);
    const uint32_t z = __shfl_xor_sync(0xffffffffu, b1 ? a1 : a3, 2);
    if (in && q * 8 < nl)
      *reinterpret_cast<uint4 *>(out + q * 8) = b1 ? make_uint4(u, z, a2, a3) : make_uint4(a0, a1, u, z);
  } else {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int l = 8 * g + 2 * q;
      if constexpr (WORDS == 2) {
        if (in && l < nl) *reinterpret_cast<uint32_t *>(out + l) = w[g];
      } else {
        if (in && l < nl) out[l] = (uint16_t)w[g];
        if (in && l + 1 < nl) out[l + 1] = (uint16_t)(w[g] >> 16);
      }
    }
  }
}
template <int DT>
__device__ __forceinline__ void store_b16(const GroupedArgs &P, long long base, int n, int nl, int id, const uint64_t (&v)[4]) {
  uint16_t *out = reinterpret_cast<uint16_t *>(P.out) + base;
  if (P.store_words == 8)
    store_b16<DT, 8>(out, P.ldo, n, nl, id, v);
  else if (P.store_words == 2)
    store_b16<DT, 2>(out, P.ldo, n, nl, id, v);
  else
    store_b16<DT, 1>(out, P.ldo, n, nl, id, v);
}
__device__ __forceinline__ void store_block(const GroupedArgs &P, long long base, int n, int nl, int id, const uint64_t (&v)[4]) {
  if (P.out_dtype == TILEQ_DT_F32) {
    float *out = reinterpret_cast<float *>(P.out) + base + 2 * (id & 3) * P.ldo + (id >> 2);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (8 * g + (id >> 2) < nl) {
        if (2 * (id & 3) < n) out[8 * g] = low(v[g]);
        if (2 * (id & 3) + 1 < n) out[P.ldo + 8 * g] = high(v[g]);
      }
  } else if (P.out_dtype == TILEQ_DT_BF16) {
    store_b16<TILEQ_DT_BF16>(P, base, n, nl, id, v);
  } else {
    store_b16<TILEQ_DT_F16>(P, base, n, nl, id, v);
  }
}

template <class G, GroupedMode MODE>
__global__ void __launch_bounds__(G::THREADS, 1) grouped_kernel(const __grid_constant__ GroupedArgs P) {
  constexpr int CG = G::CG, SQ = G::SQ, NACC = G::NACC, PARTS = G::PARTS;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle wants tiles at multiples of 1024
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + G::BAR_OFF);
  uint64_t *empty = full + SQ;
  uint64_t *acc_full = empty + SQ;
  uint64_t *acc_empty = acc_full + PARTS * NACC;  // both [PARTS][NACC]
  uint64_t *tail = acc_empty + PARTS * NACC;  // [SQ] GG_DW: the copies of a stage with foreign rows
  uint64_t *drain = tail + SQ;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  float *scale = reinterpret_cast<float *>(smem + G::SCALE_OFF);
  int *first = reinterpret_cast<int *>(smem + G::TAB_OFF), *beg = first + kGroupedMaxE + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : tc::cluster_rank();
  const int unit0 = blockIdx.x / CG, units = gridDim.x / CG;
  auto stage_a = [&](int s) { return smem + s * G::STAGE; };
  auto stage_b = [&](int s) { return smem + s * G::STAGE + G::A_BYTES; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < SQ; ++s) {
      mbar_init(&full[s], CG);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
    }
    for (int b = 0; b < PARTS * NACC; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], G::EPW / PARTS * CG);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) tc::alloc_cg<CG>(tmem_slot, G::TMEM_COLS);
  // the prologue overlaps the previous kernel's tail
  pdl_wait_and_release();
  if (warp == 2) {
    // rows and tiles of each expert; offsets outside [0, P] are cut to it, one below its predecessor is raised to it
    int before = 0, top = P.offsets ? min(max(P.offsets[0], 0), P.P) : 0;
    if (lane == 0) beg[0] = top;
    for (int e0 = 0; e0 < P.E; e0 += 32) {
      const int e = e0 + lane;
      int hi = top;
      if (e < P.E) hi = P.offsets ? min(max(P.offsets[e + 1], top), P.P) : P.P;
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, hi, d);
        if (lane >= d) hi = max(hi, o);
      }
      int lo = __shfl_up_sync(0xffffffffu, hi, 1);
      if (lane == 0) lo = top;
      int sum = e < P.E ? P.nL * (((MODE == GG_DW ? P.C : hi - lo) + G::BN - 1) / G::BN) : 0;
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      if (e < P.E) beg[e + 1] = hi, first[e + 1] = before + sum;
      before += __shfl_sync(0xffffffffu, sum, 31);
      top = __shfl_sync(0xffffffffu, hi, 31);
    }
    if (lane == 0) first[0] = 0;
  }
  tc::fence_before();
  __syncthreads();
  if constexpr (CG == 2) tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;

  Tiles<G, MODE> tiles{first, beg, P.E, P.L, P.nL, P.C};
  auto steps = [&](const Tile &t) { return ((MODE == GG_DW ? t.rows : P.R) + G::KE - 1) / G::KE; };
  // columns of one part's MMA
  auto mma_n = [&](const Tile &t) { return (t.ncols + 16 * CG * PARTS - 1) / (16 * CG * PARTS) * (16 * CG); };
  Tile t;
  bool ok = true;

  if constexpr (G::SPLIT_REGS) {
    if (warp < kFirstEpw) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsControl));
  }
  if (warp == 0) {
    // ============================================================ producer
    uint32_t qi = 0;
    for (int w = unit0; ok && tiles.get(w, t); w += units) {
      const int nk = steps(t), half = mma_n(t) / CG;
      const int l0 = t.l0 + (int)rank * 128, c0 = t.c0 + (int)rank * half;
      constexpr int ABOX = MODE == GG_FWD ? 1 : 2;         // boxes of A: 128 rows, or twice 64 columns
      constexpr int BBOX = MODE == GG_DW ? 64 : G::BOX_ROWS;  // columns of the tile in one box of B
      const int nbox = PARTS == 2 ? 2 : (half + BBOX - 1) / BBOX;
      const int bstep = PARTS == 2 ? half * CG : BBOX;  // columns from one box to the next (two parts: a box each)
      const uint32_t bytes = G::A_BYTES + nbox * BBOX * 128;
      for (int kb = 0; kb < nk; ++kb, ++qi) {
        const int s = qi % SQ;
        const int left = MODE == GG_DW ? t.rows - kb * G::KE : G::KE;
        const bool cut = left < G::KE && (left & 15);  // the last MMA of the step reaches the next expert's rows
        if (qi >= (uint32_t)SQ && !(ok = warp_wait(&empty[s], ((qi / SQ) - 1) & 1, P.status))) break;
        const uint32_t bar = cut ? smem_addr(&tail[s]) : CG == 2 ? tc::map_cta(&full[s], 0) : smem_addr(&full[s]);
        if (lane == 0) {
          if (cut || CG == 1)
            mbar_arrive_expect_tx(cut ? &tail[s] : &full[s], bytes);
          else
            tc::arrive_expect_at(bar, bytes);
        }
        // one lane per box: a single lane would need the time of a whole stage to issue five or six copies
        if (lane < ABOX + nbox) {
          const bool is_a = lane < ABOX;
          const int i = is_a ? lane : lane - ABOX;
          uint8_t *dst = is_a ? stage_a(s) + i * 8192 : stage_b(s) + i * BBOX * 128;
          const CUtensorMap *map = is_a ? &P.amap : &P.bmap;
          int x, y, z = 0;
          if (MODE == GG_FWD || (MODE == GG_DX && !is_a)) {
            x = kb * G::KE;
            y = is_a ? l0 : t.row0 + c0 + i * bstep;
          } else {
            x = (is_a ? l0 : c0) + i * 64;
            y = (MODE == GG_DW ? t.row0 : 0) + kb * 64;
          }
          if (is_a && MODE != GG_DW) z = t.e;
          tc::tma_3d<CG>(dst, map, x, y, z, bar);
        }
      }
    }
    // no copy of this CTA may land and no commit may arrive after it has gone
    if (lane == 0)
      for (uint32_t i = qi > (uint32_t)SQ ? qi - SQ : 0; ok && i < qi; ++i)
        ok = mbar_wait(&empty[i % SQ], (i / SQ) & 1, P.status);
    if (lane == 0 && !ok && rank == 0)
      for (uint32_t i = qi > (uint32_t)SQ ? qi - SQ : 0; i < qi; ++i) mbar_wait(&full[i % SQ], (i / SQ) & 1, P.status);
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    if (rank == 0) {
      constexpr bool A_MN = MODE != GG_FWD, B_MN = MODE == GG_DW;  // output dimension contiguous
      const uint32_t fmt = P.bf16 && !G::F8 ? (1u << 7) | (1u << 10) : 0u;
      uint32_t qi = 0, ai = 0;
      for (int w = unit0; ok && tiles.get(w, t); w += units) {
        const int nk = steps(t);
        if (nk == 0) continue;
        const uint32_t idesc = (1u << 4) | fmt | ((uint32_t)A_MN << 15) | ((uint32_t)B_MN << 16) |
                               ((uint32_t)(mma_n(t) >> 3) << 17) | ((uint32_t)(G::LANES >> 4) << 24);
        for (int kb = 0; kb < nk; ++kb, ++qi) {
          const int s = qi % SQ, ab = ai % NACC;
          const bool cut = MODE == GG_DW && kb == nk - 1 && (t.rows & 15);  // the producers zeroed rows
          if (!(ok = warp_wait(&full[s], (qi / SQ) & 1, P.status, cut))) break;
          // 16 (fp8: 32) reduction elements per MMA: 32 bytes along a row, or 16 rows
          const int nmma = MODE == GG_DW ? min(4, (t.rows - kb * 64 + 15) / 16) : 4;
          const uint64_t ad = tc::sdesc(smem_addr(stage_a(s)), A_MN ? 8192 : 16);
          const uint64_t bd = tc::sdesc(smem_addr(stage_b(s)), B_MN ? 8192 : 16);
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
            const int pa = part * NACC + ab;
            if ((G::F8 || kb == 0) && ai >= (uint32_t)NACC &&
                !(ok = warp_wait(&acc_empty[pa], ((ai / NACC) - 1) & 1, P.status)))
              break;
            tc::fence_after();
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (MODE != GG_DW || kk < nmma)
                  tc::mma_ss<CG, G::F8>(tmem + pa * G::PC, ad + (uint64_t)(kk * (A_MN ? 128 : 2)),
                                        bd + (uint64_t)(kk * (B_MN ? 128 : 2) + part * (8192 >> 4)), idesc,
                                        (kk || (!G::F8 && kb)) ? 1u : 0u);
              if (part == PARTS - 1) tc::commit_cg<CG>(&empty[s]);
              if (G::F8 || kb == nk - 1) tc::commit_cg<CG>(&acc_full[pa]);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (G::F8 || kb == nk - 1) ++ai;
        }
      }
      // all issued MMAs have retired before tensor memory is released
      if (tc::elect_one()) tc::commit_cg<CG>(drain);
      __syncwarp();
      warp_wait(drain, 0, P.status);
    }
  } else if (warp == 3) {
    // ============================================================ rows of the next expert (GG_DW)
    // A warp of its own, because the copies have to land first: the producer would lose that time for every tile.
    if constexpr (MODE == GG_DW) {
      uint32_t q0 = 0, phase = 0;  // phase: bit s, the use of tail[s]
      for (int w = unit0; ok && tiles.get(w, t); w += units) {
        const int nk = steps(t), left = t.rows & 63;
        q0 += nk;
        if (!(left & 15)) continue;
        const int s = (q0 - 1) % SQ, to = (left + 15) & ~15, nbox = (mma_n(t) / CG + 63) / 64;
        if (!(ok = warp_wait(&tail[s], phase >> s & 1, P.status))) break;
        phase ^= 1u << s;
        for (int i = lane; i < (to - left) * 8; i += 32) {
          const int off = (left + i / 8) * 128 + (i % 8) * 16;  // whole rows: the swizzle stays inside a row
          for (int j = 0; j < 2; ++j) *reinterpret_cast<uint4 *>(stage_a(s) + j * 8192 + off) = make_uint4(0, 0, 0, 0);
          for (int j = 0; j < nbox; ++j) *reinterpret_cast<uint4 *>(stage_b(s) + j * 8192 + off) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::arrive_at(tc::map_cta(&full[s], 0));
      }
    }
  } else if (warp >= kFirstEpw) {
    // ============================================================ epilogue
    // 128 accumulators a thread: the register file has room for them once the first four warps give theirs up
    // (168 registers a thread at launch: 384 * 168 = 128 * (56 + 2 * 224))
    if constexpr (G::SPLIT_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsEpilogue));
    const int half = (warp - kFirstEpw) >> 2;
    const uint32_t lane_addr = tc::lane_base(warp);  // TMEM lane quadrant of this warp
    uint32_t ai = 0, gi = 0;
    // (fp8: the four warps of a named barrier stay together, also after a wait that gave up)
    for (int w = unit0; (ok || G::F8) && tiles.get(w, t); w += units) {
      const int nk = steps(t), l0 = t.l0 + (int)rank * 128 + (warp & 3) * 32;
      const int cw = half * (PARTS == 2 ? mma_n(t) : G::COLS);              // first column of this warp
      const int mine = min(t.ncols - cw, PARTS == 2 ? mma_n(t) : G::COLS);  // its columns, none if <= 0
      const int nl = P.L - l0;
      const long long base = (MODE == GG_DW ? (long long)t.e * P.out_stride + (long long)(t.c0 + cw) * P.ldo
                                            : (long long)(t.row0 + t.c0 + cw) * P.ldo) + l0;
      if constexpr (!G::F8) {
        const int ab = ai % NACC;
        if (nk > 0) {
          if (!(ok = warp_wait(&acc_full[ab], (ai / NACC) & 1, P.status))) break;
          tc::fence_after();
        }
#pragma unroll 1
        for (int c = 0; c < mine; c += 32) {
          uint32_t r[2][16];
          if (nk > 0) {
            ld_block(tmem + lane_addr + ab * G::BN + cw + c, r);
            wait_block(r);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint64_t v[4];
#pragma unroll
            for (int g = 0; g < 4; ++g)  // an expert without rows: zeros
              v[g] = nk > 0 ? pair(r[g >> 1][4 * j + 2 * (g & 1)], r[g >> 1][4 * j + 2 * (g & 1) + 1]) : 0;
            store_block(P, base + (c + 8 * j) * P.ldo, mine - c - 8 * j, nl, lane, v);
          }
        }
        if (nk > 0) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::arrive_relaxed_at(tc::map_cta(&acc_empty[ab], 0));
          ++ai;
        }
      } else {
        constexpr int CH = G::CHUNK, NCH = G::COLS / CH, GROUPS = CH / 8;
        uint64_t acc[G::COLS / 8][4];  // [8 columns][lane block]: two columns, folded by one packed FMA
#pragma unroll
        for (int i = 0; i < G::COLS / 8; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) acc[i][g] = 0;
        const int part = PARTS == 2 ? half : 0, col0 = PARTS == 2 ? 0 : cw;
        // scales of kScaleGroup blocks at a time: thread tid's column (the last one where it has none) and block,
        // fetched while the group before is folded
        const int tid = threadIdx.x & 127;  // within the four warps that share these columns
        const float *xs = P.xs + t.row0 + t.c0 + (mine > 0 ? cw + min(tid, mine - 1) : 0);
        const float *ws = P.ws + ((long long)t.e * P.nLb + min((t.l0 + (int)rank * 128) / 128, P.nLb - 1)) * P.nKb;
        float sx[kScaleGroup], sw[kScaleGroup];
        auto fetch = [&](int kb) {
#pragma unroll
          for (int j = 0; j < kScaleGroup; ++j) {
            const int k = min(kb + j, nk - 1);
            sx[j] = __ldg(xs + k * P.ld_xs);
            sw[j] = __ldg(ws + k);
          }
        };
        fetch(0);
#pragma unroll 1
        for (int kg = 0; kg < nk; kg += kScaleGroup) {
          float *sc = scale + (gi++ & 1) * kScaleGroup * G::BN + half * G::COLS;
          if (G::COLS == 128 || tid < G::COLS) {
#pragma unroll
            for (int j = 0; j < kScaleGroup; ++j) sc[j * G::BN + tid] = sx[j] * sw[j];
          }
          fetch(kg + kScaleGroup);
          // also keeps these warps within one group of each other: two buffers of scales do
          named_sync(1 + half, 128);
          sc += 2 * (lane & 3);
#pragma unroll 1
          for (int kb = kg; kb < min(kg + kScaleGroup, nk); ++kb, ++ai, sc += G::BN) {
            const int pa = part * NACC + ai % NACC;
            ok = ok && warp_wait(&acc_full[pa], (ai / NACC) & 1, P.status);
            tc::fence_after();
            const uint32_t ta = tmem + lane_addr + pa * G::PC + col0;
            uint32_t r[2][2][CH / 2];
            if (mine > 0) {
              ld_block(ta, r[0]);
#pragma unroll
              for (int ch = 0; ch < NCH; ++ch) {
                if (ch * CH < mine) {
                  wait_block(r[ch & 1]);
                  if (ch + 1 < NCH && (ch + 1) * CH < mine) ld_block(ta + (ch + 1) * CH, r[(ch + 1) & 1]);
#pragma unroll
                  for (int j = 0; j < GROUPS; ++j) {
                    const uint64_t s = *reinterpret_cast<const uint64_t *>(sc + ch * CH + 8 * j);
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                      fma2(acc[ch * GROUPS + j][g],
                           pair(r[ch & 1][g >> 1][4 * j + 2 * (g & 1)], r[ch & 1][g >> 1][4 * j + 2 * (g & 1) + 1]), s);
                  }
                }
              }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::arrive_relaxed_at(tc::map_cta(&acc_empty[pa], 0));
          }
        }
#pragma unroll
        for (int j = 0; j < G::COLS / 8; ++j)
          if (ok && 8 * j < mine) store_block(P, base + 8 * j * P.ldo, mine - 8 * j, nl, lane, acc[j]);
      }
    }
  }

  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if constexpr (CG == 2) {
    // the last commit arrives in both CTAs; only here, where it is due, can a bounded wait for it start
    if (rank == 1 && warp == 1) warp_wait(drain, 0, P.status);
    __syncwarp();
    tc::cluster_sync();
  }
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc_cg<CG>(tmem, G::TMEM_COLS);
  }
}

using Narrow = GCfg<1, 64, false>;
using NarrowF8 = GCfg<1, 64, true>;
using Wide = GCfg<2, 256, false>;
using WideF8 = GCfg<2, 256, true>;

template <class G, GroupedMode MODE>
cudaError_t launch_one(const GroupedArgs &a, int grid, cudaStream_t stream) {
  auto kern = grouped_kernel<G, MODE>;
  static std::atomic<uint64_t> configured{0};  // one attribute call per instantiation and device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e != cudaSuccess) return e;
    if (G::SPLIT_REGS) {
      // the split asks for no more registers than the block is launched with, or it would wait forever
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
      if (fa.numRegs * G::THREADS < 128 * (kRegsControl + 2 * kRegsEpilogue)) return cudaErrorInvalidConfiguration;
    }
    configured.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(G::THREADS);
  cfg.dynamicSmemBytes = G::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = G::CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = G::CG == 1 ? 1 : 2;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess) return e;
  count_launches();
  return cudaGetLastError();
}

}  // namespace

int grouped_tile_cols(GroupedKernel k) { return k == GG_WIDE ? Wide::BN : Narrow::BN; }
int grouped_box_rows(GroupedKernel k) { return k == GG_WIDE ? Wide::BOX_ROWS : Narrow::BOX_ROWS; }
int grouped_tile_lanes(GroupedKernel k) { return k == GG_WIDE ? Wide::LANES : Narrow::LANES; }

cudaError_t launch_grouped(const GroupedArgs &a, GroupedKernel k, GroupedMode mode, bool fp8, int grid,
                           cudaStream_t stream) {
  if (fp8) {
    if (mode != GG_FWD) return cudaErrorInvalidValue;
    return k == GG_WIDE ? launch_one<WideF8, GG_FWD>(a, grid, stream) : launch_one<NarrowF8, GG_FWD>(a, grid, stream);
  }
  switch (mode) {
    case GG_FWD:
      return k == GG_WIDE ? launch_one<Wide, GG_FWD>(a, grid, stream) : launch_one<Narrow, GG_FWD>(a, grid, stream);
    case GG_DX:
      return k == GG_WIDE ? launch_one<Wide, GG_DX>(a, grid, stream) : launch_one<Narrow, GG_DX>(a, grid, stream);
    default:
      return k == GG_WIDE ? launch_one<Wide, GG_DW>(a, grid, stream) : launch_one<Narrow, GG_DW>(a, grid, stream);
  }
}

}  // namespace tileq
