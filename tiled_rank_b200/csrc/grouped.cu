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
// one 64- or 128-byte run of an output row in every mode (but for the wide fp8
// kernel below, where a thread stores a row of its own in pieces of 32 bytes).
//
// One persistent CTA per SM (CG = 1) or a pair of CTAs on neighbouring SMs that
// share one MMA of 256 lanes (CG = 2: each CTA loads its own 128 rows of A and
// half of B's, so an SM reads 32 KB per 64-element step of a 256 x 256 tile
// instead of 48 KB).  Warps of a CTA:
//   0      producer: TMA tiles (128-byte swizzle) of one 128-byte reduction step
//          per stage into a ring, a lane per box;
//   1      MMA issuer (first CTA of a pair), one thread: four MMAs per stage into
//          an fp32 TMEM accumulator, two or four accumulators in turn;
//   2      the table of the experts' rows and tiles, before the others start;
//          then, in wide fp8, the MMAs of the tile's second part;
//   3      in GG_DW zeroes the rows of the next expert in the last stage of a
//          tile (of both operands: 0 * NaN would be NaN);
//   4..    epilogue: TMEM to registers, one rounding, stores.
// fp8: one 128-byte stage is one scale block.  Every block gets an accumulator
// of its own, which the epilogue warps fold into fp32 registers with
// xs[block][row] * ws[e][o / 128][block]: one FMA per sum and block, as the
// scales are no powers of two in general and cannot be left to the exponent.
// In the narrow kernel a column's scale is read from shared memory; wide tiles
// are too many columns for that (the reads alone cost more than the MMAs), so
// there the operands change places: rows of x on the lanes (ROWS), each thread
// with the scale of its own row in a register.
// Few tiles, as of one expert's few rows: clusters of CTAs share the reduction of
// each (SPLIT); two units of the GPU share a tile of a last round (HALVES).
//
// What bounds them, measured on a B200 (of measured: of 6458 GB/s and 1663
// TFLOP/s), the routing skewed as far as not said otherwise:
//   one token on 8 experts, 4096 -> 14336    43 us    memory, 84 % of measured
//   64 x 4096 -> 1536, 131072 rows           1.13 ms at full clocks, tensor cores,
//                                            1460 TFLOP/s; 1.35 to 1.43 ms (1150 to
//                                            1220) under the power limit
//   gradient of 8192 rows, 60 experts        88 us    memory, 69 % of measured (76 us in a captured run of calls)
//   dW of 8192 rows, 8 x 14336 x 4096        0.72 ms at full clocks, 0.80 to 0.84 at the limit
//   fp8, 64 x 4096 -> 1536, 128 rows         64 us    memory, 90 % of measured
//   fp8, 8192 rows, 8 x 14336 -> 4096        0.46 ms at full clocks, 2080 TFLOP/s (even rows): the fold
// With equal experts the library's batched products run at 1525 TFLOP/s in one call
// and 1280 under the power limit where this kernel has 1440 and 1240 (64 x 4096 ->
// 1536, 2048 rows each), dx 1515 / 1270 and 1490 / 1270, dW 1425 / 1210 and 1385 /
// 1170 (8 x 14336 x 4096, 1024 rows each).
// The fold is why fp8 wide tiles stay at half of the tensor cores' rate: without
// its FMAs a 2048 x 5632 x 2048 product took 25.5 us instead of 34.9, without its
// TMEM reads 30.8; the sharing of a last round's tiles, which came later, brought
// the whole to 32.  (Pairs of CTAs and sixteen fold warps were no faster.)  Its 224
// registers a fold warp spill 20 bytes a thread.
// An accumulator goes back to the issuer by a relaxed arrival.  Tensor memory is no
// part of what release and acquire order: its accesses are ordered by wait::ld and
// the fences tcgen05.fence::before_thread_sync and ::after_thread_sync on either
// side of the arrival and of the wait that sees it, and nothing else is handed over
// with it.  (With release the arrival also waits for the thread's own stores: dW of
// 512 rows, 8 x 4096 x 1536, 50.6 us instead of 39.6 side by side, 8 x 14336 -> 4096
// in fp8 786 instead of 715.)
// Every wait is bounded and reports TILEQ_ERR_TIMEOUT.
#include "grouped.cuh"

#include <atomic>

#include "kernels.cuh"
#include "tc_pair.cuh"

namespace tileq {
namespace {

constexpr int kScaleGroup = 8;      // narrow fp8: blocks whose scales the fold's warps stage at a time
constexpr int kFirstEpw = 4;        // first epilogue warp
constexpr int kRegsControl = 56, kRegsEpilogue = 224;  // registers a thread where the warps split them
constexpr int kRowTileGroup = 8;    // column tiles that share a pass over the lane tiles

template <int CG_, int BN_, bool F8_, bool SPLIT_ = false>
struct GCfg {
  static constexpr int CG = CG_, BN = BN_;
  static constexpr bool F8 = F8_;
  // A cluster of CTAs shares a tile, each with a part of the reduction; their partial sums meet in shared memory.
  static constexpr bool SPLIT = SPLIT_;
  static constexpr int RED = SPLIT ? 128 * BN * 4 : 0;
  static constexpr bool ROWS = F8 && BN == 256;  // the experts' rows on the lanes, d_out on the columns
  static constexpr int LANES = 128 * CG;
  static constexpr int KE = F8 ? 128 : 64;  // reduction elements per stage (128 bytes)
  static constexpr int EPW = BN == 256 ? 8 : 4;
  static constexpr int COLS = BN / (EPW / 4);  // columns of one epilogue warp
  static constexpr int THREADS = (kFirstEpw + EPW) * 32;
  static constexpr bool SPLIT_REGS = ROWS;
  static constexpr int SCALES = F8 && !ROWS ? 2 * kScaleGroup * BN * 4 : 0;
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = BN / CG * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int TAB = (2 * kGroupedMaxE + 2) * 4;
  static constexpr int SQ = (227 * 1024 - TAB - SCALES - RED - 512) / STAGE;
  // ROWS: the columns of a tile are two MMAs, one for each 128 of d_out and so for each weight scale, with
  // accumulators of their own, folded by four epilogue warps each: while one part is folded the other's MMAs run
  static constexpr int PARTS = ROWS ? 2 : 1;
  static constexpr bool HALVES = BN == 256;  // the tiles of a last round may be shared by two units
  static constexpr int PC = BN / PARTS;  // columns of a part
  static constexpr int BOX_B = ROWS ? PC / CG : BN == 256 ? 64 : 32;  // rows of a box of B where the reduction is contiguous
  static constexpr int NACC = BN == 256 ? 2 : 4;
  static constexpr int TMEM_COLS = NACC * BN;
  static constexpr int BAR_OFF = SQ * STAGE;
  static constexpr int SCALE_OFF = BAR_OFF + ((3 * SQ + 2 * NACC * PARTS + 3) * 8 + 31) / 16 * 16;
  static constexpr int RED_OFF = SCALE_OFF + SCALES;
  static constexpr int TAB_OFF = RED_OFF + RED;
  static constexpr int SMEM = TAB_OFF + TAB;
  static_assert(!SPLIT || (CG == 1 && PARTS == 1 && EPW == 4), "the reduction's columns");
  static_assert(TMEM_COLS == 256 || TMEM_COLS == 512, "a power of two of tensor memory columns");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Position in a ring of N slots and the parity of its use there.
template <int N>
struct Ring {
  int at = 0;
  uint32_t parity = 0;
  __device__ void next() {
    if (++at == N) at = 0, parity ^= 1;
  }
  __device__ Ring after() const {
    Ring r = *this;
    r.next();
    return r;
  }
};

struct Tile {
  int e, row0, rows;  // expert and its rows
  int l0, c0, ncols;  // first lane of the tile, first column, columns
};

__host__ __device__ __forceinline__ int tiles_of(int n, int size) { return (n + size - 1) / size; }

// The tiles of the call, experts in order; first[e] = tiles before expert e.
// Within an expert the column tiles go in groups that share a pass over the lane
// tiles, so that the CTAs at work read few distinct rows of either operand.
template <class G, GroupedMode MODE>
struct Tiles {
  const int *first, *beg;
  int E, L, C, e = 0, halves = 0x7fffffff;  // halves: first tile that is shared by two (HALVES)
  // lanes and columns of an expert with `rows` rows
  __device__ int lanes(int rows) const { return G::ROWS ? rows : L; }
  __device__ int cols(int rows) const { return G::ROWS || MODE == GG_DW ? C : rows; }
  __device__ int count(int rows) const { return tiles_of(lanes(rows), G::LANES) * tiles_of(cols(rows), G::BN); }
  __device__ bool get(int w, Tile &t) {
    int half = -1;
    if constexpr (G::HALVES) {
      if (w >= halves) {
        half = (w - halves) & 1;
        w = halves + ((w - halves) >> 1);
      }
    }
    if (w >= first[E]) return false;
    while (w >= first[e + 1]) ++e;
    const int i = w - first[e], rows = beg[e + 1] - beg[e], total = cols(rows);
    const int nl = tiles_of(lanes(rows), G::LANES), nc = tiles_of(total, G::BN);
    const int step = G::ROWS ? G::BN : 16 * G::CG;  // (ROWS: whole scale blocks)
    int l = i, c = 0, tc = tiles_of(total, step) * step;
    if (nc > 1) {  // (divisions only where they are needed: every role waits for them at each tile)
      const int grp = nc <= kRowTileGroup ? 0 : (uint32_t)i / (uint32_t)(kRowTileGroup * nl);
      const int rem = i - grp * kRowTileGroup * nl, gsz = min(kRowTileGroup, nc - grp * kRowTileGroup);
      l = (uint32_t)rem / (uint32_t)gsz;
      c = grp * kRowTileGroup + rem - l * gsz;
      // equal tiles, rounded to the MMA's step: one short tile would leave its CTAs idle
      tc = G::ROWS ? step : tiles_of((uint32_t)(total + nc - 1) / (uint32_t)nc, step) * step;
    }
    t.e = e;
    t.row0 = beg[e];
    t.rows = rows;
    t.l0 = l * G::LANES;
    t.c0 = c * tc;
    t.ncols = min(tc, total - t.c0);
    if constexpr (G::HALVES) {
      const int h = G::ROWS ? G::PC : tiles_of(tiles_of(t.ncols, 2), step) * step;
      if (half == 0) t.ncols = min(t.ncols, h);
      if (half == 1) t.c0 += h, t.ncols -= h;  // none may be left
    }
    return true;
  }
};

// Has this phase of the barrier completed?  Asked without waiting; the answer takes some 100 cycles, so the loops ask
// for what they need next before the work at hand.
__device__ __forceinline__ bool test_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// TMEM to registers in the layout of 8 x 8 blocks (16x256b): of 32 lanes x 32
// columns at taddr, r[h][4 j + 2 g + i] is lane 16 h + 8 g + id / 4, column
// 8 j + 2 (id % 4) + i for thread id: what a transposing store wants.  (These
// loads run at half the rate of 32x32b, a lane for each thread: 550 against 260
// cycles for 128 columns in eight warps.  The folds use those.)  The values are
// there after wait_block of the same r.
__device__ __forceinline__ void ld_half(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void ld_block(uint32_t taddr, uint32_t (&r)[2][16]) {
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
__device__ __forceinline__ void wait_block(uint32_t (&r)[2][16]) {
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

// A wait by a whole warp with one answer: no lane leaves a loop in which the others still meet.
// (`remote`: the pair's other CTA has written memory before it arrived.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *status, bool remote = false,
                                          long long limit = kWaitLimitCycles) {
  return __all_sync(0xffffffffu,
                    remote ? tc::mbar_wait_cluster(bar, parity, status, limit) : tc::mbar_wait_for(bar, parity, status, limit));
}
// The limit of a wait for the `steps` steps of a tile's reduction: a step takes some 500 cycles, so that a sum over 3e8
// rows lasts longer than the second that suffices for a wait between neighbours in a pipeline.
__device__ __forceinline__ long long reduction_limit(int steps) { return kWaitLimitCycles + 4096ll * steps; }

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == TILEQ_DT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    return h2_as_u32(__floats2half2_rn(lo, hi));
  }
}

// Two values of neighbouring columns of a lane, rounded and transposed as 8 x 8 blocks: thread id, which had lane id / 4
// of columns 2 (id % 4) + 0, 1, gets lanes 2 (id % 4) + 0, 1 of column id / 4.
template <int DT>
__device__ __forceinline__ uint32_t transpose8(uint32_t lo, uint32_t hi) {
  uint32_t w;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n"
               : "=r"(w)
               : "r"(pack2<DT>(__uint_as_float(lo), __uint_as_float(hi))));
  return w;
}

// Stores a block of 32 columns (n of them exist) x 32 lanes (nl exist, a multiple of 8) of 16-bit results in runs of
// eight lanes, after a transposition among the four threads of a column.  The four groups of eight columns go through
// each step together: one after the other, their latencies made this the most expensive part of a tile (dW of 512 rows,
// 8 x 4096 x 1536: 48 us, together 31).
template <int DT>
__device__ __forceinline__ void store_runs(uint16_t *out, long long ldo, int n, int nl, int id, const uint32_t (&r)[2][16]) {
  uint32_t w[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) w[j][g] = transpose8<DT>(r[g >> 1][4 * j + 2 * (g & 1)], r[g >> 1][4 * j + 2 * (g & 1) + 1]);
  const int q = id & 3;
  const bool b0 = q & 1, b1 = q & 2;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = __shfl_xor_sync(0xffffffffu, b0 ? w[j][0] : w[j][1], 1);
    const uint32_t y = __shfl_xor_sync(0xffffffffu, b0 ? w[j][2] : w[j][3], 1);
    (b0 ? w[j][0] : w[j][1]) = x;
    (b0 ? w[j][2] : w[j][3]) = y;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u = __shfl_xor_sync(0xffffffffu, b1 ? w[j][0] : w[j][2], 2);
    const uint32_t z = __shfl_xor_sync(0xffffffffu, b1 ? w[j][1] : w[j][3], 2);
    (b1 ? w[j][0] : w[j][2]) = u;
    (b1 ? w[j][1] : w[j][3]) = z;
  }
  out += (id >> 2) * ldo + q * 8;
  n = q * 8 < nl ? n - (id >> 2) : 0;
#pragma unroll
  for (int j = 0; j < 4; ++j, out += 8 * ldo)
    if (8 * j < n) *reinterpret_cast<uint4 *>(out) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
}

// Stores 8 columns (n of them exist) x 32 lanes (nl exist) of 16-bit results to out + column * ldo + lane, one by one
// or (PAIR) two neighbouring lanes at a time; v[g]: this thread's two columns of lane 8 g + id / 4.
template <int DT, bool PAIR>
__device__ __forceinline__ void store_b16(uint16_t *out, long long ldo, int n, int nl, int id, const uint64_t (&v)[4]) {
  out += (id >> 2) * ldo;
  const bool in = (id >> 2) < n;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t w = transpose8<DT>((uint32_t)v[g], (uint32_t)(v[g] >> 32));
    const int l = 8 * g + 2 * (id & 3);
    if constexpr (PAIR) {
      if (in && l < nl) *reinterpret_cast<uint32_t *>(out + l) = w;
    } else {
      if (in && l < nl) out[l] = (uint16_t)w;
      if (in && l + 1 < nl) out[l + 1] = (uint16_t)(w >> 16);
    }
  }
}
template <int DT>
__device__ __forceinline__ void store_b16(const GroupedArgs &P, long long base, int n, int nl, int id, const uint64_t (&v)[4]) {
  uint16_t *out = reinterpret_cast<uint16_t *>(P.out) + base;
  if (P.store_words == 2)
    store_b16<DT, true>(out, P.ldo, n, nl, id, v);
  else
    store_b16<DT, false>(out, P.ldo, n, nl, id, v);
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

// Stores n of N columns where a thread has the values of its own lane (pairs of neighbouring columns): column j to
// out + at + j * ldo, which is this lane's (in: it exists).  16-bit results of neighbouring lanes are exchanged so that
// a store takes two of them (PAIR).
template <int N, int DT, bool PAIR>
__device__ __forceinline__ void store_lanes_b16(uint16_t *out, long long ldo, int n, bool in, int odd, const uint64_t (&v)[N / 2]) {
  if constexpr (PAIR) out += odd ? ldo - 1 : 0;
#pragma unroll
  for (int i = 0; i < N / 2; ++i, out += 2 * ldo) {
    if (2 * i >= n) break;
    const float a = low(v[i]), b = high(v[i]);
    if constexpr (PAIR) {
      const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
      const uint32_t w = pack2<DT>(odd ? got : a, odd ? b : got);
      if (in && 2 * i + odd < n) *reinterpret_cast<uint32_t *>(out) = w;
    } else {
      if (in) out[0] = (uint16_t)pack2<DT>(a, 0.f);
      if (in && 2 * i + 1 < n) out[ldo] = (uint16_t)pack2<DT>(b, 0.f);
    }
  }
}
template <int N>
__device__ __forceinline__ void store_lanes(const GroupedArgs &P, long long at, int n, bool in, int odd, const uint64_t (&v)[N / 2]) {
  if (P.out_dtype == TILEQ_DT_F32) {
    float *out = reinterpret_cast<float *>(P.out) + at;
#pragma unroll
    for (int i = 0; i < N / 2; ++i, out += 2 * P.ldo) {
      if (2 * i >= n) break;
      if (in) out[0] = low(v[i]);
      if (in && 2 * i + 1 < n) out[P.ldo] = high(v[i]);
    }
    return;
  }
  uint16_t *out = reinterpret_cast<uint16_t *>(P.out) + at;
  if (P.out_dtype == TILEQ_DT_BF16) {
    if (P.store_words >= 2)
      store_lanes_b16<N, TILEQ_DT_BF16, true>(out, P.ldo, n, in, odd, v);
    else
      store_lanes_b16<N, TILEQ_DT_BF16, false>(out, P.ldo, n, in, odd, v);
  } else {
    if (P.store_words >= 2)
      store_lanes_b16<N, TILEQ_DT_F16, true>(out, P.ldo, n, in, odd, v);
    else
      store_lanes_b16<N, TILEQ_DT_F16, false>(out, P.ldo, n, in, odd, v);
  }
}

// Stores n columns of one output row, N / 2 pairs in registers, to out + base.  A thread has a row of its own, so a
// store should fill whole 32-byte sectors where the row allows it (WORDS == 16).
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
template <int N, int DT>
__device__ __forceinline__ void store_row_b16(uint16_t *out, int words, int n, const uint64_t (&v)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N; i += 16) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack2<DT>(low(v[i / 2 + j]), high(v[i / 2 + j]));
    if (words == 16) {
      if (i < n) store32(out + i, w);
    } else if (words == 8) {
      if (i < n) *reinterpret_cast<uint4 *>(out + i) = make_uint4(w[0], w[1], w[2], w[3]);
      if (i + 8 < n) *reinterpret_cast<uint4 *>(out + i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = i + 2 * j;
        if (words == 2) {
          if (c < n) *reinterpret_cast<uint32_t *>(out + c) = w[j];
        } else {
          if (c < n) out[c] = (uint16_t)w[j];
          if (c + 1 < n) out[c + 1] = (uint16_t)(w[j] >> 16);
        }
      }
    }
  }
}
template <int N>
__device__ __forceinline__ void store_row(const GroupedArgs &P, long long base, int n, const uint64_t (&v)[N / 2]) {
  if (P.out_dtype == TILEQ_DT_F32) {
    float *out = reinterpret_cast<float *>(P.out) + base;
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      if (P.store_words >= 8) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = (uint32_t)(v[i / 2 + j / 2] >> (j & 1 ? 32 : 0));
        if (i < n) store32(out + i, w);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i + j < n) out[i + j] = __uint_as_float((uint32_t)(v[i / 2 + j / 2] >> (j & 1 ? 32 : 0)));
      }
    }
  } else if (P.out_dtype == TILEQ_DT_BF16) {
    store_row_b16<N, TILEQ_DT_BF16>(reinterpret_cast<uint16_t *>(P.out) + base, P.store_words, n, v);
  } else {
    store_row_b16<N, TILEQ_DT_F16>(reinterpret_cast<uint16_t *>(P.out) + base, P.store_words, n, v);
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
  uint64_t *red_full = drain + 1, *red_empty = red_full + 1;  // SPLIT: the partial sums are here, have been read
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(red_empty + 1);
  float *scale = reinterpret_cast<float *>(smem + G::SCALE_OFF);
  int *first = reinterpret_cast<int *>(smem + G::TAB_OFF), *beg = first + kGroupedMaxE + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : tc::cluster_rank();
  const int splits = G::SPLIT ? P.splits : 1, split = G::SPLIT ? (int)tc::cluster_rank() : 0;
  const uint32_t lead = CG == 2 ? 0 : split;  // the CTA of the cluster that issues this one's MMAs
  const int unit0 = blockIdx.x / (CG * splits), units = gridDim.x / (CG * splits);
  Tiles<G, MODE> tiles{first, beg, P.E, P.L, P.C};
  auto stage_a = [&](int s) { return smem + s * G::STAGE; };
  auto stage_b = [&](int s) { return smem + s * G::STAGE + G::A_BYTES; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < SQ; ++s) {
      mbar_init(&full[s], CG);
      mbar_init(&empty[s], PARTS);
      mbar_init(&tail[s], 1);
    }
    for (int b = 0; b < PARTS * NACC; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], G::EPW / PARTS * CG);
    }
    mbar_init(drain, PARTS);
    mbar_init(red_full, G::EPW * splits);
    mbar_init(red_empty, G::EPW * splits);
    fence_mbar_init();
  }
  if (warp == 1) tc::alloc_cg<CG>(tmem_slot, G::TMEM_COLS);
  tc::grid_wait();  // the prologue overlaps the previous kernel's tail
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
      int sum = e < P.E ? tiles.count(hi - lo) : 0;
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
  if constexpr (CG == 2 || G::SPLIT) tc::cluster_sync();
  tc::fence_after();
  // only now: a kernel that starts early finds this one's tensor memory taken, not the other way round
  tc::grid_release();
  const uint32_t tmem = *tmem_slot;
  if constexpr (G::HALVES) {
    // Where the last round would leave half of the GPU idle, two share each of its tiles, half of the columns each
    // (ROWS: a part; the second has nothing to do where there is one).  fp8 1 x 4096 -> 1536, 1024 rows: 21.0 -> 17.2 us.
    const int rest = (uint32_t)first[P.E] % (uint32_t)units;
    if (2 * rest <= units) tiles.halves = first[P.E] - rest;
  }

  auto steps = [&](const Tile &t) { return ((MODE == GG_DW ? t.rows : P.R) + G::KE - 1) / G::KE; };
  // this CTA's steps of the reduction
  auto first_step = [&](int nk) { return G::SPLIT ? nk * split / splits : 0; };
  auto end_step = [&](int nk) { return G::SPLIT ? nk * (split + 1) / splits : nk; };
  // parts of the tile that have columns, and the columns of one part's MMA
  auto parts = [&](const Tile &t) { return PARTS == 1 || t.ncols <= G::PC ? 1 : 2; };
  auto mma_n = [&](const Tile &t) { return G::ROWS ? G::PC : tiles_of(t.ncols, 16 * CG) * 16 * CG; };
  Tile t;
  bool ok = true;

  if constexpr (G::SPLIT_REGS) {
    if (warp < kFirstEpw) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsControl));
  }
  if (warp == 0) {
    // ============================================================ producer
    Ring<SQ> q;
    for (int w = unit0; ok && tiles.get(w, t); w += units) {
      if (G::HALVES && t.ncols <= 0) continue;
      const int nk = steps(t), half = mma_n(t) / CG;
      const int l0 = t.l0 + (int)rank * 128, c0 = t.c0 + (int)rank * half;
      constexpr int ABOX = MODE == GG_FWD ? 1 : 2;           // boxes of A: 128 rows, or twice 64 columns
      constexpr int BBOX = MODE == GG_DW ? 64 : G::BOX_B;    // columns of the tile in one box of B
      const int nbox = G::ROWS ? parts(t) : tiles_of(half, BBOX);
      const uint32_t bytes = G::A_BYTES + nbox * BBOX * 128;
      // One lane per box (a single lane would need the time of a whole stage to issue five or six copies):
      // this lane's box and how far it moves from one step to the next
      const bool is_a = lane < ABOX;
      const int i = is_a ? lane : lane - ABOX;
      uint8_t *dst = is_a ? stage_a(0) + i * 8192 : stage_b(0) + i * BBOX * 128;
      const CUtensorMap *map = is_a ? &P.amap : &P.bmap;
      int x, y, z = 0;
      const bool along_x = is_a ? MODE == GG_FWD : MODE != GG_DW;  // is the reduction the inner dimension?
      if (along_x) {
        x = 0;
        // rows of x (dy): from the expert's first one; of w: within the expert (a box per part: 128 apart)
        y = is_a ? l0 + (G::ROWS ? t.row0 : 0) : c0 + i * (G::ROWS ? G::PC : BBOX) + (G::ROWS ? 0 : t.row0);
      } else {
        x = (is_a ? l0 : c0) + i * 64;
        y = MODE == GG_DW ? t.row0 : 0;
      }
      if (MODE != GG_DW && is_a != G::ROWS) z = t.e;
      const int k0 = first_step(nk), k1 = end_step(nk);
      x += along_x ? k0 * G::KE : 0;
      y += along_x ? 0 : k0 * G::KE;
      for (int kb = k0; kb < k1; ++kb, q.next()) {
        const int left = MODE == GG_DW ? t.rows - kb * G::KE : G::KE;
        const bool cut = left < G::KE && (left & 15);  // the last MMA of the step reaches the next expert's rows
        if (!(ok = warp_wait(&empty[q.at], q.parity ^ 1, P.status))) break;
        const uint32_t bar = cut ? smem_addr(&tail[q.at]) : CG == 2 ? tc::map_cta(&full[q.at], 0) : smem_addr(&full[q.at]);
        if (lane == 0) {
          if (cut || CG == 1)
            mbar_arrive_expect_tx(cut ? &tail[q.at] : &full[q.at], bytes);
          else
            tc::arrive_expect_at(bar, bytes);
        }
        if (lane < ABOX + nbox) tc::tma_3d<CG>(dst + q.at * G::STAGE, map, x, y, z, bar);
        x += along_x ? G::KE : 0;
        y += along_x ? 0 : G::KE;
      }
    }
    // no copy of this CTA may land and no commit may arrive after it has gone
    if (lane == 0) {
      for (int i = 0; ok && i < SQ; ++i, q.next()) ok = mbar_wait(&empty[q.at], q.parity ^ 1, P.status);
      if (!ok && rank == 0)
        for (int i = 0; i < SQ; ++i, q.next()) mbar_wait(&full[q.at], q.parity ^ 1, P.status);
    }
  } else if (warp == 1 || (PARTS == 2 && warp == 2)) {
    // ============================================================ MMA issuer (one for each part)
    // (a stage costs the issuer some 350 cycles: with two accumulators a stage one would not keep the tensor core busy)
    if (rank == 0) {
      constexpr bool A_MN = MODE != GG_FWD, B_MN = MODE == GG_DW;  // output dimension contiguous
      const uint32_t fmt = P.bf16 && !G::F8 ? (1u << 7) | (1u << 10) : 0u;
      const int part = PARTS == 2 ? warp - 1 : 0;
      Ring<SQ> q;
      Ring<NACC> acc;
      const uint64_t ad0 = tc::sdesc(smem_addr(stage_a(0)), A_MN ? 8192 : 16);
      const uint64_t bd0 = tc::sdesc(smem_addr(stage_b(0)) + part * (G::PC / CG * 128), B_MN ? 8192 : 16);
      bool full_ready = false, acc_ready = false;
      // One thread from here on: a stage then costs it some 350 cycles, against 470 for a warp that votes on every
      // wait and elects for every issue.
      if (tc::elect_one()) {
        for (int w = unit0; ok && tiles.get(w, t); w += units) {
          if (G::HALVES && t.ncols <= 0) continue;
          const int nk = steps(t);
          const bool mine = part < parts(t);
          const uint32_t idesc = (1u << 4) | fmt | ((uint32_t)A_MN << 15) | ((uint32_t)B_MN << 16) |
                                 ((uint32_t)(mma_n(t) >> 3) << 17) | ((uint32_t)(G::LANES >> 4) << 24);
          const int k0 = first_step(nk), k1 = end_step(nk);
          for (int kb = k0; kb < k1; ++kb, q.next()) {
            const bool cut = MODE == GG_DW && kb == nk - 1 && (t.rows & 15);  // the producers zeroed rows
            const bool last = G::F8 || kb == k1 - 1, first_k = G::F8 || kb == k0;
            const int pa = part * NACC + acc.at;
            // 16 (fp8: 32) reduction elements per MMA: 32 bytes along a row, or 16 rows
            const int nmma = MODE == GG_DW ? min(4, (t.rows - kb * 64 + 15) / 16) : 4;
            const uint64_t at = (uint64_t)(q.at * (G::STAGE >> 4));
            const bool want_acc = mine && first_k;
            if (cut || !full_ready)
              ok = cut ? tc::mbar_wait_cluster(&full[q.at], q.parity, P.status) : mbar_wait(&full[q.at], q.parity, P.status);
            if (ok && want_acc && !acc_ready) ok = mbar_wait(&acc_empty[pa], acc.parity ^ 1, P.status);
            if (!ok) break;
            tc::fence_after();
            // the next stage's barriers, asked now: the answers come while this one's MMAs are issued
            const Ring<SQ> q1 = q.after();
            full_ready = test_wait(&full[q1.at], q1.parity);
            if (G::F8) {  // (a part without columns in this tile leaves its ring where it is)
              const Ring<NACC> a1 = acc.after();
              acc_ready = mine && test_wait(&acc_empty[part * NACC + a1.at], a1.parity ^ 1);
            }
            if (mine) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (MODE != GG_DW || kk < nmma)
                  tc::mma_ss<CG, G::F8>(tmem + pa * G::PC, ad0 + at + (uint64_t)(kk * (A_MN ? 128 : 2)),
                                        bd0 + at + (uint64_t)(kk * (B_MN ? 128 : 2)), idesc, (kk || !first_k) ? 1u : 0u);
              if (last) tc::commit_cg<CG>(&acc_full[pa]);
            }
            tc::commit_cg<CG>(&empty[q.at]);
            if (mine && last) acc.next();
          }
        }
        tc::commit_cg<CG>(drain);
      }
      __syncwarp();
      warp_wait(drain, 0, P.status);  // all issued MMAs have retired before tensor memory is released
    }
  } else if (warp == 3) {
    // ============================================================ rows of the next expert (GG_DW)
    // A warp of its own, because the copies have to land first: the producer would lose that time for every tile.
    if constexpr (MODE == GG_DW) {
      uint32_t q0 = 0, phase = 0;  // phase: bit s, the use of tail[s]
      for (int w = unit0; ok && tiles.get(w, t); w += units) {
        if (G::HALVES && t.ncols <= 0) continue;
        const int nk = steps(t), left = t.rows & 63;
        const int k0 = first_step(nk), k1 = end_step(nk);
        q0 += k1 - k0;
        if (!(left & 15) || k1 < nk || k0 == k1) continue;  // the last step has all its rows, or is another CTA's
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
        if (lane == 0) tc::arrive_at(tc::map_cta(&full[s], lead));
      }
    }
  } else if (warp >= kFirstEpw) {
    // ============================================================ epilogue
    // 128 accumulators a thread: the register file has room for them once the first four warps give theirs up
    // (168 registers a thread at launch: 384 * 168 = 128 * (56 + 2 * 224))
    if constexpr (G::SPLIT_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsEpilogue));
    const int half = (warp - kFirstEpw) >> 2;
    const uint32_t lane_addr = tc::lane_base(warp);  // TMEM lane quadrant of this warp
    const int part = PARTS == 2 ? half : 0;
    uint64_t *my_full = acc_full + part * NACC, *my_empty = acc_empty + part * NACC;
    Ring<NACC> acc;
    uint32_t group = 0, red_parity = 0;
    bool ready = false;
    float *red = reinterpret_cast<float *>(smem + G::RED_OFF);
    const uint32_t release_at = tc::map_cta(my_empty, lead);
    auto release = [&] {  // this warp has read the accumulator (wait::ld is the whole warp's)
      tc::fence_before();
      if (lane == 0) tc::arrive_relaxed_at(release_at + acc.at * 8);
      acc.next();
    };
    // (narrow fp8: the four warps of a named barrier stay together, also after a wait that gave up)
    for (int w = unit0; (ok || G::F8) && tiles.get(w, t); w += units) {
      if (G::HALVES && t.ncols <= 0) continue;
      const int steps_all = steps(t), k0 = first_step(steps_all), nk = end_step(steps_all) - k0;  // this CTA's steps
      const int l0 = t.l0 + (int)rank * 128 + (warp & 3) * 32;
      // this warp's columns: of eight warps (but for ROWS) four have one half of the tile's, in blocks of 32
      const int share = G::EPW == 8 && !G::ROWS ? tiles_of(t.ncols, 64) * 32 : G::COLS;
      const int cw = half * share, mine = min(t.ncols - cw, share);  // first, and how many (none if <= 0)
      if constexpr (G::ROWS) {
        if (mine <= 0) continue;  // a part without columns has no MMAs either
        // this thread's row of x and y, and its scale with the part's weight scale, fetched two blocks ahead
        const int row = min(l0 + lane, t.rows - 1);
        const float *xs = P.xs + t.row0 + row;
        const float *ws = P.ws + ((long long)t.e * P.nOb + t.c0 / 128 + part) * P.nKb;
        float sx[2], sw[2];
        auto fetch = [&](int kb) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (kb + j < nk) {
              sx[j] = __ldg(xs);
              sw[j] = __ldg(ws);
              xs += P.ld_xs;
              ++ws;
            }
          }
        };
        uint64_t v[G::COLS / 2];  // pairs of neighbouring columns: one packed FMA folds both
#pragma unroll
        for (int i = 0; i < G::COLS / 2; ++i) v[i] = 0;
        fetch(0);
#pragma unroll 1
        for (int kb = 0; kb < nk; kb += 2) {
          const float s0 = sx[0] * sw[0], s1 = sx[1] * sw[1];
          fetch(kb + 2);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (kb + j >= nk) break;
            const uint64_t ss = pair(__float_as_uint(j ? s1 : s0), __float_as_uint(j ? s1 : s0));
            ok = ok && (ready || warp_wait(&my_full[acc.at], acc.parity, P.status));
            tc::fence_after();
            const uint32_t ta = tmem + lane_addr + (part * NACC + acc.at) * G::PC;
            // 16 columns at a time: with 32 the registers do not suffice for a load beside the FMAs of the one before
            uint32_t r[2][16];
            tc::ld16_nowait(ta, r[0]);
#pragma unroll
            for (int c = 0; c < G::COLS / 16; ++c) {
              tc::wait_ld();
              tie(r[c & 1]);
              if (c + 1 < G::COLS / 16) {
                tc::ld16_nowait(ta + 16 * (c + 1), r[(c + 1) & 1]);
              } else {
                release();
                // the next block's barrier is asked before the last FMAs, which take as long as the answer
                ready = test_wait(&my_full[acc.at], acc.parity);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) fma2(v[8 * c + i], pair(r[c & 1][2 * i], r[c & 1][2 * i + 1]), ss);
            }
            ready = __all_sync(0xffffffffu, ready);
          }
        }
        if (ok && l0 + lane < t.rows)
          store_row<G::COLS>(P, (long long)(t.row0 + l0 + lane) * P.ldo + t.c0 + cw, mine, v);
      } else {
        const int nl = P.L - l0;
        const long long base = (MODE == GG_DW ? (long long)t.e * P.out_stride + (long long)(t.c0 + cw) * P.ldo
                                              : (long long)(t.row0 + t.c0 + cw) * P.ldo) + l0;
        // SPLIT: CTA i of the cluster sums columns [i, i + 1) << shift of the tile.  Each CTA sends its partial sums
        // there, [sender][four columns][128 lanes][4] so that a lane's four travel as 16 bytes (word by word the
        // sending took longer than the products); the receiver adds them in the senders' order, so the bits do not
        // depend on who comes first.
        int shift = 2;
        if constexpr (G::SPLIT) {
          while (splits << shift < t.ncols) ++shift;
          ok = ok && warp_wait(red_empty, red_parity ^ 1, P.status, true, reduction_limit(steps_all));
        }
        [[maybe_unused]] const int tid = threadIdx.x & 127;
        [[maybe_unused]] auto send = [&](int c, float a, float b, float d, float e) {  // columns c .. c + 3 of this lane
          if (c < mine)
            tc::store4_at(tc::map_cta(red, c >> shift) + ((((split << shift) + (c & ((1 << shift) - 1))) >> 2) * 128 + tid) * 16, a, b, d, e);
        };
        [[maybe_unused]] auto join = [&](long long base, int nl) {
          tc::fence_cluster();
          __syncwarp();
          if (lane < splits) tc::arrive_at(tc::map_cta(red_full, lane));
          const bool got = ok && warp_wait(red_full, red_parity, P.status, true, reduction_limit(steps_all));
          if (got) {
            const float4 *from = reinterpret_cast<const float4 *>(red) + tid;
            for (int c = split << shift; c < min((split + 1) << shift, mine); c += 4) {
              float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < splits) {
                  const float4 f = from[(((i << shift) + (c & ((1 << shift) - 1))) >> 2) * 128];
                  sum = make_float4(sum.x + f.x, sum.y + f.y, sum.z + f.z, sum.w + f.w);
                }
              const uint64_t v[2] = {pair(__float_as_uint(sum.x), __float_as_uint(sum.y)),
                                     pair(__float_as_uint(sum.z), __float_as_uint(sum.w))};
              store_lanes<4>(P, base + c * P.ldo + lane, mine - c, lane < nl, lane & 1, v);
            }
          }
          __syncwarp();
          if (lane < splits) tc::arrive_at(tc::map_cta(red_empty, lane));
          red_parity ^= 1;
          return got;
        };
        if constexpr (!G::F8) {
          if (nk > 0) {
            if (!(ok = warp_wait(&my_full[acc.at], acc.parity, P.status, false, reduction_limit(nk)))) break;
            tc::fence_after();
          }
          if constexpr (G::SPLIT) {
#pragma unroll 1
            for (int c = 0; c < mine; c += 16) {
              uint32_t r[16];
              if (nk > 0) {
                tc::ld16_nowait(tmem + lane_addr + acc.at * G::BN + c, r);
                tc::wait_ld();
                tie(r);
              }
              float v[16];  // a part without steps: zeros
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = nk > 0 ? __uint_as_float(r[i]) : 0.f;
#pragma unroll
              for (int i = 0; i < 16; i += 4) send(c + i, v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          } else {
            const bool runs = P.store_words >= 8 && P.out_dtype != TILEQ_DT_F32;
#pragma unroll 1
            for (int c = 0; c < mine; c += 32) {
              uint32_t r[2][16];
              if (nk > 0) {
                ld_block(tmem + lane_addr + acc.at * G::BN + cw + c, r);
                wait_block(r);
              } else {  // an expert without rows
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i >> 4][i & 15] = 0;
              }
              uint16_t *out = reinterpret_cast<uint16_t *>(P.out) + base + c * P.ldo;
              if (runs && P.out_dtype == TILEQ_DT_BF16) {
                store_runs<TILEQ_DT_BF16>(out, P.ldo, mine - c, nl, lane, r);
              } else if (runs) {
                store_runs<TILEQ_DT_F16>(out, P.ldo, mine - c, nl, lane, r);
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  uint64_t v[4];
#pragma unroll
                  for (int g = 0; g < 4; ++g) v[g] = pair(r[g >> 1][4 * j + 2 * (g & 1)], r[g >> 1][4 * j + 2 * (g & 1) + 1]);
                  store_block(P, base + (c + 8 * j) * P.ldo, mine - c - 8 * j, nl, lane, v);
                }
              }
            }
          }
          if (nk > 0) release();
          if constexpr (G::SPLIT) ok = join(base, nl);
        } else {
          uint64_t v[G::COLS / 2];  // pairs of neighbouring columns of this lane: one packed FMA folds both
#pragma unroll
          for (int i = 0; i < G::COLS / 2; ++i) v[i] = 0;
          // Scales of kScaleGroup blocks at a time, fetched while the group before is folded: thread tid has column
          // tid % 64 (the last one where there are fewer) of every other block.
          static_assert(G::F8 && G::COLS <= 64, "128 threads stage two blocks at a time");
          const int col = tid & 63, odd = tid >> 6;
          const float *xs = P.xs + k0 * P.ld_xs + t.row0 + t.c0 + min(col, mine - 1);
          const float *ws = P.ws + ((long long)t.e * P.nOb + min((t.l0 + (int)rank * 128) / 128, P.nOb - 1)) * P.nKb + k0;
          float sx[kScaleGroup / 2], sw[kScaleGroup / 2];
          auto fetch = [&](int kb) {
#pragma unroll
            for (int j = 0; j < kScaleGroup / 2; ++j) {
              const int k = max(min(kb + 2 * j + odd, nk - 1), 0);
              sx[j] = __ldg(xs + k * P.ld_xs);
              sw[j] = __ldg(ws + k);
            }
          };
          fetch(0);
#pragma unroll 1
          for (int kg = 0; kg < nk; kg += kScaleGroup) {
            float *sc = scale + (group++ & 1) * kScaleGroup * G::BN;
#pragma unroll
            for (int j = 0; j < kScaleGroup / 2; ++j) sc[(2 * j + odd) * G::BN + col] = sx[j] * sw[j];
            fetch(kg + kScaleGroup);
            // also keeps these warps within one group of each other: two buffers of scales do
            named_sync(1, 128);
#pragma unroll 1
            for (int kb = kg; kb < min(kg + kScaleGroup, nk); ++kb, sc += G::BN) {
              ok = ok && warp_wait(&my_full[acc.at], acc.parity, P.status);
              tc::fence_after();
              const uint32_t ta = tmem + lane_addr + acc.at * G::BN;
              uint32_t r[2][16];
              tc::ld16_nowait(ta, r[0]);
#pragma unroll
              for (int c = 0; c < G::COLS / 16; ++c) {
                if (16 * c < mine) {
                  tc::wait_ld();
                  tie(r[c & 1]);
                  if (c + 1 < G::COLS / 16 && 16 * (c + 1) < mine) tc::ld16_nowait(ta + 16 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
                  for (int i = 0; i < 16; i += 4) {
                    const ulonglong2 s = *reinterpret_cast<const ulonglong2 *>(sc + 16 * c + i);
                    fma2(v[8 * c + i / 2], pair(r[c & 1][i], r[c & 1][i + 1]), s.x);
                    fma2(v[8 * c + i / 2 + 1], pair(r[c & 1][i + 2], r[c & 1][i + 3]), s.y);
                  }
                }
              }
              release();
            }
          }
          if constexpr (G::SPLIT) {
#pragma unroll
            for (int i = 0; i < G::COLS / 2; i += 2)
              if (ok && 2 * i < mine) send(2 * i, low(v[i]), high(v[i]), low(v[i + 1]), high(v[i + 1]));
          } else if (ok) {
            store_lanes<G::COLS>(P, base + lane, mine, lane < nl, lane & 1, v);
          }
          if constexpr (G::SPLIT) ok = join(base, nl);
        }
      }
    }
  }

  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if constexpr (G::SPLIT) tc::cluster_sync();  // nothing may be sent to a CTA that has gone
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
using NarrowSplit = GCfg<1, 64, false, true>;
using NarrowSplitF8 = GCfg<1, 64, true, true>;
using Wide = GCfg<2, 256, false>;
using WideF8 = GCfg<1, 256, true>;

// The kernel, ready for a launch on the current device: one attribute call per instantiation and device.
template <class G, GroupedMode MODE>
cudaError_t configure() {
  static std::atomic<uint64_t> configured{0};
  auto kern = grouped_kernel<G, MODE>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (configured.load() & bit) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM)) != cudaSuccess) return e;
  if (G::SPLIT_REGS) {
    // the split asks for no more registers than the block is launched with, or it would wait forever
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs * G::THREADS < 128 * (kRegsControl + 2 * kRegsEpilogue)) return cudaErrorInvalidConfiguration;
  }
  configured.fetch_or(bit);
  return cudaSuccess;
}

// attr: room for two attributes
template <class G>
cudaLaunchConfig_t launch_config(int grid, int cluster, cudaLaunchAttribute *attr, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(G::THREADS);
  cfg.dynamicSmemBytes = G::SMEM;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster == 1 ? 1 : 2;
  return cfg;
}

template <class G, GroupedMode MODE>
cudaError_t launch_one(const GroupedArgs &a, int grid, cudaStream_t stream) {
  cudaError_t e = configure<G, MODE>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = launch_config<G>(grid, G::SPLIT ? a.splits : G::CG, attr, stream);
  e = cudaLaunchKernelEx(&cfg, grouped_kernel<G, MODE>, a);
  if (e != cudaSuccess) return e;
  count_launches();
  return cudaGetLastError();
}

// Asked once for each device and size; 0 where the question fails.
template <class G, GroupedMode MODE>
int clusters(int splits) {
  static std::atomic<int> known[64][3];
  const int which = splits == 2 ? 0 : splits == 4 ? 1 : 2;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
  if ((n = known[dev][which].load()) > 0) return n - 1;
  n = 0;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = launch_config<G>(splits, splits, attr, nullptr);
  cfg.attrs = attr + 1;
  cfg.numAttrs = 1;
  if (configure<G, MODE>() != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, grouped_kernel<G, MODE>, &cfg) != cudaSuccess) {
    cudaGetLastError();  // not this call's failure: it runs without clusters
    n = 0;
  }
  known[dev][which].store(n + 1);
  return n;
}

template <GroupedMode MODE>
cudaError_t launch_mode(const GroupedArgs &a, GroupedKernel k, int grid, cudaStream_t stream) {
  if (k == GG_WIDE) return launch_one<Wide, MODE>(a, grid, stream);
  return a.splits > 1 ? launch_one<NarrowSplit, MODE>(a, grid, stream) : launch_one<Narrow, MODE>(a, grid, stream);
}

}  // namespace

GroupedTile grouped_tile(GroupedKernel k, bool fp8) {
  if (k == GG_NARROW) return {Narrow::LANES, Narrow::BN, Narrow::BOX_B, false};
  return fp8 ? GroupedTile{WideF8::LANES, WideF8::BN, WideF8::BOX_B, true} : GroupedTile{Wide::LANES, Wide::BN, Wide::BOX_B, false};
}

int grouped_clusters(GroupedMode mode, bool fp8, int splits) {
  if (fp8) return clusters<NarrowSplitF8, GG_FWD>(splits);
  return mode == GG_FWD ? clusters<NarrowSplit, GG_FWD>(splits)
         : mode == GG_DX ? clusters<NarrowSplit, GG_DX>(splits)
                         : clusters<NarrowSplit, GG_DW>(splits);
}

cudaError_t launch_grouped(const GroupedArgs &a, GroupedKernel k, GroupedMode mode, bool fp8, int grid,
                           cudaStream_t stream) {
  if (fp8) {
    if (mode != GG_FWD) return cudaErrorInvalidValue;
    if (k == GG_WIDE) return launch_one<WideF8, GG_FWD>(a, grid, stream);
    return a.splits > 1 ? launch_one<NarrowSplitF8, GG_FWD>(a, grid, stream) : launch_one<NarrowF8, GG_FWD>(a, grid, stream);
  }
  switch (mode) {
    case GG_FWD: return launch_mode<GG_FWD>(a, k, grid, stream);
    case GG_DX: return launch_mode<GG_DX>(a, k, grid, stream);
    default: return launch_mode<GG_DW>(a, k, grid, stream);
  }
}

}  // namespace tileq
