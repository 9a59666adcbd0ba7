// Products of the dense layer with everything that follows them in registers:
//   y    = act(x @ W^T + delta + bias) + residual
//   rows = act(g) * u,  (g, u) = x @ [W_gate; W_up]^T + delta + bias, also in MXFP8
// over bf16 operands or over MXFP8 ones (e4m3, a scale byte per 32 values).
//
// Page "mstar.model.components.linear", FusedColumnLinear (W [out, in], the
// shards stacked along the output dimension), and page
// "mstar.engine.resources.lora.backend", LoraBackend.apply_linear_ (the delta:
// per output slice, scaling * h @ B^T of the token's adapter slot); page
// "spark_model/lora/target.rs", module overview, names kernels that add the
// delta in the base projection's epilogue. Before an activation that is the
// only place for it.
//
// Mathematics: the W rows are operand A and the x rows operand B of
// v_mfma_f32_32x32x16_bf16 or v_mfma_scale_f32_32x32x64_f8f6f4, whose products
// are exact and whose sums are fp32; a lane ends with columns of one row of y.
// A tile's sums go along K one step after the other, each lane's in its own
// accumulators: the same call gives the same bits. What follows is fp32 and is
// rounded once.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>
#include "epilogue.h"
#include "linear_choice.h"

namespace lora {

inline hipError_t dense_compute_units(int* dev, int* n) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  const hipError_t e = hipGetDevice(dev);
  if (e != hipSuccess) return e;
  if (*dev < 0 || *dev >= kMaxDevices) return hipErrorInvalidDevice;
  *n = known[*dev].load(std::memory_order_relaxed);
  if (*n > 0) return hipSuccess;
  const hipError_t a = hipDeviceGetAttribute(n, hipDeviceAttributeMultiprocessorCount, *dev);
  if (a == hipSuccess) known[*dev].store(*n, std::memory_order_relaxed);
  return a;
}

namespace {

// Operand forms: steps of a stage, 16-byte chunks a lane supplies per step.
// bf16, K 16 a step: chunk 2 j + h. MXFP8, K 64 a step: a lane's 32 bytes are
// chunks h and 2 + h of the step's four (values [16 h, 16 h + 16) of both
// blocks of 32), and its scale is that of block h.
// MXFP8 with a float32 result: the scaled instruction drops the low bits of its
// 64 products where they differ much (measured: relative error of a product
// of 4096 2e-5, 1e-7 by way of bf16), which a bf16 result hides and a float32
// one shows, and so do codes of the rows. There the values are taken to bf16,
// where each is exact with its scale, and multiplied at half the rate.
struct OpBF16 {
  static constexpr bool kMX = false, kWide = false;
  static constexpr int kSteps = 4, kParts = 1;
};
struct OpMX8 {
  static constexpr bool kMX = true, kWide = false;
  static constexpr int kSteps = 2, kParts = 2;
};
struct OpMX8Wide {
  static constexpr bool kMX = true, kWide = true;
  static constexpr int kSteps = 2, kParts = 2;
};

// the kernel's first argument, where the launch left it
typedef const __attribute__((address_space(4))) LinearArgs* ArgsPtr;

template <int J>
__device__ __forceinline__ f32x16 mfma_mx8(const u32x4* a, const u32x4* b, f32x16 c, uint32_t sa,
                                           uint32_t sb) {
  const i32x8 A = {(int)a[0].x, (int)a[0].y, (int)a[0].z, (int)a[0].w,
                   (int)a[1].x, (int)a[1].y, (int)a[1].z, (int)a[1].w};
  const i32x8 B = {(int)b[0].x, (int)b[0].y, (int)b[0].z, (int)b[0].w,
                   (int)b[1].x, (int)b[1].y, (int)b[1].z, (int)b[1].w};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 0, 0, 2 * J, (int)sa, 2 * J,
                                                         (int)sb);
}

// Bytes [8 g, 8 g + 8) of a lane's 32 (step J of a stage) as bf16; word holds
// the row's scales of the stage, one a block: g = 0, 1 are of block 2 J, g = 2,
// 3 of the next.
template <int J, int G>
__device__ __forceinline__ u32x4 wide8(const u32x4* o, uint32_t word) {
  const float s = mx8_exponent(word >> (8 * (2 * J + G / 2)) & 255u);
  const uint32_t lo = o[G / 2][G % 2 * 2], hi = o[G / 2][G % 2 * 2 + 1];
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true))};
}

// mask of the scale bytes of blocks [b, b + 4) of a row with kb blocks
__device__ __forceinline__ uint32_t keep_blocks(int b, int kb) {
  const int n = kb - b;
  return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}

// LDS of a tile kernel: NST stages of both operands' rows, and as many groups
// of scales (16 bytes of every row, the scales of 4 stages), and kWayB bytes a
// wave for the way of y from registers to memory.
constexpr int kWayB = 2048;
template <class OP, int BM, int BN, int NW, int NST>
struct Lds {
  static constexpr int kStageB = (BM + BN) * kRowB;
  static constexpr int kScaleOps = OP::kMX ? ((BM + BN) / 64 + NW - 1) / NW : 0;   // a wave and group
  static constexpr int kGroupB = kScaleOps * NW * 1024;
  static constexpr int kBytes = NST * (kStageB + kGroupB) + NW * kWayB;
  static constexpr int kPerUnit = 163840 / kBytes;
  // workgroups of a compute unit, at most 8 waves of them
  static constexpr int kOccupancy = kPerUnit * NW > 8 ? 8 / NW : kPerUnit;
};

// Schedule of a step of `reads` LDS reads, `products` matrix instructions and
// `transfers` into LDS: the reads after the first products, the transfers
// between all of them, so that the matrix unit never waits for a run of the
// others. Nothing moves into or out of the step.
template <int READS, int PRODUCTS, int TRANSFERS>
__device__ __forceinline__ void spread() {
  constexpr int RP = (2 * READS + PRODUCTS - 1) / PRODUCTS;
#pragma unroll
  for (int i = 0; i < PRODUCTS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (i * RP < READS) __builtin_amdgcn_sched_group_barrier(0x100, RP, 0);
    const int v = (i + 1) * TRANSFERS / PRODUCTS - i * TRANSFERS / PRODUCTS;
    if (v == 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    if (v == 2) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
    if (v > 2) __builtin_amdgcn_sched_group_barrier(0x020, 4, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}
// The same where the products are few: all reads before them.
template <int READS, int PRODUCTS, int TRANSFERS>
__device__ __forceinline__ void spread_deep() {
  __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
#pragma unroll
  for (int i = 0; i < PRODUCTS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    const int v = (i + 1) * TRANSFERS / PRODUCTS - i * TRANSFERS / PRODUCTS;
    if (v == 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    if (v == 2) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
    if (v > 2) __builtin_amdgcn_sched_group_barrier(0x020, 4, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// A step of K 64 by way of bf16: four products of K 16 a tile.
template <int J, int G, int TM, int TN>
__device__ __forceinline__ void wide_quarter(const u32x4 (*wo)[2], const u32x4 (*xo)[2],
                                             const uint32_t* sv, const uint32_t* sx,
                                             f32x16 (*acc)[TM]) {
  u32x4 xb[TM];
#pragma unroll
  for (int j = 0; j < TM; ++j) xb[j] = wide8<J, G>(xo[j], sx[j]);
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    const u32x4 wb = wide8<J, G>(wo[i], sv[i]);
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = mfma_bf16(wb, xb[j], acc[i][j]);
  }
}
template <int J, int TM, int TN>
__device__ __forceinline__ void wide_step(const u32x4 (*wo)[2], const u32x4 (*xo)[2],
                                          const uint32_t* sv, const uint32_t* sx,
                                          f32x16 (*acc)[TM]) {
  wide_quarter<J, 0, TM, TN>(wo, xo, sv, sx, acc);
  wide_quarter<J, 1, TM, TN>(wo, xo, sv, sx, acc);
  wide_quarter<J, 2, TM, TN>(wo, xo, sv, sx, acc);
  wide_quarter<J, 3, TM, TN>(wo, xo, sv, sx, acc);
}

}  // namespace

// BM x BN tiles (BN rows of W: of a gated product BN / 2 gates and the ups of
// the same columns) by a workgroup of WM x WN waves that walks its share of
// them. K passes in stages of 128 bytes a row through a ring of NST LDS
// stages, which runs on from one tile into the next.
//
// What bounds it, 256 x 256: a stage's products, 1.06 us at the clock that the
// power leaves, and its 64 KB on their way into LDS beside them. 8192 x 4096, K
// 14336: bf16 731 us (1.32 PFLOP/s; about 70 % of the matrix unit's cycles; 627
// without transfers), MXFP8 409 to 460 us (2.1 to 2.35 PFLOP/s; half of those
// cycles; 347 without transfers), MXFP8 by way of bf16 713 us. A tile's way out
// takes 11 to 15 us of about 120, its delta over one or two slots of 64 ranks 15.
// Smaller tiles: the time of a stage, 0.3 to 0.6 us for what its products and
// bytes would take half of.
template <class OP, bool GATED, int BM, int BN, int WM, int WN, int NST>
__global__ __launch_bounds__(64 * WM * WN, (Lds<OP, BM, BN, WM * WN, NST>::kOccupancy * WM * WN + 3) / 4)
void k_linear_tile(LinearArgs a, int sld, int mtiles, int ntiles) {
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  constexpr int OT = GATED ? TN / 2 : TN;          // tiles of a wave along y's columns
  constexpr int BNO = GATED ? BN / 2 : BN;         // y's columns of a tile
  constexpr int XI = BM / 8 / NW, WI = BN / 8 / NW;   // transfers a wave and stage
  using S = Lds<OP, BM, BN, NW, NST>;
  constexpr int KS = OP::kSteps, PT = OP::kParts;
  constexpr int KR = (TM + TN) * PT, KM = TM * TN * (OP::kWide ? 4 : 1);   // reads, products of a step
  // Operands in registers: of two steps, the one being multiplied and the one
  // being read; of two whole stages where a step is over before a read is.
  constexpr bool DEEP = TM * TN <= 2;
  // ROLL: where there are no registers for two, a tile of W is read over the one
  // whose products have just been asked for.
  constexpr bool ROLL = NW == 8 && OP::kMX && !OP::kWide && !DEEP;
  constexpr int BUF = DEEP ? 2 * KS : 2, WBUF = ROLL ? 1 : BUF;
  static_assert(NW % 2 == 0 && XI >= 1 && WI >= 1 && (!GATED || TN % 2 == 0), "");
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char* lsc = lds + NST * S::kStageB;
  const int lane = lane_id();
  const int w = wave_id();
  const uint32_t rowb = (uint32_t)a.K * (OP::kMX ? 1 : 2);
  const int kb = a.K / 32;
  const int kt = (int)((rowb + kRowB - 1) / kRowB);

  // block b runs on XCD b % 8, which takes a run of positions of an order in
  // which 8 row tiles vary fastest, so that the tiles an XCD runs at a time
  // share their operands in its L2
  const int G = mtiles * ntiles;
  const int per = (G + 7) / 8;
  const int stride = (int)gridDim.x >> 3;
  const int end = min(G - ((int)blockIdx.x & 7) * per, per);
  int pos = (int)blockIdx.x >> 3;
  if (pos >= end) return;
  struct Tile {
    int row, mrows, n0, ncols;   // first row of y (position of token_order), rows, first column, columns
  };
  auto locate = [&](int p) {
    constexpr int kGroupM = 8;
    const int L = ((int)blockIdx.x & 7) * per + p;
    const int grp = L / (kGroupM * ntiles);
    const int gsz = min(kGroupM, mtiles - grp * kGroupM);
    const int li = L - grp * kGroupM * ntiles;
    Tile t;
    t.row = (grp * kGroupM + li % gsz) * BM;
    t.mrows = min(BM, a.T - t.row);
    t.n0 = li / gsz * BNO;
    t.ncols = min(BNO, a.N - t.n0);
    return t;
  };
  // LDS row r of W: its part (gate, up) and column in the tile
  auto part_of = [](int r) { return GATED ? r % (TN * 32) / (OT * 32) : 0; };
  auto column_of = [](int r) { return r / (TN * 32) * (OT * 32) + r % (OT * 32); };
  auto token_of = [&](int p) {   // position -> row of x and y
    return a.order ? min(max(a.order[p], 0), a.T - 1) : p;
  };

  // global -> LDS without registers: an instruction of a wave fills 8 rows of
  // 128 bytes, lane L at row L / 8, physical chunk L % 8 of 16 bytes; the
  // lane fetches the logical chunk stored there, L % 8 ^ (row / 2) % 8, so
  // that the operand reads of 16 consecutive rows spread over the banks
  const int pr = lane >> 3;
  auto swz = [](int row) { return row >> 1 & 7; };
  const uint32_t pc = (uint32_t)((lane & 7) ^ swz(w * 8 + pr)) * 16u;   // of all its transfers
  rsrc_t x_r, w_r[GATED ? 2 : 1], xs_r, ws_r;
  uint32_t xoff[XI], woff[WI], soff[OP::kMX ? S::kScaleOps : 1];
  auto point_at = [&](const Tile& t) {
    // by token ids x is addressed from its first row (below 2 GiB), else from the tile's
    const int64_t first = a.order ? 0 : t.row;
    const uint32_t xrows = a.order ? (uint32_t)a.T : (uint32_t)t.mrows;
    x_r = make_rsrc(a.x + first * rowb, xrows * rowb);
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int row = (w + NW * i) * 8 + pr;
      xoff[i] = row < t.mrows ? (uint32_t)(token_of(t.row + row) - (int)first) * rowb + pc : kOOB;
    }
#pragma unroll
    for (int p = 0; p < (GATED ? 2 : 1); ++p)
      w_r[p] = make_rsrc(a.w + ((int64_t)p * a.N + t.n0) * rowb, (uint32_t)t.ncols * rowb);
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      const int c = column_of((w + NW * i) * 8 + pr);
      woff[i] = c < t.ncols ? (uint32_t)c * rowb + pc : kOOB;
    }
    if constexpr (OP::kMX) {
      xs_r = make_rsrc(a.xs + first * sld, xrows * (uint32_t)sld);
      ws_r = make_rsrc(a.ws + (int64_t)t.n0 * sld,
                       (uint32_t)((GATED ? a.N : 0) + t.ncols) * (uint32_t)sld);
#pragma unroll
      for (int i = 0; i < S::kScaleOps; ++i) {
        const int row = (w + NW * i) * 64 + lane;
        if (row < BM) {
          soff[i] = row < t.mrows ? (uint32_t)(token_of(t.row + row) - (int)first) * (uint32_t)sld
                                  : kOOB;
        } else {
          const int r = row - BM, c = column_of(r);
          soff[i] = r < BN && c < t.ncols ? (uint32_t)(part_of(r) * a.N + c) * (uint32_t)sld : kOOB;
        }
      }
    }
  };
  // the scales of stages [it, it + 4), it a multiple of 4
  auto issue_scales = [&](int it, int group) {
    if constexpr (OP::kMX) {
      const uint32_t b0 = (uint32_t)it * 4;   // below sld, a multiple of 16
#pragma unroll
      for (int i = 0; i < S::kScaleOps; ++i)
        dma16((w + NW * i) * 64 < BM ? xs_r : ws_r,
              lsc + group * S::kGroupB + (w + NW * i) * 1024, soff[i] + b0);
    }
  };
  auto issue_x = [&](int it, int slot) {
    const uint32_t k0 = (uint32_t)it * kRowB;
    const bool live = k0 + pc < rowb;
    char* sb = lds + slot * S::kStageB;
#pragma unroll
    for (int i = 0; i < XI; ++i) dma16(x_r, sb + (w + NW * i) * 1024, live ? xoff[i] + k0 : kOOB);
  };
  auto issue_w = [&](int it, int slot) {
    const uint32_t k0 = (uint32_t)it * kRowB;
    const bool live = k0 + pc < rowb;
    char* sb = lds + slot * S::kStageB;
#pragma unroll
    for (int i = 0; i < WI; ++i)
      dma16(w_r[part_of((w + NW * i) * 8)], sb + BM * kRowB + (w + NW * i) * 1024,
            live ? woff[i] + k0 : kOOB);
  };
  static_assert(!OP::kMX || BM % 64 == 0, "a transfer of scales is all of x or all of W");

  // the walk of the transfers, NST - 1 stages ahead: stage lit of the tile at
  // position pos, into the slot just freed
  Tile cur = locate(pos);
  int cpos = pos;
  bool has_ld = true;
  int lit = 0, lgroup = NST - 1;
  point_at(cur);
  auto fetch = [&](int slot) {
    if (!has_ld) return;
    if (lit == kt) {
      lit = 0;
      pos += stride;
      has_ld = pos < end;
      if (!has_ld) return;
      point_at(locate(pos));
    }
    if (lit % 4 == 0) {
      lgroup = lgroup + 1 == NST ? 0 : lgroup + 1;
      issue_scales(lit, lgroup);
    }
    issue_x(lit, slot);
    issue_w(lit, slot);
    ++lit;
  };
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) fetch(i);

  const int m = lane & 31, h = lane >> 5;
  const int wm = w % WM, wn = w / WM;
  const uint32_t xrow = (uint32_t)(wm * TM * 32 + m) * kRowB;
  const uint32_t wrow = (uint32_t)(BM + wn * TN * 32 + m) * kRowB;
  const uint32_t xsc = (uint32_t)(wm * TM * 32 + m) * 16;
  const uint32_t wsc = (uint32_t)(BM + wn * TN * 32 + m) * 16;
  const uint32_t sw = (uint32_t)(swz(m) << 4);
  f32x16 acc[TN][TM];
  u32x4 xo[BUF][TM][PT], wo[WBUF][TN][PT];
  uint32_t sx[DEEP ? 2 : 1][TM], sv[DEEP ? 2 : 1][TN];   // scale words
  // step j of the stage in `slot`, into buffer q
  auto read = [&](int slot, int j, auto qc) {
    constexpr int Q = decltype(qc)::value;
    const char* sb = lds + slot * S::kStageB;
    uint32_t c[PT];
#pragma unroll
    for (int p = 0; p < PT; ++p) c[p] = (uint32_t)((OP::kMX ? 4 * j + 2 * p + h : 2 * j + h) << 4) ^ sw;
    auto read_w = [&](int i) {
#pragma unroll
      for (int p = 0; p < PT; ++p) wo[Q % WBUF][i][p] = *(const u32x4*)(sb + wrow + i * 32 * kRowB + c[p]);
    };
    auto read_x = [&](int i) {
#pragma unroll
      for (int p = 0; p < PT; ++p) xo[Q][i][p] = *(const u32x4*)(sb + xrow + i * 32 * kRowB + c[p]);
    };
    read_w(0);   // in the order in which the products take them
#pragma unroll
    for (int i = 0; i < TM; ++i) read_x(i);
#pragma unroll
    for (int i = 1; i < TN; ++i) read_w(i);
  };
  // scale words of stage it; the byte of this half's block is then the lowest
  auto read_scales = [&](int it, int group, uint32_t* nx, uint32_t* nv) {
    if constexpr (OP::kMX) {
      const char* ss = lsc + group * S::kGroupB + (it & 3) * 4;
#pragma unroll
      for (int i = 0; i < TM; ++i) nx[i] = *(const uint32_t*)(ss + xsc + i * 512);
#pragma unroll
      for (int i = 0; i < TN; ++i) nv[i] = *(const uint32_t*)(ss + wsc + i * 512);
    }
  };
  auto take_scales = [&](int it, uint32_t* nx, uint32_t* nv, uint32_t* tx, uint32_t* tv) {
    if constexpr (OP::kMX) {
      const uint32_t keep = keep_blocks(it * 4, kb);   // the padding of a scale row is not a scale
#pragma unroll
      for (int i = 0; i < TM; ++i) tx[i] = (nx[i] & keep) >> (OP::kWide ? 0 : 8 * h);
#pragma unroll
      for (int i = 0; i < TN; ++i) tv[i] = (nv[i] & keep) >> (OP::kWide ? 0 : 8 * h);
    }
  };
  auto step = [&](auto jc, auto qc, const uint32_t* tx, const uint32_t* tv) {
    constexpr int J = decltype(jc)::value, Q = decltype(qc)::value;
    if constexpr (OP::kWide) {
      wide_step<J, TM, TN>(wo[Q % WBUF], xo[Q], tv, tx, acc);
    } else {
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          if constexpr (OP::kMX)
            acc[i][j] = mfma_mx8<J>(wo[Q % WBUF][i], xo[Q][j], acc[i][j], tv[i], tx[j]);
          else
            acc[i][j] = mfma_bf16(wo[Q % WBUF][i][0], xo[Q][j][0], acc[i][j]);
        }
    }
  };

  // Stage by stage: the products of what is in registers, while the next is
  // read from LDS and later ones are on their way into it. A stage's slot is
  // free once every wave has it in registers, which is before its last step
  // (DEEP: its first).
  constexpr int L = KS - 1;
  int slot = 0, group = NST - 1;
  auto none = [&]() {   // before a tile's first stage: operands that add nothing
    constexpr int Z = DEEP ? KS : 1;
#pragma unroll
    for (int q = 0; q < Z; ++q) {
      const int at = DEEP ? q : L % 2;
#pragma unroll
      for (int p = 0; p < PT; ++p) {
#pragma unroll
        for (int i = 0; i < TN; ++i) wo[ROLL ? 0 : at][i][p] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < TM; ++i) xo[at][i][p] = u32x4{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) sx[0][i] = 0;
#pragma unroll
    for (int i = 0; i < TN; ++i) sv[0][i] = 0;
  };
  for (;;) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
    none();
    // stage `it` is there once at most the transfers of later ones are
    // outstanding; the barrier makes every wave's part visible and frees the
    // slot of the stage before it, into which stage it + NST - 1 is asked for
    auto arrive = [&](int it, auto tail) {
      if (NST > 2 && (!decltype(tail)::value || has_ld))
        __builtin_amdgcn_s_waitcnt(vm_lds_le((NST - 2) * (XI + WI)));
      else
        __builtin_amdgcn_s_waitcnt(vm_lds_le(0));
      barrier_no_fence();
      if (it % 4 == 0) group = group + 1 == NST ? 0 : group + 1;
      if constexpr (!decltype(tail)::value) {
        if (OP::kMX && (it + NST - 1) % 4 == 0) {
          lgroup = lgroup + 1 == NST ? 0 : lgroup + 1;
          issue_scales(it + NST - 1, lgroup);
        }
      }
    };
    auto before = [&]() { return slot == 0 ? NST - 1 : slot - 1; };
    using std::integral_constant;
    auto stage = [&](int it, auto tail) {
      constexpr bool TAIL = decltype(tail)::value;
      uint32_t nx[TM], nv[TN];
      arrive(it, tail);
      if constexpr (TAIL) fetch(before());
      // the last step of the stage before
      read(slot, 0, integral_constant<int, 0>());
      read_scales(it, group, nx, nv);
      if constexpr (!TAIL) issue_x(it + NST - 1, before());
      step(integral_constant<int, L>(), integral_constant<int, L % 2>(), sx[0], sv[0]);
      spread<KR + (OP::kMX ? TM + TN : 0), KM, TAIL ? 0 : XI>();
      take_scales(it, nx, nv, sx[0], sv[0]);
      read(slot, 1, integral_constant<int, 1>());
      if constexpr (!TAIL) issue_w(it + NST - 1, before());
      step(integral_constant<int, 0>(), integral_constant<int, 0>(), sx[0], sv[0]);
      spread<KR, KM, TAIL ? 0 : WI>();
      if constexpr (KS == 4) {
        read(slot, 2, integral_constant<int, 0>());
        step(integral_constant<int, 1>(), integral_constant<int, 1>(), sx[0], sv[0]);
        spread<KR, KM, 0>();
        read(slot, 3, integral_constant<int, 1>());
        step(integral_constant<int, 2>(), integral_constant<int, 0>(), sx[0], sv[0]);
        spread<KR, KM, 0>();
      }
      slot = slot + 1 == NST ? 0 : slot + 1;
    };
    // ROLL: the products of step J, whose x is in buffer J, tile of W by tile of W,
    // and over each the same tile of step R of the stage in `slot`. The transfers
    // come before all of that: with one stage ahead they need its whole time
    // (between the products 6 % slower).
    auto roll = [&](auto jc, auto rc, auto transfers, auto scale_reads) {
      constexpr int J = decltype(jc)::value, R = decltype(rc)::value;
      constexpr int DMAS = decltype(transfers)::value, SR = decltype(scale_reads)::value;
      const char* sb = lds + slot * S::kStageB;
      uint32_t c[PT];
#pragma unroll
      for (int p = 0; p < PT; ++p) c[p] = (uint32_t)((4 * R + 2 * p + h) << 4) ^ sw;
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int p = 0; p < PT; ++p) xo[R][i][p] = *(const u32x4*)(sb + xrow + i * 32 * kRowB + c[p]);
#pragma unroll
      for (int i = 0; i < TN; ++i) {
#pragma unroll
        for (int j = 0; j < TM; ++j)
          acc[i][j] = mfma_mx8<J>(wo[0][i], xo[J][j], acc[i][j], sv[0][i], sx[0][j]);
#pragma unroll
        for (int p = 0; p < PT; ++p) wo[0][i][p] = *(const u32x4*)(sb + wrow + i * 32 * kRowB + c[p]);
      }
      if constexpr (DMAS > 0) __builtin_amdgcn_sched_group_barrier(0x020, DMAS, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, TM * PT + SR, 0);
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, TM, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, PT, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto roll_stage = [&](int it, auto tail) {
      if constexpr (ROLL) {
        constexpr bool TAIL = decltype(tail)::value;
        uint32_t nx[TM], nv[TN];
        arrive(it, tail);
        if constexpr (TAIL) {
          fetch(before());
        } else {
          issue_x(it + NST - 1, before());
          issue_w(it + NST - 1, before());
        }
        read_scales(it, group, nx, nv);
        roll(integral_constant<int, 1>(), integral_constant<int, 0>(),
             integral_constant<int, TAIL ? 0 : XI + WI>(), integral_constant<int, TM + TN>());
        take_scales(it, nx, nv, sx[0], sv[0]);
        roll(integral_constant<int, 0>(), integral_constant<int, 1>(), integral_constant<int, 0>(),
             integral_constant<int, 0>());
        slot = slot + 1 == NST ? 0 : slot + 1;
      }
    };
    // DEEP: reads into the buffers of parity P, products of the others
    auto deep_products = [&](auto pc2) {
      constexpr int O = decltype(pc2)::value;
      if constexpr (DEEP) {
        step(integral_constant<int, 0>(), integral_constant<int, O * KS>(), sx[O], sv[O]);
        step(integral_constant<int, 1>(), integral_constant<int, O * KS + 1>(), sx[O], sv[O]);
        if constexpr (KS == 4) {
          step(integral_constant<int, 2>(), integral_constant<int, O * KS + 2>(), sx[O], sv[O]);
          step(integral_constant<int, 3>(), integral_constant<int, O * KS + 3>(), sx[O], sv[O]);
        }
      }
    };
    auto deep_stage = [&](int it, auto tail, auto pc2) {
      constexpr bool TAIL = decltype(tail)::value;
      constexpr int P = decltype(pc2)::value;
      if constexpr (DEEP) {
        uint32_t nx[TM], nv[TN];
        arrive(it, tail);
        if constexpr (TAIL) fetch(before());
        read_scales(it, group, nx, nv);
        read(slot, 0, integral_constant<int, P * KS>());
        read(slot, 1, integral_constant<int, P * KS + 1>());
        if constexpr (KS == 4) {
          read(slot, 2, integral_constant<int, P * KS + 2>());
          read(slot, 3, integral_constant<int, P * KS + 3>());
        }
        if constexpr (!TAIL) {
          issue_x(it + NST - 1, before());
          issue_w(it + NST - 1, before());
        }
        deep_products(integral_constant<int, 1 - P>());
        spread_deep<KR * KS + (OP::kMX ? TM + TN : 0), KM * KS, TAIL ? 0 : XI + WI>();
        take_scales(it, nx, nv, sx[P], sv[P]);
        slot = slot + 1 == NST ? 0 : slot + 1;
      }
    };
    // all but the last NST - 1 stages are followed by one of the same tile
    int it = 0;
    if constexpr (DEEP) {   // in pairs, a parity each
      using P0 = integral_constant<int, 0>;
      using P1 = integral_constant<int, 1>;
      for (; it + NST < kt; it += 2) {
        deep_stage(it, std::false_type(), P1());
        deep_stage(it + 1, std::false_type(), P0());
      }
      if (it > 0) lit = min(it + NST - 1, kt);
      for (;; it += 2) {
        if (it == kt) {
          deep_products(P0());
          break;
        }
        deep_stage(it, std::true_type(), P1());
        if (it + 1 == kt) {
          deep_products(P1());
          break;
        }
        deep_stage(it + 1, std::true_type(), P0());
      }
    } else if constexpr (ROLL) {
      for (; it + NST - 1 < kt; ++it) roll_stage(it, std::false_type());
      if (it > 0) lit = kt;
      for (; it < kt; ++it) roll_stage(it, std::true_type());
      step(integral_constant<int, 1>(), integral_constant<int, 1>(), sx[0], sv[0]);
    } else {
      for (; it + NST - 1 < kt; ++it) stage(it, std::false_type());
      if (it > 0) lit = kt;
      for (; it < kt; ++it) stage(it, std::true_type());
      step(integral_constant<int, L>(), integral_constant<int, L % 2>(), sx[0], sv[0]);
    }

    // what follows reads its arguments here, not ahead of the main loop
    ArgsPtr ap = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(ap));
    const LinearArgs& e = *(const LinearArgs*)ap;
    // y columns of this wave are [c0w, c0w + OT 32)
    const int c0w = cur.n0 + wn * OT * 32;

    // ---- the LoRA delta, before anything else ----------------------------
    // For each slot with rows among the wave's, each slice among its columns
    // and 16 ranks at a time: scaling * h as bf16 parts (other rows 0) against
    // the slot's B, on the accumulators. A turn is a few products and its loads
    // take 2 us, so the loads of kTurns turns are on their way at a time.
    // Looking for values that are not for it, see add_unfit, takes 0 to 1 % of a
    // product; having one 4 to 6 times the product's time at 8192 rows.
    bool unfit = false;
    if (e.h) {
      // h in all its 24 bits of fraction; in 16 in gated products by the scaled
      // instruction, which has no codes to follow and loses 2^-16 itself
      constexpr int TERMS = GATED && OP::kMX && !OP::kWide ? 2 : 3;
      constexpr int PARTS = GATED ? 2 : 1;   // gates and ups have slices of their own
      constexpr int kTurns = TM * TN > 4 ? 2 : 4;   // as the registers allow
      const int SR = e.slices * e.R, out = PARTS * e.N;
      const int p0 = cur.row + wm * TM * 32, p1 = min(p0 + TM * 32, cur.row + cur.mrows);
      const rsrc_t h_r = make_rsrc(e.h, (uint32_t)e.T * (uint32_t)SR * 4u);
      uint32_t hoff[TM], boff[OT];
      int column[OT];   // of this lane's row of W tile i
#pragma unroll
      for (int j = 0; j < TM; ++j)
        hoff[j] = ((uint32_t)token_of(min(p0 + j * 32 + m, e.T - 1)) * (uint32_t)SR + 8u * h) * 4u;
#pragma unroll
      for (int i = 0; i < OT; ++i) {
        column[i] = c0w + i * 32 + m;
        boff[i] = ((uint32_t)column[i] * (uint32_t)e.R + 8u * h) * 2u;
      }
      // What a turn needs to know is held by the lanes, so that going on to the
      // next one waits for no load. Lane l: slot base + l, its rows among the
      // wave's, rank and scaling;
      int base = 0, wlo = 0, whi = 0, wrank = 0;
      float wscale = 0.0f;
      uint64_t with_rows = 0;   // the slots that have some
      bool more = false;        // slots behind these
      auto window = [&](int first) {
        base = first;
        const int s = min(base + lane, e.slots - 1);
        int beg, len;
        segment_of(e.indptr, s, e.T, beg, len);
        wrank = clamp_rank(e.ranks[s], e.R);
        wscale = e.scalings[s];
        wlo = max(beg, p0) - p0;
        whi = min(beg + len, p1) - p0;
        const bool there = base + lane < e.slots;
        with_rows = __ballot(there && wrank > 0 && wlo < whi);
        more = base + kWave < e.slots && __ballot(beg >= p1) == 0;
      };
      // and part l / slices, slice l % slices: its columns among the wave's.
      int clo = 0, chi = 0;
      uint64_t with_columns;
      {
        const int l = min(lane, PARTS * e.slices - 1), part = GATED && l >= e.slices ? 1 : 0;
        const int si = l - part * e.slices;
        clo = max(e.off[si] - part * e.N, c0w);
        chi = min(e.off[si + 1] - part * e.N, min(c0w + OT * 32, e.N));
        with_columns = __ballot(lane < PARTS * e.slices && clo < chi);
      }
      struct Turn {
        int s, lo, hi, r;   // slot, its rows of the wave's, its rank (0: no turn)
        float scale;
        int part, si, clo, chi, k0;   // part, slice and its columns, first rank
      };
      Turn t = {};
      uint64_t columns = 0;   // with_columns, those of this slot that are to come
      bool has = p0 < p1 && with_columns != 0;
      auto next = [&]() {
        t.k0 += 16;
        if (t.k0 < t.r) return;
        t.k0 = 0;
        if (columns == 0) {
          while (with_rows == 0 && more) window(base + kWave);
          has = with_rows != 0;
          if (!has) return;
          const int l = __builtin_ctzll(with_rows);
          with_rows &= with_rows - 1;
          t.s = base + l;
          t.lo = __builtin_amdgcn_readlane(wlo, l);
          t.hi = __builtin_amdgcn_readlane(whi, l);
          t.r = __builtin_amdgcn_readlane(wrank, l);
          t.scale = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wscale), l));
          columns = with_columns;
        }
        const int l = __builtin_ctzll(columns);
        columns &= columns - 1;
        t.part = GATED && l >= e.slices ? 1 : 0;
        t.si = l - t.part * e.slices;
        t.clo = __builtin_amdgcn_readlane(clo, l);
        t.chi = __builtin_amdgcn_readlane(chi, l);
      };
      auto take = [&]() {   // the turn at t, and t on to the next
        if (!has) return Turn{};
        const Turn now = t;
        next();
        return now;
      };
      auto in_tile = [&](const Turn& n, int j) { return n.lo < j * 32 + 32 && n.hi > j * 32; };
      u32x4 hb[kTurns][TM][2], bb[kTurns][OT];
      Turn turn[kTurns];
      auto load = [&](int d) {   // past the rows, the columns and the ranks: zeros
        const Turn& n = turn[d];
        const bool some = n.k0 + 8 * h < n.r;
        const rsrc_t b_r = make_rsrc((const char*)e.b + ((int64_t)n.s * out + n.part * e.N) * e.R * 2,
                                     (uint32_t)e.N * (uint32_t)e.R * 2u);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          const int row = j * 32 + m;
          const uint32_t o = row >= n.lo && row < n.hi && some
                                 ? hoff[j] + (uint32_t)(n.si * e.R + n.k0) * 4u : kOOB;
          hb[d][j][0] = bload16(h_r, o);
          hb[d][j][1] = bload16(h_r, o + 16u);
        }
#pragma unroll
        for (int i = 0; i < OT; ++i) {
          const bool in = column[i] >= n.clo && column[i] < n.chi && some;
          bb[d][i] = bload16(b_r, in ? boff[i] + (uint32_t)n.k0 * 2u : kOOB);
        }
      };
      if (has) {
        window(e.slots <= kWave ? 0 : min(wave_slot_of(e.indptr, e.slots, p0), e.slots - 1));
        next();
      }
#pragma unroll
      for (int d = 0; d < kTurns; ++d) {
        turn[d] = take();
        load(d);
      }
      while (turn[0].r > 0) {
#pragma unroll
        for (int d = 0; d < kTurns; ++d) {
          const Turn now = turn[d];
          const int n = now.r - now.k0 - 8 * h;   // ranks of this lane's eight that there are
          if (now.k0 + 16 > now.r) {   // what lies past the rank does not count
#pragma unroll
            for (int j = 0; j < TM; ++j)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (k >= n) hb[d][j][k / 4][k % 4] = 0u;
#pragma unroll
            for (int i = 0; i < OT; ++i)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (k >= n) bb[d][i][k / 2] &= (k & 1) ? 0x0000ffffu : 0xffff0000u;
          }
          uint32_t ends = 0;
#pragma unroll
          for (int i = 0; i < OT; ++i) ends |= not_finite(bb[d][i]);
          if (__builtin_expect(__ballot(ends != 0) != 0, 0)) {
            unfit = true;
#pragma unroll
            for (int i = 0; i < OT; ++i) bb[d][i] &= finite_halves(bb[d][i]);
          }
#pragma unroll
          for (int j = 0; j < TM; ++j)
            if (in_tile(now, j)) {
              float v[8];
              u32x4 hp[TERMS];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(hb[d][j][k / 4][k % 4]) * now.scale;
              split_bf16<TERMS>(v, hp);
              if (__builtin_expect(__ballot(not_finite(hp[0]) != 0) != 0, 0)) {
                unfit = true;
                const u32x4 keep = finite_halves(hp[0]);
#pragma unroll
                for (int p = 0; p < TERMS; ++p) hp[p] &= keep;
              }
#pragma unroll
              for (int part = 0; part < PARTS; ++part)
                if (now.part == part) {
#pragma unroll
                  for (int i = 0; i < OT; ++i)
#pragma unroll
                    for (int p = 0; p < TERMS; ++p)
                      acc[part * OT + i][j] = mfma_bf16(bb[d][i], hp[p], acc[part * OT + i][j]);
                }
            }
          turn[d] = take();
          load(d);
        }
      }
    }
    // wait states between the last MFMA and the first vector read of its result
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);

    // ---- bias, activation, residual or the gated product; y --------------
    // A wave's tiles of 32 x 32 go to memory one after the other by way of
    // 2 KB of LDS that are its own, as 16 rows of 32 columns (the gates', then
    // the ups'), 8 columns a lane: of the epilogue only the 16-byte writes into
    // LDS are there once for each tile. (With the whole of it unrolled over the
    // accumulators the code of a kernel was 145 KB against 64 KB of instruction
    // cache, and a tile of 256 x 256 took 34 us to finish in place of 15.) A
    // row's 16-byte chunk q is held at q ^ (row & 7) of its eight.
    char* way = lds + NST * (S::kStageB + S::kGroupB) + w * kWayB;
    auto fence = []() { asm volatile("" ::: "memory"); };   // a wave's LDS operations are done in order
    auto put = [&](const f32x16& z) {   // row m
      const int row = m % 16;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)(way + row * 128 + (((2 * q + h) ^ (row & 7)) << 4)) =
            f32x4{z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]};
    };
    auto get = [&](float* v) {   // columns [8 (lane % 4), 8 (lane % 4) + 8) of row lane / 4
      const int row = lane / 4;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const f32x4 u = *(const f32x4*)(way + row * 128 + (((lane % 4 * 2 + p) ^ (row & 7)) << 4));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * p + k] = u[k];
      }
    };
    // rows and columns of this lane in tile (j, b), half k
    auto row_in = [&](int j, int k) { return wm * TM * 32 + j * 32 + k * 16 + lane / 4; };
    // Seldom: tile by tile to LDS, what is unfit added there, and back. (In the loop
    // below, where more is held, it costs the main loop registers; so do addresses
    // that the compiler can form ahead of it, hence the lane that it cannot know.)
    if (__builtin_expect(unfit, 0)) {
      int ln = lane;
      asm volatile("" : "+v"(ln));
      const int lm = ln & 31, lr = ln / 4;
      auto chunk = [&](int row, int c) { return (f32x4*)(way + row * 128 + ((c ^ (row & 7)) << 4)); };
#pragma unroll 1
      for (int u = 0; u < TM * TN * 2; ++u) {
        const int i = u / 2 % TN, j = u / 2 / TN, k = u % 2;
#pragma unroll
        for (int q = 0; q < TM * TN; ++q)
          if (u / 2 == q && lm / 16 == k) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const f32x16& z = acc[q % TN][q / TN];
              *chunk(lm % 16, 2 * c + ln / 32) = f32x4{z[4 * c], z[4 * c + 1], z[4 * c + 2], z[4 * c + 3]};
            }
          }
        fence();
        f32x4 v[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) v[c] = *chunk(lr, ln % 4 * 2 + c);
        fence();
        const int row = wm * TM * 32 + j * 32 + k * 16 + lr, p = cur.row + row;
        if (row < cur.mrows)
          add_unfit(e, token_of(p), p, GATED ? i / OT * e.N : 0, c0w + i % OT * 32 + ln % 4 * 8,
                    GATED ? 2 * (int64_t)e.N : e.N, v);
#pragma unroll
        for (int c = 0; c < 2; ++c) *chunk(lr, ln % 4 * 2 + c) = v[c];
        fence();
#pragma unroll
        for (int q = 0; q < TM * TN; ++q)
          if (u / 2 == q && lm / 16 == k) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const f32x4 z = *chunk(lm % 16, 2 * c + ln / 32);
#pragma unroll
              for (int x = 0; x < 4; ++x) acc[q % TN][q / TN][4 * c + x] = z[x];
            }
          }
        fence();
      }
    }
    auto ahead_of = [&](int u) {
      Ahead<GATED> n;
      const int c = c0w + u % OT * 32 + lane % 4 * 8;
      n.load_bias(e, c);
      if constexpr (!GATED) {
        if (e.residual) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int row = row_in(u / OT, k);
            if (row < cur.mrows) n.load_residual(e, k, (int64_t)token_of(cur.row + row) * e.N + c, c);
          }
        }
      }
      return n;
    };
    Ahead<GATED> ahead = ahead_of(0);
#pragma unroll 1
    for (int u = 0; u < TM * OT; ++u) {
      Ahead<GATED> now = ahead;
      ahead = ahead_of(min(u + 1, TM * OT - 1));
      const int cb = c0w + u % OT * 32;
      if (cb >= e.N) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v[8], up[8];
#pragma unroll
        for (int q = 0; q < TM * OT; ++q)
          if (u == q && m / 16 == k) put(acc[q % OT][q / OT]);
        fence();
        get(v);
        fence();
        if constexpr (GATED) {
#pragma unroll
          for (int q = 0; q < TM * OT; ++q)
            if (u == q && m / 16 == k) put(acc[OT + q % OT][q / OT]);
          fence();
          get(up);
          fence();
        }
        const int row = row_in(u / OT, k);
        finish<GATED>(e, now, k, row < cur.mrows, token_of(min(cur.row + row, e.T - 1)),
                      cb + lane % 4 * 8, v, up);
      }
    }
    cpos += stride;
    if (cpos >= end) break;
    cur = locate(cpos);
  }
}

template <class OP, bool GATED, int BM, int BN, int WM, int WN, int NST>
hipError_t launch_tile(const LinearArgs& a, hipStream_t stream, int dev, int cus) {
  constexpr int NW = WM * WN;
  using S = Lds<OP, BM, BN, NW, NST>;
  constexpr int lds = S::kBytes;
  const int mt = tiles_of(a.T, BM), nt = tiles_of(a.N, GATED ? BN / 2 : BN);
  const int64_t tiles = (int64_t)mt * nt;
  if (tiles > 0x7ffffff0) return hipErrorInvalidValue;
  const int64_t grid = std::min<int64_t>(8 * ((tiles + 7) / 8), (int64_t)cus * S::kOccupancy / 8 * 8);
  const void* f = (const void*)k_linear_tile<OP, GATED, BM, BN, WM, WN, NST>;
  if (lds > 65536) {   // said once per device
    static std::atomic<uint64_t> said{0};
    if (!(said.load(std::memory_order_relaxed) >> dev & 1)) {
      const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
      said.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL((k_linear_tile<OP, GATED, BM, BN, WM, WN, NST>), dim3((unsigned)grid),
                     dim3(64 * NW), lds, stream, a, mx8_scale_row(a.K), mt, nt);
  return hipGetLastError();
}

}  // namespace lora
