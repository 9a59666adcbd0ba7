// Products over MXFP4 operands: y = x @ W^T for one weight, or per row the
// weight of the expert that the row belongs to.
//
// Page "mstar.model.components.linear", FusedColumnLinear (W [out, in], the
// shards stacked along the output dimension), and page
// "spark_model/lora/expert_apply.rs" (the experts' products on rows sorted
// by expert, before the experts' LoRA is added to them).
//
// Mathematics: v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 codes and a scale
// byte of each operand per lane and forms D += A B^T over a K step of 64.
// Products of two 4-bit values and powers of two are exact; the sums are
// fp32, in the same order of K in every tile shape, so a row's result does
// not depend on the batch it is in; y is rounded once. The W rows are operand
// A and the x rows operand B, so a lane ends with runs of 4 columns of one
// row of y.
//
// What bounds it (MI355X, 4.7 TB/s copy, 2.66 PFLOP/s largest fp8 product).
// Cards differ: a range is that of several cards, its low end with the inputs
// of the call before in the cache, its high end with other ones every time.
//   few rows: the weight's bytes. 512 rows of 8 experts x 28672 x 4096: 108
//     to 129 us, 4.1 to 4.9 TB/s of codes, scales and y.
//   many rows: 8192 x 28672 x 4096 493 to 558 us, 3.4 to 3.9 PFLOP/s; 16384
//     rows of 8 experts x 4096 x 14336 533 to 564 us (its 70 row tiles x 16
//     take 4.4 turns of the 256 units). Where the first one took 511 us, the
//     products alone were 266 of them, waiting for their LDS operands 85, for
//     the transfers 55, scales 20, and the way of y through LDS and out 70.
//   few tiles (a decode step's dense projections): the walk over K, 0.3 us a
//     stage of 256. 1 x 6144 x 4096: 8.1 to 8.9 us, of which the launch and the
//     ends of the walk are 5.
#include <algorithm>
#include <atomic>
#include <type_traits>
#include "lora_common.h"
#include "experts.h"

namespace lora {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));   // 16 bytes from any element on

// D[32x32] += A[32 x 64] . B[32 x 64]^T: lane (m = lane & 31, h = lane >> 5)
// supplies row m, one block of 32 codes, and byte J of its scale word as that
// block's scale; it receives D[8 (i / 4) + 4 h + i % 4][m] in element i.
template <int J>
__device__ __forceinline__ f32x16 mfma_mx32(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, J, (int)sa, J, (int)sb);
}

constexpr int kStageK = 256;        // K of one LDS stage
constexpr int kRowB = kStageK / 2;  // code bytes of a row in it
// an operand tile is at most 2^27 bytes, so an offset past kPastEnd, with or
// without kOOB, is outside it
constexpr uint32_t kPastEnd = 0x40000000u;

// One 4-byte global -> LDS transfer per lane: lane L to byte 4 L of dst.
__device__ __forceinline__ void dma4(rsrc_t r, char* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 4, (int)off, 0, 0, 0);
}

// scale bytes of blocks [b, b + 4) of a row with kb blocks, the rest cleared
__device__ __forceinline__ uint32_t keep_blocks(uint32_t v, int b, int kb) {
  const int n = kb - b;
  return n >= 4 ? v : n <= 0 ? 0u : v & ((1u << (8 * n)) - 1u);
}

// s_waitcnt operand: at most n vector memory operations and no LDS operation
// outstanding; 63 vector memory operations are not waited for at all.
constexpr int vm_lds(int n) { return vmcnt_le(n) & ~(15 << 8); }

// Workgroup barrier that waits for the wave's LDS operations alone, so that
// transfers and stores stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(vm_lds(63));
  barrier_no_fence();
}

// Tiles of `tile` that hold n rows or columns; n up to 2^31 - 1, whose sum with
// the tile is no int any more.
__host__ __device__ __forceinline__ int tiles_of(int n, int tile) {
  return (int)(((uint32_t)n + (uint32_t)tile - 1) / (uint32_t)tile);
}

// The current device and its compute units (asked for once per device).
constexpr int kMaxDevices = 64;
hipError_t compute_units(int* dev, int* n) {
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

}  // namespace

// Rows of y outside [offsets[0], offsets[E]), by the whole grid.
template <typename D>
__device__ __forceinline__ void zero_dead_rows(const MxArgs& a) {
  const int lo = min(max(a.offsets[0], 0), a.rows);
  const int hi = min(max(a.offsets[a.E], lo), a.rows);
  const int64_t dead = ((int64_t)lo + (a.rows - hi)) * a.N;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < dead;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t at = i < (int64_t)lo * a.N ? i : i + (int64_t)(hi - lo) * a.N;
    if constexpr (D::kBytes == 2) ((uint16_t*)a.y)[at] = 0; else ((float*)a.y)[at] = 0.0f;
  }
}

// Row tiles of BM rows over all experts, counted by every wave for itself. No
// more than bounds in order can give, whatever the bounds are.
template <int BM>
__device__ __forceinline__ int count_tiles(const MxArgs& a) {
  const int most = tiles_of(a.rows, BM) + a.E;
  int tiles = 0;
  for (int s = lane_id(); s < a.E; s += kWave) {
    int beg, len;
    segment_of(a.offsets, s, a.rows, beg, len);
    tiles = min(tiles + tiles_of(len, BM), most);
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) tiles = min(tiles + __shfl_xor(tiles, d), most);
  return __builtin_amdgcn_readfirstlane(tiles);
}

// Row tile `item` of the experts: its first row, rows and expert.
template <int BM>
__device__ __forceinline__ void find_tile(const MxArgs& a, int item, int& row, int& rows, int& e) {
  const int lane = lane_id();
  int before = 0;
  row = rows = e = 0;
  for (int s0 = 0; s0 < a.E; s0 += kWave) {
    int beg = 0, len = 0;
    if (s0 + lane < a.E) segment_of(a.offsets, s0 + lane, a.rows, beg, len);
    const int tiles = tiles_of(len, BM);
    const int upto = before + wave_inclusive_scan(tiles);
    const uint64_t past = __ballot(upto > item);
    if (past != 0) {
      const int src = __ffsll((unsigned long long)past) - 1;
      // within the segment, whatever the bounds are
      const int mine = __shfl(tiles, src);
      const int local = max(min(item - (__shfl(upto, src) - mine), mine - 1), 0);
      row = __builtin_amdgcn_readfirstlane(__shfl(beg, src) + local * BM);
      rows = __builtin_amdgcn_readfirstlane(min(BM, __shfl(len, src) - local * BM));
      e = __builtin_amdgcn_readfirstlane(s0 + src);
      return;
    }
    before = __builtin_amdgcn_readfirstlane(__shfl(upto, kWave - 1));
  }
}

// The scales in LDS: a ring of groups, each the next kRowB bytes of every
// row's. By way of registers a group serves two stages. By transfers it is a
// stage's own 8 bytes of a row, or in the tiles of 128 columns those of 4
// stages, with the first of them, which asks for a line a quarter as often:
// 256 x 6144 x 4096 12.7 us against 15.4, 16 x 28672 x 4096 in 64 x 128 tiles
// 16.1 against 18.9. In 64 x 64 tiles, which have fewer rows to a wave, 128 x
// 4096 x 4096 takes 9.1 us that way against 8.8.
template <int BM, int BN, int NW, int NST, bool SCREG>
struct Scales {
  static constexpr int kRowB = SCREG ? 16 : NST > 2 && BM < BN ? 32 : 8;
  static constexpr int kStages = kRowB / 8;                        // that a group serves
  static constexpr int kRows = 256 / kRowB;                        // of a wave's operation
  static constexpr int kOps = ((BM + BN) / kRows + NW - 1) / NW;   // of a wave and group
  static constexpr int kSlotB = kOps * NW * 256;
  // The NST stages read and on their way are of as many groups at most where a
  // group is a stage, else of 3: a tile has NST - 1 stages at least, so only
  // its last group can be of one.
  static constexpr int kSlots = kStages == 1 || NST < 3 ? NST : 3;
};

// LDS of a tile kernel (stages, scale slots), and the workgroups of it that a
// compute unit's 160 KB hold (at most 16 waves of them: with more, fewer
// registers a wave than its accumulators and operands need). The compiler is
// held to that many: with 20 registers more the 128 x 128 tile has one
// workgroup a unit, and the 512-row product above took 158 us in place of 124.
template <int BM, int BN, int NW, int NST, bool SCREG>
constexpr int lds_bytes() {
  using S = Scales<BM, BN, NW, NST, SCREG>;
  return NST * (BM + BN) * kRowB + S::kSlots * S::kSlotB;
}
template <int BM, int BN, int NW, int NST, bool SCREG>
constexpr int occupancy() {
  constexpr int by_lds = 163840 / lds_bytes<BM, BN, NW, NST, SCREG>();
  return by_lds * NW > 16 ? 16 / NW : by_lds;
}

// BM x BN tiles of y, by a workgroup of WM x WN waves that walks its share of
// them. K passes in stages of 256 (whole 128-byte lines of codes; stages of 128
// in a deeper ring: 700 us against 640 for 8192 x 28672 x 4096) through a ring
// of NST LDS stages; the ring runs on from one tile into the next, so a tile's
// first stage is on its way while the tile before it is finished and stored
// (a workgroup a tile: 590 us against 515).
template <typename D, int BM, int BN, int WM, int WN, int NST, bool SCREG>
__global__ __launch_bounds__(64 * WM * WN, ((occupancy<BM, BN, WM * WN, NST, SCREG>() * WM * WN + 3) / 4)) void
k_mx_tile(MxArgs a, int sld, int ntiles) {
  static_assert(!SCREG || NST == 2, "scale registers look one stage ahead");
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  constexpr int RPI = 8;                                    // rows of a transfer
  constexpr int kStageB = (BM + BN) * kRowB;
  constexpr int XI = BM / RPI / NW, WI = BN / RPI / NW;     // transfers a wave and stage
  using S = Scales<BM, BN, NW, NST, SCREG>;
  constexpr bool GROUPS = !SCREG && S::kStages > 1;
  constexpr int SRowB = S::kRowB, SI = S::kOps, kScaleB = S::kSlotB;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char* lsc = lds + NST * kStageB;
  const int tid = threadIdx.x;
  const int lane = lane_id();
  const int w = wave_id();
  const uint32_t rowb = (uint32_t)a.K / 2;
  const int kb = a.K / 32;
  const int kt = (a.K + kStageK - 1) / kStageK;   // at least NST - 1 (the walk looks one tile ahead)

  // the experts' row tiles; rows of no expert become zero
  int mtiles = tiles_of(a.rows, BM);
  if (a.offsets) {
    mtiles = count_tiles<BM>(a);
    zero_dead_rows<D>(a);
  }

  // block b runs on XCD b % 8, which takes a run of positions of an order in
  // which 8 row tiles vary fastest, so that the tiles an XCD runs at a time
  // share their operands in its L2
  const int G = mtiles * ntiles;
  const int per = (G + 7) / 8;
  const int stride = (int)gridDim.x >> 3;
  int end = min(G - ((int)blockIdx.x & 7) * per, per);   // positions of this XCD
  // Where the last turn of the XCD's workgroups has tiles for half of them at
  // most, it has half tiles (BN / 2 columns) for twice as many; the waves of the
  // other columns, one on every SIMD, only fetch and wait. 16384 rows of 8
  // experts x 4096 x 14336, whose last turn is 4 tenths full: 543 us in place
  // of 551; 4262 rows of 9 experts x 6521 x 6496: 181 in place of 196; 8192 x
  // 28672 x 4096, whose turns are full: 511 in place of 508.
  constexpr bool HALVES = BN == 256 && WN == 2;
  static_assert(!HALVES || NST == 2, "a half tile has fewer transfers than the waits count");
  int halves = end;                                       // the first position with a half tile
  if (HALVES && end > stride && end % stride * 2 <= stride) {
    halves = end / stride * stride;
    end += end - halves;
  }
  int pos = (int)blockIdx.x >> 3;
  if (pos >= end) return;
  struct Tile {
    int row, mrows, n0, ncols, e;   // first row of y, rows, first column, columns, expert
  };
  auto locate = [&](int p) {
    constexpr int kGroupM = 8;
    const bool half = HALVES && p >= halves;
    const int L = ((int)blockIdx.x & 7) * per + (half ? halves + (p - halves) / 2 : p);
    const int grp = L / (kGroupM * ntiles);
    const int gsz = min(kGroupM, mtiles - grp * kGroupM);
    const int li = L - grp * kGroupM * ntiles;
    const int tm = grp * kGroupM + li % gsz;
    Tile t;
    t.n0 = li / gsz * BN;
    t.ncols = min(BN, a.N - t.n0);
    if (half) {
      t.n0 += (p - halves) % 2 * (BN / 2);
      t.ncols = max(min(BN / 2, a.N - t.n0), 0);
    }
    t.e = 0;
    t.row = tm * BM;
    t.mrows = min(BM, a.rows - t.row);
    if (a.offsets) {
      find_tile<BM>(a, tm, t.row, t.mrows, t.e);
    }
    return t;
  };

  // operand and scale buffers of a tile
  rsrc_t x_r, w_r;
  auto xs_of = [&](const Tile& t) {
    return make_rsrc(a.xs + (int64_t)t.row * sld, (uint32_t)(t.mrows * sld));
  };
  auto ws_of = [&](const Tile& t) {
    return make_rsrc(a.ws + ((int64_t)t.e * a.N + t.n0) * sld, (uint32_t)(t.ncols * sld));
  };
  // global -> LDS without registers: an instruction of a wave fills 8 rows of
  // 128 bytes, lane L at row L / 8, physical chunk L % 8 of 16 bytes; the
  // lane fetches the logical chunk stored there, L % 8 ^ (row / 2) % 8, so
  // that the operand reads of 16 consecutive rows spread over the banks
  // (with row % 8 in its place rows r and r + 8 meet: 366 us against 318 us
  // for the products and reads of a 8192 x 28672 x 4096 product)
  const int pr = lane >> 3;
  auto swz = [](int row) { return row >> 1 & 7; };
  // of a wave's transfer i; the same for all of them but for a lone wave
  auto pc = [&](int i) { return (uint32_t)((lane & 7) ^ swz((w + NW * i) * RPI + pr)) * 16u; };
  // the word of a row that a lane transfers: a row's are held at word ^ 2 * sswz
  auto sswz = [](int row) { return row / S::kRows % S::kStages; };
  static_assert(SCREG || (BM % S::kRows == 0 && NW % S::kStages == 0),
                "an operation is all of x or all of W, a wave's are of one swizzle");
  const uint32_t sword = (uint32_t)(lane % (SRowB / 4)) ^ (uint32_t)(w % S::kStages * 2);
  uint32_t xoff[XI], woff[WI], soff[SCREG ? 1 : SI];
  rsrc_t xs_r, ws_r;
  int ld_cols = BN;   // columns of the tile being fetched
  auto point_at = [&](const Tile& t) {
    ld_cols = t.ncols;
    x_r = make_rsrc(a.x + (int64_t)t.row * rowb, (uint32_t)t.mrows * rowb);
    w_r = make_rsrc(a.w + ((int64_t)t.e * a.N + t.n0) * rowb, (uint32_t)t.ncols * rowb);
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int row = (w + NW * i) * RPI + pr;
      xoff[i] = row < t.mrows ? (uint32_t)row * rowb + pc(i) : kOOB;
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      const int row = (w + NW * i) * RPI + pr;
      woff[i] = row < t.ncols ? (uint32_t)row * rowb + pc(i) : kOOB;
    }
    if constexpr (!SCREG) {
      xs_r = xs_of(t);
      ws_r = ws_of(t);
#pragma unroll
      for (int i = 0; i < SI; ++i) {
        const int row = (w + NW * i) * S::kRows + lane / (SRowB / 4);
        const int rr = row < BM ? row : row - BM;
        soff[i] = rr < (row < BM ? t.mrows : row < BM + BN ? t.ncols : 0)
                      ? (uint32_t)rr * sld + sword * 4 : kOOB;
      }
    }
  };
  auto issue = [&](int it, int slot) {
    const uint32_t k0 = (uint32_t)it * kRowB;
    uint32_t ko[2];   // by the parity of the transfer
#pragma unroll
    for (int i = 0; i < 2; ++i) ko[i] = k0 + pc(i) < rowb ? k0 : kPastEnd;
    char* sb = lds + slot * kStageB;
#pragma unroll
    for (int i = 0; i < XI; ++i) dma16(x_r, sb + (w + NW * i) * 1024, xoff[i] + ko[i & 1]);
#pragma unroll
    for (int i = 0; i < WI; ++i)
      if (!HALVES || (w + NW * i) * RPI < ld_cols)
        dma16(w_r, sb + BM * kRowB + (w + NW * i) * 1024, woff[i] + ko[i & 1]);
  };
  auto issue_scales = [&](int it, int slot) {
    const uint32_t b0 = (uint32_t)it * 8;
    const uint32_t so = b0 + sword * 4 < (uint32_t)sld ? b0 : kPastEnd;
#pragma unroll
    for (int i = 0; i < SI; ++i)
      dma4((w + NW * i) * S::kRows < BM ? xs_r : ws_r, lsc + slot * kScaleB + (w + NW * i) * 256,
           soff[i] + so);
  };

  // Scales by way of registers: a group is 64 bytes (K of 2048) of every row,
  // read by 4 lanes side by side so that a line is asked for once, and handed
  // to LDS a chunk at a time by the lanes that hold it. The same bytes by
  // stage-wise transfers would ask L2 for every line many times: 512 rows of 8
  // experts x 4096 x 14336 82 us against 106 in 64 x 64 tiles.
  const int piece = lane & 3;
  u32x4 sreg[SCREG ? SI : 1];
  auto load_scales = [&](const Tile& t, int grp) {
    const int b = grp * 64 + piece * 16;
    // 16 bytes that would run past the row (sld >= 16) end with it instead
    const uint32_t o = b < sld ? (uint32_t)min(b, sld - 16) : kPastEnd;
    const rsrc_t xr = xs_of(t), wr = ws_of(t);
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      const int first = (w + NW * i) * 16;   // the 16 rows are all of x or all of W
      const int rr = first + (lane >> 2) - (first < BM ? 0 : BM);
      const int lim = first < BM ? t.mrows : first < BM + BN ? t.ncols : 0;
      sreg[i] = bload16(first < BM ? xr : wr, (rr < lim ? (uint32_t)rr * sld : kOOB) + o);
    }
  };
  auto store_scales = [&](int chunk, int slot) {
    char* cb = lsc + slot * kScaleB + (lane >> 2) * 16;
    const int back = max(chunk * 16 + 16 - sld, 0);   // bytes that load_scales moved back
    if (piece == (chunk & 3)) {
#pragma unroll
      for (int i = 0; i < SI; ++i) {
        u32x4 v = sreg[i];
        if (back > 0)
          v = back == 4 ? u32x4{v.y, v.z, v.w, 0u}
              : back == 8 ? u32x4{v.z, v.w, 0u, 0u} : u32x4{v.w, 0u, 0u, 0u};
        *(u32x4*)(cb + (w + NW * i) * 256) = v;
      }
    }
  };

  // cur: the tile being multiplied; ld: the tile being fetched, stage lit
  // next; nx: the one after it (its scales are fetched ahead of it)
  Tile cur = locate(pos), ld = cur, nx = cur;
  pos += stride;
  bool has_ld = true, has_nx = pos < end;
  if (has_nx) nx = locate(pos);
  int lit = 0, lslot = 0, chunks = 0;
  point_at(ld);
  if constexpr (SCREG) load_scales(ld, 0);
  // fetch the next stage of the walk, if there is one
  auto fetch = [&]() {
    if (lit == kt) {
      lit = 0;
      has_ld = has_nx;
      if (has_nx) {
        ld = nx;
        pos += stride;
        has_nx = pos < end;
        if (has_nx) nx = locate(pos);
        point_at(ld);
      }
    }
    if (!has_ld) return;
    if constexpr (SCREG) {
      // before the transfers, which a wait for the registers would wait for too
      if (lit % 2 == 0) {
        const int c = lit / 2;
        store_scales(c, chunks++ & 1);
        if (lit + 2 >= kt) {
          if (has_nx) load_scales(nx, 0);
        } else if (c % 4 == 3) {
          load_scales(ld, c / 4 + 1);
        }
      }
    }
    if constexpr (GROUPS) {
      if (lit % S::kStages == 0) {
        issue_scales(lit, chunks);
        chunks = chunks + 1 == S::kSlots ? 0 : chunks + 1;
      }
    }
    issue(lit, lslot);
    if constexpr (!SCREG && !GROUPS) issue_scales(lit, lslot);
    lslot = lslot + 1 == NST ? 0 : lslot + 1;
    ++lit;
  };
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) fetch();

  const int m = lane & 31, h = lane >> 5;
  const int wm = w % WM, wn = w / WM;
  const uint32_t sw = (uint32_t)(((4 * h) ^ swz(m)) << 4);   // chunk of step 0
  const uint32_t xrow = (uint32_t)(wm * TM * 32 + m) * kRowB;
  const uint32_t wrow = (uint32_t)(BM + wn * TN * 32 + m) * kRowB;
  const uint32_t xsc = (uint32_t)(wm * TM * 32 + m) * SRowB + 4 * h;
  const uint32_t wsc = (uint32_t)(BM + wn * TN * 32 + m) * SRowB + 4 * h;

  int slot = 0, cslot = S::kSlots - 1;
  f32x16 acc[TN][TM];
  u32x4 xo[2][TM], wo[2][TN];   // operands of two steps
  uint32_t sx[TM], sv[TN];      // scale words of a stage
  auto read_scales = [&](int it) {
    const char* ss = lsc + (SCREG || GROUPS ? cslot : slot) * kScaleB +
                     (it % S::kStages ^ (GROUPS ? sswz(m) : 0)) * 8;
#pragma unroll
    for (int j = 0; j < TM; ++j) sx[j] = *(const uint32_t*)(ss + xsc + j * 32 * SRowB);
#pragma unroll
    for (int i = 0; i < TN; ++i) sv[i] = *(const uint32_t*)(ss + wsc + i * 32 * SRowB);
    if (it * 8 + 8 > kb) {   // the padding of a scale row is not a scale
#pragma unroll
      for (int j = 0; j < TM; ++j) sx[j] = keep_blocks(sx[j], it * 8 + 4 * h, kb);
#pragma unroll
      for (int i = 0; i < TN; ++i) sv[i] = keep_blocks(sv[i], it * 8 + 4 * h, kb);
    }
  };
  // step j of the stage in `slot`: chunk 4 h + j of every row, into buffer j % 2
  auto read = [&](int j) {
    const char* sb = lds + slot * kStageB + (sw ^ (uint32_t)(j << 4));
#pragma unroll
    for (int i = 0; i < TN; ++i) wo[j & 1][i] = *(const u32x4*)(sb + wrow + i * 32 * kRowB);
#pragma unroll
    for (int i = 0; i < TM; ++i) xo[j & 1][i] = *(const u32x4*)(sb + xrow + i * 32 * kRowB);
  };
  auto step = [&](auto jc) {
    constexpr int J = decltype(jc)::value;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
        acc[i][j] = mfma_mx32<J>(wo[J & 1][i], xo[J & 1][j], acc[i][j], sv[i], sx[j]);
  };
  for (;;) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

    for (int it = 0; it < kt; ++it) {
      // this stage is there once at most the transfers of the later ones
      // are outstanding; then the barrier makes every wave's part visible
      // and frees the buffer read in the previous iteration
      // (a group's scales come on top and make the wait the longer one)
      constexpr int AH = NST - 2, OPS = XI + WI + (SCREG || GROUPS ? 0 : SI);
      if (AH > 0 && has_ld)
        __builtin_amdgcn_s_waitcnt(vm_lds(AH * OPS));
      else
        __builtin_amdgcn_s_waitcnt(vm_lds(0));
      barrier_no_fence();
      fetch();
      if ((SCREG || GROUPS) && it % S::kStages == 0) cslot = cslot + 1 == S::kSlots ? 0 : cslot + 1;
      if (!HALVES || wn * TN * 32 < cur.ncols) {
        read_scales(it);
        // a step's operand reads go before the products of the step before it
        read(0);
        read(1);
        step(std::integral_constant<int, 0>());
        read(2);
        step(std::integral_constant<int, 1>());
        read(3);
        step(std::integral_constant<int, 2>());
        step(std::integral_constant<int, 3>());
        __builtin_amdgcn_sched_group_barrier(0x100, TN + TM, 0);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          __builtin_amdgcn_sched_group_barrier(0x100, TN + TM, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, TN * TM, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, TN * TM, 0);
      }
      if (it + 1 < kt) slot = slot + 1 == NST ? 0 : slot + 1;
    }

    // wait states between the last MFMA and the first vector read of its result
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    // The tile goes to memory through the LDS stage just read, so that a
    // store takes whole lines of y: 16 bytes a lane, a row's lanes side by
    // side (8 bytes a lane to 32 rows at a time straight from the registers
    // took 660 us in place of 600 for 8192 x 28672 x 4096, and 49 in place of
    // 24 where y is float32 with an odd width). 16-byte chunks of a row are held at chunk ^ (row & 31), so that
    // neither the 32 rows a wave writes at a time nor the row it reads meets
    // a bank twice.
    constexpr int kElem = D::kBytes;
    constexpr int NEED = (BM * BN * kElem + kStageB - 1) / kStageB;
    constexpr int PJ = NEED < TM ? NEED : TM, PI = (NEED + PJ - 1) / PJ;   // passes
    constexpr int TPJ = TM / PJ, TPI = TN / PI;             // of a wave and pass
    constexpr int CW = TPI * 32 * kElem / 16;               // chunks of a wave's columns
    constexpr int CH = WN * CW;                             // chunks of a row
    constexpr int MASK = CH < 32 ? CH - 1 : 31;
    static_assert(WM * TPJ * 32 * CH * 16 <= kStageB && TM % PJ == 0 && TN % PI == 0 &&
                      (CH & (CH - 1)) == 0 && 64 * NW % CH == 0, "a pass fits a stage");
    char* eb = lds + slot * kStageB;
    slot = slot + 1 == NST ? 0 : slot + 1;
    const bool whole = cur.mrows == BM && cur.ncols == BN;
    char* yb = (char*)a.y + ((int64_t)cur.row * a.N + cur.n0) * kElem;
    // addresses of this part are formed here, not kept over the main loop
    int te = tid;
    asm volatile("" : "+v"(te));
    const int me = te & 31, he = te >> 5 & 1;
#pragma unroll
    for (int p = 0; p < PJ * PI; ++p) {
      const int pj = p % PJ, pi = p / PJ;
      lds_barrier();
#pragma unroll
      for (int j = 0; j < TPJ; ++j) {
        const int lr = (wm * TPJ + j) * 32 + me;
#pragma unroll
        for (int i = 0; i < TPI; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16& z = acc[pi * TPI + i][pj * TPJ + j];
            const int byte = (wn * TPI * 32 + i * 32 + 8 * q + 4 * he) * kElem;
            char* dst = eb + lr * (CH * 16) + (((byte >> 4) ^ (lr & MASK)) << 4) + (byte & 15);
            if constexpr (kElem == 2)
              *(u32x2*)dst = u32x2{pack_bf16x2(z[4 * q], z[4 * q + 1]),
                                   pack_bf16x2(z[4 * q + 2], z[4 * q + 3])};
            else
              *(f32x4*)dst = f32x4{z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]};
          }
      }
      lds_barrier();
#pragma unroll
      for (int k = 0; k < WM * TPJ * 32 * CH / (64 * NW); ++k) {
        const int lr = te / CH + k * (64 * NW / CH), ch = te % CH;
        const int r = (lr / (TPJ * 32) * TM + pj * TPJ) * 32 + lr % (TPJ * 32);
        const int c = ((ch / CW * TN + pi * TPI) * 32 * kElem / 16 + ch % CW) * (16 / kElem);
        const char* src = eb + lr * (CH * 16) + ((ch ^ (lr & MASK)) << 4);
        char* dst = yb + (uint32_t)(r * a.N + c) * (uint32_t)kElem;   // below 2^30
        // y's rows start on any element: 16 bytes go to any element's address
        if (whole || (r < cur.mrows && c + 16 / kElem <= cur.ncols)) {
          __builtin_nontemporal_store(*(const u32x4*)src, (u32x4_any*)dst);
        } else if (r < cur.mrows) {
          for (int u = 0; u < cur.ncols - c; ++u) {
            if constexpr (kElem == 2)
              ((uint16_t*)dst)[u] = ((const uint16_t*)src)[u];
            else
              ((uint32_t*)dst)[u] = ((const uint32_t*)src)[u];
          }
        }
      }
    }
    if (!has_ld) break;   // no tile was fetched after this one
    cur = ld;
  }
}

template <typename D, int BM, int BN, int WM, int WN, int NST, bool SCREG>
hipError_t launch_tile(const MxArgs& a, hipStream_t stream, int dev, int cus) {
  constexpr int NW = WM * WN;
  constexpr int lds = lds_bytes<BM, BN, NW, NST, SCREG>();
  const int64_t mt = (int64_t)tiles_of(a.rows, BM) + (a.offsets ? a.E : 0);
  const int64_t nt = tiles_of(a.N, BN);
  if (mt * nt > 0x7fffffff) return hipErrorInvalidValue;
  constexpr int occ = occupancy<BM, BN, NW, NST, SCREG>();
  const int64_t grid = std::min<int64_t>(8 * ((mt * nt + 7) / 8), (int64_t)cus * occ / 8 * 8);
  const void* f = (const void*)k_mx_tile<D, BM, BN, WM, WN, NST, SCREG>;
  if (lds > 65536) {   // said once per device
    static std::atomic<uint64_t> said{0};
    if (!(said.load(std::memory_order_relaxed) >> dev & 1)) {
      const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
      said.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL((k_mx_tile<D, BM, BN, WM, WN, NST, SCREG>), dim3((unsigned)grid),
                     dim3(64 * NW), lds, stream, a, mx_scale_row(a.K), (int)nt);
  return hipGetLastError();
}

// Tiles and depths by the sizes, mt x nt tiles of y for the compute units to
// share. Every choice gives the same y. Measured on one card, other weights
// every time (us, us of the others):
//   256 x 256, where they fill the chip: 2048 x 6144 x 4096 38 (128^2: 44,
//     64 x 128: 59)
//   128 x 128, two workgroups a unit: 512 rows of 8 experts x 28672 x 4096
//     129 (64 x 128: 140, 64^2: 148, 256^2: 158)
//   64 x 64, four stages, where every tile has a unit to itself: 1 x 6144 x
//     4096 8.8 (32 x 128: 10.3, 64 x 128, three stages: 11.7, 128^2: 21)
//   64 x 128, three stages, where those have: 40 x 18000 x 4096 15.3 (64^2:
//     19.5, 128^2: 22); of them 32 x 128, four stages, where no more rows are
//     there: 8 x 18000 x 4096 13.1 (64 x 128: 14.8)
//   64 x 64, scales by way of registers, for more tiles than units: 91 rows
//     of 14 experts x 7390 x 8576 111 (64 x 128: 114, 128^2: 120); 64 x 128
//     where the rows fill it: 600 x 5300 x 1056 9.4 (64^2: 10.0, 128^2: 10.3),
//     1024 x 4096 x 4096 21 (64^2: 23, 128^2: 21)
template <typename D>
hipError_t launch_by_size(const MxArgs& a, hipStream_t stream) {
  int dev = 0, cus = 0;
  const hipError_t ec = compute_units(&dev, &cus);
  if (ec != hipSuccess) return ec;
  const int used = std::min(a.E, a.rows);   // experts with rows, at most
  const int avg = a.rows / used;
  auto tiles = [&](int bm, int bn) {
    const int64_t mt = (int64_t)tiles_of(a.rows, bm) + (a.offsets ? used / 2 : 0);
    return std::max<int64_t>(mt, used) * tiles_of(a.N, bn);
  };
  // a group of scale registers is 16 bytes of a row at the least, and a walk
  // through NST stages needs tiles of NST - 1
  if (a.K < 512) {
    if (avg > 32 && tiles(128, 128) >= cus)
      return launch_tile<D, 128, 128, 2, 2, 2, false>(a, stream, dev, cus);
    return launch_tile<D, 64, 128, 2, 2, 2, false>(a, stream, dev, cus);
  }
  if (avg >= 192 && tiles(256, 256) * 4 >= cus * 3)
    return launch_tile<D, 256, 256, 4, 2, 2, true>(a, stream, dev, cus);
  if (avg >= 48 && tiles(128, 128) * 4 >= cus * 5)
    return launch_tile<D, 128, 128, 2, 2, 2, true>(a, stream, dev, cus);
  if (a.K > 512 && tiles(64, 64) <= cus)
    return launch_tile<D, 64, 64, 2, 2, 4, false>(a, stream, dev, cus);
  if (tiles(64, 128) <= cus) {
    if (a.K > 512 && a.rows <= 32)
      return launch_tile<D, 32, 128, 1, 4, 4, false>(a, stream, dev, cus);
    return launch_tile<D, 64, 128, 2, 2, 3, false>(a, stream, dev, cus);
  }
  if (avg > 64) return launch_tile<D, 64, 128, 2, 2, 2, true>(a, stream, dev, cus);
  return launch_tile<D, 64, 64, 2, 2, 2, true>(a, stream, dev, cus);
}

hipError_t launch_mxfp4_linear(int dtype, const MxArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  return dtype == 1 ? launch_by_size<BF16>(a, stream) : launch_by_size<F32>(a, stream);
}

}  // namespace lora
