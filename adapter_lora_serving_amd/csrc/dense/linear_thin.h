// Products of few rows (at most 64): the weight streams through LDS once.
//
// What bounds it: W's bytes, and the latency of getting them. A workgroup owns
// CT * 16 columns of y (of a gated product as many gates and ups) and its NW
// waves split K between them: wave w takes the stages w, w + NW, ... of 128
// bytes a row, so that the workgroup reads NW * 128 bytes of each row at a
// time, and sums what they have at the end. Each wave has a ring of D stages of
// its own and waits for nothing but its own transfers. No part of the sum
// leaves the workgroup: no workspace, and the same order every time. The LoRA
// delta is formed meanwhile by waves of its own, in fp32 on the vector unit.
//
// Measured: 1 x 4096, K 14336 MXFP8 10.8 us (5.6 TB/s, part of it the cache's);
// a gated pair of 14336 columns, K 4096, 1 row bf16 45 us (5.2 TB/s), 32 rows
// MXFP8 over 32 adapters 59 us; 64 x 4096, K 14336 MXFP8 31 us, where the x that
// every workgroup reads is four times its weight.
#pragma once

#include "linear_tile.h"

namespace lora {

namespace {

// D[16x16] += A[16 x 128] . B[16 x 128]^T: lane (m = lane & 15, g = lane >> 4)
// supplies row m, chunks g and 4 + g of 16 bytes and the scale of block g; it
// receives D[4 g + i][m] in element i.
__device__ __forceinline__ f32x4 mfma_mx8_16(const u32x4* a, const u32x4* b, f32x4 c, uint32_t sa,
                                             uint32_t sb) {
  const i32x8 A = {(int)a[0].x, (int)a[0].y, (int)a[0].z, (int)a[0].w,
                   (int)a[1].x, (int)a[1].y, (int)a[1].z, (int)a[1].w};
  const i32x8 B = {(int)b[0].x, (int)b[0].y, (int)b[0].z, (int)b[0].w,
                   (int)b[1].x, (int)b[1].y, (int)b[1].z, (int)b[1].w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 0, 0, 0, (int)sa, 0, (int)sb);
}
// The same in bf16, K of 32: chunk g.
__device__ __forceinline__ f32x4 mfma_bf16_16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// Eight e4m3 values (words 2 G, 2 G + 1 of a chunk) and their scale as bf16.
template <int G>
__device__ __forceinline__ u32x4 wide8_16(u32x4 o, float s) {
  const uint32_t lo = o[2 * G], hi = o[2 * G + 1];
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true))};
}

// One 4-byte global -> LDS transfer per lane: lane L to byte 4 L of dst.
__device__ __forceinline__ void dma4(rsrc_t r, char* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 4, (int)off, 0, 0, 0);
}

// XD transfers of 8 rows hold x: up to 8 XD rows.
template <class OP, bool GATED, int XD, int CT, int NW, int D>
struct Thin {
  static constexpr int kXT = (XD + 1) / 2;                 // tiles of 16 rows of x
  static constexpr int kWT = CT * (GATED ? 2 : 1);         // tiles of 16 rows of W
  static constexpr int kRowsB = (kWT * 2 + XD) * 1024;     // both operands' rows of a stage
  static constexpr int kSlotB = kRowsB + (OP::kMX ? 512 : 0);   // and their scales
  static constexpr int kOps = kWT * 2 + XD + (OP::kMX ? 2 : 0);
  static constexpr int kRingB = NW * D * kSlotB;
  static constexpr int kPartB = kWT * kXT * 1024;          // a wave's sums
  static constexpr int kSumB = NW * kPartB;
  static constexpr int kBytes = (kRingB > kSumB ? kRingB : kSumB) + kPartB;   // and the whole sums
  // waves for the delta: up to 4, for 128 sums each
  static constexpr int kDelta = XD * kWT > 4 ? 4 : XD * kWT;
  // waves of a SIMD with as many workgroups as the unit's LDS holds
  static constexpr int kWaves = (163840 / kBytes * (NW + kDelta) + 3) / 4;
};

// The LoRA delta of T tokens and the workgroup's columns by `waves` waves, kU
// of the sums a lane, 16 ranks of each at a time. Under the weight's stream a
// vector load takes 7 us (that is how much of it is on its way), so slots,
// ranks and scalings come by scalar loads, which do not queue behind it.
template <bool GATED, int XT, int WT, int CT>
__device__ __forceinline__ void thin_delta(const LinearArgs& a, int n0, int w, int waves, float* whole) {
  const int lane = lane_id();
  const int p = min(lane, a.T - 1);   // lane t knows token t's
  int slot = 0, token = 0, rank = 0;
  float scale = 0.0f;
  if (a.slots <= 256) {
    for (int s0 = 1; s0 <= a.slots; s0 += 16) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int s = min(s0 + k, a.slots);
        slot += s0 + k <= a.slots && a.indptr[s] <= p;
      }
    }
  } else {
    slot = slot_of_position(a.indptr, a.slots, p);
  }
  for (int t0 = 0; t0 < a.T; t0 += 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = min(t0 + k, a.T - 1);
      const int s = __builtin_amdgcn_readlane(slot, t), sm = min(s, a.slots - 1);
      const int r = a.ranks[sm], tok = a.order[t];
      const float c = a.scalings[sm];
      if (lane == t) {
        rank = s < a.slots ? clamp_rank(r, a.R) : 0;
        scale = c;
        token = min(max(tok, 0), a.T - 1);
      }
    }
  }
  const int out = a.N * (GATED ? 2 : 1);
  constexpr int kU = 2, kCols = WT * 16;
  for (int o0 = w * 64 * kU; o0 < a.T * kCols; o0 += waves * 64 * kU) {
    const uint16_t* bp[kU];
    const float* hp[kU];
    int r[kU], at[kU], most = 0;
    float d[kU], sc[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int o = o0 + u * 64 + lane, t = o / kCols, q = o % kCols / 16;
      const bool in = t < a.T;
      const int s = __shfl(slot, t & 63);
      const int c = n0 + q % CT * 16 + o % 16, row = q / CT * a.N + c;   // row of W and B
      r[u] = __shfl(rank, t & 63);
      if (!in || c >= a.N) r[u] = 0;
      at[u] = in ? (q * XT * 16 + t) * 16 + o % 16 : -1;
      int si = 0;
      for (int i = 1; i < a.slices; ++i) si += a.off[i] <= row;
      hp[u] = a.h + (int64_t)__shfl(token, t & 63) * a.slices * a.R + si * a.R;
      bp[u] = (const uint16_t*)a.b + ((int64_t)s * out + row) * a.R;
      sc[u] = __shfl(scale, t & 63);
      d[u] = 0.0f;
      most = max(most, r[u]);
    }
    for (int k0 = 0; k0 < most; k0 += 16) {
      u32x4 bv[kU][2];
      f32x4 hv[kU][4];
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v)
          if (k0 + 8 * v < r[u]) {
            bv[u][v] = *(const u32x4*)(bp[u] + k0 + 8 * v);
            hv[u][2 * v] = *(const f32x4*)(hp[u] + k0 + 8 * v);
            hv[u][2 * v + 1] = *(const f32x4*)(hp[u] + k0 + 8 * v + 4);
          }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (k0 + k < r[u]) {
            const uint32_t b = bv[u][k / 8][k % 8 / 2];
            d[u] = fmaf(hv[u][k / 4][k % 4], k & 1 ? bf16hi(b) : bf16lo(b), d[u]);
          }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (at[u] >= 0) whole[at[u]] = r[u] > 0 ? sc[u] * d[u] : 0.0f;
  }
}

}  // namespace

template <class OP, bool GATED, int XD, int CT, int NW, int D>
__global__ __launch_bounds__(64 * (NW + Thin<OP, GATED, XD, CT, NW, D>::kDelta),
                             (Thin<OP, GATED, XD, CT, NW, D>::kWaves)) void k_linear_thin(LinearArgs a, int sld) {
  using S = Thin<OP, GATED, XD, CT, NW, D>;
  constexpr int XT = S::kXT, WT = S::kWT;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = lane_id(), w = wave_id();
  const uint32_t rowb = (uint32_t)a.K * (OP::kMX ? 1 : 2);
  const int kb = a.K / 32;
  const int kt = (int)((rowb + kRowB - 1) / kRowB);
  const int n0 = (int)blockIdx.x * CT * 16;
  const int ncols = min(CT * 16, a.N - n0);
  auto token_of = [&](int p) { return a.order ? min(max(a.order[p], 0), a.T - 1) : p; };
  char* ring = lds + w * D * S::kSlotB;

  // transfers of 8 rows of 128 bytes, chunk c of row r held at c ^ (r / 2) % 8
  const int pr = lane >> 3;
  auto swz = [](int row) { return row >> 1 & 7; };
  rsrc_t w_r[GATED ? 2 : 1];
#pragma unroll
  for (int p = 0; p < (GATED ? 2 : 1); ++p)
    w_r[p] = make_rsrc(a.w + ((int64_t)p * a.N + n0) * rowb, (uint32_t)ncols * rowb);
  const rsrc_t x_r = make_rsrc(a.x, (uint32_t)a.T * rowb);
  uint32_t xoff[XD], woff[CT * 2], xsoff = kOOB, wsoff = kOOB;
  uint32_t pc[2];   // by the parity of the transfer
#pragma unroll
  for (int i = 0; i < 2; ++i) pc[i] = (uint32_t)((lane & 7) ^ swz(i * 8 + pr)) * 16u;
#pragma unroll
  for (int i = 0; i < XD; ++i) {
    const int row = i * 8 + pr;
    xoff[i] = row < a.T ? (uint32_t)token_of(min(row, a.T - 1)) * rowb + pc[i & 1] : kOOB;
  }
#pragma unroll
  for (int i = 0; i < CT * 2; ++i) {
    const int row = i * 8 + pr;
    woff[i] = row < ncols ? (uint32_t)row * rowb + pc[i & 1] : kOOB;
  }
  rsrc_t xs_r = x_r, ws_r = x_r;
  if constexpr (OP::kMX) {
    xs_r = make_rsrc(a.xs, (uint32_t)a.T * (uint32_t)sld);
    ws_r = make_rsrc(a.ws + (int64_t)n0 * sld, (uint32_t)((GATED ? a.N : 0) + ncols) * (uint32_t)sld);
    if (lane < a.T) xsoff = (uint32_t)token_of(lane) * (uint32_t)sld;
    const int c = lane % (CT * 16);
    if (lane < WT * 16 && c < ncols) wsoff = (uint32_t)(lane / (CT * 16) * a.N + c) * (uint32_t)sld;
  }
  auto issue = [&](int it, int slot) {
    const uint32_t k0 = (uint32_t)it * kRowB;
    char* sb = ring + slot * S::kSlotB;
    const bool live[2] = {k0 + pc[0] < rowb, k0 + pc[1] < rowb};
#pragma unroll
    for (int i = 0; i < WT * 2; ++i)
      dma16(w_r[i / (CT * 2)], sb + i * 1024, live[i & 1] ? woff[i % (CT * 2)] + k0 : kOOB);
#pragma unroll
    for (int i = 0; i < XD; ++i)
      dma16(x_r, sb + (WT * 2 + i) * 1024, live[i & 1] ? xoff[i] + k0 : kOOB);
    if constexpr (OP::kMX) {
      dma4(ws_r, sb + S::kRowsB, wsoff + (uint32_t)it * 4);
      dma4(xs_r, sb + S::kRowsB + 256, xsoff + (uint32_t)it * 4);
    }
  };

  float* whole = (float*)(lds + S::kBytes - S::kPartB);   // [tile of W][token][16 columns]
  if (w >= NW) {   // only with a delta
    thin_delta<GATED, XT, WT, CT>(a, n0, w - NW, S::kDelta, whole);
    __syncthreads();
    __syncthreads();
    __syncthreads();
    return;
  }

  f32x4 acc[WT][XT];
#pragma unroll
  for (int i = 0; i < WT; ++i)
#pragma unroll
    for (int j = 0; j < XT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int m = lane & 15, g = lane >> 4;
  const int n = w < kt ? (kt - w + NW - 1) / NW : 0;   // stages of this wave
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (i < n) issue(w + i * NW, i);

  // what the sums meet at the end is asked for now: a lane's 8 columns of a row
  constexpr int RUNS = CT * 2;
  const int et = tid / RUNS, ec = n0 + tid % RUNS * 8;
  const bool elive = et < a.T;
  const int64_t erow = token_of(min(et, a.T - 1));
  Ahead<GATED> ahead;
  if (elive) {
    ahead.load_bias(a, ec);
    if (!GATED && a.residual) ahead.load_residual(a, 0, erow * a.N + ec, ec);
  }

  int slot = 0;
  for (int i = 0; i < n; ++i) {
    if (i + D - 1 < n)
      __builtin_amdgcn_s_waitcnt(vmcnt_le((D - 1) * S::kOps));
    else
      __builtin_amdgcn_s_waitcnt(vmcnt_le(0));
    asm volatile("" ::: "memory");
    const char* sb = ring + slot * S::kSlotB;
    u32x4 wo[WT][2], xo[XT][2];
    uint32_t sv[WT], sx[XT];
    // rows of x past the transfers' have no slot: the last tile reads its first half twice
    auto x_row = [&](int j) { return XD % 2 && j == XT - 1 ? j * 16 + m % 8 : j * 16 + m; };
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t c = (uint32_t)(((4 * p + g) ^ swz(m)) << 4);
#pragma unroll
      for (int q = 0; q < WT; ++q) wo[q][p] = *(const u32x4*)(sb + (q * 16 + m) * kRowB + c);
#pragma unroll
      for (int j = 0; j < XT; ++j) {
        const int r = x_row(j);
        const uint32_t cx = (uint32_t)(((4 * p + g) ^ swz(r)) << 4);
        xo[j][p] = *(const u32x4*)(sb + (WT * 16 + r) * kRowB + cx);
      }
    }
    const int it = w + i * NW;
    if constexpr (OP::kMX) {
      const uint32_t keep = keep_blocks(it * 4, kb);   // the padding of a scale row is not a scale
#pragma unroll
      for (int q = 0; q < WT; ++q)
        sv[q] = *(const uint32_t*)(sb + S::kRowsB + (q * 16 + m) * 4) & keep;
#pragma unroll
      for (int j = 0; j < XT; ++j)
        sx[j] = *(const uint32_t*)(sb + S::kRowsB + 256 + (j * 16 + m) * 4) & keep;
    }
    // the slot is free once its operands are in registers
    __builtin_amdgcn_s_waitcnt(vm_lds_le(63));
    asm volatile("" ::: "memory");
    if (i + D < n) issue(w + (i + D) * NW, slot);
    slot = slot + 1 == D ? 0 : slot + 1;
    if constexpr (!OP::kMX) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int q = 0; q < WT; ++q)
#pragma unroll
          for (int j = 0; j < XT; ++j) acc[q][j] = mfma_bf16_16(wo[q][p], xo[j][p], acc[q][j]);
    } else if constexpr (!OP::kWide) {
#pragma unroll
      for (int q = 0; q < WT; ++q)
#pragma unroll
        for (int j = 0; j < XT; ++j)
          acc[q][j] = mfma_mx8_16(wo[q], xo[j], acc[q][j], sv[q] >> (8 * g), sx[j] >> (8 * g));
    } else {
      // chunk p of this lane is of block 2 p + g / 2
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int q = 0; q < WT; ++q)
#pragma unroll
          for (int j = 0; j < XT; ++j) {
            const float s = mx8_exponent(sv[q] >> (8 * (2 * p + g / 2)) & 255u);
            const float t = mx8_exponent(sx[j] >> (8 * (2 * p + g / 2)) & 255u);
            acc[q][j] = mfma_bf16_16(wide8_16<0>(wo[q][p], s), wide8_16<0>(xo[j][p], t), acc[q][j]);
            acc[q][j] = mfma_bf16_16(wide8_16<1>(wo[q][p], s), wide8_16<1>(xo[j][p], t), acc[q][j]);
          }
    }
  }
  // wait states between the last MFMA and the first vector read of its result
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);

  // the waves' sums, and what they come to
  __syncthreads();   // the sums take the rings' place
#pragma unroll
  for (int q = 0; q < WT; ++q)
#pragma unroll
    for (int j = 0; j < XT; ++j)
      *(f32x4*)(lds + w * S::kPartB + ((q * XT + j) * 16 + m) * 64 + g * 16) = acc[q][j];
  __syncthreads();
  for (int o = tid; o < S::kPartB / 4; o += 64 * NW) {
    float z = a.h ? whole[o] : 0.0f;
#pragma unroll
    for (int p = 0; p < NW; ++p) z += *(const float*)(lds + p * S::kPartB + o * 4);
    whole[o] = z;
  }
  __syncthreads();
  if (tid < XT * 16 * RUNS) {
    float v[8], up[8];
    const int q = tid % RUNS / 2, half = tid % 2;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = whole[(q * XT * 16 + et) * 16 + half * 8 + k];
      if constexpr (GATED) up[k] = whole[((CT + q) * XT * 16 + et) * 16 + half * 8 + k];
    }
    finish<GATED>(a, ahead, 0, elive, erow, ec, v, up);
  }
}

template <class OP, bool GATED, int XD, int CT, int NW, int D>
hipError_t launch_thin(const LinearArgs& a, hipStream_t stream, int dev) {
  using S = Thin<OP, GATED, XD, CT, NW, D>;
  static_assert(S::kXT * 16 * CT * 2 <= 64 * NW && S::kBytes <= 163840, "");
  const void* f = (const void*)k_linear_thin<OP, GATED, XD, CT, NW, D>;
  if (S::kBytes > 65536) {   // said once per device
    static std::atomic<uint64_t> said{0};
    if (!(said.load(std::memory_order_relaxed) >> dev & 1)) {
      const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
      if (e != hipSuccess) return e;
      said.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL((k_linear_thin<OP, GATED, XD, CT, NW, D>), dim3((unsigned)tiles_of(a.N, CT * 16)),
                     dim3(64 * (NW + (a.h ? S::kDelta : 0))), S::kBytes, stream, a, mx8_scale_row(a.K));
  return hipGetLastError();
}

template <class OP, bool GATED, int XD>
hipError_t launch_thin_by_width(const LinearArgs& a, hipStream_t stream, int dev) {
  // as many waves as leave two workgroups a unit
  if constexpr (GATED) return launch_thin<OP, GATED, XD, 2, XD == 2 ? 3 : 4, 2>(a, stream, dev);
  else return launch_thin<OP, GATED, XD, 1, XD == 4 ? 6 : 8, 2>(a, stream, dev);
}

// The kernel that linear_choice.h names.
template <class OP, bool GATED>
hipError_t launch_by_size(const LinearArgs& a, hipStream_t stream) {
  int dev = 0, cus = 0;
  const hipError_t e = dense_compute_units(&dev, &cus);
  if (e != hipSuccess) return e;
  const LinearChoice c = choose_linear<OP::kMX, GATED>(a, cus);
  if (c.each == 0) {
    if (c.rows == 8) return launch_thin_by_width<OP, GATED, 1>(a, stream, dev);
    if (c.rows == 16) return launch_thin_by_width<OP, GATED, 2>(a, stream, dev);
    if (c.rows == 32) return launch_thin_by_width<OP, GATED, 4>(a, stream, dev);
    if constexpr (!GATED) {
      if (c.cols == 16) return launch_thin<OP, GATED, 8, 1, 4, 3>(a, stream, dev);
      return launch_thin<OP, GATED, 8, 2, 5, 2>(a, stream, dev);
    }
    return hipErrorInvalidValue;   // not reached: gated ones have 32 rows at most
  }
  // Eight waves, two for each SIMD, one of which multiplies while the other
  // reads; four where the conversions of a float32 result take the registers of
  // eight, and where a wave would be left with one tile of gates (55 us for 60).
  if (c.rows == 256 && c.cols == 256)
    return launch_tile<OP, GATED, 256, 256, OP::kWide ? 2 : 4, 2, 2>(a, stream, dev, cus);
  if constexpr (OP::kMX) {
    if (c.rows == 256) return launch_tile<OP, GATED, 256, 128, 4, 2, 2>(a, stream, dev, cus);
  } else {
    if (c.each == 2) return launch_tile<OP, GATED, 128, 128, 2, 2, 2>(a, stream, dev, cus);
  }
  if (c.rows == 128) return launch_tile<OP, GATED, 128, 128, GATED ? 2 : 4, 2, 3>(a, stream, dev, cus);
  if (c.cols == 128) return launch_tile<OP, GATED, 64, 128, 2, GATED ? 2 : 4, 4>(a, stream, dev, cus);
  if constexpr (!GATED) return launch_tile<OP, GATED, 64, 64, 2, 2, 4>(a, stream, dev, cus);
  return hipErrorInvalidValue;   // not reached: gated ones have 128 columns at least
}

}  // namespace lora
