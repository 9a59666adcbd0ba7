// Which kernel forms a product of the dense layer: a rule on its sizes, its
// operands and the card's compute units.
#pragma once

#include <algorithm>

#include "dense.h"

namespace lora {

constexpr int kRowB = 128;       // bytes of a row in one LDS stage: K of 64 (bf16) or 128

__host__ __device__ __forceinline__ int tiles_of(int n, int tile) {
  return (int)(((uint32_t)n + (uint32_t)tile - 1) / (uint32_t)tile);
}

// Tiles of rows x cols (of a gated product cols / 2 gates and as many ups), `each`
// workgroups of them a compute unit; each == 0: the kernel for up to `rows` rows
// of x, with cols columns of y (gated: gates) a workgroup.
struct LinearChoice {
  int rows, cols, each;
};

// What a product in tiles of BM x BN takes, in quarters of the time of a stage
// of a 64 x 64 tile that has its compute unit for itself (0.29 us in bf16, 0.36
// in MXFP8): `stage` times the stages and what a tile's y and residual take, for
// as many rounds as the units need, with EACH tiles a unit at a time.
template <bool GATED, int BM, int BN, int EACH = 1>
int64_t cost_of(const LinearArgs& a, int cus, int stages, int stage) {
  const int64_t tiles = (int64_t)tiles_of(a.T, BM) * tiles_of(a.N, GATED ? BN / 2 : BN);
  const int bytes = (a.y_f32 ? 4 : 2) * (a.residual ? 2 : 1);
  return (tiles + EACH * cus - 1) / (EACH * cus) *
         ((int64_t)stages * stage + EACH * BM * BN / (GATED ? 2 : 1) * bytes / 800);
}

// Larger tiles read each operand less often and have more products for every
// barrier; smaller ones leave fewer compute units idle. Measured, us, 64 x 64 /
// 64 x 128 / 128 x 128 / 256 x 128 / 256 x 256, MXFP8:
//   256 x  6144, K  4096:  28.5 /  21.3 /  27.6 /       /  76.7
//   512 x  6144, K  4096:  42.0 /  41.5 /  28.2 /  47.8 /
//  1024 x  6144, K  4096:  76.2 /  60.5 /  53.4 /  49.2 /  76.5
//   256 x  4096, K 14336:  45.2 /  61.6 /  79.0 /       / 224.9
//  1024 x  4096, K 14336: 154.0 / 117.0 /  82.2 / 148.2 / 208.6
// and of gated pairs of 14336 columns, K 4096, from 64 x 128 on:
//   256 rows 80.5 / 55.0 / 51.4 / 75.8, 512 rows 135.7 / 98.8 / 87.5 / 69.9.
template <bool MX, bool GATED>
LinearChoice choose_linear(const LinearArgs& a, int cus) {
  const int narrow = GATED ? 32 : 16;
  if (a.T <= 8) return {8, narrow, 0};
  if (a.T <= 16) return {16, narrow, 0};
  if (a.T <= 32) return {32, narrow, 0};
  // Up to 64 rows where that is one round of workgroups, all of whose x each of
  // them reads: 64 x 4096, K 14336 31 us (tiles of 64 x 64: 46), 64 x 6144, K
  // 4096 14.9 (17.0); gated pairs of 14336 columns 41 (tiles: 33).
  if (!GATED && a.T <= 64 && tiles_of(a.N, 16) <= cus) return {64, 16, 0};
  if (!GATED && a.T <= 64 && tiles_of(a.N, 32) <= cus) return {64, 32, 0};
  const int stages = tiles_of(a.K * (MX ? 1 : 2), kRowB);
  const int64_t c256 = cost_of<GATED, 256, 256>(a, cus, stages, 20);
  // Between the two: 256 x 128 in MXFP8; in bf16 two workgroups of 128 x 128 a
  // unit with two stages each instead of three (1024 x 6144, K 4096: 70 us, in 256
  // x 128 80; MXFP8 76 and 49, for the room that scales take in LDS).
  const int64_t c384 = MX ? cost_of<GATED, 256, 128>(a, cus, stages, 15)
                          : cost_of<GATED, 128, 128, 2>(a, cus, stages, 14);
  const int64_t c128 = cost_of<GATED, 128, 128>(a, cus, stages, 8);
  const int64_t c192 = cost_of<GATED, 64, 128>(a, cus, stages, 6);
  const int64_t c64 = GATED ? c192 + 1 : cost_of<GATED, 64, 64>(a, cus, stages, 4);
  const int64_t least = std::min({c256, c384, c128, c192, c64});
  if (c256 == least) return {256, 256, 1};
  if (c128 == least) return {128, 128, 1};
  if (c384 == least) return MX ? LinearChoice{256, 128, 1} : LinearChoice{128, 128, 2};
  if (c192 == least) return {64, 128, 1};
  return {64, 64, 1};
}

}  // namespace lora
