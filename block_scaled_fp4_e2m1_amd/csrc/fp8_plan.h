// Which kernel an E4M3 product runs on, dense or grouped by expert.
#pragma once

#include "fp8_rows_gemm.h"

namespace bsfp4 {
namespace {

// Costs as in kTileCosts, fitted to 5795 timed (shape, kernel, split) combinations (profiles/fp8_tile_plan_timings.csv) by
// least squares of log(tile_time and the split's cost / time), residuals past 0.1 weighted down:
// M 33 .. 4096, N 512 .. 14336, K 512 .. 7168, 11 % rms.  The choice among those is 0.6 % slower than the best of each shape on
// average (1.3 % with a scale per row of B), 1.6 % with the 8-bit integer products' figures.  With a scale per row the FMAs are
// twice as many instructions, and the 256 x 256 tile's accumulators leave no registers for them (4096 x 4096 x 7168: 150 us, 128
// on 256 x 128).
constexpr TileCost kBlockCosts[kTileKinds] = {{256, 256, 1, {1.25, 0}, 6.5},   {256, 128, 1, {0.69, 0}, 5.1},
                                              {128, 128, 2, {0.67, 0.96}, 3.9}, {128, 128, 1, {0.51, 0}, 4.5},
                                              {64, 128, 2, {0.35, 0.65}, 4.1},  {64, 64, 2, {0.30, 0.48}, 3.7}};
constexpr TileCost kRowCosts[kTileKinds] = {{256, 256, 1, {0, 0}, 0},          {256, 128, 1, {0.85, 0}, 5.7},
                                            {128, 128, 2, {0.65, 1.08}, 4.8}, {128, 128, 1, {0.61, 0}, 4.4},
                                            {64, 128, 2, {0.45, 0.74}, 4.2},  {64, 64, 2, {0.29, 0.51}, 3.8}};

inline TilePlan plan_fp8(bool row_b, int64_t M, int64_t N, int64_t K, int cus) {
  if (row_b) return plan_tile(M, N, K, cus, kRowCosts, ~(1u << kTile256), 2.7);
  return plan_tile(M, N, K, cus, kBlockCosts, ~0u, 2.5);
}

// Time of na workgroups of ta and then nb of tb that share `slots` places: the first end of a place's last one by which
// all of b's have run, each starting where a place is free.
inline double two_time(int64_t na, double ta, int64_t nb, double tb, int64_t slots) {
  const int64_t late = na % slots;  // places with one more of a's
  const double t0 = (double)(na / slots) * ta;
  auto all = [&](double t) {  // b's that have ended by t
    auto of = [&](double from) { return t + 1e-9 < from ? 0 : (int64_t)((t + 1e-9 - from) / tb); };
    return of(t0) * (slots - late) + of(t0 + ta) * late;
  };
  double best = 1e300;
  for (const double from : {t0, t0 + ta})
    for (int64_t k = nb / slots > 1 ? nb / slots - 1 : 0; from + (double)k * tb < best; k++)
      if (all(from + (double)k * tb) >= nb) best = from + (double)k * tb;
  return std::max(best, t0 + (late ? ta : 0.0));
}

// Time of a linear layer's two gradients (dx [M, K], a sum over N; dW [N, K], over M) on kernel k in one launch, two
// workgroups a CU of either.
inline double fp8_two_us(TileKind k, int64_t M, int64_t N, int64_t K, int cus) {
  const TileCost &a = kBlockCosts[k], &b = kRowCosts[k];
  const int64_t cols = (K + a.bn - 1) / a.bn, na = (M + a.bm - 1) / a.bm * cols, nb = (N + a.bm - 1) / a.bm * cols;
  const bool alone = na + nb <= cus;  // none shares its CU
  const double sa = (double)fp8_blocks(N), tb = (double)fp8_blocks(M) * b.us[!alone];
  double ta = sa * a.us[!alone];
  if (!alone && na <= cus) {  // a workgroup of a's shares its CU with b's, and is alone when they have run
    const double shared = (double)nb * tb / (double)(2 * cus - na);
    if (shared < ta) ta = shared + (sa - shared / a.us[1]) * a.us[0];
  }
  return std::max(a.round_us, b.round_us) + two_time(na, ta, nb, tb, 2 * cus);
}

// The kernel that runs both in one launch; kTileKinds: one after the other (a launch more, 1 us) is faster.  Over 78 shapes (M 64 ..
// 4096, N 256 .. 7168, K 512 .. 4096) the choice takes 1 % more than the best of the three, one after the other 13 %: 353 x
// 5936 x 1856 37.6 us with the quantiser against 46.2, 1163 x 5072 x 3728 86.5 against 100, 827 x 560 x 1024 15.7 against
// 18.4; but 3797 x 1056 x 784 42 against 37.
inline TileKind plan_fp8_gradients(int64_t M, int64_t N, int64_t K, int cus) {
  double best = plan_fp8(false, M, K, N, cus).us + plan_fp8(true, N, K, M, cus).us + 1.0;
  TileKind kind = kTileKinds;
  for (const TileKind k : {kTile64x128, kTile128}) {
    const double fit = k == kTile128 ? 0.9 : 1.0;  // unlike products side by side stall less than like ones
    const double t = fp8_two_us(k, M, N, K, cus) * fit;
    if (t < best) best = t, kind = k;
  }
  return kind;
}

// Grouped by expert, N columns of results: whether a tile has up to 256 rows, or 64.
//
// Tiles of 64 rows while each expert has few, and while they all run at once (rows / 64 and half a tile an expert;
// one workgroup a CU of the gated kernel, two of the other): a taller tile only leaves CUs idle then.  Beyond, a
// taller tile reads the weight less often.  us, tiles of 64 against up to 256 rows (H, I, experts x rows each):
//   up    1024, 512, 16 x 192: 12 against 23; 4096, 2048, 8 x 96: 34, 41; 7168, 2048, 16 x 64: 127, 94;
//         4096, 1024, 32 x 32: 88, 66 (an expert with more than 64); 4096, 2048, 128 x 16: the same
//   down  2048, 2048, 16 x 96: 19 against 26; 3584, 1024, 60 x 16: 52, 57; 4096, 512, 128 x 128: 157, 122
inline bool fp8_tall_tiles(bool gated, int64_t rows, int64_t N, int64_t E, int cus) {
  const int64_t slots = gated ? cus : 2 * cus;
  const int64_t mean = rows / std::min<int64_t>(E, std::max<int64_t>(rows, 1));
  const int64_t tiles = (rows + 32 * E) / 64 * ((N + 127) / 128);
  return mean > 24 && tiles > slots;
}

// Few rows: a scale per block of B, a bf16 result.  That is what a token's projection is; fp8_rows has no other ending, and
// binary32 results (weights' gradients) and scales by row (the same) come with many rows.
inline bool fp8_on_rows(bool row_b, bool f32, int64_t M, int64_t N, int64_t K) {
  return !row_b && !f32 && fp8_rows_ok(M, N, K);
}

}  // namespace
}  // namespace bsfp4
