// The gated feed-forward product in bf16 and its backward pass.
//
//   [G | U] = x W^T,  h = bf16(act(G) * U)            W [2 I, H]: gate rows, then up rows
//   dG = dh U act'(G),  dU = dh act(G)
//   dx = [dG | dU] W,   dW = [dG | dU]^T x
//
// Forward: one kernel, both projections of a column in one wave's accumulators, so
// the activation and the product happen on the binary32 sums; [G | U] is written
// only when the backward pass is to follow, and in binary32: rounded to bf16 it
// would put a second error of 2^-8 beside that of [dG | dU] into every gradient
// (measured at 4096 x 4096 x 7168: 2-norm error 0.30 % against 0.17 % of the
// output's own rounding; so 0.24 %).
// Backward: one pass writes [dG | dU] in bf16, the matrix cores' operand type, then
// the two products read W, x and [dG | dU] as they lie (transposed operands of
// tile_gemm), with binary32 sums.
// Measured at 4096 tokens, H 4096, I 7168 (481 GFLOP each product): forward with its sums
// kept 382 us (the 294 MB written are 55 of them), the [dG | dU] pass 80 (411 MB, at a
// copy's rate), dx 314 and dW 343.
#include "rows_gemm.h"

namespace bsfp4 {
namespace {

__global__ void __launch_bounds__(256)
    gated_grad(const uint16_t* __restrict__ dh, const float* __restrict__ gate_up, int act, int64_t M, int I,
               uint16_t* __restrict__ dgu) {
  const int chunks = I / 8;
  const int64_t all = M * chunks, stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < all; idx += stride) {
    const int64_t m = idx / chunks;
    const int64_t n = (idx - m * chunks) * 8, row = m * 2 * I;
    float d[8], g[8], u[8], dg[8], du[8];
    unpack8(*reinterpret_cast<const uint4*>(dh + m * I + n), d);
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const float4 gv = reinterpret_cast<const float4*>(gate_up + row + n)[k];
      const float4 uv = reinterpret_cast<const float4*>(gate_up + row + I + n)[k];
      g[4 * k] = gv.x, g[4 * k + 1] = gv.y, g[4 * k + 2] = gv.z, g[4 * k + 3] = gv.w;
      u[4 * k] = uv.x, u[4 * k + 1] = uv.y, u[4 * k + 2] = uv.z, u[4 * k + 3] = uv.w;
    }
#pragma unroll
    for (int k = 0; k < 8; k++) {
      float a, da;
      act_value_grad(act, g[k], a, da);
      dg[k] = d[k] * u[k] * da;
      du[k] = d[k] * a;
    }
    *reinterpret_cast<uint4*>(dgu + row + n) = pack8(dg);
    *reinterpret_cast<uint4*>(dgu + row + I + n) = pack8(du);
  }
}

// Both products of a small layer in one launch: the workgroups of one fill the units
// that the other leaves free.  The product of longer sums goes first.
__global__ void __launch_bounds__(256, (tile_waves_simd<64, 128, 3, 4>()))
    gated_products(const TileArgs dx, const TileArgs dw, int dw_first) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[tile_smem<64, 128, 3>()];
  const int n_dx = dx.tiles_m * dx.tiles_n, n_dw = dw.tiles_m * dw.tiles_n;
  const int lead = dw_first ? n_dw : n_dx;
  const bool first = (int)blockIdx.x < lead;
  const int block = first ? blockIdx.x : blockIdx.x - lead;
  if (first == (dw_first != 0)) tile_body<false, 64, 128, 2, 2, 3, true, true, kTileStore>(dw, block, smem);
  else tile_body<false, 64, 128, 2, 2, 3, false, true, kTileStore>(dx, block, smem);
}

struct BwdPlan {
  TilePlan dx, dw;
  bool joint;        // both in one launch of gated_products
  size_t dgu, part;  // workspace bytes of [dG | dU] and of the larger product's partials
};

// One launch where each of the 64 x 128 tile's slots (two per unit) has no more K stages
// than this to do.  Whole backward passes, one launch against two: 256 x 4096 x 1024 (M,
// H, I; 16 stages) 20.9 us against 25.0, 777 x 2048 x 776 (20) 27.6 against 29.4, 4096 x
// 512 x 1024 (32) 39.2 against 43.4, 1024 x 2048 x 1536 (48) 42.3 against 44.6; beyond,
// larger tiles win: 1500 x 3000 x 1000 (72) 69.6 against 59.7.  Only where neither
// product alone is split over K, so that a gradient's bits do not depend on whether the
// other one is asked for.
constexpr int64_t kJointStages = 48;

int64_t joint_tiles(int64_t m, int64_t n) {
  const TileCost& c = kTileCosts[kTile64x128];
  return (m + c.bm - 1) / c.bm * ((n + c.bn - 1) / c.bn);
}

hipError_t launch_products(TileArgs dx, TileArgs dw, hipStream_t stream) {
  for (TileArgs* a : {&dx, &dw}) {
    a->tiles_m = (a->M + 63) / 64;
    a->tiles_n = (a->N + 127) / 128;
    a->splits = 1;
  }
  const unsigned grid = (unsigned)(dx.tiles_m * dx.tiles_n + dw.tiles_m * dw.tiles_n);
  gated_products<<<grid, 256, 0, stream>>>(dx, dw, dw.kend > dx.kend);
  return hipGetLastError();
}

BwdPlan plan_bwd(int64_t M, int64_t H, int64_t I) {
  const int cus = device_cu_count();
  BwdPlan b;
  b.dx = plan_tile(M, H, 4 * I, cus);
  b.dw = plan_tile(2 * I, H, 2 * M, cus);
  const int64_t stages = joint_tiles(M, H) * ((4 * I + kTileStage - 1) / kTileStage) +
                         joint_tiles(2 * I, H) * ((2 * M + kTileStage - 1) / kTileStage);
  b.joint = b.dx.splits == 1 && b.dw.splits == 1 && stages <= kJointStages * 2 * cus;
  b.dgu = ((size_t)M * 2 * I * 2 + 255) / 256 * 256;
  b.part = std::max(tile_workspace(b.dx, M, H), tile_workspace(b.dw, 2 * I, H));
  return b;
}

}  // namespace

size_t gated_ffn_workspace(int64_t M, int64_t I, int64_t H) {
  if (rows_ok(M, 2 * I, 2 * H)) return 0;
  return tile_workspace(plan_tile(M, 2 * I, 2 * H, device_cu_count()), M, 2 * I);
}

hipError_t launch_gated_ffn(const uint16_t* x, const uint16_t* W, int act, uint16_t* h, float* gate_up, int64_t M,
                            int64_t I, int64_t H, void* ws, hipStream_t stream) {
  TileArgs a{};
  a.A = reinterpret_cast<const uint8_t*>(x);
  a.B = reinterpret_cast<const uint8_t*>(W);
  a.lda = a.ldb = 2 * H;
  a.M = (int)M;
  a.N = (int)I;
  a.kend = 2 * H;
  a.act = act;
  a.D = h;
  a.gate_up = gate_up;
  a.part = ws;
  if (rows_ok(M, 2 * I, 2 * H)) return launch_rows<false, kTileGated>(a, stream);
  return launch_tile<false, false, false, kTileGated>(a, plan_tile(M, 2 * I, 2 * H, device_cu_count()), stream);
}

size_t gated_ffn_bwd_workspace(int64_t M, int64_t I, int64_t H) {
  const BwdPlan b = plan_bwd(M, H, I);
  return b.dgu + b.part;
}

hipError_t launch_gated_ffn_bwd(const uint16_t* dh, const uint16_t* x, const uint16_t* W, const float* gate_up,
                                int act, uint16_t* dx, uint16_t* dW, int64_t M, int64_t I, int64_t H, void* ws,
                                hipStream_t stream) {
  const BwdPlan b = plan_bwd(M, H, I);
  uint16_t* dgu = static_cast<uint16_t*>(ws);
  void* part = static_cast<uint8_t*>(ws) + b.dgu;
  const int64_t items = M * (I / 8);
  hipError_t e = hipSuccess;
  if (M > 0) {
    gated_grad<<<(unsigned)std::min<int64_t>((items + 255) / 256, 8192), 256, 0, stream>>>(dh, gate_up, act, M,
                                                                                           (int)I, dgu);
    e = hipGetLastError();
  }
  TileArgs ax{}, aw{};
  ax.A = aw.A = reinterpret_cast<const uint8_t*>(dgu);
  ax.lda = aw.lda = 4 * I;
  ax.B = reinterpret_cast<const uint8_t*>(W);
  aw.B = reinterpret_cast<const uint8_t*>(x);
  ax.ldb = aw.ldb = 2 * H;
  ax.M = (int)M;
  aw.M = (int)(2 * I);
  ax.N = aw.N = (int)H;
  ax.kend = 2 * I;  // k rows of W
  aw.kend = M;      // k rows of dgu and x
  ax.D = dx;
  aw.D = dW;
  ax.part = aw.part = part;
  if (e == hipSuccess && dx != nullptr && dW != nullptr && b.joint) return launch_products(ax, aw, stream);
  if (e == hipSuccess && dx != nullptr) e = launch_tile<false, false, true, kTileStore>(ax, b.dx, stream);
  if (e == hipSuccess && dW != nullptr) e = launch_tile<false, true, true, kTileStore>(aw, b.dw, stream);
  return e;
}

}  // namespace bsfp4
