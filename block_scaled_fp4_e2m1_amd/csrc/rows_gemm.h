// Products of few rows (M <= 32): the weight is read once, straight from memory
// into the matrix cores' operand registers.
//
// Bound by the weight's bytes.  A workgroup owns 16 NB weight rows (gated: 16 gate
// and 16 up rows) and all M activation rows; its waves take the 128-byte steps of
// K in turn, so that the workgroup reads whole stretches of its rows and a
// thousand and more 16-byte loads per compute unit are in flight without any LDS
// ring or barrier in the loop.  v_mfma_*_16x16x{32, 64} takes the weight as its first
// operand: lane l supplies 16 bytes of weight row l % 16 and of activation row
// l % 16, K group l / 16 (the same bytes of both, so any order of K is right), and
// ends with weight rows 4 (l / 16) .. + 3 of activation row l % 16.  The waves'
// sums meet in LDS and are added in wave order; one wave per 16 activation rows
// finishes them.  Activation rows beyond M repeat the last row and are dropped.
//
// kQuant (8-bit, M K <= kRowsQuantBytes): the activations come in bf16 and every
// workgroup quantises all of them into LDS itself, its first weight loads already
// under way: one launch and no intermediate for a token's projection.
#pragma once

#include "tile_gemm.h"

namespace bsfp4 {
namespace {

constexpr int kRowsMaxM = 32;
constexpr int kRowsStep = 128;             // bytes of K per wave and step: two MFMAs
constexpr int kRowsUnroll = 4;             // steps loaded before any is multiplied
constexpr int kRowsQuantBytes = 64 * 1024;  // quantised activations kept in LDS

// MB blocks of 16 activation rows, NB blocks of 16 weight rows (gated: NB = 2, gate
// and up), WAVES waves.  p as for tile_gemm (operands along K), splits unused.
template <bool kInt8, int EPI, int MB, int NB, int WAVES, bool kQuant>
__global__ void __launch_bounds__(64 * WAVES, WAVES / 4)
    rows_gemm(const TileArgs p, const uint16_t* __restrict__ x) {
  typedef Mma<kInt8> MM;
  constexpr bool kGated = EPI == kTileGated;
  static_assert(!kGated || NB == 2, "gate and up blocks");
  static_assert(!kQuant || (kInt8 && MB == 1 && !kGated), "fused quantiser");
  constexpr int kTiles = MB * NB;
  extern __shared__ __attribute__((aligned(16))) uint8_t rows_smem[];  // quantised rows, then (reused) the sums
  __shared__ uint32_t red_max[kQuant ? 4 * WAVES : 1];
  __shared__ float row_scale[kQuant ? 16 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, kg = lane >> 4;
  const int n0 = blockIdx.x * (kGated ? 16 : 16 * NB);
  const int kb = (int)p.kend;

  const uint8_t* w[NB];
#pragma unroll
  for (int j = 0; j < NB; j++) {
    // rows past N repeat the last one; their columns are not stored
    const int64_t row = kGated ? (int64_t)j * p.N + min(n0 + lr, p.N - 1) : min(n0 + 16 * j + lr, p.N - 1);
    w[j] = p.B + row * p.ldb + kg * 16;
  }
  const uint8_t* a[MB];
#pragma unroll
  for (int i = 0; i < MB; i++) a[i] = p.A + (int64_t)min(16 * i + lr, p.M - 1) * p.lda + kg * 16;

  typename MM::Acc acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; i++)
#pragma unroll
    for (int j = 0; j < NB; j++) acc[i][j] = typename MM::Acc{};

  const int full = kb / kRowsStep;
  v4i wr[kRowsUnroll][2][NB];
  auto load_w = [&](int u, int s) {
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int j = 0; j < NB; j++)
        wr[u][h][j] = *reinterpret_cast<const v4i*>(w[j] + (int64_t)s * kRowsStep + h * 64);
  };
  auto load_a = [&](int i, int s, int h) -> v4i {
    if constexpr (kQuant)
      return *reinterpret_cast<const v4i*>(rows_smem + min(lr, p.M - 1) * kb + s * kRowsStep + h * 64 + kg * 16);
    else
      return *reinterpret_cast<const v4i*>(a[i] + (int64_t)s * kRowsStep + h * 64);
  };

  int s = wave;
  if constexpr (kQuant) {
    // the first weight steps are on their way while the rows are quantised
#pragma unroll
    for (int u = 0; u < kRowsUnroll; u++)
      if (s + u * WAVES < full) load_w(u, s + u * WAVES);
    const int chunks = kb / 8;  // 16-byte bf16 chunks of a row
    for (int m0 = 0; m0 < p.M; m0 += 4) {
      uint32_t mx[4] = {0, 0, 0, 0};
      for (int m = 0; m < 4 && m0 + m < p.M; m++) {
        const uint4* row = reinterpret_cast<const uint4*>(x + (int64_t)(m0 + m) * kb);
        for (int c = threadIdx.x; c < chunks; c += 64 * WAVES) mx[m] = amax_bits8(row[c], mx[m]);
      }
#pragma unroll
      for (int m = 0; m < 4; m++) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) mx[m] = max(mx[m], (uint32_t)__shfl_xor((int)mx[m], o, 64));
        if (lane == 0) red_max[m * WAVES + wave] = mx[m];
      }
      __syncthreads();
      for (int m = 0; m < 4 && m0 + m < p.M; m++) {
        uint32_t v = red_max[m * WAVES];
#pragma unroll
        for (int k = 1; k < WAVES; k++) v = max(v, red_max[m * WAVES + k]);
        const Int8Row r(v);
        const uint4* row = reinterpret_cast<const uint4*>(x + (int64_t)(m0 + m) * kb);
        for (int c = threadIdx.x; c < chunks; c += 64 * WAVES)
          *reinterpret_cast<uint2*>(rows_smem + (m0 + m) * kb + c * 8) = r.codes8(row[c]);
        if (threadIdx.x == 0) row_scale[m0 + m] = r.s;
      }
      __syncthreads();
    }
  }
  for (bool first = kQuant; s < full; s += kRowsUnroll * WAVES, first = false) {
    v4i ar[kRowsUnroll][2][MB];
    if (!first) {
#pragma unroll
      for (int u = 0; u < kRowsUnroll; u++)
        if (s + u * WAVES < full) load_w(u, s + u * WAVES);
    }
#pragma unroll
    for (int u = 0; u < kRowsUnroll; u++)
      if (s + u * WAVES < full)
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int i = 0; i < MB; i++) ar[u][h][i] = load_a(i, s + u * WAVES, h);
#pragma unroll
    for (int u = 0; u < kRowsUnroll; u++)
      if (s + u * WAVES < full)
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int i = 0; i < MB; i++)
#pragma unroll
            for (int j = 0; j < NB; j++) acc[i][j] = MM::run(wr[u][h][j], ar[u][h][i], acc[i][j]);
  }
  // K past the last whole step: the wave whose turn it is, chunk by chunk
  if (full * kRowsStep < kb && wave == full % WAVES) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const bool in = full * kRowsStep + h * 64 + kg * 16 < kb;
      v4i wv[NB], av[MB];
#pragma unroll
      for (int j = 0; j < NB; j++)
        wv[j] = in ? *reinterpret_cast<const v4i*>(w[j] + (int64_t)full * kRowsStep + h * 64) : v4i{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < MB; i++) {
        av[i] = v4i{0, 0, 0, 0};
        if (in) av[i] = load_a(i, full, h);
      }
#pragma unroll
      for (int i = 0; i < MB; i++)
#pragma unroll
        for (int j = 0; j < NB; j++) acc[i][j] = MM::run(wv[j], av[i], acc[i][j]);
    }
  }

  if constexpr (kQuant) __syncthreads();  // the quantised rows are done with
  typename MM::Acc* red = reinterpret_cast<typename MM::Acc*>(rows_smem);
#pragma unroll
  for (int i = 0; i < MB; i++)
#pragma unroll
    for (int j = 0; j < NB; j++) red[(wave * kTiles + i * NB + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  constexpr int kOut = kGated ? MB : kTiles;  // output blocks of 16 x 16
  if (wave >= kOut) return;
  auto total = [&](int tile) -> typename MM::Acc {
    typename MM::Acc v = red[tile * 64 + lane];
#pragma unroll
    for (int k = 1; k < WAVES; k++) v += red[(k * kTiles + tile) * 64 + lane];
    return v;
  };
  const int i = kGated ? wave : wave / NB, j = kGated ? 0 : wave % NB;
  const int m = 16 * i + lr, n = n0 + 16 * j + 4 * kg;
  if (m >= p.M || n >= p.N) return;  // N % 8 == 0: four columns are in or out together
  float sa = 1.0f;
  if constexpr (kInt8) sa = kQuant ? row_scale[m] : p.sa[m];
  auto scaled = [&](const typename MM::Acc& v, int64_t col) -> float4 {
    if constexpr (kInt8) {
      const float4 sb = *reinterpret_cast<const float4*>(p.sb + col);
      return make_float4((float)v[0] * sa * sb.x, (float)v[1] * sa * sb.y, (float)v[2] * sa * sb.z,
                         (float)v[3] * sa * sb.w);
    } else {
      return make_float4(v[0], v[1], v[2], v[3]);
    }
  };
  float4 v = scaled(total(i * NB + j), n);
  if constexpr (kGated) {
    const float4 u = scaled(total(i * NB + 1), (int64_t)p.N + n);
    if (!kInt8 && p.gate_up) {
      *reinterpret_cast<float4*>(p.gate_up + (int64_t)m * 2 * p.N + n) = v;
      *reinterpret_cast<float4*>(p.gate_up + (int64_t)m * 2 * p.N + p.N + n) = u;
    }
    v = make_float4(act_value(p.act, v.x) * u.x, act_value(p.act, v.y) * u.y, act_value(p.act, v.z) * u.z,
                    act_value(p.act, v.w) * u.w);
  } else if (kInt8 && p.bias) {
    const uint2 b = *reinterpret_cast<const uint2*>(p.bias + n);
    v = make_float4(v.x + bf16_lo(b.x), v.y + bf16_hi(b.x), v.z + bf16_lo(b.y), v.w + bf16_hi(b.y));
  }
  *reinterpret_cast<uint2*>(p.D + (int64_t)m * p.N + n) =
      make_uint2(pack_bf16x2_ieee(v.x, v.y), pack_bf16x2_ieee(v.z, v.w));
}

// Whether a product of M rows runs on rows_gemm.
inline bool rows_ok(int64_t M) { return M <= kRowsMaxM; }

template <bool kInt8, int EPI, int MB, int NB, bool kQuant>
hipError_t launch_rows_shape(const TileArgs& a, const uint16_t* x, hipStream_t stream) {
  constexpr int kPer = EPI == kTileGated ? 16 : 16 * NB;
  const unsigned grid = (unsigned)((a.N + kPer - 1) / kPer);
  const size_t quant = kQuant ? (size_t)a.M * a.kend : 0;
  auto lds = [&](int waves) { return std::max(quant, (size_t)waves * MB * NB * 1024); };
  // waves: as many as have a whole round of steps each; four operand blocks take
  // more registers than 16 waves have
  const int64_t steps = a.kend / kRowsStep;
  if constexpr (MB * NB < 4) {
    if (steps >= 16 * kRowsUnroll) {
      rows_gemm<kInt8, EPI, MB, NB, 16, kQuant><<<grid, 1024, lds(16), stream>>>(a, x);
      return hipGetLastError();
    }
  }
  if (steps >= 4 * kRowsUnroll)
    rows_gemm<kInt8, EPI, MB, NB, 8, kQuant><<<grid, 512, lds(8), stream>>>(a, x);
  else
    rows_gemm<kInt8, EPI, MB, NB, 4, kQuant><<<grid, 256, lds(4), stream>>>(a, x);
  return hipGetLastError();
}

template <bool kInt8, int EPI>
hipError_t launch_rows(const TileArgs& a, hipStream_t stream) {
  constexpr int NB = EPI == kTileGated ? 2 : 1;
  if (a.M <= 16) return launch_rows_shape<kInt8, EPI, 1, NB, false>(a, nullptr, stream);
  return launch_rows_shape<kInt8, EPI, 2, NB, false>(a, nullptr, stream);
}

}  // namespace
}  // namespace bsfp4
