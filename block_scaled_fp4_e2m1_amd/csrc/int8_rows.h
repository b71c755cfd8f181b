// Row helpers shared by the 8-bit quantiser and the block norms: 128-bit row
// chunks, sums and maxima over the threads of a row, and the per-token 8-bit
// integer rounding.
#pragma once

#include "device_common.h"

#pragma clang fp contract(off)

namespace bsfp4 {

// Rounds to bf16 nearest-even, NaN kept (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16x2_ieee(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi});
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4& c, float (&v)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    v[2 * j] = bf16_lo(w[j]);
    v[2 * j + 1] = bf16_hi(w[j]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2_ieee(v[0], v[1]), pack_bf16x2_ieee(v[2], v[3]), pack_bf16x2_ieee(v[4], v[5]),
                    pack_bf16x2_ieee(v[6], v[7]));
}

// Largest |bits| of a chunk of eight bf16 values: ordered like the magnitudes,
// infinities above every finite value and NaNs above those.
__device__ __forceinline__ uint32_t amax_bits8(const uint4& c, uint32_t m) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    m = max(m, w[j] & 0x7FFFu);
    m = max(m, (w[j] >> 16) & 0x7FFFu);
  }
  return m;
}

// A value of another lane of the wave: neighbours at 1, 2 (lane xor) and at the
// mirrored places of 8 and 16 lanes by a data-parallel move, 16 and 32 apart
// through LDS hardware.  Combining with all six in turn gives every lane the same
// bits (both partners of a step form the same pair).
template <int kStep>
__device__ __forceinline__ int lane_partner(int v) {
  if constexpr (kStep == 0) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);        // xor 1
  else if constexpr (kStep == 1) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);   // xor 2
  else if constexpr (kStep == 2) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);  // mirror of 8
  else if constexpr (kStep == 3) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);  // mirror of 16
  else return __shfl_xor(v, kStep == 4 ? 16 : 32, 64);
}
template <int kStep>
__device__ __forceinline__ double lane_partner(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)lane_partner<kStep>((int)(uint32_t)u);
  const uint32_t hi = (uint32_t)lane_partner<kStep>((int)(uint32_t)(u >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

struct AddOp {
  __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};
struct MaxOp {
  __device__ __forceinline__ int operator()(int a, int b) const { return max(a, b); }
};

// Over groups of 2^kSteps lanes (64 with all six steps).
template <int kSteps, class Op, class T>
__device__ __forceinline__ T lanes_reduce(T v, Op op) {
  if constexpr (kSteps > 0) v = op(v, lane_partner<0>(v));
  if constexpr (kSteps > 1) v = op(v, lane_partner<1>(v));
  if constexpr (kSteps > 2) v = op(v, lane_partner<2>(v));
  if constexpr (kSteps > 3) v = op(v, lane_partner<3>(v));
  if constexpr (kSteps > 4) v = op(v, lane_partner<4>(v));
  if constexpr (kSteps > 5) v = op(v, lane_partner<5>(v));
  return v;
}

constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }

// N values over the NT threads that hold one row (NT 64: a wave of its own, no
// barrier; else the whole workgroup), every thread with the same bits.  The waves'
// values meet in `red` (N NT / 64 of them), where each group of NT / 64 lanes
// combines them: one value in a register at a time.  `red` must not be in use by
// an earlier call still being read: two calls that alternate use two buffers.
template <int NT, class Op, class T, int N>
__device__ __forceinline__ void row_reduce(T (&v)[N], T* red, Op op) {
  constexpr int W = NT / 64;
  static_assert((W & (W - 1)) == 0 && W <= 16, "waves of a row");
#pragma unroll
  for (int k = 0; k < N; k++) v[k] = lanes_reduce<6>(v[k], op);
  if constexpr (W > 1) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < N; k++) red[k * W + wave] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; k++) v[k] = lanes_reduce<log2_of(W)>(red[k * W + (lane & (W - 1))], op);
  }
}

template <int NT, int N>
__device__ __forceinline__ void row_sum(double (&v)[N], double* red) { row_reduce<NT>(v, red, AddOp{}); }

template <int NT>
__device__ __forceinline__ uint32_t row_max(uint32_t m, int* red) {
  int v[1] = {(int)m};
  row_reduce<NT>(v, red, MaxOp{});
  return (uint32_t)v[0];
}

// Per-token 8-bit rounding of a row of bf16 values with largest magnitude amax:
// q = round-to-even(127 x / amax), s = amax / 127.
//
// The quotient is formed as a correctly rounded binary32 division would: with
// r = fl(1 / amax), q0 = t r, e = t - q0 amax (exact in an FMA), q1 = q0 + e r
// (Markstein's step).  t = 127 x has 15 significant bits and amax 8, so t / amax
// is either exactly half-way between two integers or further than 2^-16 of its
// value from it, and q1, within one unit of 2^-24 and exact where the quotient
// is representable, always rounds to the right integer.  Rows whose amax is far
// from 1 are scaled by 2^+-64 first, so that neither 127 x nor 1 / amax leaves
// the binary32 range; both sides are multiplied, the quotient is unchanged.
struct Int8Row {
  float mul;   // 127 * 2^k
  float amax;  // amax * 2^k
  float r;     // 1 / (amax * 2^k), 0 for a row without codes
  float s;     // amax / 127 (NaN for a row with an infinity or a NaN)
  __device__ __forceinline__ explicit Int8Row(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits << 16);
    const bool finite = amax_bits < 0x7F80u;
    const float k = a < 0x1p-60f ? 0x1p64f : a > 0x1p60f ? 0x1p-64f : 1.0f;
    mul = 127.0f * k;
    amax = a * k;
    r = (amax_bits != 0 && finite) ? 1.0f / amax : 0.0f;
    s = finite ? a / 127.0f : __uint_as_float(0x7FC00000u);
  }
  __device__ __forceinline__ int code(float x) const {
    const float t = x * mul;
    const float q0 = t * r;
    const float q1 = __builtin_fmaf(__builtin_fmaf(-q0, amax, t), r, q0);
    // a row with r == 0 has t * 0: NaN for its infinities and NaNs
    return r == 0.0f ? 0 : (int)__builtin_rintf(q1);
  }
  __device__ __forceinline__ uint2 codes8(const uint4& c) const {
    float v[8];
    unpack8(c, v);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; h++)
      w[h] = (uint32_t)(code(v[4 * h]) & 0xFF) | (uint32_t)(code(v[4 * h + 1]) & 0xFF) << 8 |
             (uint32_t)(code(v[4 * h + 2]) & 0xFF) << 16 | (uint32_t)code(v[4 * h + 3]) << 24;
    return make_uint2(w[0], w[1]);
  }
};

}  // namespace bsfp4
