// bf16 -> E4M3 with one FP32 scale per 128 values along a row, along a column, or per 128 x 128 block:
//
//   amax = max |x| over the block,  s = fl32(amax / 448),  q = rne_e4m3(448 x / amax)      (Fp8Block)
//
// Bound by memory: 2 bytes read and 1 written per element and direction.  Everything is read once and kept in
// registers between the maximum and the rounding.  The codes are of the exact quotient (correctly rounded, no double
// rounding through binary32); scales are rounded to binary32, 2^-24 of their value.  Rows of 4096 x 7168: 17 us, 5.2 TB/s.
#include "fp8_rows.h"
#include "launchers.h"

namespace bsfp4 {
namespace {

constexpr int kThreads = 256;

// bits of the largest |x| of eight bf16 values, as binary32
__device__ __forceinline__ uint32_t amax8(const uint4& c) { return amax_of_pairs(amax_pairs8(c, 0)) << 16; }

// ---- rows only -------------------------------------------------------------
// A workgroup takes 16 rows x 4 blocks: a wave reads four blocks of a row at a time (1 KB), 16 lanes each, and
// the scales, which lie block by block, meet in LDS so that 16 rows' are written together.
constexpr int kQRows = 16, kQBlocks = 4;

__global__ void __launch_bounds__(kThreads)
    fp8_quant_rows(const uint16_t* __restrict__ x, int64_t M, int64_t K, uint8_t* __restrict__ q,
                   float* __restrict__ s) {
  __shared__ float scale[kQBlocks][kQRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m0 = (int64_t)blockIdx.x * kQRows;
  const int64_t kb0 = (int64_t)blockIdx.y * kQBlocks, kb = kb0 + lane / 16;
  const int64_t k = kb * kFp8Block + (lane & 15) * 8;
  uint4 c[kQRows / 4];
#pragma unroll
  for (int i = 0; i < kQRows / 4; i++) {
    const int64_t m = m0 + i * 4 + wave;
    c[i] = m < M && k < K ? *reinterpret_cast<const uint4*>(x + m * K + k) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kQRows / 4; i++) {
    const int64_t m = m0 + i * 4 + wave;
    const Fp8Block b((uint32_t)lanes_reduce<4>((int)amax8(c[i]), MaxOp{}));
    if (m < M && k < K) *reinterpret_cast<uint2*>(q + m * K + k) = fp8_codes8(b, c[i]);
    if ((lane & 15) == 0) scale[lane / 16][i * 4 + wave] = b.s;
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < kQBlocks * kQRows) {
    const int64_t m = m0 + t % kQRows, b = kb0 + t / kQRows;
    if (m < M && b * kFp8Block < K) s[b * M + m] = scale[t / kQRows][t % kQRows];
  }
}

// ---- 128 x 128 tiles -------------------------------------------------------
// Columns (transposed codes), columns and rows, or one scale for the tile (codes as they lie, transposed, or both).
// Thread t holds rows 8 (t / 16) .. + 7, columns 8 (t % 16) .. + 7: a column's eight codes are eight consecutive
// bytes of a transposed row, which the tile passes through LDS so that 128 bytes of it are written together.  There the
// 16-byte pieces of row c stand at their place xor c / 16, so that a wave's stores reach all banks.  4096 x 7168 both
// ways and 4096 x 4096 columns in one launch: 34 us, 4.9 TB/s (38 with conflicts, 50 in two launches).
constexpr int kTile = kFp8Block, kPitch = kTile + 16;

template <bool kBlock>
__device__ __forceinline__ void quant_tile(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                           uint8_t* __restrict__ q, float* __restrict__ s, uint8_t* __restrict__ qt,
                                           float* __restrict__ st, int64_t ldt, int64_t mb, int64_t kb) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[kTile * kPitch];
  __shared__ int col_max[4][kTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, rg = tid / 16, cg = tid % 16;
  const int64_t m0 = mb * kTile + rg * 8, k0 = kb * kTile + cg * 8;
  uint4 c[8];
#pragma unroll
  for (int i = 0; i < 8; i++)
    c[i] = m0 + i < M && k0 < K ? *reinterpret_cast<const uint4*>(x + (m0 + i) * K + k0) : make_uint4(0, 0, 0, 0);

  if (!kBlock && q != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const Fp8Block b((uint32_t)lanes_reduce<4>((int)amax8(c[i]), MaxOp{}));
      if (m0 + i < M && k0 < K) *reinterpret_cast<uint2*>(q + (m0 + i) * K + k0) = fp8_codes8(b, c[i]);
      if (cg == 0 && m0 + i < M) s[kb * M + m0 + i] = b.s;
    }
  }
  Fp8Block one(0);
  if constexpr (kBlock) {
    const int64_t MB = gridDim.x, KB = gridDim.y;
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) mx = amax_pairs8(c[i], mx);
    one = Fp8Block(row_max<kThreads>(amax_of_pairs(mx), col_max[0]) << 16);
    if (tid == 0) {
      if (q != nullptr) s[mb * KB + kb] = one.s;
      if (qt != nullptr) st[kb * MB + mb] = one.s;
    }
    if (q != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (m0 + i < M && k0 < K) *reinterpret_cast<uint2*>(q + (m0 + i) * K + k0) = fp8_codes8(one, c[i]);
    }
    if (qt == nullptr) return;
  } else {
    // largest magnitude of each of the thread's columns, two at a time: its eight rows, the wave's four row groups
    // (then the waves, in LDS)
    typedef uint16_t v2u16 __attribute__((ext_vector_type(2)));
    uint32_t mx[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      v2u16 m{0, 0};
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
        m = __builtin_elementwise_max(m, __builtin_bit_cast(v2u16, w[e] & 0x7FFF7FFFu));
      }
#pragma unroll
      for (int s = 16; s < 64; s *= 2)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(v2u16, __shfl_xor(__builtin_bit_cast(int, m), s, 64)));
      mx[e] = __builtin_bit_cast(uint32_t, m);
    }
    if (lane < 16) {
#pragma unroll
      for (int e = 0; e < 8; e++) col_max[wave][e * 16 + cg] = (int)(mx[e / 2] >> (16 * (e & 1)) & 0xFFFFu);
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 8; e++) {
    Fp8Block b = one;
    if constexpr (!kBlock) {
      const int at = e * 16 + cg;  // neighbouring lanes, neighbouring banks
      b = Fp8Block((uint32_t)max(max(col_max[0][at], col_max[1][at]), max(col_max[2][at], col_max[3][at])) << 16);
      if (rg == 0 && k0 + e < K) st[mb * K + k0 + e] = b.s;
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
      v[i] = e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    }
    *reinterpret_cast<uint2*>(tile + (cg * 8 + e) * kPitch + (rg ^ (cg / 2 * 2)) * 8) =
        make_uint2(fp8_codes4<true>(b, v[0], v[1], v[2], v[3]), fp8_codes4<true>(b, v[4], v[5], v[6], v[7]));
  }
  __syncthreads();
  // rows past M are zeros up to ldt, a multiple of 16
#pragma unroll
  for (int i = tid; i < kTile * kTile / 16; i += kThreads) {
    const int r = i / (kTile / 16), p = i % (kTile / 16) * 16;
    if (kb * kTile + r < K && mb * kTile + p < ldt)
      *reinterpret_cast<uint4*>(qt + (kb * kTile + r) * ldt + mb * kTile + p) =
          *reinterpret_cast<const uint4*>(tile + r * kPitch + (p ^ (r / 16 * 16)));
  }
}

// One matrix per third index.  4096 x 7168 as it lies 19-21 us (4.1-4.7 TB/s), transposed too 25-30 (4.0-4.6); 128 of 4096 x
// 2048 591-623 (5.2-5.4), 814-868 (5.0-5.3); a copy's rate is 5.3.
__global__ void __launch_bounds__(kThreads)
    fp8_quant_blocks(const uint16_t* __restrict__ x, int64_t M, int64_t K, uint8_t* __restrict__ q,
                     float* __restrict__ s, uint8_t* __restrict__ qt, float* __restrict__ st, int64_t ldt) {
  const int64_t e = blockIdx.z, scales = (int64_t)gridDim.x * gridDim.y;
  if (q != nullptr) q += e * M * K, s += e * scales;
  if (qt != nullptr) qt += e * K * ldt, st += e * scales;
  quant_tile<true>(x + e * M * K, M, K, q, s, qt, st, ldt, blockIdx.x, blockIdx.y);
}

// One matrix, or two of M rows: the second's column blocks behind the first's.  A linear layer's gradients take dy
// (both ways) and x (columns) in one launch.
__global__ void __launch_bounds__(kThreads)
    fp8_quant_columns(Fp8Columns a, Fp8Columns b, int64_t M, int64_t ldt) {
  int64_t kb = blockIdx.y;
  if (kb >= (a.K + kTile - 1) / kTile) {
    kb -= (a.K + kTile - 1) / kTile;
    a = b;
  }
  quant_tile<false>(a.x, M, a.K, a.q, a.s, a.qt, a.st, ldt, blockIdx.x, kb);
}

}  // namespace

hipError_t launch_fp8_quant_columns(const Fp8Columns& a, const Fp8Columns& b, int64_t M, hipStream_t stream) {
  const dim3 grid((unsigned)fp8_blocks(M), (unsigned)(fp8_blocks(a.K) + fp8_blocks(b.K)));
  fp8_quant_columns<<<grid, kThreads, 0, stream>>>(a, b, M, fp8_padded(M));
  return hipGetLastError();
}

hipError_t launch_fp8_quant(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* s, uint8_t* qt, float* st,
                            hipStream_t stream) {
  if (qt != nullptr) return launch_fp8_quant_columns({x, q, s, qt, st, K}, {}, M, stream);
  const dim3 grid((unsigned)((M + kQRows - 1) / kQRows), (unsigned)((fp8_blocks(K) + kQBlocks - 1) / kQBlocks));
  fp8_quant_rows<<<grid, kThreads, 0, stream>>>(x, M, K, q, s);
  return hipGetLastError();
}

hipError_t launch_fp8_quant_weight(const uint16_t* W, int64_t E, int64_t N, int64_t K, uint8_t* q, float* s,
                                   uint8_t* qt, float* st, hipStream_t stream) {
  const dim3 grid((unsigned)fp8_blocks(N), (unsigned)fp8_blocks(K), (unsigned)E);
  fp8_quant_blocks<<<grid, kThreads, 0, stream>>>(W, N, K, q, s, qt, st, fp8_padded(N));
  return hipGetLastError();
}

}  // namespace bsfp4
