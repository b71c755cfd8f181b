// E4M3 products of few rows with a scale for each block of 128, bound by the weight's bytes.
//
// As rows_gemm: a workgroup owns 16 weight rows and all M activation rows; its waves take the 128-byte steps of K,
// which are the blocks, in turn, each through a ring of its own in LDS, and their sums meet at the end.  A step is one
// v_mfma_f32_16x16x128_f8f6f4 for each 16 activation rows, started from zero, and one multiply-add a value with the
// product of the step's two scales.  The activations' scales of a step come with it (4 bytes a lane, row by row); the
// weight's, one a step, are loaded into LDS ahead of everything.
//
// kQuant: the activations come in bf16 and every workgroup quantises all of them into LDS itself, its first weight
// loads already under way.
//
// 1 x 4096 x 7168, bf16 in: 7.3 us with other weights in turn, 7.8-8.2 behind other data (29 MB: 4.0 TB/s and 3.6; 15.1
// on tiles, quantised apart).  16 x 131072 x 4096: 106 us, 5.1 TB/s.
#pragma once

#include "fp8_tile.h"
#include "rows_gemm.h"

namespace bsfp4 {
namespace {

constexpr int kFp8RowsMaxM = 32;
constexpr int kFp8RowsQuantBytes = 28 * 1024;  // kQuant: activations, their codes and scales in LDS

// AQ: 1 KB loads of activations per step, eight rows each (1, 2 or 4); 0: kQuant.  Two workgroups share a compute unit.
template <int AQ>
struct Fp8RowsShape {
  static constexpr int kWaves = AQ <= 2 ? 8 : 4;
  static constexpr int kRing = AQ == 2 ? 2 : 3;
  static constexpr int kSlot = (2 + AQ) * 1024 + (AQ > 0 ? 256 : 0);
  static constexpr int kBlocks = AQ <= 2 ? 1 : AQ / 2;  // of 16 activation rows
  static constexpr int kRings = kWaves * kRing * kSlot;
  // weight scales of 64 steps a wave
  static constexpr int kSmem = kRings + kWaves * 256 + (AQ == 0 ? kFp8RowsQuantBytes : 0);
  static_assert(2 * kSmem <= 160 * 1024, "two workgroups per compute unit");
};

template <int AQ>
__global__ void __launch_bounds__(64 * Fp8RowsShape<AQ>::kWaves, Fp8RowsShape<AQ>::kWaves / 2)
    fp8_rows(const Fp8Args p, const uint16_t* __restrict__ x) {
  typedef Fp8RowsShape<AQ> S;
  constexpr bool kQuant = AQ == 0;
  constexpr int W = S::kWaves, RING = S::kRing, kSlot = S::kSlot, MB = S::kBlocks, kL = 2 + AQ + (kQuant ? 0 : 1);
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kSmem];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, kg = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int kb = (int)p.K, total = p.kb;

  const int row8 = lane >> 3;  // row of a load
  const v4u32 rw = make_rsrc4(p.B + (int64_t)n0 * p.K, (int64_t)min(16, p.N - n0) * p.K);
  const v4u32 ra = make_rsrc4(p.A, (int64_t)p.M * p.K);
  const uint32_t c16 = (uint32_t)((lane & 7) ^ tile_swz(row8)) * 16;
  uint32_t ow[2], oa[AQ > 0 ? AQ : 1];
#pragma unroll
  for (int q = 0; q < 2; q++) ow[q] = n0 + 8 * q + row8 < p.N ? (uint32_t)((8 * q + row8) * p.K) + c16 : kBufOOB;
#pragma unroll
  for (int q = 0; q < AQ; q++) oa[q] = 8 * q + row8 < p.M ? (uint32_t)((8 * q + row8) * p.K) + c16 : kBufOOB;
  const uint32_t os = lane < p.M ? (uint32_t)lane * 4 : kBufOOB;
  const uint32_t ring0 = lds_offset(smem) + (uint32_t)wave * RING * kSlot;
  const uint8_t* const ring = smem + wave * RING * kSlot;
  float* const weight_scales = reinterpret_cast<float*>(smem + S::kRings) + wave * 64;

  const int mine = wave < total ? (total - 1 - wave) / W + 1 : 0;  // turns wave, wave + W, ...; 64 at most
  const int first = (int)(blockIdx.x % (unsigned)total);           // each workgroup begins a step further on in K
  auto step_of = [&](int i) {
    const int s = wave + i * W + first;
    return s < total ? s : s - total;
  };
  auto issue = [&](int s, int slot) {
    const uint32_t soff = (uint32_t)s * kTileStage, lds = ring0 + (uint32_t)slot * kSlot;
    const bool in = (int)c16 < kb - (int)soff;  // a partial last step masks its chunks past K
#pragma unroll
    for (int q = 0; q < 2; q++) buf_lds16(rw, in ? ow[q] : kBufOOB, soff, lds + q * 1024);
#pragma unroll
    for (int q = 0; q < AQ; q++) buf_lds16(ra, in ? oa[q] : kBufOOB, soff, lds + (2 + q) * 1024);
    if constexpr (!kQuant)
      buf_lds4(make_rsrc4(p.sa + (int64_t)s * p.M, (int64_t)p.M * 4), os, 0u, lds + (2 + AQ) * 1024);
  };
  {
    const v4u32 rs = make_rsrc4(p.sb + (int64_t)(n0 / kFp8Block) * total, (int64_t)total * 4);
    buf_lds4(rs, lane < mine ? (uint32_t)step_of(lane) * 4 : kBufOOB, 0u, lds_offset(weight_scales));
  }
  // kQuant: codes of whole steps, then scales, then the activations as they came
  uint8_t* const codes = smem + S::kRings + W * 256;
  float* const scales = reinterpret_cast<float*>(codes + p.M * total * kTileStage);
  uint8_t* const raw = codes + (p.M * total * (kTileStage + 4) + 15) / 16 * 16;
  if constexpr (kQuant) {
    const int raw_bytes = p.M * kb * 2;
    const v4u32 rx = make_rsrc4(x, raw_bytes);
    for (int q = wave; q * 1024 < raw_bytes; q += W)
      buf_lds16(rx, (uint32_t)(q * 1024 + lane * 16), 0u, lds_offset(raw) + q * 1024);
  }
#pragma unroll
  for (int r = 0; r < RING; r++)
    if (r < mine) issue(step_of(r), r);

  if constexpr (kQuant) {
    const int chunks = kb / 8, kept = total * (kTileStage / 8);
    const uint4* const rows = reinterpret_cast<const uint4*>(raw);
    wait_vmcnt_upto(kL * min(RING, mine));  // all but the ring's loads
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    for (int m = 0; m < p.M; m++)
      for (int c = threadIdx.x; c < kept; c += 64 * W) {  // 16 lanes hold a block
        const uint4 v = c < chunks ? rows[m * chunks + c] : make_uint4(0, 0, 0, 0);
        const Fp8Block b((uint32_t)lanes_reduce<4>((int)amax_of_pairs(amax_pairs8(v, 0)), MaxOp{}) << 16);
        *reinterpret_cast<uint2*>(codes + (m * kept + c) * 8) = fp8_codes8(b, v);
        if ((c & 15) == 0) scales[m * total + c / 16] = b.s;
      }
    // the codes are in LDS; the weight loads stay in flight
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  v4f acc[MB] = {};
  uint32_t off[2];  // the lane's two chunks of a row: row lr, chunk 4 h + kg
#pragma unroll
  for (int h = 0; h < 2; h++) off[h] = (uint32_t)(lr * kTileStage + (((4 * h + kg) ^ tile_swz(lr)) * 16));
  auto step = [&](int i, int slot) {
    const uint8_t* s = ring + slot * kSlot;
    v4i w[2], a[2][MB];
    float sa[MB];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      w[h] = *reinterpret_cast<const v4i*>(s + off[h]);
      if constexpr (kQuant) {
        const int at = (min(lr, p.M - 1) * total + step_of(i)) * kTileStage + h * 64 + kg * 16;
        a[h][0] = *reinterpret_cast<const v4i*>(codes + at);
      } else {
        // M <= 8: the upper eight rows of the fragment repeat the lower (outputs not stored)
#pragma unroll
        for (int b = 0; b < MB; b++)
          a[h][b] = *reinterpret_cast<const v4i*>(s + 2048 + b * 2048 + (AQ == 1 ? off[h] & 1023u : off[h]));
      }
    }
#pragma unroll
    for (int b = 0; b < MB; b++)
      sa[b] = kQuant ? scales[min(lr, p.M - 1) * total + step_of(i)]
                     : reinterpret_cast<const float*>(s + (2 + AQ) * 1024)[b * 16 + lr];
    const float sb = weight_scales[i];
    // all is in registers before the slot is filled again
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (i + RING < mine) issue(step_of(i + RING), slot);
#pragma unroll
    for (int b = 0; b < MB; b++) {
      const v4f part = mfma_fp8(fp8_frag(w[0], w[1]), fp8_frag(a[0][b], a[1][b]));
      const float f = sa[b] * sb;
#pragma unroll
      for (int e = 0; e < 4; e++) acc[b][e] = __builtin_fmaf(part[e], f, acc[b][e]);
    }
  };
  int i = 0, slot = 0;
  for (; i + RING <= mine; i++) {
    wait_vmcnt<(RING - 1) * kL>();  // the loads of the RING - 1 steps after this one may be under way
    step(i, slot);
    slot = slot + 1 == RING ? 0 : slot + 1;
  }
  if constexpr (RING > 2) {
    if (mine - i == 2) {
      wait_vmcnt<kL>();
      step(i++, slot);
      slot = slot + 1 == RING ? 0 : slot + 1;
    }
  }
  if (mine - i == 1) {
    wait_vmcnt<0>();
    step(i, slot);
  }

  __syncthreads();  // every ring is done with
  v4f* red = reinterpret_cast<v4f*>(smem);
#pragma unroll
  for (int b = 0; b < MB; b++) red[(wave * MB + b) * 64 + lane] = acc[b];
  __syncthreads();
  if (wave >= MB) return;  // wave b finishes activation rows 16 b .. + 15
  v4f v = red[wave * 64 + lane];
#pragma unroll
  for (int k = 1; k < W; k++) v += red[(k * MB + wave) * 64 + lane];
  const int m = 16 * wave + lr, n = n0 + 4 * kg;
  if (m >= p.M || n >= p.N) return;  // N % 8 == 0: four columns are in or out together
  if (p.bias) {
    const uint2 b = *reinterpret_cast<const uint2*>(p.bias + n);
    v += v4f{bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y)};
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.D) + (int64_t)m * p.N + n) =
      make_uint2(pack_bf16x2_ieee(v[0], v[1]), pack_bf16x2_ieee(v[2], v[3]));
}

template <int AQ>
void launch_fp8_rows_shape(const Fp8Args& a, const uint16_t* x, hipStream_t stream) {
  fp8_rows<AQ><<<(unsigned)((a.N + 15) / 16), 64 * Fp8RowsShape<AQ>::kWaves, 0, stream>>>(a, x);
}

inline hipError_t launch_fp8_rows(const Fp8Args& a, hipStream_t stream) {
  if (a.M <= 8) launch_fp8_rows_shape<1>(a, nullptr, stream);
  else if (a.M <= 16) launch_fp8_rows_shape<2>(a, nullptr, stream);
  else launch_fp8_rows_shape<4>(a, nullptr, stream);
  return hipGetLastError();
}

// Up to four rows in bf16, quantised inside: what fits in LDS, and where it is cheaper than a launch of its own.  us,
// inside against two launches: 1 x 4096 x 7168 7.8, 10.1; 4 x 512 x 512 4.0, 4.9; 2 x 14336 x 4096 13.4, 15.2; but 3 x
// 65536 x 1024 26.6, 21.8.
//
// Every workgroup of 16 columns quantises all M K values: what the launch saves is lost again when N is large, sooner with
// more rows and later with longer sums, which the last bound follows by fit.  It keeps to the safe side: one row is faster
// inside up to some N = 16384, 24576, 60000 of K 512, 1024, 2048 and past 131072 of 3584 (bound: 16384, 16384, 32768, 100352),
// and calls just past it lose up to a third to it (2 x 10000 x 1024 inside 6.1, apart 8.1; 3 x 8192 x 512 4.6, 5.8).
inline bool fp8_rows_quant_ok(int64_t M, int64_t N, int64_t K) {
  const int64_t lds = (M * fp8_blocks(K) * (kFp8Block + 4) + 15) / 16 * 16 + (2 * M * K + 1023) / 1024 * 1024;
  return M <= 4 && fp8_blocks(K) <= 512 && lds <= kFp8RowsQuantBytes &&
         (M * N <= ((int64_t)1 << 14) || M * M * M * N <= K * K / 128);
}

// Whether M rows run on fp8_rows: 64 steps a wave at most, and few enough columns that its workgroups, which read all
// activations each, beat tiles.  us against tiles, other weights in turn: 1 x 4096 x 7168 7.3, 11.1; 16 x 512 x 512 2.6,
// 4.0; 32 x 4096 x 7168 9.3, 12.4; 16 x 131072 x 4096 106, 116; but 32 x 14336 x 4096 16.7, 15.1; 24 x 16384 x 7168 29,
// 25.5.  Short K leaves its workgroups little beside their start: 1 x 65536 x 1024 19.2, 16; 8 x 32768 x 1024 10.4, 8.9;
// 8 x 16384 x 2048 8.4, 8.8; 16 x 8192 x 512 3.4, 4.4.
//
// What may be quantised inside always runs here, so that the product alone sums in the same order and gives the same bits.
// Beyond the other bounds that is one row of more columns (10000 x 512 4.2, 4.4; 16384 x 512 4.8, 4.6; 16384 x 1024 6.5, 6.3;
// 32768 x 2048 15.2, 15.5; 49152 x 2560 24.9, 30.6; quantised inside 5.1, 5.8, 7.4, 15.4, 25.1, on tiles behind the quantiser
// 6.7, 7.0, 9.0, 17.1, 30.5).
inline bool fp8_rows_ok(int64_t M, int64_t N, int64_t K) {
  const int64_t waves = M <= 16 ? 8 : 4;
  if (M > kFp8RowsMaxM || fp8_blocks(K) > 64 * waves) return false;
  if (M <= 16 && K >= 4096) return M * N <= (int64_t)1 << 21;
  return (M * N <= (int64_t)1 << 18 && N <= std::max<int64_t>(8192, 8 * K)) || fp8_rows_quant_ok(M, N, K);
}

inline hipError_t launch_fp8_rows_quant(const Fp8Args& a, const uint16_t* x, hipStream_t stream) {
  launch_fp8_rows_shape<0>(a, x, stream);
  return hipGetLastError();
}

}  // namespace
}  // namespace bsfp4
