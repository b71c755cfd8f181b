// Products of few rows (M <= 64), bound by the weight's bytes.
//
// A workgroup owns 16 weight rows (gated: 8 gate rows and their 8 up rows) and all M
// activation rows; its waves take the 128-byte steps of K in turn.  Each wave
// runs a ring of its own in LDS, filled by direct loads of eight rows x 128 bytes, so
// there is no barrier until the waves' sums meet at the end.  The loads go through
// LDS, though every byte is used by one wave only, because the memory pipeline
// takes a request per 128-byte line: operands loaded straight into the MFMA's
// registers (16 rows x 64 bytes per load, twice the lines) ran at 33 GB/s per
// compute unit against 70 this way (measured; 48 workgroups, bf16 gated 1 x 2048 x 768
// 6.4 us that way).
//
// v_mfma_*_16x16x{32, 64} takes the weight as its first operand: lane l ends with
// weight rows 4 (l / 16) .. + 3 of activation row l % 16.  Rows outside the operands
// and chunks past K are zeros through the buffers' range check.  The waves' sums are
// added in wave order by one wave, which finishes the outputs.
//
// Bound by the weight's bytes from some 20 MB on: bf16 gated 1 x 14336 x 4096 (117 MB) 21
// us, 5.6 TB/s, behind other data (42 where that was written just before: its lines go back
// to memory meanwhile); int8 8 x 65536 x 4096 (268 MB) 48 us, 5.6 TB/s.  Smaller ones are a launch and two memory
// latencies (int8 16 x 1024 x 4096 3.5 us).
//
// kQuant (8-bit): the activations come in bf16 and every workgroup quantises all of
// them into LDS itself, its first weight loads already under way: one launch and no
// intermediate for a token's projection.
#pragma once

#include "tile_gemm.h"

namespace bsfp4 {
namespace {

constexpr int kRowsMaxM = 64;
constexpr int kRowsQuantBytes = 28 * 1024;  // kQuant: activations and their codes in LDS

// AQ: 1 KB loads of activations per step, eight rows each (1, 2, 4 or 8); 0: kQuant.
// Waves and ring slots per wave so that two workgroups share a compute unit (80 KB
// each).
template <int AQ>
struct RowsShape {
  static constexpr int kWaves = AQ <= 2 ? 8 : 4;
  static constexpr int kRing = AQ == 2 || AQ == 8 ? 2 : 3;
  static constexpr int kSlot = (2 + AQ) * 1024;
  static constexpr int kBlocks = AQ <= 2 ? 1 : AQ / 2;  // of 16 activation rows
};

// p as for tile_gemm (operands along K), splits unused.
template <bool kInt8, int EPI, int AQ>
__global__ void __launch_bounds__(64 * RowsShape<AQ>::kWaves, RowsShape<AQ>::kWaves / 2)
    rows_gemm(const TileArgs p, const uint16_t* __restrict__ x) {
  typedef Mma<kInt8> MM;
  constexpr bool kGated = EPI == kTileGated, kQuant = AQ == 0;
  static_assert(!kQuant || (kInt8 && !kGated), "fused quantiser");
  constexpr int W = RowsShape<AQ>::kWaves, RING = RowsShape<AQ>::kRing, kSlot = RowsShape<AQ>::kSlot, kL = 2 + AQ,
                MB = RowsShape<AQ>::kBlocks;
  constexpr int kRings = W * RING * kSlot;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kRings + (kQuant ? kRowsQuantBytes : 0)];
  __shared__ int red_max[kQuant ? 4 * W : 1];
  __shared__ float row_scale[kQuant ? 4 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, kg = lane >> 4;
  const int n0 = blockIdx.x * (kGated ? 8 : 16);
  const int kb = (int)p.kend;

  // weight rows: buffers of the two loads (gated: gate, up), lane offsets inside
  const int row8 = lane >> 3;  // row of a load
  const v4u32 rw0 = make_rsrc4(p.B + (int64_t)n0 * p.ldb, (int64_t)min(kGated ? 8 : 16, p.N - n0) * p.ldb);
  const v4u32 rw1 = kGated ? make_rsrc4(p.B + ((int64_t)p.N + n0) * p.ldb, 8 * p.ldb) : rw0;
  const v4u32 ra = make_rsrc4(p.A, (int64_t)p.M * p.lda);
  uint32_t c16[2], ow[2], oa[AQ > 0 ? AQ : 1];
#pragma unroll
  for (int q = 0; q < 2; q++) {
    const int r = 8 * q + row8;
    c16[q] = (uint32_t)((lane & 7) ^ tile_swz(r)) * 16;
    ow[q] = (uint32_t)((kGated ? row8 : r) * p.ldb) + c16[q];
  }
#pragma unroll
  for (int q = 0; q < AQ; q++) {
    const int r = 8 * q + row8;
    oa[q] = r < p.M ? (uint32_t)(r * p.lda) + c16[q & 1] : kBufOOB;
  }
  const uint32_t ring0 = lds_offset(smem) + (uint32_t)wave * RING * kSlot;
  const uint8_t* const ring = smem + wave * RING * kSlot;
  auto issue = [&](int s, int slot) {
    const uint32_t soff = (uint32_t)s * kTileStage, lds = ring0 + (uint32_t)slot * kSlot;
    const int left = kb - (int)soff;  // a partial last step masks its chunks past K
#pragma unroll
    for (int q = 0; q < 2; q++)
      buf_lds16(q ? rw1 : rw0, (int)c16[q] < left ? ow[q] : kBufOOB, soff, lds + q * 1024);
#pragma unroll
    for (int q = 0; q < AQ; q++) buf_lds16(ra, (int)c16[q & 1] < left ? oa[q] : kBufOOB, soff, lds + (2 + q) * 1024);
  };
  const int total = (kb + kTileStage - 1) / kTileStage;
  const int mine = wave < total ? (total - 1 - wave) / W + 1 : 0;  // turns wave, wave + W, ...
  // Each workgroup begins a step further on in K: rows of 4096 bytes and the like put
  // one step of every row on the same few memory channels (int8 16 x 4096 x 14336
  // 13.5 us with one start for all, 10.7 so).
  const int first = (int)(blockIdx.x % (unsigned)total);
  auto step_of = [&](int i) {
    const int s = wave + i * W + first;
    return s < total ? s : s - total;
  };
  // kQuant: the activations go ahead of the weight, into LDS behind their codes.  Loads
  // return in order: read into registers, behind the ring's first loads, the
  // activations arrived with those, and nothing flew while they were quantised (1 x
  // 4096 x 7168 8.3 us that way, 7.1 so).
  const int kept = total * (kTileStage / 8);  // chunks of a row's codes
  uint8_t* const raw = smem + kRings + p.M * kept * 8;
  const int raw_bytes = p.M * kb * 2;
  if constexpr (kQuant) {
    const v4u32 rx = make_rsrc4(x, raw_bytes);
    for (int q = wave; q * 1024 < raw_bytes; q += W)
      buf_lds16(rx, (uint32_t)(q * 1024 + lane * 16), 0u, lds_offset(raw) + q * 1024);
  }
#pragma unroll
  for (int r = 0; r < RING; r++)
    if (r < mine) issue(step_of(r), r);

  if constexpr (kQuant) {
    // all M <= 4 rows, a chunk of eight values at a time; a row's codes are kept in
    // whole steps of 128 bytes, its chunks past K zero
    const int chunks = kb / 8;
    const uint4* const rows = reinterpret_cast<const uint4*>(raw);
    wait_vmcnt_upto(kL * min(RING, mine));  // all but the ring's loads
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    int mx[4] = {0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < 4; m++)
      if (m < p.M)
        for (int c = threadIdx.x; c < chunks; c += 64 * W)
          mx[m] = (int)amax_bits8(rows[m * chunks + c], (uint32_t)mx[m]);
    row_reduce<64 * W>(mx, red_max, MaxOp{});
#pragma unroll
    for (int m = 0; m < 4; m++)
      if (m < p.M) {
        const Int8Row r((uint32_t)mx[m]);
        for (int c = threadIdx.x; c < kept; c += 64 * W)
          *reinterpret_cast<uint2*>(smem + kRings + m * kept * 8 + c * 8) =
              c < chunks ? r.codes8(rows[m * chunks + c]) : make_uint2(0, 0);
        if (threadIdx.x == 0) row_scale[m] = r.s;
      }
    // the codes are in LDS; the weight loads stay in flight
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  typename MM::Acc acc[MB] = {};
  // lane offsets of the two K halves of a step: row lr, chunk 4 h + kg
  uint32_t off[2];
#pragma unroll
  for (int h = 0; h < 2; h++) off[h] = (uint32_t)(lr * kTileStage + (((4 * h + kg) ^ tile_swz(lr)) * 16));
  auto step = [&](int i, int slot) {
    const uint8_t* s = ring + slot * kSlot;
    v4i w[2], a[2][MB];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      w[h] = *reinterpret_cast<const v4i*>(s + off[h]);
      if constexpr (kQuant) {
        const int at = min(lr, p.M - 1) * total * kTileStage + step_of(i) * kTileStage + h * 64 + kg * 16;
        a[h][0] = *reinterpret_cast<const v4i*>(smem + kRings + at);
      } else {
        // M <= 8: the upper eight rows of the fragment repeat the lower (outputs not stored)
#pragma unroll
        for (int b = 0; b < MB; b++)
          a[h][b] = *reinterpret_cast<const v4i*>(s + 2048 + b * 2048 + (AQ == 1 ? off[h] & 1023u : off[h]));
      }
    }
    // the fragments are in registers before the slot is filled again
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (i + RING < mine) issue(step_of(i + RING), slot);
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int b = 0; b < MB; b++) acc[b] = MM::run(w[h], a[h][b], acc[b]);
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
  typename MM::Acc* red = reinterpret_cast<typename MM::Acc*>(smem);
#pragma unroll
  for (int b = 0; b < MB; b++) red[(wave * MB + b) * 64 + lane] = acc[b];
  __syncthreads();
  if (wave >= MB) return;  // wave b finishes activation rows 16 b .. + 15
  // weight rows 4 kg .. + 3; gated: of the lanes kg < 2 the gate rows, the up rows 8 on
  auto total_of = [&](int l) -> typename MM::Acc {
    typename MM::Acc v = red[wave * 64 + l];
#pragma unroll
    for (int k = 1; k < W; k++) v += red[(k * MB + wave) * 64 + l];
    return v;
  };
  const int m = 16 * wave + lr, n = n0 + 4 * kg;
  if (m >= p.M || n >= p.N || (kGated && kg >= 2)) return;  // N % 8 == 0: four columns are in or out together
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
  float4 v = scaled(total_of(lane), n);
  if constexpr (kGated) {
    const float4 u = scaled(total_of(lane + 32), (int64_t)p.N + n);
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

template <bool kInt8, int EPI, int AQ>
void launch_rows_shape(const TileArgs& a, const uint16_t* x, hipStream_t stream) {
  constexpr int kPer = EPI == kTileGated ? 8 : 16;
  rows_gemm<kInt8, EPI, AQ>
      <<<(unsigned)((a.N + kPer - 1) / kPer), 64 * RowsShape<AQ>::kWaves, 0, stream>>>(a, x);
}

template <bool kInt8, int EPI>
hipError_t launch_rows(const TileArgs& a, hipStream_t stream) {
  if (a.M <= 8) launch_rows_shape<kInt8, EPI, 1>(a, nullptr, stream);
  else if (a.M <= 16) launch_rows_shape<kInt8, EPI, 2>(a, nullptr, stream);
  else if (a.M <= 32) launch_rows_shape<kInt8, EPI, 4>(a, nullptr, stream);
  else launch_rows_shape<kInt8, EPI, 8>(a, nullptr, stream);
  return hipGetLastError();
}

// Whether a product of M rows with n weight rows (gated: both halves) of kbytes runs
// on rows_gemm.  Every workgroup reads all activation rows, so past some M n the tiles
// are faster: int8 32 x 4096 x 14336 10.8 us against 14.8, 64 x 4096 x 4096 6.2 against
// 8.9, but 64 x 7168 x 4096 9.9 against 9.1.  Few rows keep it longer, where K has steps
// enough for the waves' rings (4096 bytes): int8 8 x 131072 x 4096 96 against 117, 16 x
// 65536 x 4096 53 against 63, bf16 gated 1 x 32768 x 4096 49 against 63; but bf16 gated
// 16 x 131072 x 4096 194 against 175, int8 4 x 131072 x 1024 35 against 27.
// And past some M kbytes the activations are most of what a workgroup reads, where the
// tiles split K: bf16 gated 32 x 4096 x 14336 29 against 27, 64 x 4096 x 14336 40 against
// 29, 48 x 1024 x 14336 22 against 18; 32 x 2048 x 14336 17 against 21, int8 48 x 4096 x
// 14336 13.4 against 15.9.
inline bool rows_ok(int64_t M, int64_t n, int64_t kbytes) {
  const bool few = M <= 16 && kbytes >= 4096;
  return M <= kRowsMaxM && M * n <= ((int64_t)1 << (few ? 20 : 18)) &&
         M * kbytes <= (M <= 32 ? (int64_t)4 << 18 : (int64_t)3 << 18);
}

// 8-bit, the activations x in bf16, up to four rows: where they and their codes (whole
// 128-byte steps) fit kRowsQuantBytes, K <= 9216 / M.  More of them are quantised faster
// once than by every workgroup; read from memory, 2 x 4096 x 7168 ran 9.6 us against 9.5
// and 4 x 4096 x 7168 12.5 against 9.6.  The same holds of many workgroups: each quantises
// the M K values again, against one launch saved.  Device time, fused against two
// launches, other weights in turn: 1 x 4096 x 7168 8.0 us against 10.2, 4 x 3584 x 2304
// 6.0 against 6.2, 2 x 8192 x 1024 5.2 against 6.0, 1 x 131072 x 7168 147 against 153; but
// 4 x 8192 x 1024 6.5 against 5.9, 4 x 131072 x 1024 69 against 30, 1 x 49152 x 1024 19.0
// against 17.5.  At either border the two are within 5 %, and the grid stays far below
// the 2^32 threads of a launch.
inline bool rows_quant_ok(int64_t M, int64_t N, int64_t K) {
  return M <= 4 && M * ((K + 127) / 128 * 128) + (2 * M * K + 1023) / 1024 * 1024 <= kRowsQuantBytes &&
         (M * N <= ((int64_t)1 << 14) || M * M * M * N <= K * K / 128);
}

inline hipError_t launch_rows_quant(const TileArgs& a, const uint16_t* x, hipStream_t stream) {
  launch_rows_shape<true, kTileStore, 0>(a, x, stream);
  return hipGetLastError();
}

}  // namespace
}  // namespace bsfp4
