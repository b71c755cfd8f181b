// Tiled matrix product for bf16 and 8-bit integer operands, shared by the 8-bit
// GEMM, the gated feed-forward products and their backward pass.
//
//   acc[m, n] = sum_k A(m, k) B(n, k)
//
// bf16 and int8 are the same kernel: a 16-byte chunk is 8 bf16 or 16 int8
// values, v_mfma_f32_16x16x32_bf16 and v_mfma_i32_16x16x64_i8 each take one such
// chunk per lane and operand, and both run 16 cycles, so everything is laid out
// in bytes and only the instruction differs.  The part is power-limited under
// these products and the 16 x 16 forms take less power per operation than 32 x 32:
// from registers, on random operands, 1.95 PFLOP/s bf16 and 3.86 POP/s int8
// against 1.65 and 3.33 (measured).
//
// Each operand is stored either with its rows along K (a row of A is one m, K
// contiguous) or, for bf16, transposed (a row is one k): the backward pass reads
// the weight and the activations that way.  A transposed tile stays k-major in
// LDS and ds_read_b64_tr_b16 hands every lane its four consecutive k values, so
// no transposed copy is ever written.
//
// Structure: a BM x BN tile per workgroup of WGM x WGN waves, K in stages of 128
// bytes per row, RING LDS slots filled by direct-to-LDS buffer loads (1 KB each),
// the loads of the RING - 1 stages that follow in flight while a stage is multiplied.
// LDS layout of a stage, A first:
//   rows along K   [rows][8 chunks of 16 B], chunk c of row r at position
//                  c ^ tile_swz(r): the 16 rows of a fragment read hit
//                  distinct bank groups
//   transposed     [64 k][BM or BN values] in 32-byte units, exchanged by row
//                  (tile_tswz): the k rows of a transposing read hit distinct
//                  banks
// Both swizzles are applied to the global address of each lane's 16 bytes, as the
// LDS side of a direct load is always consecutive.
//
// Rows past the operand's end and chunks past K are read as zeros through the
// buffer range check (kBufOOB lanes), so any M, any N and any K of whole 16-byte
// chunks run through the same loop.
//
// Measured at 4096 x 4096 x 7168 (256 x 256 tiles): bf16 158 us, 1.52 PFLOP/s; int8
// 85.7 us, 2.81 POP/s (98, 2.45, on the slowest card seen).  The matrix cores are busy 62
// to 75 % of the time (counters: gated forward 62, int8 71, the gradients 73 and 75) at
// 1.7 to 1.9 GHz; the rest is the wait at each stage's barrier, which two slots of 64 KB
// do not cover, and the epilogue.
#pragma once

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "int8_rows.h"
#include "launchers.h"
#include "lds_dma.h"

namespace bsfp4 {
namespace {

constexpr int kTileStage = 128;  // bytes of K per row and stage (rows along K)
constexpr int kTileStageK = 64;  // k rows per stage (transposed bf16)

template <bool kInt8>
struct Mma;
template <>
struct Mma<false> {
  typedef v4f Acc;
  typedef float Elem;
  __device__ static __forceinline__ Acc run(v4i a, v4i b, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
};
template <>
struct Mma<true> {
  typedef v4i Acc;
  typedef int Elem;
  __device__ static __forceinline__ Acc run(v4i a, v4i b, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};

// ---- activations -----------------------------------------------------------
// sigmoid with the hardware exp2 and reciprocal (a few binary32 ulp; results
// are rounded to bf16)
__device__ __forceinline__ float sigmoid_f(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f));
}

// tanh form: 0.5 (1 + tanh u) = sigmoid(2 u), 2 u = kGeluC (g + 0.044715 g^3)
constexpr float kGeluC = 1.59576912160573071f;  // sqrt(8 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float act_value(int act, float g) {
  if (act == kActSilu) return g * sigmoid_f(g);
  if (act == kActGelu) return 0.5f * g * erfcf(g * -0.70710678118654752f);
  return g * sigmoid_f(kGeluC * (g + kGeluA * g * g * g));
}

// act(g) and act'(g)
__device__ __forceinline__ void act_value_grad(int act, float g, float& a, float& da) {
  if (act == kActSilu) {
    const float s = sigmoid_f(g);
    a = g * s;
    da = s * (1.0f + g * (1.0f - s));
  } else if (act == kActGelu) {
    const float cdf = 0.5f * erfcf(g * -0.70710678118654752f);
    a = g * cdf;
    da = cdf + g * 0.39894228040143268f * __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f);
  } else {
    const float s = sigmoid_f(kGeluC * (g + kGeluA * g * g * g));
    a = g * s;
    // s (1 - s) is 0 in binary32 beyond |g| = 10: the polynomial is held there
    const float c = fminf(fmaxf(g, -10.0f), 10.0f);
    da = s + c * s * (1.0f - s) * kGeluC * (1.0f + 3.0f * kGeluA * c * c);
  }
}

// ---- one operand of a tile -------------------------------------------------
// Position of 16-byte chunk c of row r inside its 128 bytes is c ^ tile_swz(r).  A
// fragment's read (row lane % 16, chunk lane / 16) is served 16 lanes at a time,
// lanes 0-3, 12-15 and 20-27 first, 4-11, 16-19 and 28-31 next: with r % 8 each of these
// sixteen meets other banks (r ^ r / 8 % 2 doubled every read; of a kernel's LDS cycles 1
// to 5 % are counted as conflicts, half were so).
__device__ __forceinline__ constexpr int tile_swz(int r) { return r & 7; }

// Transposed: 32-byte unit u (16 values) of k row k is kept at u ^ tile_tswz(k).  A
// transposing read takes, for each 16 lanes, one unit of four consecutive k rows;
// 32 lanes read the rows k .. k + 3 and k + 8 .. k + 11.  Rows of 256 bytes or more
// start at the same bank, those of 128 bytes (ROWS 64) alternate between two halves.
template <int ROWS>
__device__ __forceinline__ constexpr int tile_tswz(int k) {
  return 2 * (ROWS == 64 ? (k >> 1) & 1 : k & 3) + ((k >> 3) & 1);
}

// ROWS tile rows (m or n) of one operand, its 1 KB loads shared by WAVES waves
// (load q = wave * kLoads + j).
//   rows along K: load q holds tile rows 8q .. 8q + 7; lane l brings position
//     l % 8 of row 8q + l / 8.  With kPairs the tile rows are blocks of 16
//     alternating between two row ranges (gate and up), each its own buffer.
//   transposed: load q holds 512 / ROWS k rows.
template <int ROWS, bool kTrans, bool kPairs, int WAVES>
struct TileLoader {
  static constexpr int kBytes = ROWS * kTileStage;
  static constexpr int kLoads = kBytes / 1024 / WAVES;
  static_assert(kLoads * WAVES * 1024 == kBytes, "whole loads per wave");
  static_assert(!(kTrans && kPairs), "a gated weight has its rows along K");

  uint32_t off[kLoads];
  uint32_t c16[kTrans ? 1 : kLoads];  // byte position of the lane's chunk in the row's 128
  v4u32 rsrc[kPairs ? 2 : 1];
  const uint8_t* base;  // transposed: tile's first column of k row 0
  int64_t ld;
  int cols;             // transposed: bytes left of the tile's first column
  int q0;

  // rows along K: `p` the first tile row (`p2` that of the second range), `rows`
  // valid rows left.  transposed: `p` the operand, first column `first` of `rows`.
  __device__ __forceinline__ void init(const uint8_t* p, const uint8_t* p2, int64_t ld_, int rows, int first, int wave,
                                       int lane) {
    q0 = wave * kLoads;
    ld = ld_;
    if constexpr (kTrans) {
      base = p + (int64_t)first * 2;
      cols = first * 2;
      constexpr int kLanesRow = ROWS / 8;  // 16-byte pieces of a k row
#pragma unroll
      for (int j = 0; j < kLoads; j++) {
        const int k = (q0 + j) * (64 / kLanesRow) + lane / kLanesRow;
        const int pos = lane % kLanesRow;
        const int col = ((pos >> 1) ^ tile_tswz<ROWS>(k)) * 16 + (pos & 1) * 8;
        off[j] = first + col < rows ? (uint32_t)(k * ld + col * 2) : kBufOOB;
      }
    } else {
      const int lim = min(rows, kPairs ? ROWS / 2 : ROWS);
      rsrc[0] = make_rsrc4(p, (int64_t)lim * ld);
      if constexpr (kPairs) rsrc[1] = make_rsrc4(p2, (int64_t)lim * ld);
#pragma unroll
      for (int j = 0; j < kLoads; j++) {
        const int q = q0 + j, r = 8 * q + lane / 8;
        const int row = kPairs ? (q >> 2) * 16 + (r & 15) : r;
        c16[j] = (uint32_t)((lane & 7) ^ tile_swz(r)) * 16;
        off[j] = row < lim ? (uint32_t)(row * ld) + c16[j] : kBufOOB;
      }
    }
  }

  // Before the loads of the last stage, `left` bytes of K wide: chunks past K read as zeros.
  __device__ __forceinline__ void mask_tail(int left) {
    if constexpr (!kTrans) {
#pragma unroll
      for (int j = 0; j < kLoads; j++) off[j] = (int)c16[j] < left ? off[j] : kBufOOB;
    }
  }

  // The buffer of a stage (transposed: `k0` its first k row, `left` rows of it)
  __device__ __forceinline__ v4u32 stage_rsrc(int64_t k0, int64_t left) const {
    if constexpr (kTrans) return make_rsrc4(base + k0 * ld, min(left, (int64_t)kTileStageK) * ld - cols);
    else return rsrc[0];
  }

  // Load j of stage `st` into LDS at `lds`.
  __device__ __forceinline__ void issue(int j, int st, v4u32 r, uint32_t lds) const {
    if (kPairs && (((q0 + j) >> 1) & 1)) r = rsrc[kPairs ? 1 : 0];
    buf_lds16(r, off[j], kTrans ? 0u : (uint32_t)st * kTileStage, lds + (uint32_t)(q0 + j) * 1024);
  }
};

// Fragments of 16-row blocks from a stage in LDS: 16 bytes per lane, K chunk
// 4 kk + lane / 16 of row lane % 16 (kk 0, 1).
template <int ROWS, bool kTrans>
struct TileReader {
  // LDS byte offsets inside the operand's stage.  transposed: of blocks 0 .. 7 of
  // the wave's range (whose first block is a multiple of 8, or the range is short)
  static constexpr int kBlocks = 8;
  uint32_t off[kTrans ? kBlocks : 2];
  __device__ __forceinline__ void init(int block0, int lane) {
    const int lr = lane & 15, kg = lane >> 4;
    if constexpr (kTrans) {
      const int k = 8 * kg + (lr >> 2);
#pragma unroll
      for (int i = 0; i < kBlocks; i++)
        off[i] = (uint32_t)(k * ROWS * 2 + ((block0 + i) ^ tile_tswz<ROWS>(k)) * 32 + (lr & 3) * 8);
    } else {
#pragma unroll
      for (int kk = 0; kk < 2; kk++)
        off[kk] = (uint32_t)((block0 * 16 + lr) * kTileStage + (((4 * kk + kg) ^ tile_swz(lr)) * 16));
    }
  }
  __device__ __forceinline__ v4i read(const uint8_t* stage, int i, int kk) const {
    if constexpr (kTrans) {
      typedef short v4s __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4s lds_v4s;
      lds_v4s* p = (lds_v4s*)(const __attribute__((address_space(3))) uint8_t*)(stage + off[i] + kk * 32 * ROWS * 2);
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + ROWS);  // four k rows on (8 bytes per element)
      const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
      return v4i{(int)a.x, (int)a.y, (int)b.x, (int)b.y};
    } else {
      return *reinterpret_cast<const v4i*>(stage + off[kk] + i * 16 * kTileStage);
    }
  }
};

// ---- the kernel ------------------------------------------------------------
constexpr int kTileStore = 0;  // D = bf16 rows (scales and bias for 8-bit operands)
constexpr int kTileGated = 1;  // columns are gate / up pairs: act(gate) * up

struct TileArgs {
  const uint8_t* A;
  const uint8_t* B;
  int64_t lda, ldb;    // bytes from one stored row to the next
  int M;               // output rows
  int N;               // output columns (gated: of h; B holds N gate rows, then N up rows)
  int64_t kend;        // K in bytes (both operands along K) or in k rows (any transposed)
  const float* sa;     // 8-bit: scale per row of A
  const float* sb;     // 8-bit: scale per row of B
  const uint16_t* bias;  // [N] or null (store)
  uint16_t* D;         // [M, N]
  float* gate_up;      // gated: the sums [M, 2 N] or null
  int act;
  int m_base, n_base;  // first row and column of this launch
  int tiles_m, tiles_n, splits;
  void* part;          // splits > 1: float / int32 [splits][M][N or 2 N]
};

template <int BM, int BN, int RING>
constexpr int tile_smem() {
  const int ring = RING * (BM + BN) * kTileStage;
  const int out = BM * (BN * 2 + 16);
  return ring > out ? ring : out;
}

// Waves per SIMD that the LDS lets in: what the registers are sized for.  Every
// kernel has two at least: with the 512 registers of a single one the compiler keeps
// accumulators in the second bank and copies them around (measured 24 % slower, int8
// 128 x 128 with four slots on four waves against eight).
template <int BM, int BN, int RING, int WAVES>
constexpr int tile_waves_simd() {
  constexpr int w = 160 * 1024 / tile_smem<BM, BN, RING>() * WAVES / 4;
  static_assert(w >= 2, "two waves per SIMD");
  return w;
}

// Work item of a workgroup.  Workgroups are dispatched round-robin over the 8
// XCDs; consecutive items go to one XCD and run down bands of `band` tile rows, so
// an XCD's items share few A and B panels in its L2.
__device__ __forceinline__ void tile_item(const TileArgs& p, int item, int& tile_m, int& tile_n, int& split) {
  const int items = p.tiles_m * p.tiles_n * p.splits;
  // the first 8 * (items / 8) workgroups are remapped, the rest keep their index
  const int per = items / 8;
  if (item < per * 8) item = (item % 8) * per + item / 8;
  split = item % p.splits;
  const int tile = item / p.splits;
  constexpr int kBand = 4;
  const int band_tiles = kBand * p.tiles_n;
  const int band = tile / band_tiles, in_band = tile % band_tiles;
  const int rows = min(kBand, p.tiles_m - band * kBand);
  tile_m = band * kBand + in_band % rows;
  tile_n = in_band / rows;
}

// Work item `block` of p, in tile_smem bytes of LDS.
template <bool kInt8, int BM, int BN, int WGM, int WGN, int RING, bool kTransA, bool kTransB, int EPI>
__device__ __forceinline__ void tile_body(const TileArgs& p, int block, uint8_t* smem) {
  typedef Mma<kInt8> MM;
  constexpr int NT = 64 * WGM * WGN, WAVES = WGM * WGN;
  constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 16, TN = WN / 16;
  constexpr int kStageA = BM * kTileStage, kStage = (BM + BN) * kTileStage;
  constexpr bool kGated = EPI == kTileGated;
  static_assert(RING >= 2 && RING <= 4, "ring depth");
  static_assert(!kGated || TN % 2 == 0, "a wave holds pairs of gate and up blocks");
  static_assert(!kInt8 || (!kTransA && !kTransB), "8-bit operands have their rows along K");

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave % WGN, kg = lane >> 4, lr = lane & 15;
  int tile_m, tile_n, split;
  tile_item(p, block, tile_m, tile_n, split);
  constexpr int kCols = kGated ? BN / 2 : BN;  // output columns of a tile
  const int m0 = p.m_base + tile_m * BM, n0 = p.n_base + tile_n * kCols;

  constexpr int64_t kStep = (kTransA || kTransB) ? kTileStageK : kTileStage;
  const int total = (int)((p.kend + kStep - 1) / kStep);
  const int s0 = (int)((int64_t)total * split / p.splits), s1 = (int)((int64_t)total * (split + 1) / p.splits);

  TileLoader<BM, kTransA, false, WAVES> la;
  TileLoader<BN, kTransB, kGated, WAVES> lb;
  if constexpr (kTransA) la.init(p.A, nullptr, p.lda, p.M, m0, wave, lane);
  else la.init(p.A + (int64_t)m0 * p.lda, nullptr, p.lda, p.M - m0, 0, wave, lane);
  if constexpr (kTransB) lb.init(p.B, nullptr, p.ldb, p.N, n0, wave, lane);
  else lb.init(p.B + (int64_t)n0 * p.ldb, p.B + ((int64_t)p.N + n0) * p.ldb, p.ldb, p.N - n0, 0, wave, lane);
  // an operand along K beside a transposed one: K counted in bytes there
  const int64_t kend_a = !kTransA && kTransB ? p.kend * 2 : p.kend;
  const int64_t kend_b = !kTransB && kTransA ? p.kend * 2 : p.kend;
  static_assert(TM <= 8 && TN <= 8, "transposed readers hold eight blocks");
  TileReader<BM, kTransA> ra;
  TileReader<BN, kTransB> rb;
  ra.init(wm * TM, lane);
  rb.init(wn * TN, lane);
  const uint32_t lds0 = lds_offset(smem);
  typename MM::Acc acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[i][j] = typename MM::Acc{};

  // A stage is 2 kParts groups of MFMAs: two K halves kk, and in each the wave's
  // rows of A in kParts parts.  The fragments of the next group are read, and the
  // loads of the stage RING on issued, between a group's MFMAs.  The one barrier of
  // a stage stands late in its last group but one, where the wave has all fragments
  // of the stage in registers: past it every wave's loads of the next stage have
  // landed and the slot just read is free, so the last group already reads the next
  // stage and the MFMAs run on across it.
  constexpr int kParts = TM >= 2 ? 2 : 1, TP = TM / kParts, kGroups = 2 * kParts;
  constexpr int kMfma = TP * TN, kReads = TP + TN;
  constexpr int kIssues = decltype(la)::kLoads + decltype(lb)::kLoads;
  v4i fa[2][TP], fb[2][TN];
  // fragment r of group `grp`: its A rows, then, with a new kk, B's
  auto read_one = [&](int r, int slot, int grp) {
    const uint8_t* q = smem + slot * kStage;
    const int kk = grp / kParts, part = grp % kParts;
    if (r < TP) fa[grp & 1][r] = ra.read(q, part * TP + r, kk);
    else if (part == 0) fb[kk & 1][r - TP] = rb.read(q + kStageA, r - TP, kk);
  };
  v4u32 rsa, rsb;
  auto begin_issue = [&](int st) {  // before the loads of stage st
    if (st + 1 == total) {
      la.mask_tail((int)(kend_a - (int64_t)st * kTileStage));
      lb.mask_tail((int)(kend_b - (int64_t)st * kTileStage));
    }
    rsa = la.stage_rsrc((int64_t)st * kTileStageK, kend_a - (int64_t)st * kTileStageK);
    rsb = lb.stage_rsrc((int64_t)st * kTileStageK, kend_b - (int64_t)st * kTileStageK);
  };
  auto issue_one = [&](int j, int st, int in) {  // load j of stage st into slot `in`
    const uint32_t slot = lds0 + (uint32_t)in * kStage;
    if (j < decltype(la)::kLoads) la.issue(j, st, rsa, slot);
    else lb.issue(j - decltype(la)::kLoads, st, rsb, slot + kStageA);
  };
  // `flying`: loads, after those of the next stage, that may still be under way
  auto arrive = [&](auto flying) {
    // this wave's loads of the next stage and its last reads of this one
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(flying)::value) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // Position of the barrier among a stage's MFMAs, and of the loads after it: the memory
  // pipeline takes 1 KB in 17 clocks, so they are spread over most of a stage's time
  // and reach into the next stage's MFMAs (kNow of them do not); with two slots over
  // half of it, for they have to land within that stage.  Loads right behind the
  // barrier held the MFMAs up: bf16 777 x 4096 x 4096 on 256 x 256 tiles 79 -> 67 us, on
  // 128 x 128 34 -> 32 with these positions and tile_swz.
  constexpr int kStageMfma = kGroups * kMfma;
  constexpr int kBarrier = (kGroups - 2) * kMfma + (kMfma > 1 ? kMfma * 3 / 4 - 1 : 0);
  constexpr int kSpread = kStageMfma * (RING == 2 ? 8 : 15) / 16 - 1;
  constexpr int kNow = [] {
    int n = 0;
    while (n < kIssues && kBarrier + 1 + n * kSpread / kIssues < kStageMfma) n++;
    return n;
  }();
  static_assert(kBarrier + 1 + (kIssues - 1) * kSpread / kIssues - kStageMfma < kBarrier / kMfma * kMfma,
                "a stage's loads are issued before the next one's begin");
  // kLeft: stages that follow (RING: that many or more, so stage st + RING is issued)
  auto group = [&](auto left_c, int grp, int st, int slot) {
    constexpr int kLeft = decltype(left_c)::value;
    constexpr bool kNext = kLeft > 0, kAfter = kLeft >= RING;
    const int kk = grp / kParts, part = grp % kParts;
    const bool last = grp == kGroups - 1;
    if (kAfter && grp == kBarrier / kMfma) begin_issue(st + RING);
#pragma unroll
    for (int t = 0; t < kMfma; t++) {
      const int i = t / TN, j = t % TN;
      // the B fragment as first operand: a lane ends with four consecutive columns
      // of one row in its four registers
      acc[part * TP + i][j] = MM::run(fb[kk & 1][j], fa[grp & 1][i], acc[part * TP + i][j]);
      if (!last || kNext) {
#pragma unroll
        for (int r = 0; r < kReads; r++)
          if (r * (kMfma / 2) / kReads == t) read_one(r, !last ? slot : slot + 1 == RING ? 0 : slot + 1, (grp + 1) % kGroups);
      }
      const int q = grp * kMfma + t;
      if (kNext && q == kBarrier) arrive(std::integral_constant<int, (kLeft < RING ? kLeft - 1 : RING - 2) * kIssues>{});
#pragma unroll
      for (int l = 0; l < kIssues; l++) {
        const int at = kBarrier + 1 + l * kSpread / kIssues;
        if (kAfter && at == q) issue_one(l, st + RING, slot);
        // what is left of the stage before's
        if (kLeft >= RING - 1 && at - kStageMfma == q) issue_one(l, st - 1 + RING, slot == 0 ? RING - 1 : slot - 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto stage = [&](auto left_c, int st, int slot) {
#pragma unroll
    for (int grp = 0; grp < kGroups; grp++) group(left_c, grp, st, slot);
  };
  const int nst = s1 - s0;
  if (nst > 0) {
#pragma unroll
    for (int r = 0; r < RING; r++)
      if (r < nst) {
        begin_issue(s0 + r);
#pragma unroll
        for (int l = 0; l < (r == RING - 1 ? kNow : kIssues); l++) issue_one(l, s0 + r, r);
      }
    // the first stage has landed when the loads after it are all that is out
    if (nst >= RING) arrive(std::integral_constant<int, (RING - 2) * kIssues + kNow>{});
    else arrive(std::integral_constant<int, 0>{});
#pragma unroll
    for (int r = 0; r < kReads; r++) read_one(r, 0, 0);
    int st = s0, slot = 0;
    auto advance = [&] {
      st++;
      slot = slot + 1 == RING ? 0 : slot + 1;
    };
    for (; st + RING < s1; advance()) stage(std::integral_constant<int, RING>{}, st, slot);
    if constexpr (RING > 3) {
      if (st + 3 < s1) {
        stage(std::integral_constant<int, 3>{}, st, slot);
        advance();
      }
    }
    if constexpr (RING > 2) {
      if (st + 2 < s1) {
        stage(std::integral_constant<int, 2>{}, st, slot);
        advance();
      }
    }
    if (st + 1 < s1) {
      stage(std::integral_constant<int, 1>{}, st, slot);
      advance();
    }
    stage(std::integral_constant<int, 0>{}, st, slot);
  }

  // register e of block (i, j): row wm WM + 16 i + lr, tile column wn WN + 16 j + 4 kg + e;
  // gated: even j gate, odd j up, output column wn WN / 2 + 16 (j / 2) + 4 kg + e
  auto out_col = [&](int j) { return (kGated ? wn * (WN / 2) + (j / 2) * 16 : wn * WN + j * 16) + 4 * kg; };
  if (p.splits > 1) {
    const int64_t width = kGated ? 2 * (int64_t)p.N : p.N;
    float* dst = reinterpret_cast<float*>(p.part) + (int64_t)split * p.M * width;
#pragma unroll
    for (int i = 0; i < TM; i++) {
      const int m = m0 + wm * WM + i * 16 + lr;
      if (m >= p.M) continue;
#pragma unroll
      for (int j = 0; j < TN; j++) {
        const int n = n0 + out_col(j);
        if (n < p.N)
          *reinterpret_cast<uint4*>(dst + (int64_t)m * width + (kGated && (j & 1) ? p.N : 0) + n) =
              __builtin_bit_cast(uint4, acc[i][j]);
      }
    }
    return;
  }

  // bf16 through LDS: each lane's four-column runs into a row-major tile, then
  // whole 16-byte row segments per lane to memory
  constexpr int kPitch = kCols * 2 + 16;
  __syncthreads();  // the stages are done with
  auto flush = [&](uint16_t* dst, int64_t pitch) {
    __syncthreads();
    constexpr int kChunksRow = kCols / 8;
    for (int idx = tid; idx < BM * kChunksRow; idx += NT) {
      const int r = idx / kChunksRow, c = (idx % kChunksRow) * 8;
      if (m0 + r < p.M && n0 + c < p.N)
        *reinterpret_cast<uint4*>(dst + (int64_t)(m0 + r) * pitch + n0 + c) =
            *reinterpret_cast<const uint4*>(smem + r * kPitch + c * 2);
    }
  };
  float sa[TM];
#pragma unroll
  for (int i = 0; i < TM; i++) {
    const int m = m0 + wm * WM + i * 16 + lr;
    sa[i] = kInt8 && m < p.M ? p.sa[m] : 0.0f;
  }
  auto quad = [&](int i, int j, const float4& sb) -> float4 {
    const auto& a = acc[i][j];
    if constexpr (kInt8)
      return make_float4((float)a[0] * sa[i] * sb.x, (float)a[1] * sa[i] * sb.y, (float)a[2] * sa[i] * sb.z,
                         (float)a[3] * sa[i] * sb.w);
    else
      return make_float4(a[0], a[1], a[2], a[3]);
  };
  auto scales = [&](int n) -> float4 {  // of B rows n .. n + 3
    if constexpr (kInt8) return *reinterpret_cast<const float4*>(p.sb + n);
    else return make_float4(1.0f, 1.0f, 1.0f, 1.0f);
  };
  auto put4 = [&](int i, int c, const float4& v) {
    *reinterpret_cast<uint2*>(smem + (wm * WM + i * 16 + lr) * kPitch + c * 2) =
        make_uint2(pack_bf16x2_ieee(v.x, v.y), pack_bf16x2_ieee(v.z, v.w));
  };
  if constexpr (!kGated) {
#pragma unroll
    for (int j = 0; j < TN; j++) {
      const int c = out_col(j), n = min(n0 + c, p.N - 4);
      const float4 sb = scales(n);
      float4 bv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (kInt8 && p.bias) {
        const uint2 b = *reinterpret_cast<const uint2*>(p.bias + n);
        bv = make_float4(bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y));
      }
#pragma unroll
      for (int i = 0; i < TM; i++) {
        float4 v = quad(i, j, sb);
        if (kInt8) v = make_float4(v.x + bv.x, v.y + bv.y, v.z + bv.z, v.w + bv.w);
        put4(i, c, v);
      }
    }
    flush(p.D, p.N);
  } else {
#pragma unroll
    for (int j = 0; j < TN; j += 2) {
      const int c = out_col(j), n = min(n0 + c, p.N - 4);
      const float4 sg = scales(n), su = scales(p.N + n);
#pragma unroll
      for (int i = 0; i < TM; i++) {
        const float4 gv = quad(i, j, sg), uv = quad(i, j + 1, su);
        put4(i, c, make_float4(act_value(p.act, gv.x) * uv.x, act_value(p.act, gv.y) * uv.y,
                               act_value(p.act, gv.z) * uv.z, act_value(p.act, gv.w) * uv.w));
      }
    }
    flush(p.D, p.N);
    if constexpr (!kInt8) {
      if (p.gate_up) {  // the sums as they are, gate then up, in whole row segments as well
        constexpr int kPitch4 = kCols * 4 + 16;
        static_assert(BM * kPitch4 <= tile_smem<BM, BN, RING>(), "a binary32 half tile fits in LDS");
#pragma unroll
        for (int half = 0; half < 2; half++) {
          __syncthreads();
#pragma unroll
          for (int j = half; j < TN; j += 2)
#pragma unroll
            for (int i = 0; i < TM; i++)
              *reinterpret_cast<v4f*>(smem + (wm * WM + i * 16 + lr) * kPitch4 + out_col(j) * 4) = acc[i][j];
          __syncthreads();
          constexpr int kChunksRow = kCols / 4;
          for (int idx = tid; idx < BM * kChunksRow; idx += NT) {
            const int r = idx / kChunksRow, c = (idx % kChunksRow) * 4;
            if (m0 + r < p.M && n0 + c < p.N)
              *reinterpret_cast<float4*>(p.gate_up + (int64_t)(m0 + r) * 2 * p.N + half * p.N + n0 + c) =
                  *reinterpret_cast<const float4*>(smem + r * kPitch4 + c * 4);
          }
        }
      }
    }
  }
}

template <bool kInt8, int BM, int BN, int WGM, int WGN, int RING, bool kTransA, bool kTransB, int EPI>
__global__ void __launch_bounds__(64 * WGM * WGN, (tile_waves_simd<BM, BN, RING, WGM * WGN>()))
    tile_gemm(const TileArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[tile_smem<BM, BN, RING>()];
  tile_body<kInt8, BM, BN, WGM, WGN, RING, kTransA, kTransB, EPI>(p, blockIdx.x, smem);
}

// ---- split K ---------------------------------------------------------------
// Sums the splits' partials in split order (8-bit: exact integers) and finishes
// the rows as the tile's epilogue would.  One thread: eight output columns.
template <bool kInt8, int EPI>
__global__ void __launch_bounds__(256)
    tile_reduce(const TileArgs p) {
  typedef typename Mma<kInt8>::Elem T;
  constexpr bool kGated = EPI == kTileGated;
  const int64_t width = kGated ? 2 * (int64_t)p.N : p.N;
  const int64_t mn = (int64_t)p.M * width;
  const int64_t chunks = p.N / 8, all = (int64_t)p.M * chunks;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < all; idx += stride) {
    const int64_t m = idx / chunks;
    const int n = (int)(idx - m * chunks) * 8;
    auto sum8 = [&](int64_t col, const float* sb, float (&v)[8]) {
      const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.part) + m * width + col);
      T t[8] = {};
#pragma unroll 4
      for (int s = 0; s < p.splits; s++) {
        const uint4 a = src[s * (mn / 4)], b = src[s * (mn / 4) + 1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 8; k++) t[k] += __builtin_bit_cast(T, w[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; k++) v[k] = kInt8 ? (float)t[k] * p.sa[m] * sb[col + k] : (float)t[k];
    };
    float v[8];
    sum8(n, p.sb, v);
    if constexpr (kGated) {
      float u[8];
      sum8(p.N + n, p.sb, u);
      if (p.gate_up) {
        float4* dg = reinterpret_cast<float4*>(p.gate_up + m * width + n);
        float4* du = reinterpret_cast<float4*>(p.gate_up + m * width + p.N + n);
        dg[0] = make_float4(v[0], v[1], v[2], v[3]);
        dg[1] = make_float4(v[4], v[5], v[6], v[7]);
        du[0] = make_float4(u[0], u[1], u[2], u[3]);
        du[1] = make_float4(u[4], u[5], u[6], u[7]);
      }
#pragma unroll
      for (int k = 0; k < 8; k++) v[k] = act_value(p.act, v[k]) * u[k];
    } else if (kInt8 && p.bias) {
      float b[8];
      unpack8(*reinterpret_cast<const uint4*>(p.bias + n), b);
#pragma unroll
      for (int k = 0; k < 8; k++) v[k] += b[k];
    }
    *reinterpret_cast<uint4*>(p.D + m * (int64_t)p.N + n) = pack8(v);
  }
}

// ---- planning --------------------------------------------------------------
// The kernels of a product.  A large tile does the most with each byte in LDS; a
// small one with more slots has more loads under way per multiplied stage, which is
// what a product of few workgroups waits for.
enum TileKind { kTile256, kTile256x128, kTile128, kTile128Deep, kTile64x128, kTile64, kTileKinds };

struct TilePlan {
  TileKind kind;
  int splits;
  // Whole rounds of workgroups only: the output rows (or columns, of weight rows)
  // from `cut` on are a second launch of kernel `rest`.  0: everything in one.
  int64_t cut_m, cut_n;
  TileKind rest;
  double us;  // the estimate
};

// Kernel and K split of an M x N (x K bytes) product: the choice with the least
// estimated time.  A stage takes a workgroup us[c - 1] microseconds when c share a
// compute unit, its start and end round_us; a split's second kernel costs kSplitUs
// and its partials their bytes.  The figures are a least-squares fit to 2034 timed
// (shape, kernel, split) combinations (profiles/tile_plan_timings.csv), M 48 .. 4096, weights of 1536 x 2048 .. 14336 x
// 4096, bf16 and int8 (9 % rms); the plan's choice is 0.4 % slower than the best of
// each shape on average, 8 % at worst.  N counts weight rows (gated: both halves).
struct TileCost {
  int bm, bn, per_cu;
  double us[2], round_us;
};
constexpr TileCost kTileCosts[kTileKinds] = {{256, 256, 1, {1.03, 0}, 4.1},  {256, 128, 1, {0.62, 0}, 3.0},
                                             {128, 128, 2, {0.542, 0.767}, 2.1}, {128, 128, 1, {0.423, 0}, 2.7},
                                             {64, 128, 2, {0.279, 0.533}, 2.6}, {64, 64, 2, {0.214, 0.342}, 2.3}};

// Estimated time of `items` workgroups of `stages` stages each.
inline double tile_time(const TileCost& c, int64_t items, double stages, int cus) {
  const int64_t slots = (int64_t)cus * c.per_cu, full = items / slots, rest = (items % slots + cus - 1) / cus;
  return c.round_us + full * stages * c.us[c.per_cu - 1] + (rest ? stages * c.us[rest - 1] : 0.0);
}

inline TilePlan plan_tile(int64_t M, int64_t N, int64_t kbytes, int cus) {
  constexpr double kSplitUs = 3.8, kPartBytesUs = 5.0e6;
  const int64_t stages = (kbytes + kTileStage - 1) / kTileStage;
  auto tiles = [](const TileCost& c, int64_t m, int64_t n) { return ((m + c.bm - 1) / c.bm) * ((n + c.bn - 1) / c.bn); };
  TilePlan best{kTile256, 1, 0, 0, kTile256, 1e300};
  auto consider = [&](const TilePlan& pl) {
    if (pl.us < best.us * 0.999) best = pl;
  };
  for (int c = 0; c < kTileKinds; c++) {
    const TileCost& cd = kTileCosts[c];
    const int64_t all = tiles(cd, M, N), slots = (int64_t)cus * cd.per_cu;
    for (int sp = 1; sp <= 16; sp++) {
      if (sp > 1 && (stages / sp < 4 || all * (sp - 1) >= slots)) break;
      double t = tile_time(cd, all * sp, (double)((stages + sp - 1) / sp), cus);
      if (sp > 1) t += kSplitUs + 2.0 * sp * M * N * 4 / kPartBytesUs;
      consider(TilePlan{(TileKind)c, sp, 0, 0, kTile256, t});
    }
    // a part-filled last round (896 tiles of 256 x 256 on 256 units: 3.5 rounds) goes
    // to smaller tiles: bf16 gated with its sums kept, 4096 x 14336 x 4096, 412 -> 382
    // us, a weight's gradient 14336 x 4096 x 4096 358 -> 343
    const int64_t full = all / slots * slots;
    if (c > kTile128 || full == 0 || full == all) continue;
    const int64_t tm = (M + cd.bm - 1) / cd.bm, tn = (N + cd.bn - 1) / cd.bn;
    for (int dir = 0; dir < 2; dir++) {
      const int64_t lines = full / (dir ? tm : tn);  // whole tile rows (0) or columns (1) of the main part
      if (lines == 0) continue;
      const int64_t cut = lines * (dir ? cd.bn : cd.bm);
      const double t_main = tile_time(cd, lines * (dir ? tm : tn), (double)stages, cus);
      for (int r = 0; r < kTileKinds; r++) {
        const TileCost& rd = kTileCosts[r];
        const int64_t left = dir ? tiles(rd, M, N - cut) : tiles(rd, M - cut, N);
        consider(TilePlan{(TileKind)c, 1, dir ? 0 : cut, dir ? cut : 0, (TileKind)r,
                          t_main + tile_time(rd, left, (double)stages, cus)});
      }
    }
  }
  return best;
}

inline size_t tile_workspace(const TilePlan& pl, int64_t M, int64_t N) {
  return pl.splits > 1 ? (size_t)pl.splits * M * N * 4 : 0;
}

template <bool kInt8, bool kTransA, bool kTransB, int EPI>
hipError_t launch_tile_part(const TileArgs& a, TileKind kind, hipStream_t stream) {
  const unsigned grid = (unsigned)((int64_t)a.tiles_m * a.tiles_n * a.splits);
#define BSFP4_TILE(BM, BN, WGM, WGN, RING) \
  tile_gemm<kInt8, BM, BN, WGM, WGN, RING, kTransA, kTransB, EPI><<<grid, 64 * WGM * WGN, 0, stream>>>(a)
  switch (kind) {
    case kTile256: BSFP4_TILE(256, 256, 2, 4, 2); break;
    case kTile256x128: BSFP4_TILE(256, 128, 4, 2, 3); break;
    case kTile128: BSFP4_TILE(128, 128, 2, 2, 2); break;
    case kTile128Deep: BSFP4_TILE(128, 128, 2, 4, 4); break;
    case kTile64x128: BSFP4_TILE(64, 128, 2, 2, 3); break;
    default: BSFP4_TILE(64, 64, 2, 2, 4); break;
  }
#undef BSFP4_TILE
  return hipGetLastError();
}

template <bool kInt8, bool kTransA, bool kTransB, int EPI>
hipError_t launch_tile(TileArgs a, const TilePlan& pl, hipStream_t stream) {
  constexpr int kHalf = EPI == kTileGated ? 2 : 1;  // weight rows per output column
  const int64_t brows = kHalf * (int64_t)a.N;
  auto part = [&](TileKind kind, int64_t m0, int64_t m1, int64_t n0, int64_t n1) {
    const TileCost& c = kTileCosts[kind];
    a.m_base = (int)m0;
    a.n_base = (int)(n0 / kHalf);
    a.tiles_m = (int)((m1 - m0 + c.bm - 1) / c.bm);
    a.tiles_n = (int)((n1 - n0 + c.bn - 1) / c.bn);
    return launch_tile_part<kInt8, kTransA, kTransB, EPI>(a, kind, stream);
  };
  a.splits = pl.splits;
  const int64_t m1 = pl.cut_m ? pl.cut_m : a.M, n1 = pl.cut_n ? pl.cut_n : brows;
  hipError_t e = part(pl.kind, 0, m1, 0, n1);
  if (e == hipSuccess && m1 < a.M) e = part(pl.rest, m1, a.M, 0, brows);
  if (e == hipSuccess && n1 < brows) e = part(pl.rest, 0, a.M, n1, brows);
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t items = (int64_t)a.M * (a.N / 8);
  tile_reduce<kInt8, EPI><<<(unsigned)std::min<int64_t>((items + 255) / 256, 8192), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace
}  // namespace bsfp4
