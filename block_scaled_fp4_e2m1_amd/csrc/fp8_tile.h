// Tiled matrix product of E4M3 operands with a scale for each block of 128 along K, dense and grouped by
// expert:
//
//   D[m, n] = sum_b sa[b, m] sb[b, n] P_b[m, n],   P_b[m, n] = sum_{k in block b} A[m, k] B[n, k]
//
// sb is one value per 128 rows of B (weights) or one per row (both operands quantised along K: a weight's
// gradient).  A stage of the K loop is one block: 128 bytes of every row, one v_mfma_f32_16x16x128_f8f6f4 per 16 x 16
// block started from zero, and P_b is added into the binary32 sums by vector FMAs, each P_b times the product of
// its two scales.  The FMAs of a block run while the matrix core works on the blocks after it.
//
// The loads, the LDS layout and the ring with one barrier per stage are those of tile_gemm.  A stage's scales come
// with it: every wave loads 64 of them (4 bytes a lane) into the stage's LDS slot, those of A's rows first, then
// those of B's rows; sa lies block by block ([K / 128, rows]), so that 64 rows' are two cache lines.
//
// Measured: 4096 x 4096 x 7168 on 256 x 256 tiles 99 us hot (2.4 PFLOP/s; MFMAs alone 69, without the FMAs 94, without
// loads 85), 105-108 behind other data, matrix cores busy 63 %, vector units 51 %.  With a scale per row of B each value
// takes a second multiply: 128 us on 256 x 128, busy 47 % and 66 %.  128 experts of 4096 x 4096, 64 rows each 401 us
// (5.3 TB/s of weights), 256 rows 607, 512 rows 1090 (2 PFLOP/s).
//
// Grouped: rows are sorted by expert, offsets[e] the first of expert e.  Row tiles start at an expert's first row;
// each workgroup finds the expert of its tile from the offsets.  A's rows may be gathered through an index.
#pragma once

#include "fp8_rows.h"
#include "tile_gemm.h"

namespace bsfp4 {
namespace {

constexpr int kFp8Bf16 = 0;   // D = bf16 rows, plus a bias
constexpr int kFp8F32 = 1;    // D = binary32 rows
constexpr int kFp8Gated = 2;  // columns are gate / up pairs: silu(gate) * up, quantised in blocks of 128 columns

struct Fp8Args {
  const uint8_t* A;      // [a_rows, K]
  const float* sa;       // [kb, a_rows]
  const uint8_t* B;      // [N, K] (gated: N gate rows, then N up rows), one per expert
  const float* sb;       // [ceil(rows of B / 128), kb] per expert, or (kRowB) [kb, N]
  const uint16_t* bias;  // [N] or null
  void* D;               // [M, N]
  uint8_t* q;            // gated: codes [M, N] and
  float* s;              // scales [N / 128, M]
  float* part;           // splits > 1: [splits][M][N]
  int64_t a_rows;
  int64_t K;             // bytes of a row
  int64_t b_stride, sb_stride;  // from one expert's weight (scales) to the next
  const int32_t* a_index;  // grouped: row of A that a row reads (outside [0, a_rows): zeros), or null
  const int32_t* offsets;  // grouped: [E + 1]
  int E;
  int M, N, kb;
  int m_base, n_base, tiles_m, tiles_n, splits;
};

template <int BM, int BN, int WAVES>
constexpr int fp8_slot() {
  return (BM + BN) * kTileStage + WAVES * 256;
}

template <int BM, int BN, int RING, int WAVES, int EPI>
constexpr int fp8_smem() {
  const int ring = RING * fp8_slot<BM, BN, WAVES>();
  const int out = EPI == kFp8Bf16 ? BM * (BN * 2 + 16) : EPI == kFp8F32 ? 0 : BM * (BN / 2 + 16) + BM * 16;
  return ring > out ? ring : out;
}

template <int BM, int BN, int RING, int WAVES, int EPI>
constexpr int fp8_waves_simd() {
  constexpr int w = 160 * 1024 / fp8_smem<BM, BN, RING, WAVES, EPI>() * WAVES / 4;
  static_assert(w >= 1, "fits in LDS");
  return w < 2 ? 2 : w;
}

// The experts' row tiles: those of expert e cover rows [offsets[e], offsets[e + 1]), those behind the last expert's rows
// are expert E's.  Offsets are held to [0, M], whatever the caller's list says.
struct Fp8Group {
  int e, row0, row1;
};
template <int BM>
struct Fp8Groups {
  const int32_t* offsets;
  int E, M;
  // tiles of expert e0 + lane, its rows in lo, hi
  __device__ __forceinline__ int tiles(int e, int& lo, int& hi) const {
    lo = hi = M;
    if (e <= E) {
      lo = min(max(offsets[e], 0), M);
      if (e < E) hi = min(max(offsets[e + 1], 0), M);
    }
    return hi > lo ? (hi - lo + BM - 1) / BM : 0;
  }
  // how many there are
  __device__ __forceinline__ int count() const {
    int n = 0, lo, hi;
    for (int e = threadIdx.x & 63; e <= E; e += 64) n += tiles(e, lo, hi);
    return __builtin_amdgcn_readfirstlane(lanes_reduce<6>(n, [](int a, int b) { return a + b; }));
  }
  // tile `tile` < count()
  __device__ __forceinline__ Fp8Group find(int tile) const {
    const int lane = threadIdx.x & 63;
    int before = 0;  // tiles of the experts of earlier turns
    for (int e0 = 0; e0 <= E; e0 += 64) {
      int lo, hi;
      const int n = tiles(e0 + lane, lo, hi);
      int upto = n;  // tiles of this turn's experts up to this lane's
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const int o = __shfl_up(upto, s, 64);
        if (lane >= s) upto += o;
      }
      const uint64_t past = __ballot(before + upto > tile);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        const int first = before + __shfl(upto - n, l, 64), of = __shfl(n, l, 64);
        const int from = __shfl(lo, l, 64), to = __shfl(hi, l, 64);
        // alike in size: tiles that run in step read the expert's weight out of L2 together
        const int step = (to - from + of - 1) / of, row0 = from + (tile - first) * step;
        return Fp8Group{__builtin_amdgcn_readfirstlane(e0 + l), __builtin_amdgcn_readfirstlane(row0),
                        __builtin_amdgcn_readfirstlane(min(row0 + step, to))};
      }
      before += __shfl(upto, 63, 64);
    }
    return Fp8Group{E + 1, 0, 0};
  }
};

// At most this many row tiles: every expert with rows has one that may be part-filled.
inline int64_t fp8_group_tiles(int64_t M, int64_t E, int bm) {
  const int64_t n = std::min(E + 1, M);
  return (M - n) / bm + n;
}

typedef int v8i32 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma_fp8(v8i32 a, v8i32 b) {
  // both operands E4M3, no scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// The same on binary16 (E4M3 values are exact in it), whose matrix instructions keep all of a product: for values that are
// rounded to codes again, where the other's cut turns some codes over (binary32 sums in another order only those within their
// roundings of a border).  Four times the matrix cores' time, and the conversions: where a weight's bytes are what a kernel
// waits for.
__device__ __forceinline__ v4f mfma_fp8_wide(v8i32 a, v8i32 b) {
  typedef _Float16 v2 __attribute__((ext_vector_type(2)));
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  auto wide = [](int lo, int hi) {
    const v2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false), p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const v2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false), p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return v8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  };
  v4f p{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int t = 0; t < 4; t++)
    p = __builtin_amdgcn_mfma_f32_16x16x32_f16(wide(a[2 * t], a[2 * t + 1]), wide(b[2 * t], b[2 * t + 1]), p, 0, 0, 0);
  return p;
}

__device__ __forceinline__ v8i32 fp8_frag(v4i lo, v4i hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

__device__ __forceinline__ float silu_f(float g) { return g * sigmoid_f(g); }

// What a tile is: rows m0 .. m1 - 1 (BM of them at most), columns from n0, its part of K, its expert's weight.
struct Fp8Tile {
  int m0, m1, n0, split;
  const uint8_t* B;
  const float* sb;
};

// CM: the rows that are multiplied; BM - CM more, which there are not, are only loaded (as zeros), so that each wave's
// loads are whole.
template <int BM, int BN, int WGM, int WGN, int RING, bool kRowB, int EPI, bool kGrouped, int CM = BM>
__device__ __forceinline__ void fp8_body(const Fp8Args& p, const Fp8Tile& tile, uint8_t* smem) {
  constexpr int NT = 64 * WGM * WGN, WAVES = WGM * WGN;
  constexpr int WM = CM / WGM, WN = BN / WGN, TM = WM / 16, TN = WN / 16;
  constexpr int kStageA = BM * kTileStage, kSlot = fp8_slot<BM, BN, WAVES>(), kScales = (BM + BN) * kTileStage;
  constexpr bool kGated = EPI == kFp8Gated;
  constexpr int kCols = kGated ? BN / 2 : BN;  // output columns of a tile
  constexpr int kLoadsA = BM / 8 / WAVES, kLoadsB = BN / 8 / WAVES, kIssues = kLoadsA + kLoadsB + 1;
  static_assert(kLoadsA * WAVES * 8 == BM && kLoadsB * WAVES * 8 == BN, "whole loads per wave");
  static_assert(BM + BN <= 64 * WAVES, "one load of scales per wave");
  static_assert(BM % 64 == 0 && BN % 64 == 0, "a wave's scales are all of one operand");
  static_assert(!kGated || (TN % 2 == 0 && kCols == kFp8Block && !kRowB), "a quantised block per tile row");
  static_assert(WN <= 128 && 128 % WN == 0, "a wave's columns are inside one block of B");

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave % WGN, kg = lane >> 4, lr = lane & 15;
  const int m0 = tile.m0, m1 = tile.m1, n0 = tile.n0, split = tile.split;
  const uint8_t* const Bp = tile.B;
  const float* const sbp = tile.sb;
  const int s0 = (int)((int64_t)p.kb * split / p.splits), s1 = (int)((int64_t)p.kb * (split + 1) / p.splits);
  const int K = (int)p.K;

  // ---- a stage: kGroups groups of TP rows of blocks x TN, B's fragments held for the stage, A's read a group ahead.
  constexpr int TP = TM == 4 && RING == 2 ? 2 : 1, kGroups = TM / TP, kMfma = TP * TN;
  constexpr int kStageMfma = kGroups * kMfma;
  // The next stage's first fragments go where the last group's are not: with an odd number of groups the places of
  // A's fragments are exchanged from stage to stage, which takes its code twice (and two stages at least).
  constexpr bool kOdd = kGroups % 2 != 0;
  static_assert(kGroups >= 2, "a group is read ahead");
  // With two slots a stage's own slot is filled again while it is read: past kFree, a first barrier, all waves hold B's
  // fragments and A's of the first half of their rows, so B's rows, those rows and the scales of stage st + 2 may come;
  // the rest past the stage's barrier.  (All of it past the one barrier: a stage's loads had too little time to land.)
  constexpr bool kTwoStep = RING == 2 && kGroups >= 4;
  constexpr int kFree = std::max(kMfma - 1, (TM / 2 / TP - 2) * kMfma + kMfma / 2);

  // ---- loads of 8 rows each: B's, then A's (kTwoStep: the half of A's rows that is free first, then the others)
  uint32_t offa[kLoadsA], offb[kLoadsB];
  const uint32_t c16 = (uint32_t)((lane & 7) ^ tile_swz(lane / 8)) * 16;  // byte position of the lane's chunk in a row's 128
  constexpr int kEarlyA = kTwoStep ? CM * kLoadsA / BM / 2 : 0, kLateA = kLoadsA - kEarlyA;
  constexpr int kEarlyRows = kEarlyA * WAVES / WGM * 8;  // of each wave row's WM
  static_assert(kEarlyRows <= WM / 2 && kEarlyRows % 8 == 0, "early rows are free early");
  auto first_row_a = [&](int j) {  // of this wave's load j
    const bool early = j < kEarlyA;
    const int unit = early ? wave * kEarlyA + j : wave * kLateA + j - kEarlyA;
    const int per = (early ? kEarlyRows : WM - kEarlyRows) / 8;  // loads of a wave row
    if (CM < BM && unit >= WGM * per) return CM + (unit - WGM * per) * 8;
    return unit / per * WM + (early ? 0 : kEarlyRows) + unit % per * 8;
  };
  const bool gather = kGrouped && p.a_index != nullptr;
  const v4u32 ra = gather ? make_rsrc4(p.A, p.a_rows * p.K)
                          : make_rsrc4(p.A + (int64_t)m0 * p.K, (int64_t)min(BM, m1 - m0) * p.K);
  const int bcols = min(kCols, p.N - n0);
  const v4u32 rb0 = make_rsrc4(Bp + (int64_t)n0 * p.K, (int64_t)bcols * p.K);
  const v4u32 rb1 = kGated ? make_rsrc4(Bp + ((int64_t)p.N + n0) * p.K, (int64_t)bcols * p.K) : rb0;
  auto a_row = [&](int r) -> int64_t {  // tile row r in A, from A's first row (gather) or the tile's; -1: none
    if (m0 + r >= m1) return -1;
    if (!gather) return r;
    const int src = p.a_index[m0 + r];
    return src >= 0 && src < p.a_rows ? src : -1;
  };
#pragma unroll
  for (int j = 0; j < kLoadsA; j++) {
    const int64_t row = a_row(first_row_a(j) + lane / 8);
    offa[j] = row >= 0 ? (uint32_t)(row * p.K) + c16 : kBufOOB;
  }
#pragma unroll
  for (int j = 0; j < kLoadsB; j++) {
    const int q = wave * kLoadsB + j, r = 8 * q + lane / 8;
    const int row = kGated ? (q >> 2) * 16 + (r & 15) : r;
    offb[j] = row < bcols ? (uint32_t)(row * p.K) + c16 : kBufOOB;
  }
  // scales: wave w loads those of tile rows 64 w .. of A, then of B (gated: of a column's gate, then its up row)
  const uint8_t* scale_base;
  int64_t scale_step, scale_bytes, scale_less;  // from one stage's to the next: base, and bytes left behind it
  uint32_t offs;
  if (wave * 64 < BM) {
    const int64_t row = a_row(wave * 64 + lane);
    scale_base = reinterpret_cast<const uint8_t*>(p.sa + (gather ? 0 : m0));
    scale_step = p.a_rows * 4;
    scale_bytes = (p.a_rows - (gather ? 0 : m0)) * 4;
    scale_less = 0;
    offs = row >= 0 ? (uint32_t)(row * 4) : kBufOOB;
  } else {
    const int c = wave * 64 - BM + lane;  // row of B's part of the tile; past BN: none
    scale_base = reinterpret_cast<const uint8_t*>(sbp);
    if constexpr (kRowB) {
      scale_step = (int64_t)p.N * 4;
      scale_bytes = (int64_t)p.N * 4;
      scale_less = 0;
      offs = c < BN && n0 + c < p.N ? (uint32_t)(n0 + c) * 4 : kBufOOB;
    } else {
      // gated: entries 0 .. kCols - 1 the gate rows', kCols .. the up rows'
      const int col = kGated ? c % kCols : c;
      const int64_t row = (int64_t)n0 + col + (kGated && c >= kCols ? p.N : 0);
      const int64_t nb = ((int64_t)p.N * (kGated ? 2 : 1) + kFp8Block - 1) / kFp8Block;
      scale_step = 4;
      scale_bytes = nb * p.kb * 4;
      scale_less = 4;
      offs = c < BN && col < bcols ? (uint32_t)(row / kFp8Block * p.kb) * 4 : kBufOOB;
    }
  }
  const uint32_t lds0 = lds_offset(smem);
  TileReader<BM, false> reada;
  TileReader<BN, false> readb;
  reada.init(wm * TM, lane);
  readb.init(wn * TN, lane);

  v4u32 rss;
  auto begin_issue = [&](int st) {  // before the loads of stage st
    // chunks past K read as zeros.  No branch: the compiler would sink a stage's FMAs behind it.
    const uint32_t past = st + 1 == p.kb && (int)c16 >= K - st * kTileStage ? kBufOOB : 0u;
#pragma unroll
    for (int j = 0; j < kLoadsA; j++) offa[j] |= past;
#pragma unroll
    for (int j = 0; j < kLoadsB; j++) offb[j] |= past;
    rss = make_rsrc4(scale_base + st * scale_step, scale_bytes - st * scale_less);
  };
  auto issue_one = [&](int j, int st, int in) {  // load j of stage st into slot `in`
    const uint32_t slot = lds0 + (uint32_t)in * kSlot, soff = (uint32_t)st * kTileStage;
    if (j == 0) buf_lds4(rss, offs, 0u, slot + kScales + (uint32_t)wave * 256);
    else if (j <= kLoadsB) {
      const int q = wave * kLoadsB + j - 1;
      buf_lds16(kGated && ((q >> 1) & 1) ? rb1 : rb0, offb[j - 1], soff, slot + kStageA + (uint32_t)q * 1024);
    } else {
      const int i = j - 1 - kLoadsB;
      buf_lds16(ra, offa[i], soff, slot + (uint32_t)first_row_a(i) * kTileStage);
    }
  };
  auto arrive = [&](auto flying) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(flying)::value) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // ---- multiplication.  In the last group, past the barrier, the next stage's first fragments of A are read and, as
  // each of B's is done with, the next stage's.  The barrier stands in the last group but one, where the wave has read
  // all of the stage.
  // MFMAs from a block's own to its FMAs: with fewer than three between, the wave stands until the result is there
  // (one wave, per MFMA and four FMAs: 64 clocks right behind it, 43, 36.5 with three; the MFMA alone takes 32).  The last
  // ones' FMAs run in the next stage.
  constexpr int kLag = 3;
  static_assert(kStageMfma % (kLag + 1) == 0, "the pending products keep their registers from stage to stage");
  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  v8i32 fa[2][TP], fb[TN];
  constexpr int kSb = kGated ? 2 : 1;
  struct {
    float a[TM], b[kSb];
    v4f row_b[kRowB ? TN : 1];
  } sc;
  v4f prod[kLag + 1];
  // rows whose last FMAs are done when a stage's last MFMA is issued: their next scales are read then
  constexpr int kEarly = kMfma > kLag ? TM - TP : 0;
  float pend[kRowB ? 1 : kLag];  // scales of the pending products
  v4f pend_row[kRowB ? kLag : 1];
#pragma unroll
  for (int u = 0; u < kLag; u++) {
    prod[kLag - u] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    pend[kRowB ? 0 : u] = 0.0f;
    pend_row[kRowB ? u : 0] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }

  auto read_a = [&](int r, int slot, int grp, int place) {
    const uint8_t* q = smem + slot * kSlot;
    fa[place][r] = fp8_frag(reada.read(q, grp * TP + r, 0), reada.read(q, grp * TP + r, 1));
  };
  auto read_b = [&](int j, int slot) {
    const uint8_t* q = smem + slot * kSlot + kStageA;
    fb[j] = fp8_frag(readb.read(q, j, 0), readb.read(q, j, 1));
  };
  auto read_scales_a = [&](int slot, int i0, int i1) {
    const float* q = reinterpret_cast<const float*>(smem + slot * kSlot + kScales);
#pragma unroll
    for (int i = i0; i < i1; i++) sc.a[i] = q[wm * WM + i * 16 + lr];
  };
  auto read_scales_b = [&](int slot, auto& to) {
    const float* q = reinterpret_cast<const float*>(smem + slot * kSlot + kScales) + BM;
    if constexpr (kRowB) {
#pragma unroll
      for (int j = 0; j < TN; j++) to.row_b[j] = *reinterpret_cast<const v4f*>(q + wn * WN + j * 16 + 4 * kg);
    } else if constexpr (kGated) {
      to.b[0] = q[wn * (WN / 2)];
      to.b[1] = q[kCols + wn * (WN / 2)];
    } else {
      to.b[0] = q[wn * WN];
    }
  };
  // MFMA q of a stage: group q / kMfma, in it column t / TP, row t % TP (t = q % kMfma)
  auto row_of = [](int q) { return q / kMfma * TP + q % kMfma % TP; };
  auto col_of = [](int q) { return q % kMfma / TP; };
  auto scale = [&](int q) { return sc.a[row_of(q)] * sc.b[kGated ? col_of(q) & 1 : 0]; };
  auto add = [&](int q) {  // MFMA q's products into its sums
    v4f& to = acc[row_of(q)][col_of(q)];
    const v4f& pr = prod[q % (kLag + 1)];
    if constexpr (kRowB) {
#pragma unroll
      for (int e = 0; e < 4; e++) to[e] = __builtin_fmaf(pr[e], sc.a[row_of(q)] * sc.row_b[col_of(q)][e], to[e]);
    } else {
      const float f = scale(q);
#pragma unroll
      for (int e = 0; e < 4; e++) to[e] = __builtin_fmaf(pr[e], f, to[e]);
    }
  };
  auto add_pending = [&](int u) {  // the u-th of the stage before's last kLag
    const int q = kStageMfma - kLag + u;
    v4f& to = acc[row_of(q)][col_of(q)];
    const v4f& pr = prod[q % (kLag + 1)];
#pragma unroll
    for (int e = 0; e < 4; e++) to[e] = __builtin_fmaf(pr[e], kRowB ? pend_row[kRowB ? u : 0][e] : pend[kRowB ? 0 : u], to[e]);
  };
  auto keep_pending = [&] {
#pragma unroll
    for (int u = 0; u < kLag; u++) {
      const int q = kStageMfma - kLag + u;
      if constexpr (kRowB) pend_row[u] = sc.a[row_of(q)] * sc.row_b[col_of(q)];
      else pend[u] = scale(q);
    }
  };

  constexpr int kBarrier = (kGroups - 2) * kMfma + (kMfma > 1 ? kMfma * 3 / 4 - 1 : 0);
  static_assert(!kTwoStep || kFree < kBarrier, "the first barrier is the first");
  // before which of a stage's MFMAs its load l goes out; past kStageMfma: in the next stage
  constexpr int kSpread = kStageMfma * 15 / 16 - 1, kEarlyLoads = kTwoStep ? 1 + kLoadsB + kEarlyA : 0;
  constexpr auto issue_at = [](int l) {
    if (!kTwoStep) return kBarrier + 1 + l * (RING == 2 ? kStageMfma / 2 - 1 : kSpread) / kIssues;
    if (l < kEarlyLoads) return kFree + 1 + l * (kBarrier - kFree) / (kEarlyLoads > 0 ? kEarlyLoads : 1);
    return kBarrier + 1 + (l - kEarlyLoads) * (kStageMfma - 1 - kBarrier) / (kIssues - kEarlyLoads);
  };
  constexpr auto issued_by = [issue_at](int q) {  // loads that go out at MFMA q or before
    int n = 0;
    while (n < kIssues && issue_at(n) <= q) n++;
    return n;
  };
  constexpr int kNow = issued_by(kStageMfma - 1), kBefore = issued_by(kBarrier - 1), kBegin = kTwoStep ? kFree : kBarrier;
  static_assert(kNow == kIssues || issue_at(kIssues - 1) - kStageMfma < kBegin,
                "a stage's loads are issued before the next one's begin");
  // kLeft: stages that follow (RING: that many or more, so stage st + RING is issued); kFirst: where A's first fragments are
  auto stage = [&](auto left_c, auto first_c, int st, int slot) {
    constexpr int kLeft = decltype(left_c)::value, kFirst = decltype(first_c)::value;
    constexpr bool kNext = kLeft > 0, kAfter = kLeft >= RING;
    const int next = slot + 1 == RING ? 0 : slot + 1;
    struct {
      float b[kSb];
      v4f row_b[kRowB ? TN : 1];
    } sb_next;
#pragma unroll
    for (int q = 0; q < kStageMfma; q++) {
      const int grp = q / kMfma, t = q % kMfma, j = t / TP, r = t % TP;
      const bool last = grp == kGroups - 1;
      if (kAfter && q == kBegin) begin_issue(st + RING);
      prod[q % (kLag + 1)] = mfma_fp8(fb[j], fa[(grp + kFirst) & 1][r]);
      if (q >= kLag) add(q - kLag);
      else add_pending(q);
      if (!last) {
#pragma unroll
        for (int x = 0; x < TP; x++)
          if (x * (kMfma / 2) / TP == t) read_a(x, slot, grp + 1, (grp + 1 + kFirst) & 1);
      } else if (kNext) {
        if (r == TP - 1) read_b(j, next);
#pragma unroll
        for (int x = 0; x < TP; x++)
          if (x * (kMfma / 2) / TP == t) read_a(x, next, 0, (kGroups + kFirst) & 1);
        if (t == kMfma - 1) {
          read_scales_a(next, 0, kEarly);
          read_scales_b(next, sb_next);
        }
      }
      if (kTwoStep && kAfter && q == kFree) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      if (kNext && q == kBarrier)
        arrive(std::integral_constant<int, kLeft < RING ? (kLeft - 1) * kIssues : (RING - 2) * kIssues + kBefore>{});
#pragma unroll
      for (int l = 0; l < kIssues; l++) {
        const int at = issue_at(l);
        if (kAfter && at == q) issue_one(l, st + RING, slot);
        if (kLeft >= RING - 1 && at - kStageMfma == q) issue_one(l, st - 1 + RING, slot == 0 ? RING - 1 : slot - 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    keep_pending();
    if constexpr (kNext) {
      read_scales_a(next, kEarly, TM);
#pragma unroll
      for (int k = 0; k < kSb; k++) sc.b[k] = sb_next.b[k];
#pragma unroll
      for (int j = 0; j < (kRowB ? TN : 1); j++) sc.row_b[j] = sb_next.row_b[j];
    }
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
    if (nst >= RING) arrive(std::integral_constant<int, (RING - 2) * kIssues + kNow>{});
    else arrive(std::integral_constant<int, 0>{});
    read_scales_a(0, 0, TM);
    read_scales_b(0, sc);
#pragma unroll
    for (int r = 0; r < TP; r++) {
      read_a(r, 0, 0, 0);
      if (kOdd) fa[1][r] = fa[0][r];  // an odd number of stages begins at the other place
    }
#pragma unroll
    for (int j = 0; j < TN; j++) read_b(j, 0);
    int st = s0, slot = 0;
    auto run = [&](auto left_c, auto first_c) {
      stage(left_c, first_c, st, slot);
      st++;
      slot = slot + 1 == RING ? 0 : slot + 1;
    };
    std::integral_constant<int, RING> full;
    std::integral_constant<int, 0> even;
    std::integral_constant<int, 1> odd;
    if constexpr (kOdd) {
      static_assert(RING == 2, "two stages at the end");
      if (nst & 1) run(full, odd);
      while (st + RING < s1) {
        run(full, even);
        run(full, odd);
      }
      run(std::integral_constant<int, 1>{}, even);
      run(std::integral_constant<int, 0>{}, odd);
    } else {
      while (st + RING < s1) run(full, even);
      if constexpr (RING > 3) {
        if (st + 3 < s1) run(std::integral_constant<int, 3>{}, even);
      }
      if constexpr (RING > 2) {
        if (st + 2 < s1) run(std::integral_constant<int, 2>{}, even);
      }
      if (st + 1 < s1) run(std::integral_constant<int, 1>{}, even);
      run(std::integral_constant<int, 0>{}, even);
    }
#pragma unroll
    for (int u = 0; u < kLag; u++) add_pending(u);
  }

  // ---- epilogue.  Register e of block (i, j): row wm WM + 16 i + lr, tile column wn WN + 16 j + 4 kg + e;
  // gated: even j gate, odd j up, output column wn WN / 2 + 16 (j / 2) + 4 kg + e
  auto out_col = [&](int j) { return (kGated ? wn * (WN / 2) + (j / 2) * 16 : wn * WN + j * 16) + 4 * kg; };
  if constexpr (!kGated) {
    if (p.splits > 1 || EPI == kFp8F32) {
      float* dst = p.splits > 1 ? p.part + (int64_t)split * p.M * p.N : static_cast<float*>(p.D);
#pragma unroll
      for (int i = 0; i < TM; i++) {
        const int m = m0 + wm * WM + i * 16 + lr;
        if (m >= m1) continue;
#pragma unroll
        for (int j = 0; j < TN; j++) {
          const int n = n0 + out_col(j);
          if (n < p.N) *reinterpret_cast<v4f*>(dst + (int64_t)m * p.N + n) = acc[i][j];
        }
      }
      return;
    }
  }
  __syncthreads();  // the stages are done with
  if constexpr (EPI == kFp8Bf16) {
    constexpr int kPitch = kCols * 2 + 16;
#pragma unroll
    for (int j = 0; j < TN; j++) {
      const int c = out_col(j), n = min(n0 + c, p.N - 4);
      float4 bv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.bias) {
        const uint2 b = *reinterpret_cast<const uint2*>(p.bias + n);
        bv = make_float4(bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y));
      }
#pragma unroll
      for (int i = 0; i < TM; i++) {
        const v4f& a = acc[i][j];
        *reinterpret_cast<uint2*>(smem + (wm * WM + i * 16 + lr) * kPitch + c * 2) =
            make_uint2(pack_bf16x2_ieee(a[0] + bv.x, a[1] + bv.y), pack_bf16x2_ieee(a[2] + bv.z, a[3] + bv.w));
      }
    }
    __syncthreads();
    constexpr int kChunksRow = kCols / 8;
    uint16_t* D = static_cast<uint16_t*>(p.D);
    for (int idx = tid; idx < BM * kChunksRow; idx += NT) {
      const int r = idx / kChunksRow, c = (idx % kChunksRow) * 8;
      if (m0 + r < m1 && n0 + c < p.N)
        *reinterpret_cast<uint4*>(D + (int64_t)(m0 + r) * p.N + n0 + c) =
            *reinterpret_cast<const uint4*>(smem + r * kPitch + c * 2);
    }
  }
  if constexpr (kGated) {
    // silu(gate) * up in binary32 up to its codes: the row's largest over the lanes, then over the waves
    constexpr int kPitch = kCols + 16;
    float* top = reinterpret_cast<float*>(smem + BM * kPitch);  // [BM][4]
    static_assert(WGN <= 4, "four waves across");
    uint32_t mx[TM];
#pragma unroll
    for (int i = 0; i < TM; i++) {
      mx[i] = 0;
#pragma unroll
      for (int j = 0; j < TN; j += 2)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float h = silu_f(acc[i][j][e]) * acc[i][j + 1][e];
          acc[i][j][e] = h;
          mx[i] = max(mx[i], __float_as_uint(h) & 0x7FFFFFFFu);
        }
      mx[i] = max(mx[i], (uint32_t)__shfl_xor((int)mx[i], 16, 64));
      mx[i] = max(mx[i], (uint32_t)__shfl_xor((int)mx[i], 32, 64));
      if (kg == 0) top[(wm * WM + i * 16 + lr) * 4 + wn] = __uint_as_float(mx[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; i++) {
      const int r = wm * WM + i * 16 + lr;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(top) + r * 4;
      uint32_t m = w[0];
#pragma unroll
      for (int k = 1; k < WGN; k++) m = max(m, w[k]);
      const Fp8Block b(m);
#pragma unroll
      for (int j = 0; j < TN; j += 2) {
        const v4f& h = acc[i][j];
        *reinterpret_cast<uint32_t*>(smem + r * kPitch + out_col(j)) =
            fp8_codes4<false>(b, h[0], h[1], h[2], h[3]);
      }
      if (wn == 0 && kg == 0 && m0 + r < m1) p.s[(int64_t)(n0 / kFp8Block) * p.M + m0 + r] = b.s;
    }
    __syncthreads();
    constexpr int kChunksRow = kCols / 16;
    for (int idx = tid; idx < BM * kChunksRow; idx += NT) {
      const int r = idx / kChunksRow, c = (idx % kChunksRow) * 16;
      if (m0 + r < m1)
        *reinterpret_cast<uint4*>(p.q + (int64_t)(m0 + r) * p.N + n0 + c) =
            *reinterpret_cast<const uint4*>(smem + r * kPitch + c);
    }
  }
}

template <int BM, int BN, int WGM, int WGN, int RING, bool kRowB, int EPI>
__global__ void __launch_bounds__(64 * WGM * WGN, (fp8_waves_simd<BM, BN, RING, WGM * WGN, EPI>()))
    fp8_tile(const Fp8Args p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[fp8_smem<BM, BN, RING, WGM * WGN, EPI>()];
  int tile_m, tile_n, split;
  tile_item(p, blockIdx.x, tile_m, tile_n, split);
  const Fp8Tile tile{p.m_base + tile_m * BM, p.M, p.n_base + tile_n * BN, split, p.B, p.sb};
  fp8_body<BM, BN, WGM, WGN, RING, kRowB, EPI, false>(p, tile, smem);
}

// Two products in one launch: a's workgroups, then (from `first`, a multiple of 8) those of b, which has a scale per row of B.
template <int BM, int BN, int WGM, int WGN, int RING, int EPI>
__global__ void __launch_bounds__(64 * WGM * WGN, (fp8_waves_simd<BM, BN, RING, WGM * WGN, kFp8Bf16>()))
    fp8_two(const Fp8Args a, const Fp8Args b, int first) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[fp8_smem<BM, BN, RING, WGM * WGN, kFp8Bf16>()];
  int tile_m, tile_n, split;
  if ((int)blockIdx.x < first) {
    if ((int)blockIdx.x >= a.tiles_m * a.tiles_n) return;
    tile_item(a, blockIdx.x, tile_m, tile_n, split);
    fp8_body<BM, BN, WGM, WGN, RING, false, kFp8Bf16, false>(a, Fp8Tile{tile_m * BM, a.M, tile_n * BN, split, a.B, a.sb}, smem);
  } else {
    tile_item(b, blockIdx.x - first, tile_m, tile_n, split);
    fp8_body<BM, BN, WGM, WGN, RING, true, EPI, false>(b, Fp8Tile{tile_m * BM, b.M, tile_n * BN, split, b.B, b.sb}, smem);
  }
}

// Rows of no expert: zeros.
template <int EPI>
__device__ __forceinline__ void fp8_zeros(const Fp8Args& p, int m0, int m1, int n0, int cols) {
  cols = min(cols, p.N - n0);
  for (int i = threadIdx.x; i < (m1 - m0) * cols; i += blockDim.x) {
    const int64_t at = (int64_t)(m0 + i / cols) * p.N + n0 + i % cols;
    if constexpr (EPI == kFp8Bf16) static_cast<uint16_t*>(p.D)[at] = 0;
    else if constexpr (EPI == kFp8F32) static_cast<float*>(p.D)[at] = 0.0f;
    else p.q[at] = 0;
  }
  if constexpr (EPI == kFp8Gated)
    for (int i = threadIdx.x; i < m1 - m0; i += blockDim.x) p.s[(int64_t)(n0 / kFp8Block) * p.M + m0 + i] = 0.0f;
}

// The tile of this workgroup among the experts' row tiles of BM rows; false: it has none, or zeros that are written.
template <int BM, int kCols, int EPI>
__device__ __forceinline__ bool fp8_grouped_tile(const Fp8Args& p, Fp8Tile& tile) {
  // the grid holds as many row tiles as there may be: those there are go to all XCDs alike
  const Fp8Groups<BM> groups{p.offsets, p.E, p.M};
  Fp8Args there = p;
  there.tiles_m = groups.count();
  if ((int)blockIdx.x >= there.tiles_m * p.tiles_n) return false;
  int tile_m, tile_n;
  tile_item(there, blockIdx.x, tile_m, tile_n, tile.split);
  const Fp8Group g = groups.find(tile_m);
  if (g.e > p.E) return false;
  tile.m0 = g.row0;
  tile.m1 = g.row1;
  tile.n0 = tile_n * kCols;
  if (g.e == p.E) {
    fp8_zeros<EPI>(p, tile.m0, tile.m1, tile.n0, kCols);
    return false;
  }
  tile.B = p.B + (int64_t)g.e * p.b_stride;
  tile.sb = p.sb + (int64_t)g.e * p.sb_stride;
  return true;
}

// Few rows an expert.
template <int BM, int BN, int WGM, int WGN, int RING, int EPI>
__global__ void __launch_bounds__(64 * WGM * WGN, (fp8_waves_simd<BM, BN, RING, WGM * WGN, EPI>()))
    fp8_grouped_few(const Fp8Args p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[fp8_smem<BM, BN, RING, WGM * WGN, EPI>()];
  Fp8Tile tile;
  if (fp8_grouped_tile<BM, EPI == kFp8Gated ? BN / 2 : BN, EPI>(p, tile))
    fp8_body<BM, BN, WGM, WGN, RING, false, EPI, true>(p, tile, smem);
}

// Many: tiles of up to 256 rows, by what the expert's rows come to, in steps of 32 where the matrix cores and not the
// weight's bytes bound them (the layer of 4096 tokens on 8 of 128 experts 1317 us, 1345 in steps of 64).
template <int EPI>
__global__ void __launch_bounds__(512, 2)
    fp8_grouped_many(const Fp8Args p) {
  constexpr int kSmem =
      std::max({fp8_smem<256, 256, 2, 8, EPI>(), fp8_smem<192, 256, 2, 8, EPI>(), fp8_smem<128, 256, 3, 8, EPI>(), fp8_smem<64, 256, 3, 8, EPI>()});
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kSmem];
  Fp8Tile tile;
  if (!fp8_grouped_tile<256, EPI == kFp8Gated ? 128 : 256, EPI>(p, tile)) return;
  const int rows = tile.m1 - tile.m0;
  const bool two = p.kb >= 2;  // stages
  if (rows > 224 || (rows > 192 && !two)) fp8_body<256, 256, 2, 4, 2, false, EPI, true>(p, tile, smem);
  else if (rows > 192) fp8_body<256, 256, 2, 4, 2, false, EPI, true, 224>(p, tile, smem);
  else if (rows > 160 || (rows > 128 && !two)) fp8_body<192, 256, 2, 4, 2, false, EPI, true>(p, tile, smem);
  else if (rows > 128) fp8_body<192, 256, 2, 4, 2, false, EPI, true, 160>(p, tile, smem);
  else if (rows > 64) fp8_body<128, 256, 2, 4, 3, false, EPI, true>(p, tile, smem);
  else fp8_body<64, 256, 2, 4, 3, false, EPI, true>(p, tile, smem);
}

// Sums the splits' partials in split order and finishes the rows.  One thread: eight columns.
template <int EPI>
__global__ void __launch_bounds__(256)
    fp8_reduce(const Fp8Args p) {
  const int64_t mn = (int64_t)p.M * p.N, all = mn / 8, stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < all; idx += stride) {
    const float4* src = reinterpret_cast<const float4*>(p.part) + idx * 2;
    float v[8] = {};
#pragma unroll 4
    for (int s = 0; s < p.splits; s++) {
      const float4 a = src[s * (mn / 4)], b = src[s * (mn / 4) + 1];
      const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; k++) v[k] += w[k];
    }
    if constexpr (EPI == kFp8F32) {
      float4* d = reinterpret_cast<float4*>(p.D) + idx * 2;
      d[0] = make_float4(v[0], v[1], v[2], v[3]);
      d[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      if (p.bias) {
        float b[8];
        unpack8(*reinterpret_cast<const uint4*>(p.bias + idx * 8 % p.N), b);
#pragma unroll
        for (int k = 0; k < 8; k++) v[k] += b[k];
      }
      reinterpret_cast<uint4*>(p.D)[idx] = pack8(v);
    }
  }
}

}  // namespace
}  // namespace bsfp4
