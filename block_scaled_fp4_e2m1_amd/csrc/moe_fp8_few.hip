// The E4M3 expert layer for a handful of tokens, bound by the bytes of the experts that they meet: two launches, or three.
//
// Every wave finds the distinct experts of the (token, slot) pairs itself (64 pairs at most, a lane each; equal ids by
// ballots over their bits), in order of first appearance, so nothing is sorted.  The matrix cores' rows of activations
// are the tokens: tokens that do not go to an expert take part in its products and are left out of the results.
//
//   up    a workgroup owns 8 gate and the 8 up rows of one expert (fp8_rows with a gated end): silu(gate) * up in
//         binary32, to the token's pair rows.  Up to what fits in LDS the tokens are quantised in the workgroup.
//   down  a workgroup owns 16 output columns for all experts: it quantises all pairs' rows into LDS, its waves take the
//         (expert, 128-byte step) pairs in turn, and a product enters its token's sum with both scales and the
//         routing weight, so that the sum over experts needs no further pass.
#include "fp8_rows_gemm.h"

namespace bsfp4 {
namespace {

struct FewArgs {
  const uint16_t* x;   // [T, H] (kQuant), or
  const uint8_t* xq;   // codes [T, H] and
  const float* xs;     // scales [HB, T]
  const int32_t* ids;  // [T, topk]
  const float* weights;
  const uint8_t *w13, *w2;
  const float *w13s, *w2s;
  float* h;       // [T topk, I]
  uint16_t* out;  // [T, H]
  int T, topk, E, H, I;
};

// The pairs' distinct experts.  Lane i is pair i; same: the lanes of its expert (none for a dropped pair).
struct FewExperts {
  uint64_t same, firsts;
  int dense;  // lane a: the a-th distinct expert
  // table: 64 entries of this wave's own
  __device__ __forceinline__ FewExperts(const FewArgs& p, int* table) {
    const int lane = threadIdx.x & 63, n = p.T * p.topk;
    const int key = lane < n ? p.ids[lane] : -1;
    const bool there = (uint32_t)key < (uint32_t)p.E;
    same = __ballot(there);
    for (int b = 0; b < 32 - __clz(p.E); b++) {
      const uint64_t set = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? set : ~set;
    }
    if (!there) same = 0;
    firsts = __ballot(there && (same & ((1ull << lane) - 1)) == 0);
    if (firsts >> lane & 1) table[__popcll(firsts & ((1ull << lane) - 1))] = key;
    // another lane's store: neither the compiler nor the wave may read before it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    dense = lane < count() ? table[lane] : 0;
  }
  __device__ __forceinline__ int count() const { return __popcll(firsts); }
  __device__ __forceinline__ int expert(int a) const { return __builtin_amdgcn_readlane(dense, a); }
};

constexpr int kFewPairs = 64, kFewTokens = 8;
constexpr int kFewSteps = 32;  // of a wave: K up to 8 * 32 * 128
constexpr int kOwnScales = 3 * 1024;  // quantised tokens: their scales behind gate, up and token rows in a slot

// ---- up --------------------------------------------------------------------
// One token of eight experts, 134 MB: 33.9 us, 4.0 TB/s; 31.6 on E4M3 matrix instructions, which turned some codes of
// silu(gate) * up over (the layer off by up to 0.0042 of itself; 0.0017, the output's own rounding, now).  256 workgroups
// that go through the tiles, their rings running on: 35.8 against 31.6, for they meet at each tile's end.
template <int AQ>
struct FewUpShape {
  static constexpr int kWaves = 8, kRing = 3, kSlot = (2 + AQ) * 1024 + (AQ > 0 ? 256 : 0);
  static constexpr int kRings = kWaves * kRing * kSlot, kScales = kWaves * 2 * kFewSteps * 4;
  static constexpr int kSmem = kRings + kScales + (AQ == 0 ? kFp8RowsQuantBytes : 0);
  static_assert(2 * kSmem <= 160 * 1024, "two workgroups per compute unit");
};

template <int AQ>  // 1: quantised tokens; 0: quantised here
__global__ void __launch_bounds__(512, 4)
    fp8_few_up(const FewArgs p) {
  typedef FewUpShape<AQ> S;
  constexpr bool kQuant = AQ == 0;
  constexpr int W = S::kWaves, RING = S::kRing, kSlot = S::kSlot, kL = 2 + AQ + (kQuant ? 0 : 1);
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kSmem];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, kg = lane >> 4;
  const int tiles = p.I / 8, n0 = (int)(blockIdx.x % (unsigned)tiles) * 8;
  const FewExperts ex(p, reinterpret_cast<int*>(smem) + wave * 64);
  const int a = (int)(blockIdx.x / (unsigned)tiles);
  if (a >= ex.count()) return;
  const int e = ex.expert(a);
  __syncthreads();  // the tables are done with
  const int kb = p.H, total = (p.H + kFp8Block - 1) / kFp8Block;

  const uint8_t* const w13 = p.w13 + (int64_t)e * 2 * p.I * p.H;
  const int row8 = lane >> 3;
  const v4u32 rg = make_rsrc4(w13 + (int64_t)n0 * p.H, (int64_t)8 * p.H);
  const v4u32 ru = make_rsrc4(w13 + ((int64_t)p.I + n0) * p.H, (int64_t)8 * p.H);
  const v4u32 rx = make_rsrc4(p.xq, (int64_t)p.T * p.H);
  // the gate rows are the fragment's rows 0 .. 7, the up rows 8 .. 15: row8 has the same swizzle in both
  const uint32_t c16 = (uint32_t)((lane & 7) ^ tile_swz(row8)) * 16, ow = (uint32_t)(row8 * p.H) + c16;
  const uint32_t oa = row8 < p.T ? ow : kBufOOB, os = lane < p.T ? (uint32_t)lane * 4 : kBufOOB;
  const uint32_t ring0 = lds_offset(smem) + (uint32_t)wave * RING * kSlot;
  const uint8_t* const ring = smem + wave * RING * kSlot;
  float* const weight_scales = reinterpret_cast<float*>(smem + S::kRings) + wave * 2 * kFewSteps;

  const int mine = wave < total ? (total - 1 - wave) / W + 1 : 0;
  const int first = (int)(blockIdx.x % (unsigned)total);
  auto step_of = [&](int i) {
    const int s = wave + i * W + first;
    return s < total ? s : s - total;
  };
  auto issue = [&](int s, int slot) {
    const uint32_t soff = (uint32_t)s * kTileStage, lds = ring0 + (uint32_t)slot * kSlot;
    const bool in = (int)c16 < kb - (int)soff;
    buf_lds16(rg, in ? ow : kBufOOB, soff, lds);
    buf_lds16(ru, in ? ow : kBufOOB, soff, lds + 1024);
    if constexpr (!kQuant) {
      buf_lds16(rx, in ? oa : kBufOOB, soff, lds + 2048);
      buf_lds4(make_rsrc4(p.xs + (int64_t)s * p.T, (int64_t)p.T * 4), os, 0u, lds + kOwnScales);
    }
  };
  {  // the wave's weight scales: lanes 0 .. 31 its steps of the gate rows, 32 .. 63 of the up rows
    const int64_t nb = 2 * p.I / kFp8Block, gate = n0 / kFp8Block, up = (p.I + n0) / kFp8Block;
    const v4u32 rs = make_rsrc4(p.w13s + (int64_t)e * nb * total, nb * total * 4);
    const int i = lane % kFewSteps;
    buf_lds4(rs, i < mine ? (uint32_t)((lane < kFewSteps ? gate : up) * total + step_of(i)) * 4 : kBufOOB, 0u,
             lds_offset(weight_scales));
  }
  uint8_t* const codes = smem + S::kRings + S::kScales;
  float* const scales = reinterpret_cast<float*>(codes + p.T * total * kTileStage);
  uint8_t* const raw = codes + (p.T * total * (kTileStage + 4) + 15) / 16 * 16;
  if constexpr (kQuant) {
    const int raw_bytes = p.T * kb * 2;
    const v4u32 rr = make_rsrc4(p.x, raw_bytes);
    for (int q = wave; q * 1024 < raw_bytes; q += W)
      buf_lds16(rr, (uint32_t)(q * 1024 + lane * 16), 0u, lds_offset(raw) + q * 1024);
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
    for (int m = 0; m < p.T; m++)
      for (int c = threadIdx.x; c < kept; c += 64 * W) {
        const uint4 v = c < chunks ? rows[m * chunks + c] : make_uint4(0, 0, 0, 0);
        const Fp8Block b((uint32_t)lanes_reduce<4>((int)amax_of_pairs(amax_pairs8(v, 0)), MaxOp{}) << 16);
        *reinterpret_cast<uint2*>(codes + (m * kept + c) * 8) = fp8_codes8(b, v);
        if ((c & 15) == 0) scales[m * total + c / 16] = b.s;
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  v4f acc = {};
  uint32_t off[2];
#pragma unroll
  for (int h = 0; h < 2; h++) off[h] = (uint32_t)(lr * kTileStage + (((4 * h + kg) ^ tile_swz(lr)) * 16));
  const int token = min(lr, p.T - 1);
  auto step = [&](int i, int slot) {
    const uint8_t* s = ring + slot * kSlot;
    v4i w[2], x[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      w[h] = *reinterpret_cast<const v4i*>(s + off[h]);
      if constexpr (kQuant)
        x[h] = *reinterpret_cast<const v4i*>(codes + (token * total + step_of(i)) * kTileStage + h * 64 + kg * 16);
      else
        x[h] = *reinterpret_cast<const v4i*>(s + 2048 + (off[h] & 1023u));  // rows past the eighth repeat
    }
    const float sx = kQuant ? scales[token * total + step_of(i)] : reinterpret_cast<const float*>(s + kOwnScales)[lr];
    const float sw = weight_scales[(kg >> 1) * kFewSteps + i];  // this lane's rows are gate (kg < 2) or up rows
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (i + RING < mine) issue(step_of(i + RING), slot);
    const v4f part = mfma_fp8_wide(fp8_frag(w[0], w[1]), fp8_frag(x[0], x[1]));
    const float f = sx * sw;
#pragma unroll
    for (int k = 0; k < 4; k++) acc[k] = __builtin_fmaf(part[k], f, acc[k]);
  };
  int i = 0, slot = 0;
  for (; i + RING <= mine; i++) {
    wait_vmcnt<(RING - 1) * kL>();
    step(i, slot);
    slot = slot + 1 == RING ? 0 : slot + 1;
  }
  if (mine - i == 2) {
    wait_vmcnt<kL>();
    step(i++, slot);
    slot = slot + 1 == RING ? 0 : slot + 1;
  }
  if (mine - i == 1) {
    wait_vmcnt<0>();
    step(i, slot);
  }
  __syncthreads();
  v4f* red = reinterpret_cast<v4f*>(smem);
  red[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  auto sum = [&](int l) {
    v4f v = red[l];
#pragma unroll
    for (int k = 1; k < W; k++) v += red[k * 64 + l];
    return v;
  };
  if (kg >= 2 || lr >= p.T) return;
  const v4f g = sum(lane), u = sum(lane + 32);
  v4f h;
#pragma unroll
  for (int k = 0; k < 4; k++) h[k] = silu_f(g[k]) * u[k];
  for (int j = 0; j < p.topk; j++)
    if (p.ids[lr * p.topk + j] == e) *reinterpret_cast<v4f*>(p.h + (int64_t)(lr * p.topk + j) * p.I + n0 + 4 * kg) = h;
}

// ---- down ------------------------------------------------------------------
constexpr int kFewCodes = 72 * 1024;  // the pairs' codes and scales in LDS
constexpr int kDownRing = 4, kDownWaves = 8;
constexpr int kDownItems = 128;  // of a wave
constexpr int kDownSmem =
    kDownWaves * kDownRing * 2048 + kFewCodes + kFewPairs * kFewTokens * 8 + kDownWaves * kDownItems * 4;
static_assert(kFewCodes / kFp8Block / kDownWaves + 1 <= kDownItems, "experts times steps, shared by the waves");
static_assert(kDownSmem <= 160 * 1024, "one workgroup per compute unit");

__global__ void __launch_bounds__(512, 2)
    fp8_few_down(const FewArgs p) {
  constexpr int W = kDownWaves, RING = kDownRing, kSlot = 2048, kL = 2;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kDownSmem];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, kg = lane >> 4, n0 = blockIdx.x * 16;
  const int steps = p.I / kFp8Block, pairs = p.T * p.topk;
  const FewExperts ex(p, reinterpret_cast<int*>(smem) + wave * 64);
  const int items = ex.count() * steps;
  uint8_t* const codes = smem + W * RING * kSlot;  // [pairs][I]
  float* const scales = reinterpret_cast<float*>(codes + pairs * p.I);  // [pairs][steps]
  int* const row_at = reinterpret_cast<int*>(smem + W * RING * kSlot + kFewCodes);  // [distinct][kFewTokens]: pair or -1
  float* const weight_at = reinterpret_cast<float*>(row_at + kFewPairs * kFewTokens);

  // items wave, wave + W, ...: expert a = item / steps, each workgroup beginning further on
  const int mine = wave < items ? (items - 1 - wave) / W + 1 : 0;
  const int first = items > 0 ? (int)(blockIdx.x % (unsigned)items) : 0;
  auto item_of = [&](int i) {
    const int s = wave + i * W + first;
    return s < items ? s : s - items;
  };
  const int row8 = lane >> 3;
  const uint32_t c16 = (uint32_t)((lane & 7) ^ tile_swz(row8)) * 16;
  uint32_t ow[2];
#pragma unroll
  for (int q = 0; q < 2; q++) ow[q] = n0 + 8 * q + row8 < p.H ? (uint32_t)((8 * q + row8) * p.I) + c16 : kBufOOB;
  const uint32_t ring0 = lds_offset(smem) + (uint32_t)wave * RING * kSlot;
  const uint8_t* const ring = smem + wave * RING * kSlot;
  auto issue = [&](int item, int slot) {
    const int a = item / steps, s = item - a * steps;
    const uint8_t* w = p.w2 + ((int64_t)ex.expert(a) * p.H + n0) * p.I;
    const v4u32 rw = make_rsrc4(w, (int64_t)min(16, p.H - n0) * p.I);
#pragma unroll
    for (int q = 0; q < 2; q++)
      buf_lds16(rw, ow[q], (uint32_t)s * kTileStage, ring0 + (uint32_t)(slot * kSlot + q * 1024));
  };
  // the wave's weight scales, an item a lane
  float* const weight_scales = reinterpret_cast<float*>(weight_at + kFewPairs * kFewTokens) + wave * kDownItems;
  const int64_t sb_expert = (int64_t)((p.H + kFp8Block - 1) / kFp8Block) * steps;
  int* const dense = reinterpret_cast<int*>(smem) + wave * 64;
  uint32_t scale_off[2];
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int i = lane + 64 * k, item = item_of(i < mine ? i : 0), a = steps > 0 ? item / steps : 0;
    scale_off[k] = i < mine ? (uint32_t)(dense[a] * sb_expert + (n0 / kFp8Block) * steps + item - a * steps) * 4 : kBufOOB;
  }
  __syncthreads();  // the tables of the experts are done with
  {
    const v4u32 rs = make_rsrc4(p.w2s, p.E * sb_expert * 4);
    buf_lds4(rs, scale_off[0], 0u, lds_offset(weight_scales));
    buf_lds4(rs, scale_off[1], 0u, lds_offset(weight_scales + 64));
  }
#pragma unroll
  for (int r = 0; r < RING; r++)
    if (r < mine) issue(item_of(r), r);

  if (wave == 0) {
    for (int i = lane; i < kFewPairs * kFewTokens; i += 64) {
      row_at[i] = -1;
      weight_at[i] = 0.0f;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    // one lane of a token's pairs of an expert (a token may name one twice): the first, with their weights' sum
    const int t = lane / p.topk;
    uint64_t mates = ex.same == 0 ? 0 : ex.same & (((p.topk < 64 ? 1ull << p.topk : 0ull) - 1) << (t * p.topk));
    if (mates != 0 && __builtin_ctzll(mates) == lane) {
      float w = 0.0f;
      for (; mates != 0; mates &= mates - 1) w += p.weights[__builtin_ctzll(mates)];
      const int a = __popcll(ex.firsts & ((1ull << __builtin_ctzll(ex.same)) - 1));
      row_at[a * kFewTokens + t] = lane;
      weight_at[a * kFewTokens + t] = w;
    }
  }
  // all pairs' rows, 16 lanes a block; a dropped pair's row holds anything and is never used
  const int chunks = p.I / 8;
  for (int c = threadIdx.x; c < pairs * chunks; c += 64 * W) {
    const float4* src = reinterpret_cast<const float4*>(p.h) + (int64_t)c * 2;
    const float4 v0 = src[0], v1 = src[1];
    uint32_t m = 0;
    const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int k = 0; k < 8; k++) m = max(m, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    const Fp8Block b((uint32_t)lanes_reduce<4>((int)m, MaxOp{}));
    *reinterpret_cast<uint2*>(codes + c * 8) =
        make_uint2(fp8_codes4<false>(b, v[0], v[1], v[2], v[3]), fp8_codes4<false>(b, v[4], v[5], v[6], v[7]));
    if ((c & 15) == 0) scales[c / 16] = b.s;
  }
  __syncthreads();

  v4f acc = {};
  uint32_t off[2];
#pragma unroll
  for (int h = 0; h < 2; h++) off[h] = (uint32_t)(lr * kTileStage + (((4 * h + kg) ^ tile_swz(lr)) * 16));
  auto step = [&](int i, int slot) {
    const uint8_t* w8 = ring + slot * kSlot;
    const int item = item_of(i), a = item / steps, s = item - a * steps;
    const float sw = weight_scales[i];
    const int r = lr < kFewTokens ? row_at[a * kFewTokens + lr] : -1, row = max(r, 0);
    const float wt = lr < kFewTokens ? weight_at[a * kFewTokens + lr] : 0.0f, sx = scales[row * steps + s];
    v4i w[2], x[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      w[h] = *reinterpret_cast<const v4i*>(w8 + off[h]);
      x[h] = *reinterpret_cast<const v4i*>(codes + row * p.I + s * kTileStage + h * 64 + kg * 16);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (i + RING < mine) issue(item_of(i + RING), slot);
    const v4f part = mfma_fp8(fp8_frag(w[0], w[1]), fp8_frag(x[0], x[1]));
    // a token that does not go there keeps its sum: its row is another's, and a NaN among the weight's codes or scales would
    // outlast a factor of zero
    const float f = sx * sw * wt;
#pragma unroll
    for (int k = 0; k < 4; k++) acc[k] = r >= 0 ? __builtin_fmaf(part[k], f, acc[k]) : acc[k];
  };
  int i = 0, slot = 0;
  for (; i < mine; i++) {
    if (i + RING <= mine) wait_vmcnt<(RING - 1) * kL>();
    else wait_vmcnt<0>();
    step(i, slot);
    slot = slot + 1 == RING ? 0 : slot + 1;
  }
  __syncthreads();
  v4f* red = reinterpret_cast<v4f*>(smem);
  red[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  v4f v = red[lane];
#pragma unroll
  for (int k = 1; k < W; k++) v += red[k * 64 + lane];
  const int n = n0 + 4 * kg;
  if (lr >= p.T || n >= p.H) return;  // H % 16 == 0
  *reinterpret_cast<uint2*>(p.out + (int64_t)lr * p.H + n) =
      make_uint2(pack_bf16x2_ieee(v[0], v[1]), pack_bf16x2_ieee(v[2], v[3]));
}

// Tokens in bf16 that fit in LDS with their codes are quantised in every workgroup.
bool few_quant_ok(int64_t T, int64_t H) {
  const int64_t lds = (T * fp8_blocks(H) * (kFp8Block + 4) + 15) / 16 * 16 + (2 * T * H + 1023) / 1024 * 1024;
  return T <= 4 && lds <= kFp8RowsQuantBytes;
}

}  // namespace

// down's H / 16 workgroups each read and quantise all T topk rows of I, so that more of them need a wider H.  us against
// the sorted way (H, I, experts of which topk; T): 4096, 2048, 128, 8: 1 50, 62; 2 88, 84; 4 154, 148.  4096, 1024, 64, 4:
// 8 74, 81.  2048, 2048, 60, 2: 2 21, 32; 4 35, 34; 8 59, 51.  512, 2048, 16, 2: 2 17, 25; 4 26, 26; 6 31, 27.  1024, 512,
// 16, 2: 8 17, 24.
bool fp8_moe_few_ok(int64_t T, int64_t topk, int64_t H, int64_t I, int64_t E) {
  return E * fp8_blocks(H) * (I / kFp8Block) < (int64_t)1 << 29 && T <= kFewTokens && T * topk <= kFewPairs &&
         fp8_blocks(H) <= 8 * kFewSteps && T * topk * (I + I / kFp8Block * 4) <= kFewCodes &&
         T * topk * I <= std::max<int64_t>(12288, 8 * H);
}

size_t fp8_moe_few_workspace(int64_t T, int64_t topk, int64_t H, int64_t I) {
  const size_t h = (size_t)(T * topk * I) * 4;
  return h + (few_quant_ok(T, H) ? 0 : (size_t)((T * H + 15) / 16 * 16 + fp8_blocks(H) * T * 4));
}

hipError_t launch_fp8_moe_few(const uint16_t* x, const int32_t* ids, const float* weights, const uint8_t* w13,
                              const float* w13s, const uint8_t* w2, const float* w2s, uint16_t* out, int64_t T, int64_t H,
                              int64_t I, int64_t E, int64_t topk, void* ws, hipStream_t stream) {
  FewArgs p{};
  p.x = x;
  p.ids = ids;
  p.weights = weights;
  p.w13 = w13;
  p.w13s = w13s;
  p.w2 = w2;
  p.w2s = w2s;
  p.out = out;
  p.T = (int)T;
  p.topk = (int)topk;
  p.E = (int)E;
  p.H = (int)H;
  p.I = (int)I;
  p.h = static_cast<float*>(ws);
  const unsigned grid = (unsigned)(std::min(E, T * topk) * (I / 8));
  if (few_quant_ok(T, H)) {
    fp8_few_up<0><<<grid, 512, 0, stream>>>(p);
  } else {
    uint8_t* xq = static_cast<uint8_t*>(ws) + T * topk * I * 4;
    float* xs = reinterpret_cast<float*>(xq + (T * H + 15) / 16 * 16);
    p.xq = xq;
    p.xs = xs;
    if (hipError_t e = launch_fp8_quant(x, T, H, xq, xs, nullptr, nullptr, stream)) return e;
    fp8_few_up<1><<<grid, 512, 0, stream>>>(p);
  }
  fp8_few_down<<<(unsigned)((H + 15) / 16), 512, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace bsfp4
