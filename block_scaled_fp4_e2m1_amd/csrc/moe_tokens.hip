// Tokens sorted by expert and back, in bf16 or binary32, and the gradients of both.
//
// The T topk (token, slot) pairs are sorted by expert, in flat order t topk + j within one, those whose id is
// outside [0, E) behind all others; row_of is where each pair went, a permutation of 0 .. T topk - 1.  With
// keep(t, j) true for ids inside the range, r = row_of[t, j] and w the routing weights (1 without them):
//
//   permute              xs[r] = keep ? x[t] : 0
//   unpermute            out[t] = sum_j keep ? w[t, j] ys[r] : 0
//   unpermute, backward  dys[r] = keep ? w[t, j] dout[t] : 0,  dw[t, j] = keep ? <dout[t], ys[r]> : 0
//   permute, backward    unpermute of dxs without weights
//
// Rows of pairs that are not kept start at offsets[E]; they are never read, whatever they hold.
//
// All are bound by memory.  A workgroup takes a token (or a part of its columns), so x, out and dout pass once
// and only the rows of the sorted side move topk times; nothing is gathered through an intermediate.  Sums are
// binary32, in slot order, rounded once; the dot products are summed per thread, then over the workgroup in a fixed
// order.  No atomics on results.
//
// 4096 x 7168 bf16 to 8 of 128 experts: permute 107 us (4.9 TB/s, most of it writes), unpermute 95 (5.6), its backward
// 202 (5.0), the permutation's 95; sort 11.  2011 x 1032 binary32 to 2 of 60: 14 with the sort, 8, 12, 8.
#include "int8_rows.h"
#include "launchers.h"

namespace bsfp4 {
namespace {

constexpr int kThreads = 256;

// ---- element types: a 16-byte chunk as binary32 values ---------------------
template <class T>
struct Rows;
template <>
struct Rows<uint16_t> {
  static constexpr int kPer = 8;
  __device__ static __forceinline__ void load(const uint4& c, float (&v)[8]) { unpack8(c, v); }
  __device__ static __forceinline__ uint4 store(const float (&v)[8]) { return pack8(v); }
};
template <>
struct Rows<float> {
  static constexpr int kPer = 4;
  __device__ static __forceinline__ void load(const uint4& c, float (&v)[4]) {
    v[0] = __uint_as_float(c.x), v[1] = __uint_as_float(c.y), v[2] = __uint_as_float(c.z), v[3] = __uint_as_float(c.w);
  }
  __device__ static __forceinline__ uint4 store(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

// ---- rows past the caches --------------------------------------------------
// Sorted rows of 64 MiB or more are written and read without a place in the last-level cache (256 MiB for all tensors
// of a step): a copy there only pushes others out.  There and back with gradients, bf16, us, without and with:
// 5600 rows of 7168 (80 MB) 113, 99; 32768 553, 512; there and back only, 28000 rows of 4096 124, 99; but 8024 of 4096
// (66 MB), which the next call finds in the cache, 33, 35.  The rows of sort_permute_few are written as any others: its 4096
// pairs at most come to 64 MiB only in rows of 16 KiB and more.
inline bool streamed(int64_t rows, int64_t row_bytes) { return rows * row_bytes >= (int64_t)64 << 20; }

template <bool kStream>
__device__ __forceinline__ uint4 load_row(const uint4* p) {
  typedef uint32_t v4 __attribute__((ext_vector_type(4)));
  if constexpr (!kStream) return *p;
  const v4 v = __builtin_nontemporal_load(reinterpret_cast<const v4*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <bool kStream>
__device__ __forceinline__ void store_row(uint4* p, const uint4& v) {
  typedef uint32_t v4 __attribute__((ext_vector_type(4)));
  if constexpr (kStream) __builtin_nontemporal_store(v4{v.x, v.y, v.z, v.w}, reinterpret_cast<v4*>(p));
  else *p = v;
}

// ---- sort ------------------------------------------------------------------
// A counting sort over chunks of kChunk pairs: the chunks' counts of each expert (E: dropped pairs), then every chunk
// ranks its own pairs behind those of lower experts and of earlier chunks.  A pair's rank among the 64 of its wave's
// step is found by comparing ids bit by bit (ballots); steps follow each other in order, so equal ids stay in order.
// Every chunk sums all counts itself, two launches, or a launch between sums them once (sort_direct).  32768 pairs of
// 128 experts: 9.3 us, 19 with one workgroup an expert that reads all ids.
constexpr int kChunk = 1024, kSteps = kChunk / kThreads;
constexpr int kMaxKeys = 1025;

// us, two launches against three: 32768 pairs of 8 experts 7.7, 10.5; of 128 9.3, 11.5; of 1024 16.5, 13.9; 2^18 of 128
// 16.9, 14.4; 2^22 of 128 566, 95.
inline bool sort_direct(int64_t chunks, int64_t E) { return chunks <= 128 && E < 256; }

__device__ __forceinline__ int pair_key(const int32_t* ids, int i, int n, int E) {
  return i < n ? (int)min((uint32_t)ids[i], (uint32_t)E) : -1;  // past the pairs: no key
}

__global__ void __launch_bounds__(kThreads)
    sort_count(const int32_t* __restrict__ ids, int n, int E, int32_t* __restrict__ counts) {
  __shared__ int count[kMaxKeys];
  for (int e = threadIdx.x; e <= E; e += kThreads) count[e] = 0;
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kSteps; s++) {
    const int key = pair_key(ids, blockIdx.x * kChunk + s * kThreads + threadIdx.x, n, E);
    if (key >= 0) atomicAdd(&count[key], 1);  // sums do not depend on the order
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kThreads) counts[(int64_t)blockIdx.x * (E + 1) + e] = count[e];
}

// The chunks' counts of an expert to those of the chunks before, their sum to a last line.  64 experts a workgroup, one
// a lane; the waves share the chunks.
constexpr int kScanThreads = 1024;

__global__ void __launch_bounds__(kScanThreads)
    sort_scan(int32_t* __restrict__ counts, int chunks, int E) {
  constexpr int kWaves = kScanThreads / 64, kLoads = 8;
  __shared__ int part[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = min((int)blockIdx.x * 64 + lane, E);
  const bool writes = blockIdx.x * 64 + lane <= E;
  const int each = (chunks + kWaves - 1) / kWaves, c0 = min(wave * each, chunks), c1 = min(c0 + each, chunks);
  int32_t* const at = counts + e;
  const int64_t line = E + 1;
  int sum = 0;
#pragma unroll 8
  for (int c = c0; c < c1; c++) sum += at[c * line];
  part[wave][lane] = sum;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; w++) {
    const int v = part[w][lane];
    before += w < wave ? v : 0;
    all += v;
  }
  if (!writes) return;
  for (int c = c0; c < c1; c += kLoads) {
    int v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; u++) v[u] = c + u < c1 ? at[(c + u) * line] : 0;
#pragma unroll
    for (int u = 0; u < kLoads; u++) {
      if (c + u < c1) at[(c + u) * line] = before;
      before += v[u];
    }
  }
  if (wave == 0) at[chunks * line] = all;
}

// kScanned: counts as sort_scan leaves them.
template <bool kScanned>
__global__ void __launch_bounds__(kThreads)
    sort_place(const int32_t* __restrict__ ids, int n, int topk, int E, const int32_t* __restrict__ counts,
               int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_ids, int32_t* __restrict__ sorted_tokens,
               int32_t* __restrict__ row_of) {
  constexpr int kWaves = kThreads / 64, kPer = (kMaxKeys + kThreads - 1) / kThreads;
  __shared__ int next[kWaves][kMaxKeys];  // the wave's next row of each expert
  __shared__ int every[kMaxKeys], sooner[kMaxKeys];  // an expert's pairs, those of them in earlier chunks
  __shared__ int wave_sum[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, chunks = gridDim.x, mine = blockIdx.x;
  // wave w takes pairs 64 kSteps w .. of the chunk, 64 at a time
  int key[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; s++) key[s] = pair_key(ids, mine * kChunk + (wave * kSteps + s) * 64 + lane, n, E);
  for (int i = tid; i <= E; i += kThreads) {
    every[i] = sooner[i] = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) next[w][i] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kSteps; s++)
    if (key[s] >= 0) atomicAdd(&next[wave][key[s]], 1);
  if constexpr (kScanned) {
    for (int e = tid; e <= E; e += kThreads) {
      every[e] = counts[(int64_t)chunks * (E + 1) + e];
      sooner[e] = counts[(int64_t)mine * (E + 1) + e];
    }
  }
  // an expert a lane, the chunks shared by the waves
  for (int e = lane; !kScanned && e <= E; e += 64) {
    int all = 0, earlier = 0;
#pragma unroll 8
    for (int c = wave; c < chunks; c += kWaves) {
      const int v = counts[(int64_t)c * (E + 1) + e];
      all += v;
      earlier += c < mine ? v : 0;
    }
    atomicAdd(&every[e], all);
    atomicAdd(&sooner[e], earlier);
  }
  __syncthreads();
  // first rows: a scan over the experts, kPer consecutive ones a thread
  int all[kPer], sum = 0;
  const int e0 = tid * kPer;
#pragma unroll
  for (int k = 0; k < kPer; k++) all[k] = e0 + k <= E ? every[e0 + k] : 0;
#pragma unroll
  for (int k = 0; k < kPer; k++) sum += all[k];
  int upto = sum;  // of this thread's experts and lower ones
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const int o = __shfl_up(upto, s, 64);
    if (lane >= s) upto += o;
  }
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  int base = upto - sum;
  for (int w = 0; w < wave; w++) base += wave_sum[w];
#pragma unroll
  for (int k = 0; k < kPer; k++) {
    const int e = e0 + k;
    if (e > E) break;
    if (mine == 0) offsets[e] = base;
    int at = base + sooner[e];
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
      const int c = next[w][e];
      next[w][e] = at;
      at += c;
    }
    base += all[k];
  }
  __syncthreads();
  const int bits = 32 - __clz(E);
#pragma unroll
  for (int s = 0; s < kSteps; s++) {
    uint64_t same = __ballot(key[s] >= 0);  // lanes with this lane's key
    for (int b = 0; b < bits; b++) {
      const uint64_t set = __ballot((key[s] >> b) & 1);
      same &= (key[s] >> b) & 1 ? set : ~set;
    }
    if (key[s] >= 0) {
      const int before = __popcll(same & ((1ull << lane) - 1));
      const int row = next[wave][key[s]] + before, flat = mine * kChunk + (wave * kSteps + s) * 64 + lane;
      row_of[flat] = row;
      sorted_ids[row] = flat;
      if (sorted_tokens) sorted_tokens[row] = flat / topk;
      // the last of the lanes moves the counter on (the wave's reads of it are done: LDS serves a wave in order)
      if (before == __popcll(same) - 1) next[wave][key[s]] = row + 1;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the next step reads what other lanes have written
  }
}

// ---- permute ---------------------------------------------------------------
// Workgroup (token, column part): the token's chunks once from x, to each of its rows.
template <bool kStream>
__global__ void __launch_bounds__(kThreads)
    permute_rows(const uint4* __restrict__ x, const int32_t* __restrict__ offsets, int E,
                 const int32_t* __restrict__ row_of, int topk, int chunks, uint4* __restrict__ xs) {
  const int64_t t = blockIdx.x;
  const int first_gone = offsets[E];
  const int32_t* rows = row_of + t * topk;
  for (int c = blockIdx.y * kThreads + threadIdx.x; c < chunks; c += gridDim.y * kThreads) {
    const uint4 v = x[t * chunks + c];
#pragma unroll 4
    for (int j = 0; j < topk; j++) {
      const int r = rows[j];
      store_row<kStream>(xs + (int64_t)r * chunks + c, r < first_gone ? v : make_uint4(0, 0, 0, 0));
    }
  }
}

// Sort and permute in one launch, for few pairs: every workgroup ranks its own token's pairs, kGroup at a time, by
// counting the pairs in front of each (expert, then flat index, in one number), and copies its part of the row.  The
// last workgroup of the grid's first axis counts the experts' pairs and writes the offsets instead.
// The work grows with the square of the pairs.  4022 pairs, rows of 256 binary32: 13.6 us in one launch and 35 us for
// a pass forward and back, 42 in the three launches below; 8024 pairs, rows of 1024 bf16: 21.9 us and 37.3 against 36.5.
constexpr int kFewPairs = 4096, kPairBits = 12;
static_assert(1 << kPairBits == kFewPairs, "an expert and a flat index in one number");

__global__ void __launch_bounds__(kThreads)
    sort_permute_few(const int32_t* __restrict__ ids, int T, int topk, int E, const uint4* __restrict__ x, int chunks,
                     uint4* __restrict__ xs, int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_ids,
                     int32_t* __restrict__ sorted_tokens, int32_t* __restrict__ row_of) {
  constexpr int kGroup = 8, kWaves = kThreads / 64, kLoads = 8, kPer = (kMaxKeys + kThreads - 1) / kThreads;
  __shared__ int count[kMaxKeys];  // the last workgroup's; else the group's ranks
  __shared__ int part[kWaves][kGroup / 2];
  const int n = T * topk, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // each id of the list, kLoads loads at a time
  auto for_all = [&](auto f) {
    for (int i0 = 0; i0 < n; i0 += kThreads * kLoads) {
      int id[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; u++) id[u] = ids[min(i0 + u * kThreads + tid, n - 1)];
#pragma unroll
      for (int u = 0; u < kLoads; u++) f(i0 + u * kThreads + tid, (int)min((uint32_t)id[u], (uint32_t)E));
    }
  };
  if ((int)blockIdx.x == T) {
    if (blockIdx.y != 0) return;
    for (int e = tid; e <= E; e += kThreads) count[e] = 0;
    __syncthreads();
    if (n > 0)
      for_all([&](int i, int key) {
        if (i < n) atomicAdd(&count[key], 1);
      });
    __syncthreads();
    int all[kPer], sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; k++) {
      all[k] = tid * kPer + k <= E ? count[tid * kPer + k] : 0;
      sum += all[k];
    }
    int upto = sum;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      const int o = __shfl_up(upto, s, 64);
      if (lane >= s) upto += o;
    }
    if (lane == 63) part[wave][0] = upto;
    __syncthreads();
    int base = upto - sum;
    for (int w = 0; w < wave; w++) base += part[w][0];
#pragma unroll
    for (int k = 0; k < kPer; k++) {
      if (tid * kPer + k <= E) offsets[tid * kPer + k] = base;
      base += all[k];
    }
    return;
  }
  const int t = blockIdx.x;
  for (int j0 = 0; j0 < topk; j0 += kGroup) {
    int mine[kGroup], in_front[kGroup] = {};
#pragma unroll
    for (int u = 0; u < kGroup; u++) {
      const int self = t * topk + j0 + u;
      mine[u] = j0 + u < topk ? (int)min((uint32_t)ids[self], (uint32_t)E) << kPairBits | self : 0;  // 0: none in front
    }
    for_all([&](int i, int key) {
      const int at = i < n ? key << kPairBits | i : 0x7FFFFFFF;
#pragma unroll
      for (int u = 0; u < kGroup; u++) in_front[u] += at < mine[u];
    });
    // two counts a register: 4096 fits in 16 bits
    auto add = [](int a, int b) { return a + b; };
#pragma unroll
    for (int u = 0; u < kGroup; u += 2) {
      const int two = lanes_reduce<6>(in_front[u] | in_front[u + 1] << 16, add);
      if (lane == 0) part[wave][u / 2] = two;
    }
    __syncthreads();
    if (tid < kGroup && j0 + tid < topk) {
      int r = 0;
#pragma unroll
      for (int w = 0; w < kWaves; w++) r += part[w][tid / 2] >> (16 * (tid & 1)) & 0xFFFF;
      const int self = t * topk + j0 + tid;
      const bool kept = (uint32_t)ids[self] < (uint32_t)E;
      count[tid] = kept ? r : ~r;
      if (blockIdx.y == 0) {
        row_of[self] = r;
        sorted_ids[r] = self;
        if (sorted_tokens) sorted_tokens[r] = t;
      }
    }
    __syncthreads();
    if (xs != nullptr)
      for (int c = blockIdx.y * kThreads + tid; c < chunks; c += gridDim.y * kThreads) {
        const uint4 v = x[(int64_t)t * chunks + c];
#pragma unroll
        for (int u = 0; u < kGroup; u++) {
          if (j0 + u >= topk) break;
          const int r = count[u];
          xs[(int64_t)(r < 0 ? ~r : r) * chunks + c] = r < 0 ? make_uint4(0, 0, 0, 0) : v;
        }
      }
    __syncthreads();
  }
}

// Rows that belong to an expert.  Whatever the caller's lists hold, no row past the n there are is touched.
__device__ __forceinline__ uint32_t kept_rows(const int32_t* offsets, int E, int64_t n) {
  return (uint32_t)min((int64_t)max(offsets[E], 0), n);
}

// ---- unpermute -------------------------------------------------------------
template <class In, class Out, bool kStream>
__global__ void __launch_bounds__(kThreads)
    unpermute_rows(const In* __restrict__ ys, const int32_t* __restrict__ offsets, int E,
                   const int32_t* __restrict__ row_of, const float* __restrict__ weights, int topk, int H,
                   Out* __restrict__ out) {
  constexpr int kPer = Rows<In>::kPer, kGroup = 8;
  const int64_t t = blockIdx.x;
  const uint32_t kept = kept_rows(offsets, E, (int64_t)gridDim.x * topk);
  const int chunks = H / kPer;
  const int32_t* rows = row_of + t * topk;
  const float* w = weights == nullptr ? nullptr : weights + t * topk;
  for (int c = blockIdx.y * kThreads + threadIdx.x; c < chunks; c += gridDim.y * kThreads) {
    float sum[kPer] = {};
    if (kept != 0) {
      // eight slots' loads ahead of their use, a row that is not kept read as row 0 and left out
      for (int j0 = 0; j0 < topk; j0 += kGroup) {
        uint4 in[kGroup];
#pragma unroll
        for (int u = 0; u < kGroup; u++) {
          const uint32_t r = j0 + u < topk ? (uint32_t)rows[j0 + u] : kept;
          in[u] = load_row<kStream>(reinterpret_cast<const uint4*>(ys + (int64_t)(r < kept ? r : 0) * H) + c);
        }
#pragma unroll
        for (int u = 0; u < kGroup; u++) {
          if (j0 + u >= topk || (uint32_t)rows[j0 + u] >= kept) continue;
          float v[kPer];
          Rows<In>::load(in[u], v);
          const float wj = w == nullptr ? 1.0f : w[j0 + u];
#pragma unroll
          for (int k = 0; k < kPer; k++) sum[k] = __builtin_fmaf(wj, v[k], sum[k]);
        }
      }
    }
    if constexpr (sizeof(In) == sizeof(Out)) {
      reinterpret_cast<uint4*>(out + t * H)[c] = Rows<Out>::store(sum);
    } else {
      static_assert(kPer == 4 && sizeof(Out) == 2, "binary32 rows to bf16");
      reinterpret_cast<uint2*>(out + t * H)[c] =
          make_uint2(pack_bf16x2_ieee(sum[0], sum[1]), pack_bf16x2_ieee(sum[2], sum[3]));
    }
  }
}

// ---- unpermute, backward ---------------------------------------------------
// One workgroup per token.  Slots in groups of kGroup: the group's dot products are in registers, met in LDS.
template <class T, bool kStream>
__global__ void __launch_bounds__(kThreads)
    unpermute_backward_rows(const T* __restrict__ dout, const T* __restrict__ ys, const int32_t* __restrict__ offsets,
                            int E, const int32_t* __restrict__ row_of, const float* __restrict__ weights, int topk,
                            int H, T* __restrict__ dys, float* __restrict__ dweights) {
  constexpr int kPer = Rows<T>::kPer, kGroup = 8, kWaves = kThreads / 64;
  __shared__ float red[kWaves][kGroup];
  const int64_t t = blockIdx.x, n = (int64_t)gridDim.x * topk;
  const uint32_t kept = kept_rows(offsets, E, n);
  const int chunks = H / kPer;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint4* d = reinterpret_cast<const uint4*>(dout + t * H);
  for (int j0 = 0; j0 < topk; j0 += kGroup) {
    float dot[kGroup] = {};
    for (int c = threadIdx.x; c < chunks; c += kThreads) {
      float g[kPer];
      Rows<T>::load(d[c], g);
#pragma unroll
      for (int u = 0; u < kGroup; u++) {
        if (j0 + u >= topk) break;
        const uint32_t r = (uint32_t)row_of[t * topk + j0 + u];
        if (r >= n) continue;
        uint4 o = make_uint4(0, 0, 0, 0);
        if (r < kept) {
          const float w = weights == nullptr ? 1.0f : weights[t * topk + j0 + u];
          float v[kPer];
          if (dweights != nullptr) {
            Rows<T>::load(load_row<kStream>(reinterpret_cast<const uint4*>(ys + (int64_t)r * H) + c), v);
#pragma unroll
            for (int k = 0; k < kPer; k++) dot[u] = __builtin_fmaf(g[k], v[k], dot[u]);
          }
#pragma unroll
          for (int k = 0; k < kPer; k++) v[k] = w * g[k];
          o = Rows<T>::store(v);
        }
        store_row<kStream>(reinterpret_cast<uint4*>(dys + (int64_t)r * H) + c, o);
      }
    }
    if (dweights == nullptr) continue;
#pragma unroll
    for (int u = 0; u < kGroup; u++) {
      float v = dot[u];
#pragma unroll
      for (int s = 1; s < 64; s *= 2) v += __shfl_xor(v, s, 64);
      if (lane == 0) red[wave][u] = v;
    }
    __syncthreads();
    if ((int)threadIdx.x < kGroup && j0 + (int)threadIdx.x < topk) {
      float v = red[0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < kWaves; k++) v += red[k][threadIdx.x];
      dweights[t * topk + j0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

// Column parts of a token's workgroups: a chunk a thread (4096 tokens of 7168 to 8 rows each: 80 us, 97 with four).
unsigned column_parts(int chunks) { return (unsigned)((chunks + kThreads - 1) / kThreads); }

}  // namespace

size_t moe_permute_workspace(int64_t T, int64_t topk, int64_t E) {
  if (T * topk <= kFewPairs) return 0;
  return (size_t)((T * topk + kChunk - 1) / kChunk + 1) * (E + 1) * sizeof(int32_t);
}

hipError_t launch_moe_permute(const int32_t* ids, int64_t T, int64_t topk, int64_t E, const void* x, int64_t row_bytes,
                              void* xs, int32_t* offsets, int32_t* sorted_ids, int32_t* sorted_tokens, int32_t* row_of,
                              void* ws, hipStream_t stream) {
  const int chunks_row = (int)(row_bytes / 16);
  if (T * topk <= kFewPairs) {
    // a workgroup ranks its token's pairs however little of the row it copies
    const dim3 grid((unsigned)T + 1, x == nullptr || T >= 512 ? 1 : column_parts(chunks_row));
    sort_permute_few<<<grid, kThreads, 0, stream>>>(ids, (int)T, (int)topk, (int)E, static_cast<const uint4*>(x),
                                                    chunks_row, static_cast<uint4*>(xs), offsets, sorted_ids,
                                                    sorted_tokens, row_of);
    return hipGetLastError();
  }
  const int64_t n = T * topk;
  const unsigned chunks = (unsigned)((n + kChunk - 1) / kChunk);
  int32_t* counts = static_cast<int32_t*>(ws);
  sort_count<<<chunks, kThreads, 0, stream>>>(ids, (int)n, (int)E, counts);
  if (sort_direct(chunks, E)) {
    sort_place<false><<<chunks, kThreads, 0, stream>>>(ids, (int)n, (int)topk, (int)E, counts, offsets, sorted_ids,
                                                       sorted_tokens, row_of);
  } else {
    sort_scan<<<(unsigned)((E + 64) / 64), kScanThreads, 0, stream>>>(counts, (int)chunks, (int)E);
    sort_place<true><<<chunks, kThreads, 0, stream>>>(ids, (int)n, (int)topk, (int)E, counts, offsets, sorted_ids,
                                                      sorted_tokens, row_of);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || x == nullptr) return e;
  const dim3 grid((unsigned)T, column_parts(chunks_row));
  auto* const kernel = streamed(n, row_bytes) ? permute_rows<true> : permute_rows<false>;
  kernel<<<grid, kThreads, 0, stream>>>(static_cast<const uint4*>(x), offsets, (int)E, row_of, (int)topk, chunks_row,
                                        static_cast<uint4*>(xs));
  return hipGetLastError();
}

namespace {

template <class In, class Out>
void launch_unpermute(const void* ys, const int32_t* offsets, int64_t E, const int32_t* row_of, const float* weights,
                      int64_t T, int64_t topk, int64_t H, void* out, hipStream_t stream) {
  const dim3 grid((unsigned)T, column_parts((int)(H / Rows<In>::kPer)));
  auto* const kernel = streamed(T * topk, H * (int64_t)sizeof(In)) ? unpermute_rows<In, Out, true>
                                                                   : unpermute_rows<In, Out, false>;
  kernel<<<grid, kThreads, 0, stream>>>(static_cast<const In*>(ys), offsets, (int)E, row_of, weights, (int)topk, (int)H,
                                        static_cast<Out*>(out));
}

template <class T>
void launch_unpermute_backward(const void* dout, const void* ys, const int32_t* offsets, int64_t E, const int32_t* row_of,
                               const float* weights, int64_t tokens, int64_t topk, int64_t H, void* dys, float* dweights,
                               hipStream_t stream) {
  auto* const kernel = streamed(tokens * topk, H * (int64_t)sizeof(T)) ? unpermute_backward_rows<T, true>
                                                                       : unpermute_backward_rows<T, false>;
  kernel<<<(unsigned)tokens, kThreads, 0, stream>>>(static_cast<const T*>(dout), static_cast<const T*>(ys), offsets, (int)E,
                                                    row_of, weights, (int)topk, (int)H, static_cast<T*>(dys), dweights);
}

}  // namespace

hipError_t launch_moe_unpermute(bool in_f32, bool out_f32, const void* ys, const int32_t* offsets, int64_t E,
                                const int32_t* row_of, const float* weights, int64_t T, int64_t topk, int64_t H,
                                void* out, hipStream_t stream) {
  auto* const launch = !in_f32   ? launch_unpermute<uint16_t, uint16_t>
                       : out_f32 ? launch_unpermute<float, float>
                                 : launch_unpermute<float, uint16_t>;
  launch(ys, offsets, E, row_of, weights, T, topk, H, out, stream);
  return hipGetLastError();
}

hipError_t launch_moe_unpermute_backward(bool f32, const void* dout, const void* ys, const int32_t* offsets, int64_t E,
                                         const int32_t* row_of, const float* weights, int64_t T, int64_t topk,
                                         int64_t H, void* dys, float* dweights, hipStream_t stream) {
  auto* const launch = f32 ? launch_unpermute_backward<float> : launch_unpermute_backward<uint16_t>;
  launch(dout, ys, offsets, E, row_of, weights, T, topk, H, dys, dweights, stream);
  return hipGetLastError();
}

}  // namespace bsfp4
