// RMS norms around a block, fused with the gate, the branch scale and the
// residual add, forward and backward.
//
// Forward, per row (token) of H values:
//   n  = x * rstd(x) * w_post                 (x itself without w_post)
//   r' = bf16(r + (gate * scale) * n)
//   z  = bf16(r' * rstd(r') * w_pre)           (bf16 rows, or 8-bit rows with a scale)
//   rstd(v) = fl32(1 / sqrt(mean(v^2) + eps))
// gate is [G, H]: T / G consecutive rows share a gate row.  The next norm reads
// the residual row as it is stored (rounded to bf16).
//
// Every elementwise step is one binary32 operation in the order written.  The
// mean squares are summed in 64 bits: squares of bf16 values are exact there and
// the order of the sum moves the 32-bit rstd practically never, so a row's bytes
// (its 8-bit codes in particular) do not depend on how many threads hold it.
//
// Backward, with rs = rstd(r'), xs = rstd(x), zh = r' rs, xh = x xs, mean over the row:
//   gz = dz w_pre,  d = dr' + rs (gz - zh mean(gz zh)),  dr = bf16(d)
//   dn = d (gate scale),  gx = dn w_post,  dx = xs (gx - xh mean(gx xh))
//   dw_pre = sum_rows dz zh,  dw_post = sum_rows dn xh,  dgate = sum_group d scale n
// Both means need only sums of stored values (mean(gz zh) = rs sum(gz r') / H),
// so a row takes two reductions: {sum x^2, sum r'^2, sum gz r'} and {sum gx x}.
//
// Bound by memory: forward 4 H bytes read and 4 H (3 H) written per row, backward
// 8 H read and 4 H written; the row stays in registers between the reductions.
// 8192 x 4096, other data in the caches before: forward 45 us (6.0 TB/s; 41 without post-norm and
// gate, 22 the pre-norm alone), backward 74 (5.4 TB/s) and 6 for the sums over the strips: a
// row's two reductions are waited for with one row ahead in registers.  With parts left
// out the backward kernel branches on them at run time and spills 14 registers: 110 us
// without post-norm and gate, 60 the pre-norm alone.
#include <algorithm>

#include "int8_rows.h"
#include "launchers.h"

#pragma clang fp contract(off)

namespace bsfp4 {
namespace {

// fl32(1 / sqrt(sum inv_h + eps)), inv_h = 1 / H: the hardware's 64-bit estimate and two Newton
// steps, y (1.5 - 0.5 v y^2), leave an error far below half a 32-bit unit.
__device__ __forceinline__ float rstd_of(double sum, double inv_h, double eps) {
  const double v = sum * inv_h + eps;
  double y = __builtin_amdgcn_rsq(v);
  if (v < __builtin_inf()) {
#pragma unroll
    for (int i = 0; i < 2; i++) y = y * (1.5 - 0.5 * v * y * y);
  }
  return (float)y;
}

__device__ __forceinline__ double sumsq8(const uint4& c, double s) {
  float v[8];
  unpack8(c, v);
#pragma unroll
  for (int j = 0; j < 8; j++) s = __builtin_fma((double)v[j], (double)v[j], s);
  return s;
}

__device__ __forceinline__ uint4 chunk_or_zero(const uint16_t* row, int i, bool live) {
  return live ? reinterpret_cast<const uint4*>(row)[i] : make_uint4(0, 0, 0, 0);
}

// A row as a buffer: lanes past its end read zeros and write nothing, and the
// address is four scalars and a 32-bit lane offset for every array.
struct RowBuf {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ RowBuf(const uint16_t* p, int64_t m, int H, bool live = true)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p) + m * H, (short)0, live ? 2 * H : 0, 0x00020000)) {}
  __device__ __forceinline__ uint4 load(int i) const {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, i * 16, 0, 0));
  }
  __device__ __forceinline__ void store(int i, const uint4& v) const {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{v.x, v.y, v.z, v.w}, r, i * 16, 0, 0);
  }
};

// Keeps a chunk packed: unpacked copies of loop invariants would cost twice the
// registers (and a workgroup per compute unit in the backward pass).
__device__ __forceinline__ void keep_packed(uint4& c) {
  asm volatile("" : "+v"(c.x), "+v"(c.y), "+v"(c.z), "+v"(c.w));
}

template <int NT, int CH, bool kInt8>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT)
    block_norm_fwd(const BlockNormArgs p) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  static_assert(kRows == 1 || NT == 64, "several rows per workgroup: a wave each");
  __shared__ double red[2][NT / 64];
  __shared__ int redm[NT / 64];
  const int t = kRows > 1 ? (int)(threadIdx.x % NT) : (int)threadIdx.x;
  const int64_t m = (int64_t)blockIdx.x * kRows + (kRows > 1 ? threadIdx.x / NT : 0);
  if (m >= p.T) return;
  const int H = p.H, chunks = H / 8;
  const int64_t off = m * (int64_t)H;
  uint4 x[CH], r[CH], wp[CH], gt[CH], wn[CH];
#pragma unroll
  for (int j = 0; j < CH; j++) {
    const int i = t + j * NT;
    const bool live = i < chunks;
    if (p.x) x[j] = chunk_or_zero(p.x + off, i, live);
    r[j] = chunk_or_zero(p.residual + off, i, live);
    if (p.w_post) wp[j] = chunk_or_zero(p.w_post, i, live);
    if (p.gate) gt[j] = chunk_or_zero(p.gate + (m / p.group_rows) * H, i, live);
    if (p.w_pre) wn[j] = chunk_or_zero(p.w_pre, i, live);
  }
  if (p.x) {
    float xs = 1.0f;
    if (p.w_post) {
      double s[1] = {0.0};
#pragma unroll
      for (int j = 0; j < CH; j++) s[0] = sumsq8(x[j], s[0]);
      row_sum<NT>(s, red[0]);
      xs = rstd_of(s[0], p.inv_h, p.eps);
    }
#pragma unroll
    for (int j = 0; j < CH; j++) {
      float xv[8], rv[8], wv[8], gv[8];
      unpack8(x[j], xv);
      unpack8(r[j], rv);
      if (p.w_post) unpack8(wp[j], wv);
      if (p.gate) unpack8(gt[j], gv);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float n = p.w_post ? xv[k] * xs * wv[k] : xv[k];
        const float g = p.gate ? gv[k] * p.scale : p.scale;
        rv[k] = rv[k] + g * n;
      }
      r[j] = pack8(rv);
      const int i = t + j * NT;
      if (i < chunks) reinterpret_cast<uint4*>(p.res_out + off)[i] = r[j];
    }
  }
  if (!p.w_pre) return;
  double s[1] = {0.0};
#pragma unroll
  for (int j = 0; j < CH; j++) s[0] = sumsq8(r[j], s[0]);
  row_sum<NT>(s, red[1]);
  const float rs = rstd_of(s[0], p.inv_h, p.eps);
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < CH; j++) {
    float rv[8], wv[8];
    unpack8(r[j], rv);
    unpack8(wn[j], wv);
#pragma unroll
    for (int k = 0; k < 8; k++) rv[k] = rv[k] * rs * wv[k];
    r[j] = pack8(rv);
    const int i = t + j * NT;
    if constexpr (kInt8) {
      // lanes past the row hold zeros times a finite or infinite rstd: keep them out
      if (i < chunks) mx = amax_bits8(r[j], mx);
    } else {
      if (i < chunks) reinterpret_cast<uint4*>(p.z + off)[i] = r[j];
    }
  }
  if constexpr (kInt8) {
    const Int8Row q(row_max<NT>(mx, redm));
#pragma unroll
    for (int j = 0; j < CH; j++) {
      const int i = t + j * NT;
      if (i < chunks) reinterpret_cast<uint2*>(p.q + off)[i] = q.codes8(r[j]);
    }
    if (t == 0) p.s[m] = q.s;
  }
}

// One workgroup of NT threads walks the rows of a strip with its columns' three
// vector gradients in registers.  Strips are either 1 / S of a gate group (the
// group's dgate is then summed over S partials), or whole groups (its dgate is
// final).  CH 16-byte chunks per thread: 1 up to H = 8 NT.
template <int NT, int CH, bool kAll>
__global__ void __launch_bounds__(NT, 4)
    block_norm_bwd(const BlockNormArgs p) {
  // with w_post the second reduction's barrier stands between a row's reads of red_a and
  // the next row's writes; without, red_a alternates row by row
  __shared__ double red_a[kAll ? 1 : 2][3 * (NT / 64)];
  __shared__ double red_b[NT / 64];
  int parity = 0;
  const int t = threadIdx.x;
  const int H = p.H, chunks = H / 8;
  const bool has_x = kAll || p.x != nullptr, has_post = kAll || p.w_post != nullptr, has_pre = kAll || p.w_pre != nullptr,
             has_gate = kAll || p.gate != nullptr, has_dres = kAll || p.dres_out != nullptr;
  const int64_t strip = blockIdx.x;
  int64_t g0, g1, part = 0, parts = 1;
  if (p.strips_per_group > 1) {
    parts = p.strips_per_group;
    g0 = strip / parts;
    g1 = g0 + 1;
    part = strip % parts;
  } else {
    g0 = strip * p.groups_per_strip;
    g1 = min(g0 + p.groups_per_strip, p.groups);
  }
  float apost[CH][8] = {}, apre[CH][8] = {};
  // Two chunks per thread leave no registers for a row ahead nor for the vectors,
  // which are then read again with every row (from the caches).
  constexpr bool kAhead = CH == 1;
  uint4 wp[CH] = {}, wn[CH] = {}, gt[CH] = {};
  auto vectors = [&](int64_t g) {
#pragma unroll
    for (int j = 0; j < CH; j++) {
      const int i = t + j * NT;
      if (has_post) wp[j] = RowBuf(p.w_post, 0, H).load(i);
      if (has_pre) wn[j] = RowBuf(p.w_pre, 0, H).load(i);
      if (has_gate) gt[j] = RowBuf(p.gate, g, H).load(i);
    }
  };
  for (int64_t g = g0; g < g1; g++) {
    const int64_t ra = g * p.group_rows + p.group_rows * part / parts;
    const int64_t rb = g * p.group_rows + p.group_rows * (part + 1) / parts;
    float agate[CH][8] = {};
    if (kAhead) vectors(g);
    uint4 nx[CH], nr[CH], nz[CH], nd[CH];  // the next row's chunks
    auto load = [&](int64_t m) {
#pragma unroll
      for (int j = 0; j < CH; j++) {
        const int i = t + j * NT;
        if (has_x) nx[j] = RowBuf(p.x, m, H, m < rb).load(i);
        if (has_pre) nr[j] = RowBuf(p.res, m, H, m < rb).load(i);
        if (has_pre) nz[j] = RowBuf(p.dz, m, H, m < rb).load(i);
        if (has_dres) nd[j] = RowBuf(p.dres_out, m, H, m < rb).load(i);
      }
    };
    if (kAhead) load(ra);
    for (int64_t m = ra; m < rb; m++) {
      if (!kAhead) {
        load(m);
        vectors(g);
      }
      uint4 x[CH], r[CH], z[CH], d4[CH];
#pragma unroll
      for (int j = 0; j < CH; j++) {
        x[j] = nx[j];
        r[j] = nr[j];
        z[j] = nz[j];
        d4[j] = nd[j];
        keep_packed(wp[j]);
        keep_packed(wn[j]);
        keep_packed(gt[j]);
      }
      if (kAhead) load(m + 1);
      double s[3] = {0.0, 0.0, 0.0};
#pragma unroll
      for (int j = 0; j < CH; j++) {
        if (has_x && has_post) s[0] = sumsq8(x[j], s[0]);
        if (has_pre) {
          s[1] = sumsq8(r[j], s[1]);
          float rv[8], zv[8], wv[8], dot = 0.0f;
          unpack8(r[j], rv);
          unpack8(z[j], zv);
          unpack8(wn[j], wv);
#pragma unroll
          for (int k = 0; k < 8; k++) dot = __builtin_fmaf(zv[k] * wv[k], rv[k], dot);
          s[2] += (double)dot;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      row_sum<NT>(s, red_a[parity]);
      if (!kAll) parity ^= 1;
      __builtin_amdgcn_sched_barrier(0);
      const float xs = has_x && has_post ? rstd_of(s[0], p.inv_h, p.eps) : 1.0f;
      const float rs = has_pre ? rstd_of(s[1], p.inv_h, p.eps) : 1.0f;
      const float mz = (float)(s[2] * p.inv_h) * rs;  // mean(gz zh)
      float d[CH][8];
      double sb[1] = {0.0};
#pragma unroll
      for (int j = 0; j < CH; j++) {
        keep_packed(x[j]);
        keep_packed(r[j]);
        keep_packed(z[j]);
        keep_packed(wn[j]);
        float rv[8], zv[8], wv[8];
        if (has_dres) {
          unpack8(d4[j], d[j]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; k++) d[j][k] = 0.0f;
        }
        if (has_pre) {
          unpack8(r[j], rv);
          unpack8(z[j], zv);
          unpack8(wn[j], wv);
#pragma unroll
          for (int k = 0; k < 8; k++) {
            const float zh = rv[k] * rs;
            d[j][k] += rs * (zv[k] * wv[k] - zh * mz);
            apre[j][k] += zv[k] * zh;
          }
        }
        const int i = t + j * NT;
        RowBuf(p.dres, m, H).store(i, pack8(d[j]));
        if (has_x) {
          float xv[8], pv[8], gv[8], dot = 0.0f;
          unpack8(x[j], xv);
          if (has_post) unpack8(wp[j], pv);
          if (has_gate) unpack8(gt[j], gv);
#pragma unroll
          for (int k = 0; k < 8; k++) {
            const float xh = xv[k] * xs;
            const float n = has_post ? xh * pv[k] : xh;
            if (has_gate) agate[j][k] += d[j][k] * p.scale * n;
            const float dn = d[j][k] * (has_gate ? gv[k] * p.scale : p.scale);
            if (has_post) apost[j][k] += dn * xh;
            d[j][k] = has_post ? dn * pv[k] : dn;  // gx from here on
            dot = __builtin_fmaf(d[j][k], xv[k], dot);
          }
          sb[0] += (double)dot;
        }
      }
      if (has_x) {
        float mx = 0.0f;  // mean(gx xh) xs
        if (has_post) {
          __builtin_amdgcn_sched_barrier(0);
          row_sum<NT>(sb, red_b);
          __builtin_amdgcn_sched_barrier(0);
          mx = (float)(sb[0] * p.inv_h) * xs;
        }
#pragma unroll
        for (int j = 0; j < CH; j++) {
          keep_packed(x[j]);
          if (has_post) {
            float xv[8];
            unpack8(x[j], xv);
#pragma unroll
            for (int k = 0; k < 8; k++) d[j][k] = xs * (d[j][k] - xv[k] * xs * mx);
          }
          RowBuf(p.dx, m, H).store(t + j * NT, pack8(d[j]));
        }
      }
    }
    if (has_gate) {
      float* dst = parts > 1 ? p.part_gate + strip * H : p.dgate + g * H;
#pragma unroll
      for (int j = 0; j < CH; j++) {
        const int i = t + j * NT;
        if (i < chunks) {
          reinterpret_cast<float4*>(dst)[2 * i] = make_float4(agate[j][0], agate[j][1], agate[j][2], agate[j][3]);
          reinterpret_cast<float4*>(dst)[2 * i + 1] = make_float4(agate[j][4], agate[j][5], agate[j][6], agate[j][7]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < CH; j++) {
    const int i = t + j * NT;
    if (i >= chunks) continue;
    if (has_post) {
      float4* dst = reinterpret_cast<float4*>(p.part_post + strip * H);
      dst[2 * i] = make_float4(apost[j][0], apost[j][1], apost[j][2], apost[j][3]);
      dst[2 * i + 1] = make_float4(apost[j][4], apost[j][5], apost[j][6], apost[j][7]);
    }
    if (has_pre) {
      float4* dst = reinterpret_cast<float4*>(p.part_pre + strip * H);
      dst[2 * i] = make_float4(apre[j][0], apre[j][1], apre[j][2], apre[j][3]);
      dst[2 * i + 1] = make_float4(apre[j][4], apre[j][5], apre[j][6], apre[j][7]);
    }
  }
}

// out[h] = sum over strips of part[strip][h], in a fixed order: workgroups of 64
// columns, 16 threads of four columns each on every 64th strip.  blockIdx.y: 0
// dw_post, 1 dw_pre, 2 + g dgate of group g.
__global__ void __launch_bounds__(1024)
    block_norm_sum(const BlockNormArgs p, int64_t strips) {
  __shared__ __attribute__((aligned(16))) float red[64][64];
  const int which = blockIdx.y;
  const float* src;
  float* dst;
  int64_t n = strips;
  if (which == 0) {
    src = p.part_post;
    dst = p.dw_post;
  } else if (which == 1) {
    src = p.part_pre;
    dst = p.dw_pre;
  } else {
    n = p.strips_per_group;
    src = p.part_gate ? p.part_gate + (int64_t)(which - 2) * n * p.H : nullptr;
    dst = p.dgate ? p.dgate + (int64_t)(which - 2) * p.H : nullptr;
  }
  if (src == nullptr) return;
  const int c4 = threadIdx.x & 15, w = threadIdx.x >> 4;
  const int h = blockIdx.x * 64 + c4 * 4;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (h < p.H) {  // H % 8 == 0: four columns are in or out together
#pragma unroll 4
    for (int64_t s = w; s < n; s += 64) {
      const float4 v = *reinterpret_cast<const float4*>(src + s * p.H + h);
      acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
    }
  }
  *reinterpret_cast<float4*>(&red[w][c4 * 4]) = acc;
  const int c = threadIdx.x & 63, k = threadIdx.x >> 6;
  __syncthreads();
  const float v = (red[k][c] + red[k + 16][c]) + (red[k + 32][c] + red[k + 48][c]);
  __syncthreads();
  red[k][c] = v;
  __syncthreads();
  if (k == 0 && blockIdx.x * 64 + c < p.H) {
    float t = red[0][c];
#pragma unroll
    for (int i = 1; i < 16; i++) t += red[i][c];
    dst[blockIdx.x * 64 + c] = t;
  }
}

struct Strips {
  int64_t per_group, groups_per_strip, count;
};

// Threads of a row in the backward pass: one chunk each up to H = 8192, else two.
int bwd_threads(int64_t H) {
  const int64_t chunks = H / 8;
  int nt = 64;
  while (nt < 1024 && nt < chunks) nt *= 2;
  return nt;
}

// As many strips as workgroups are resident at once (16 waves of 128 registers per
// compute unit), at most one per row: a row's two reductions cost some 2 us of
// latency, so few rows are spread wide; past one per compute unit a strip takes
// four rows, as its partial vectors cost the bytes of one.  More than 1024 strips cost more in the sum
// of their vectors than they save (4000 x 512 with 4000 strips 38 us, with 250 25).
Strips plan_strips(int64_t T, int64_t H, int64_t groups) {
  const int64_t resident = std::min<int64_t>(1024, (int64_t)device_cu_count() * (1024 / bwd_threads(H)));
  const int64_t cus = device_cu_count();
  const int64_t want = std::min<int64_t>(resident, std::max<int64_t>(std::max<int64_t>(1, std::min(T, cus)), T / 4));
  const int64_t rows = T / groups;
  Strips s;
  if (groups >= want) {
    s.per_group = 1;
    s.groups_per_strip = (groups + want - 1) / want;
    s.count = (groups + s.groups_per_strip - 1) / s.groups_per_strip;
  } else {
    s.per_group = std::min<int64_t>(rows, (want + groups - 1) / groups);
    s.groups_per_strip = 1;
    s.count = groups * s.per_group;
  }
  return s;
}

}  // namespace

size_t block_norm_bwd_workspace(int64_t T, int64_t H, int64_t groups) {
  return (size_t)plan_strips(T, H, groups).count * H * 3 * sizeof(float);
}

hipError_t launch_block_norm(const BlockNormArgs& p, hipStream_t stream) {
  const int chunks = p.H / 8;
#define BSFP4_FWD(NT, CH)                                                                              \
  do {                                                                                                 \
    const unsigned grid = (unsigned)(NT < 256 ? (p.T + 256 / NT - 1) / (256 / NT) : p.T);              \
    if (p.q)                                                                                           \
      block_norm_fwd<NT, CH, true><<<grid, NT < 256 ? 256 : NT, 0, stream>>>(p);                       \
    else                                                                                               \
      block_norm_fwd<NT, CH, false><<<grid, NT < 256 ? 256 : NT, 0, stream>>>(p);                      \
  } while (0)
  // Many rows: two chunks per thread keep more bytes in flight (8192 x 4096 40.6 us
  // against 45.2 with one, 4000 x 7168 36.5 against 43.0); few rows or short ones: one
  // chunk, more threads, less latency (1 x 4096 3.5 against 4.5, 1024 x 2048 5.9
  // against 6.6).
  const bool many = p.T >= 1024;
  if (chunks <= 64) BSFP4_FWD(64, 1);
  else if (chunks <= 256) BSFP4_FWD(256, 1);
  else if (chunks <= 512 && many) BSFP4_FWD(256, 2);
  else if (chunks <= 512) BSFP4_FWD(512, 1);
  else if (chunks <= 1024 && many) BSFP4_FWD(512, 2);
  else if (chunks <= 1024) BSFP4_FWD(1024, 1);
  else BSFP4_FWD(1024, 2);
#undef BSFP4_FWD
  return hipGetLastError();
}

hipError_t launch_block_norm_bwd(BlockNormArgs p, float* ws, hipStream_t stream) {
  const Strips s = plan_strips(p.T, p.H, p.groups);
  p.strips_per_group = s.per_group;
  p.groups_per_strip = s.groups_per_strip;
  const size_t n = (size_t)s.count * p.H;
  p.part_post = p.w_post ? ws : nullptr;
  p.part_pre = p.w_pre ? ws + n : nullptr;
  p.part_gate = p.gate && s.per_group > 1 ? ws + 2 * n : nullptr;
  const int chunks = p.H / 8;
  const unsigned grid = (unsigned)s.count;
  const bool all = p.x && p.w_post && p.w_pre && p.gate && p.dres_out && p.T > 0;
#define BSFP4_BWD(NT, CH)                                        \
  do {                                                           \
    if (all) block_norm_bwd<NT, CH, true><<<grid, NT, 0, stream>>>(p); \
    else block_norm_bwd<NT, CH, false><<<grid, NT, 0, stream>>>(p);    \
  } while (0)
  switch (bwd_threads(p.H)) {
    case 64: BSFP4_BWD(64, 1); break;
    case 128: BSFP4_BWD(128, 1); break;
    case 256: BSFP4_BWD(256, 1); break;
    case 512: BSFP4_BWD(512, 1); break;
    default:
      if (chunks <= 1024) BSFP4_BWD(1024, 1);
      else BSFP4_BWD(1024, 2);
  }
#undef BSFP4_BWD
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!p.part_post && !p.part_pre && !p.part_gate) return hipSuccess;
  const dim3 sg((unsigned)((p.H + 63) / 64), (unsigned)(2 + (p.part_gate ? p.groups : 0)));
  block_norm_sum<<<sg, 1024, 0, stream>>>(p, s.count);
  return hipGetLastError();
}

}  // namespace bsfp4
