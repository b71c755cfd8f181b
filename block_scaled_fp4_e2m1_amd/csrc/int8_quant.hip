// bf16 -> 8-bit integers with one scale per row (token).
//
//   amax_m = max_k |x[m,k]|,  s_m = amax_m / 127,  q[m,k] = rne(127 x[m,k] / amax_m)
//
// q is the correctly rounded quotient (Int8Row), so the codes are a function of
// the values alone.  An all-zero row gives s = 0 and zero codes; a row holding
// an infinity or a NaN gives s = NaN and zero codes, so whatever is computed
// from it is NaN as well.
//
// Bound by memory: 2 bytes read and 1 written per element.  A row is read once
// and kept in registers between the maximum and the rounding, by 64, 256 or 1024
// threads with at most four 16-byte chunks each (rows of 2048, 8192, 32768
// values); longer rows are read a second time, from the caches.  4096 x 7168: 17 us,
// 5.2 TB/s, what a copy reaches.
#include "int8_rows.h"
#include "launchers.h"

namespace bsfp4 {
namespace {

constexpr int kChunks = 4;

// NT threads per row, 256 / NT rows per workgroup when NT < 256.
template <int NT>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT)
    int8_quant_rows(const uint16_t* __restrict__ x, int64_t M, int K, int8_t* __restrict__ q,
                    float* __restrict__ s) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  __shared__ int red[NT / 64];
  const int t = kRows > 1 ? (int)(threadIdx.x % NT) : (int)threadIdx.x;
  const int64_t m = (int64_t)blockIdx.x * kRows + (kRows > 1 ? threadIdx.x / NT : 0);
  if (m >= M) return;  // a whole wave (rows shared by several waves fill the grid exactly)
  const int chunks = K / 8;
  const uint4* row = reinterpret_cast<const uint4*>(x + m * (int64_t)K);
  uint2* out = reinterpret_cast<uint2*>(q + m * (int64_t)K);
  uint4 c[kChunks];
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < kChunks; j++) {
    const int i = t + j * NT;
    c[j] = i < chunks ? row[i] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < kChunks; j++) mx = amax_bits8(c[j], mx);
  for (int i = t + kChunks * NT; i < chunks; i += NT) mx = amax_bits8(row[i], mx);
  const Int8Row r(row_max<NT>(mx, red));
#pragma unroll
  for (int j = 0; j < kChunks; j++) {
    const int i = t + j * NT;
    if (i < chunks) out[i] = r.codes8(c[j]);
  }
  for (int i = t + kChunks * NT; i < chunks; i += NT) out[i] = r.codes8(row[i]);
  if (t == 0) s[m] = r.s;
}

}  // namespace

hipError_t launch_int8_quant(const uint16_t* x, int64_t M, int64_t K, int8_t* q, float* s, hipStream_t stream) {
  if (K <= 64 * 8 * kChunks)
    int8_quant_rows<64><<<(unsigned)((M + 3) / 4), 256, 0, stream>>>(x, M, (int)K, q, s);
  else if (K <= 256 * 8 * kChunks)
    int8_quant_rows<256><<<(unsigned)M, 256, 0, stream>>>(x, M, (int)K, q, s);
  else
    int8_quant_rows<1024><<<(unsigned)M, 1024, 0, stream>>>(x, M, (int)K, q, s);
  return hipGetLastError();
}

}  // namespace bsfp4
