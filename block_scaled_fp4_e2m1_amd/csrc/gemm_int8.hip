// 8-bit integer products with one scale per token and per output channel:
//
//   D[m, n] = bf16(acc[m, n] * sa[m] * sb[n] + bias[n]),  acc = sum_k A[m, k] B[n, k]
//
// acc is exact: 32-bit integers in the matrix cores, and K <= 131056 keeps
// |acc| <= 2^14 K below 2^31.  Its conversion to binary32 and the two scale
// products round once each; split K adds integers, so D does not depend on the
// split.
#include "rows_gemm.h"

namespace bsfp4 {
size_t int8_gemm_workspace(int64_t M, int64_t N, int64_t K) {
  if (rows_ok(M, N, K)) return 0;
  return tile_workspace(plan_tile(M, N, K, device_cu_count()), M, N);
}

bool int8_fused_quant_ok(int64_t M, int64_t N, int64_t K) { return rows_quant_ok(M, N, K); }

hipError_t launch_int8_fused_quant_gemm(const uint16_t* x, const int8_t* B, const float* sb, const uint16_t* bias,
                                        uint16_t* D, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  TileArgs a{};
  a.B = reinterpret_cast<const uint8_t*>(B);
  a.ldb = K;
  a.M = (int)M;
  a.N = (int)N;
  a.kend = K;
  a.sb = sb;
  a.bias = bias;
  a.D = D;
  return launch_rows_quant(a, x, stream);
}

size_t int8_gated_workspace(int64_t M, int64_t I, int64_t K) { return int8_gemm_workspace(M, 2 * I, K); }

hipError_t launch_int8_gemm(const int8_t* A, const float* sa, const int8_t* B, const float* sb, const uint16_t* bias,
                            uint16_t* D, int64_t M, int64_t N, int64_t K, void* ws, hipStream_t stream) {
  TileArgs a{};
  a.A = reinterpret_cast<const uint8_t*>(A);
  a.B = reinterpret_cast<const uint8_t*>(B);
  a.lda = a.ldb = K;
  a.M = (int)M;
  a.N = (int)N;
  a.kend = K;
  a.sa = sa;
  a.sb = sb;
  a.bias = bias;
  a.D = D;
  a.part = ws;
  if (rows_ok(M, N, K)) return launch_rows<true, kTileStore>(a, stream);
  return launch_tile<true, false, false, kTileStore>(a, plan_tile(M, N, K, device_cu_count()), stream);
}

hipError_t launch_int8_gated(const int8_t* A, const float* sa, const int8_t* W, const float* sw, int act, uint16_t* D,
                             int64_t M, int64_t I, int64_t K, void* ws, hipStream_t stream) {
  TileArgs a{};
  a.A = reinterpret_cast<const uint8_t*>(A);
  a.B = reinterpret_cast<const uint8_t*>(W);
  a.lda = a.ldb = K;
  a.M = (int)M;
  a.N = (int)I;
  a.kend = K;
  a.sa = sa;
  a.sb = sw;
  a.act = act;
  a.D = D;
  a.part = ws;
  if (rows_ok(M, 2 * I, K)) return launch_rows<true, kTileGated>(a, stream);
  return launch_tile<true, false, false, kTileGated>(a, plan_tile(M, 2 * I, K, device_cu_count()), stream);
}

}  // namespace bsfp4
