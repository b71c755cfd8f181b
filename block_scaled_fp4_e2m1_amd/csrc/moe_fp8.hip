// E4M3 products over rows sorted by expert, each expert with its own weight: gate and up with silu(gate) * up quantised
// again in the epilogue, and down.
#include "fp8_plan.h"

namespace bsfp4 {
namespace {

template <int EPI>
hipError_t launch_by_rows(Fp8Args a, hipStream_t stream) {
  a.splits = 1;
  auto grid = [&](int bm, int cols) {
    a.tiles_m = (int)fp8_group_tiles(a.M, a.E, bm);
    a.tiles_n = (a.N + cols - 1) / cols;
    return (unsigned)((int64_t)a.tiles_m * a.tiles_n);
  };
  if (fp8_tall_tiles(EPI == kFp8Gated, a.M, a.N, a.E, device_cu_count())) {
    const unsigned n = grid(256, EPI == kFp8Gated ? 128 : 256);
    fp8_grouped_many<EPI><<<n, 512, 0, stream>>>(a);
  } else if constexpr (EPI == kFp8Gated) {
    const unsigned n = grid(64, 128);
    fp8_grouped_few<64, 256, 2, 4, 3, EPI><<<n, 512, 0, stream>>>(a);
  } else {
    const unsigned n = grid(64, 128);
    fp8_grouped_few<64, 128, 2, 2, 3, EPI><<<n, 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_grouped(const uint8_t* A, const float* sa, int64_t a_rows, const int32_t* a_index,
                              const int32_t* offsets, int64_t E, int64_t rows, const uint8_t* W, const float* sw,
                              int64_t N, int64_t K, void* D, bool f32, uint8_t* out_q, float* out_s,
                              hipStream_t stream) {
  Fp8Args a{};
  a.A = A;
  a.sa = sa;
  a.a_rows = a_rows;
  a.a_index = a_index;
  a.offsets = offsets;
  a.E = (int)E;
  a.M = (int)rows;
  a.B = W;
  a.sb = sw;
  a.K = K;
  a.kb = (int)fp8_blocks(K);
  a.b_stride = N * K;
  a.sb_stride = fp8_blocks(N) * a.kb;
  a.N = (int)(out_q != nullptr ? N / 2 : N);
  a.D = D;
  a.q = out_q;
  a.s = out_s;
  if (out_q != nullptr) return launch_by_rows<kFp8Gated>(a, stream);
  return f32 ? launch_by_rows<kFp8F32>(a, stream) : launch_by_rows<kFp8Bf16>(a, stream);
}

}  // namespace bsfp4
