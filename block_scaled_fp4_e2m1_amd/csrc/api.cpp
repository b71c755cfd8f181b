// C ABI of libbsfp4: argument validation, device check, dispatch.
//
// Every entry point validates all arguments before launching anything and
// reports the first violation through a status code plus a per-thread
// message.  Checks follow the pages' entry points (vLLM `sm103` branch
// comparison page: `scaled_fp4_quant_sm103a_impl` requires a row length
// divisible by 16 and bf16/fp16 input; `cutlass_scaled_fp4_mm_sm103a_impl`
// requires equal K, K % 32 == 0 and N % 32 == 0, contiguous scale tensors;
// "feat: sm100 cute_dsl w4a16 gemm" review: bf16 activations, aligned
// pointers, exact scale sizes) restated for this library's unpadded layouts.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "../../include/bsfp4.h"
#include "launchers.h"

namespace {

thread_local char g_err[512] = "";

bsfp4_status fail(bsfp4_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return s;
}

bsfp4_status ok() {
  g_err[0] = '\0';
  return BSFP4_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The MXFP4 kernels address an operand with 32-bit buffer offsets from its
// base (one expert's weights in the grouped form), so each must stay below
// 2^31 bytes.
constexpr int64_t kLim31 = (int64_t)1 << 31;

#define REQUIRE_PTR(p)                                                             \
  do {                                                                             \
    if ((p) == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "%s is NULL", #p);      \
    if (!aligned((p), 16)) return fail(BSFP4_ERR_ALIGNMENT, "%s is not 16-byte aligned", #p); \
  } while (0)

#define REQUIRE_SCALAR_PTR(p)                                                      \
  do {                                                                             \
    if ((p) == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "%s is NULL", #p);      \
    if (!aligned((p), 4)) return fail(BSFP4_ERR_ALIGNMENT, "%s is not 4-byte aligned", #p); \
  } while (0)

// The current device must be a gfx950; the answer is cached per device id.
bsfp4_status check_device() {
  static std::mutex mu;
  static int known[64] = {0};  // 0 unknown, 1 gfx950, 2 other
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess || dev < 0)
    return fail(BSFP4_ERR_DEVICE, "no HIP device: %s", hipGetErrorString(e));
  if (dev < 64) {
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev] == 0) {
      hipDeviceProp_t prop;
      e = hipGetDeviceProperties(&prop, dev);
      if (e != hipSuccess) return fail(BSFP4_ERR_DEVICE, "hipGetDeviceProperties: %s", hipGetErrorString(e));
      known[dev] = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    }
    if (known[dev] == 1) return BSFP4_OK;
  }
  return fail(BSFP4_ERR_DEVICE, "device %d is not a gfx950 GPU", dev);
}

bsfp4_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(BSFP4_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int bsfp4_version(void) { return 100; }

const char* bsfp4_status_string(int s) {
  switch (s) {
    case BSFP4_OK: return "ok";
    case BSFP4_ERR_INVALID_ARG: return "invalid argument";
    case BSFP4_ERR_SHAPE: return "unsupported shape";
    case BSFP4_ERR_ALIGNMENT: return "misaligned pointer";
    case BSFP4_ERR_WORKSPACE: return "workspace too small";
    case BSFP4_ERR_DEVICE: return "unsupported device";
    case BSFP4_ERR_HIP: return "HIP error";
    default: return "unknown status";
  }
}

const char* bsfp4_last_error(void) { return g_err; }

// ------------------------------------------------------------------ global scale

size_t fp4_global_scale_workspace_size(int64_t numel) {
  if (numel <= 0) return 0;
  return sizeof(float) * (size_t)bsfp4::global_scale_parts(numel);
}

bsfp4_status fp4_global_scale(const uint16_t* x, int64_t numel, float* gs_out, void* ws,
                              size_t ws_bytes, void* stream) {
  if (numel <= 0) return fail(BSFP4_ERR_SHAPE, "numel must be > 0 (got %lld)", (long long)numel);
  REQUIRE_PTR(x);
  REQUIRE_SCALAR_PTR(gs_out);
  REQUIRE_SCALAR_PTR(ws);
  const size_t need = fp4_global_scale_workspace_size(numel);
  if (ws_bytes < need)
    return fail(BSFP4_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws_bytes, need);
  if (bsfp4_status s = check_device()) return s;
  return launched(bsfp4::launch_global_scale(x, numel, gs_out, static_cast<float*>(ws), as_stream(stream)),
                  "fp4_global_scale launch");
}

// ------------------------------------------------------------------ quantiser

bsfp4_status fp4_quantize(int fmt, const uint16_t* x, int64_t rows_in, int64_t K, const float* gs,
                          const int32_t* row_map, int64_t rows_out, uint8_t* q, uint8_t* sf,
                          void* stream) {
  if (fmt != BSFP4_NVFP4 && fmt != BSFP4_MXFP4) return fail(BSFP4_ERR_INVALID_ARG, "unknown format %d", fmt);
  if (rows_in < 0 || rows_out < 0 || K <= 0)
    return fail(BSFP4_ERR_SHAPE, "need rows >= 0 and K > 0 (rows_in=%lld rows_out=%lld K=%lld)",
                (long long)rows_in, (long long)rows_out, (long long)K);
  const int blk = fmt == BSFP4_NVFP4 ? 16 : 32;
  if (K % blk) return fail(BSFP4_ERR_SHAPE, "K=%lld is not a multiple of %d", (long long)K, blk);
  if (row_map == nullptr && rows_out != rows_in)
    return fail(BSFP4_ERR_SHAPE, "without row_map rows_out (%lld) must equal rows_in (%lld)",
                (long long)rows_out, (long long)rows_in);
  if (fmt == BSFP4_NVFP4) {
    REQUIRE_SCALAR_PTR(gs);
  } else if (gs != nullptr) {
    return fail(BSFP4_ERR_INVALID_ARG, "MXFP4 takes no global scale (gs must be NULL)");
  }
  if (rows_out == 0) return ok();
  if (rows_in > 0) REQUIRE_PTR(x);
  if (row_map != nullptr && !aligned(row_map, 4)) return fail(BSFP4_ERR_ALIGNMENT, "row_map is not 4-byte aligned");
  REQUIRE_PTR(q);
  if (sf == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "sf is NULL");
  if (bsfp4_status s = check_device()) return s;
  return launched(bsfp4::launch_quantize(fmt, x, rows_in, K, gs, row_map, rows_out, q, sf, as_stream(stream)),
                  "fp4_quantize launch");
}

// ------------------------------------------------------------------ GEMM

size_t fp4_gemm_workspace_size(int fmt, int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N <= 0 || K <= 0) return 0;
  if (fmt == BSFP4_NVFP4) return bsfp4::nvfp4_gemm_workspace(M, N, K);
  return 0;
}

// Argument checks shared by fp4_gemm and fp4_gemm_noalloc (everything but the
// workspace).
static bsfp4_status check_gemm_args(int fmt, const uint8_t* A, const uint8_t* SFA, const uint8_t* B,
                                    const uint8_t* SFB, const float* alpha, const uint16_t* D, int64_t M, int64_t N,
                                    int64_t K) {
  if (fmt != BSFP4_NVFP4 && fmt != BSFP4_MXFP4) return fail(BSFP4_ERR_INVALID_ARG, "unknown format %d", fmt);
  if (M < 0 || N <= 0 || K <= 0)
    return fail(BSFP4_ERR_SHAPE, "need M >= 0, N > 0, K > 0 (M=%lld N=%lld K=%lld)", (long long)M,
                (long long)N, (long long)K);
  if (K % 32) return fail(BSFP4_ERR_SHAPE, "K=%lld is not a multiple of 32", (long long)K);
  if (N % 32) return fail(BSFP4_ERR_SHAPE, "N=%lld is not a multiple of 32", (long long)N);
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
    return fail(BSFP4_ERR_SHAPE, "dimensions must fit in 31 bits");
  if (fmt == BSFP4_MXFP4 && (M * (K / 2) >= kLim31 || N * (K / 2) >= kLim31))
    return fail(BSFP4_ERR_SHAPE, "MXFP4 operands must stay below 2^31 bytes (M*K/2=%lld, N*K/2=%lld)",
                (long long)(M * (K / 2)), (long long)(N * (K / 2)));
  if (M > 0) {
    REQUIRE_PTR(A);
    REQUIRE_PTR(SFA);
    REQUIRE_PTR(D);
  }
  REQUIRE_PTR(B);
  REQUIRE_PTR(SFB);
  if (alpha != nullptr && !aligned(alpha, 4)) return fail(BSFP4_ERR_ALIGNMENT, "alpha is not 4-byte aligned");
  return BSFP4_OK;
}

static bsfp4_status launch_gemm(int fmt, const uint8_t* A, const uint8_t* SFA, const uint8_t* B, const uint8_t* SFB,
                                const float* alpha, uint16_t* D, int64_t M, int64_t N, int64_t K, void* ws,
                                size_t ws_bytes, hipStream_t st) {
  if (fmt == BSFP4_NVFP4)
    return launched(bsfp4::launch_nvfp4_gemm(A, SFA, B, SFB, alpha, D, M, N, K, ws, ws_bytes, st), "fp4_gemm launch");
  return launched(bsfp4::launch_mxfp4_gemm(A, SFA, B, SFB, alpha, D, M, N, K, st), "fp4_gemm launch");
}

bsfp4_status fp4_gemm(int fmt, const uint8_t* A, const uint8_t* SFA, const uint8_t* B,
                      const uint8_t* SFB, const float* alpha, uint16_t* D, int64_t M, int64_t N,
                      int64_t K, void* ws, size_t ws_bytes, void* stream) {
  if (bsfp4_status s = check_gemm_args(fmt, A, SFA, B, SFB, alpha, D, M, N, K)) return s;
  const size_t need = fp4_gemm_workspace_size(fmt, M, N, K);
  if (need > 0) {
    if (ws == nullptr || ws_bytes < need)
      return fail(BSFP4_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws == nullptr ? 0 : ws_bytes, need);
    if (!aligned(ws, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ws is not 16-byte aligned");
  }
  if (M == 0) return ok();
  if (bsfp4_status s = check_device()) return s;
  return launch_gemm(fmt, A, SFA, B, SFB, alpha, D, M, N, K, ws, ws_bytes, as_stream(stream));
}

size_t fp4_gemm_noalloc_max_workspace(void) { return bsfp4::kScratchBytes; }

bsfp4_status fp4_gemm_noalloc(int fmt, const uint8_t* A, const uint8_t* SFA, const uint8_t* B, const uint8_t* SFB,
                              const float* alpha, uint16_t* D, int64_t M, int64_t N, int64_t K, void* stream) {
  if (bsfp4_status s = check_gemm_args(fmt, A, SFA, B, SFB, alpha, D, M, N, K)) return s;
  const size_t need = fp4_gemm_workspace_size(fmt, M, N, K);
  if (need > bsfp4::kScratchBytes)
    return fail(BSFP4_ERR_WORKSPACE,
                "this shape needs %zu bytes of split-K partials, above the %zu-byte static scratch of "
                "fp4_gemm_noalloc (use fp4_gemm with a caller workspace)",
                need, bsfp4::kScratchBytes);
  if (M == 0) return ok();
  if (bsfp4_status s = check_device()) return s;
  void* ws = nullptr;
  if (need > 0) {
    const hipError_t e = bsfp4::scratch_device_ptr(&ws);
    if (e != hipSuccess) return fail(BSFP4_ERR_HIP, "hipGetSymbolAddress(scratch): %s", hipGetErrorString(e));
  }
  return launch_gemm(fmt, A, SFA, B, SFB, alpha, D, M, N, K, ws, need > 0 ? bsfp4::kScratchBytes : 0,
                     as_stream(stream));
}

// ------------------------------------------------------------------ W4A16

size_t w4a16_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  if (bsfp4::w4a16_rows64_ok(M, N, K)) return bsfp4::w4a16_rows64_workspace(M, N, K);
  if (bsfp4::w4a16_tiled_ok(M, N, K)) return bsfp4::w4a16_tiled_workspace(M, N, K);
  // rows run in chunks of at most kSkinnyMaxM; the partials of one chunk are
  // reduced before the next chunk starts on the same stream
  const int64_t mc = M < bsfp4::kSkinnyMaxM ? M : bsfp4::kSkinnyMaxM;
  size_t need = bsfp4::skinny_workspace(mc, N, K, false);
  const int64_t tail = M % bsfp4::kSkinnyMaxM;
  if (M > bsfp4::kSkinnyMaxM && tail > 0) {
    const size_t t = bsfp4::skinny_workspace(tail, N, K, false);
    if (t > need) need = t;
  }
  return need;
}

bsfp4_status w4a16_gemm(const uint16_t* A, const uint8_t* B, const uint8_t* SFB, const float* alpha,
                        uint16_t* D, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                        void* stream) {
  if (M < 0 || N <= 0 || K <= 0)
    return fail(BSFP4_ERR_SHAPE, "need M >= 0, N > 0, K > 0 (M=%lld N=%lld K=%lld)", (long long)M,
                (long long)N, (long long)K);
  if (K % 32) return fail(BSFP4_ERR_SHAPE, "K=%lld is not a multiple of 32", (long long)K);
  if (N % 32) return fail(BSFP4_ERR_SHAPE, "N=%lld is not a multiple of 32", (long long)N);
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
    return fail(BSFP4_ERR_SHAPE, "dimensions must fit in 31 bits");
  if (M > 0) {
    REQUIRE_PTR(A);
    REQUIRE_PTR(D);
  }
  REQUIRE_PTR(B);
  REQUIRE_PTR(SFB);
  if (alpha != nullptr && !aligned(alpha, 4)) return fail(BSFP4_ERR_ALIGNMENT, "alpha is not 4-byte aligned");
  const size_t need = w4a16_gemm_workspace_size(M, N, K);
  if (need > 0) {
    if (ws == nullptr || ws_bytes < need)
      return fail(BSFP4_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws == nullptr ? 0 : ws_bytes, need);
    if (!aligned(ws, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ws is not 16-byte aligned");
  }
  if (M == 0) return ok();
  if (bsfp4_status s = check_device()) return s;
  if (bsfp4::w4a16_rows64_ok(M, N, K))
    return launched(bsfp4::launch_w4a16_rows64(A, B, SFB, alpha, D, M, N, K, static_cast<float*>(ws), ws_bytes,
                                               as_stream(stream)),
                    "w4a16_gemm launch");
  if (bsfp4::w4a16_tiled_ok(M, N, K))
    return launched(bsfp4::launch_w4a16_tiled(A, B, SFB, alpha, D, M, N, K, static_cast<float*>(ws), ws_bytes,
                                              as_stream(stream)),
                    "w4a16_gemm launch");
  // rows in chunks of kSkinnyMaxM (the weight stream is re-read once per chunk)
  for (int64_t m0 = 0; m0 < M; m0 += bsfp4::kSkinnyMaxM) {
    const int64_t mc = (M - m0 < bsfp4::kSkinnyMaxM) ? (M - m0) : bsfp4::kSkinnyMaxM;
    hipError_t e = bsfp4::launch_skinny_w4a16(A + m0 * K, B, SFB, alpha, D + m0 * N, mc, N, K,
                                              static_cast<float*>(ws), as_stream(stream));
    if (e != hipSuccess) return launched(e, "w4a16_gemm launch");
  }
  return ok();
}

// ------------------------------------------------------------------ 8-bit integers

namespace {

// Largest row of a tiled operand in bytes (32-bit lane offsets over 256 rows).
constexpr int64_t kTileRowBytes = (int64_t)1 << 23;

bsfp4_status check_rows_cols(const char* rows_name, int64_t M, const char* cols_name, int64_t N, int64_t n_step,
                             const char* k_name, int64_t K, int64_t k_step) {
  if (M < 0 || N <= 0 || K <= 0)
    return fail(BSFP4_ERR_SHAPE, "need %s >= 0, %s > 0, %s > 0 (%lld, %lld, %lld)", rows_name, cols_name, k_name,
                (long long)M, (long long)N, (long long)K);
  if (N % n_step)
    return fail(BSFP4_ERR_SHAPE, "%s=%lld is not a multiple of %lld", cols_name, (long long)N, (long long)n_step);
  if (K % k_step)
    return fail(BSFP4_ERR_SHAPE, "%s=%lld is not a multiple of %lld", k_name, (long long)K, (long long)k_step);
  if (M > ((int64_t)1 << 40) / N) return fail(BSFP4_ERR_SHAPE, "%s * %s exceeds 2^40", rows_name, cols_name);
  // a last tile's rows are counted past M: room for one tile
  if (M > INT32_MAX - 256 || N > (INT32_MAX - 256) / 2) return fail(BSFP4_ERR_SHAPE, "dimensions must fit in 31 bits");
  return BSFP4_OK;
}

bsfp4_status check_int8_k(int64_t K) {
  if (K > 131056)
    return fail(BSFP4_ERR_SHAPE, "K=%lld exceeds 131056 (the 32-bit integer sum)", (long long)K);
  return BSFP4_OK;
}

bsfp4_status check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return BSFP4_OK;
  if (ws == nullptr || ws_bytes < need)
    return fail(BSFP4_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws == nullptr ? 0 : ws_bytes, need);
  if (!aligned(ws, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ws is not 16-byte aligned");
  return BSFP4_OK;
}

bsfp4_status check_act(int act) {
  if (act != BSFP4_ACT_SILU && act != BSFP4_ACT_GELU && act != BSFP4_ACT_GELU_TANH)
    return fail(BSFP4_ERR_INVALID_ARG, "unknown activation %d", act);
  return BSFP4_OK;
}

// A launch holds fewer than 2^32 threads.  The row kernels of one wave per row launch
// (rows + 3) / 4 workgroups of 256, the others at most four threads per eight values.
bsfp4_status check_row_count(int64_t rows, int64_t cols) {
  constexpr int64_t kMostRows = ((int64_t)1 << 26) - 4;
  if (rows > kMostRows || rows * cols >= (int64_t)1 << 33)
    return fail(BSFP4_ERR_SHAPE, "%lld rows of %lld: need at most 2^26 - 4 rows and fewer than 2^33 values in a call",
                (long long)rows, (long long)cols);
  return BSFP4_OK;
}

struct Span {
  const void* p;  // null: not given
  int64_t bytes;
  const char* name;
  bool rowwise = false;
};

bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return pa < pb + (uintptr_t)b.bytes && pb < pa + (uintptr_t)a.bytes;
}

// No output may share memory with an input that other workgroups still read, nor with
// another output.  A rowwise output is written by the threads that have read the same
// place of the rowwise inputs: it may be one of them, but not overlap it otherwise.
bsfp4_status check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); o++) {
    for (const Span& i : ins)
      if (overlap(*o, i) && !(o->rowwise && i.rowwise && o->p == i.p))
        return fail(BSFP4_ERR_INVALID_ARG, "%s overlaps %s%s", o->name, i.name,
                    o->rowwise && i.rowwise ? " without being it" : "");
    for (const Span* other = outs.begin(); other != o; other++)
      if (overlap(*o, *other)) return fail(BSFP4_ERR_INVALID_ARG, "%s overlaps %s", o->name, other->name);
  }
  return BSFP4_OK;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

bsfp4_status bsfp4_int8_quantize(const uint16_t* x, int64_t M, int64_t K, int8_t* q, float* s, void* stream) {
  if (M < 0 || K <= 0)
    return fail(BSFP4_ERR_SHAPE, "need M >= 0 and K > 0 (M=%lld K=%lld)", (long long)M, (long long)K);
  if (K % 8) return fail(BSFP4_ERR_SHAPE, "K=%lld is not a multiple of 8", (long long)K);
  if (K > INT32_MAX) return fail(BSFP4_ERR_SHAPE, "dimensions must fit in 31 bits");
  if (bsfp4_status e = check_row_count(M, K)) return e;
  if (M == 0) return ok();
  REQUIRE_PTR(x);
  REQUIRE_PTR(q);
  REQUIRE_SCALAR_PTR(s);
  if (bsfp4_status e = check_apart({{q, M * K, "q"}, {s, M * 4, "s"}}, {{x, M * K * 2, "x"}})) return e;
  if (bsfp4_status e = check_device()) return e;
  return launched(bsfp4::launch_int8_quant(x, M, K, q, s, as_stream(stream)), "bsfp4_int8_quantize launch");
}

size_t bsfp4_int8_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return bsfp4::int8_gemm_workspace(M, N, K);
}

bsfp4_status bsfp4_int8_gemm(const int8_t* A, const float* sa, const int8_t* B, const float* sb, const uint16_t* bias,
                             uint16_t* D, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes, void* stream) {
  if (bsfp4_status e = check_rows_cols("M", M, "N", N, 8, "K", K, 16)) return e;
  if (bsfp4_status e = check_int8_k(K)) return e;
  if (M > 0) {
    REQUIRE_PTR(A);
    REQUIRE_SCALAR_PTR(sa);
    REQUIRE_PTR(D);
  }
  REQUIRE_PTR(B);
  REQUIRE_PTR(sb);
  if (bias != nullptr && !aligned(bias, 16)) return fail(BSFP4_ERR_ALIGNMENT, "bias is not 16-byte aligned");
  if (bsfp4_status e = check_workspace(ws, ws_bytes, bsfp4_int8_gemm_workspace_size(M, N, K))) return e;
  if (M == 0) return ok();
  if (bsfp4_status e = check_apart({{D, M * N * 2, "D"}}, {{A, M * K, "A"},
                                                           {sa, M * 4, "sa"},
                                                           {B, N * K, "B"},
                                                           {sb, N * 4, "sb"},
                                                           {bias, N * 2, "bias"}}))
    return e;
  if (bsfp4_status e = check_device()) return e;
  return launched(bsfp4::launch_int8_gemm(A, sa, B, sb, bias, D, M, N, K, ws, as_stream(stream)),
                  "bsfp4_int8_gemm launch");
}

size_t bsfp4_int8_quantize_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || bsfp4::int8_fused_quant_ok(M, N, K)) return 0;
  return round256((size_t)M * K) + round256((size_t)M * sizeof(float)) + bsfp4::int8_gemm_workspace(M, N, K);
}

bsfp4_status bsfp4_int8_quantize_gemm(const uint16_t* x, const int8_t* B, const float* sb, const uint16_t* bias,
                                      uint16_t* D, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                                      void* stream) {
  if (bsfp4_status e = check_rows_cols("M", M, "N", N, 8, "K", K, 16)) return e;
  if (bsfp4_status e = check_int8_k(K)) return e;
  if (bsfp4_status e = check_row_count(M, K)) return e;
  if (M > 0) {
    REQUIRE_PTR(x);
    REQUIRE_PTR(D);
  }
  REQUIRE_PTR(B);
  REQUIRE_PTR(sb);
  if (bias != nullptr && !aligned(bias, 16)) return fail(BSFP4_ERR_ALIGNMENT, "bias is not 16-byte aligned");
  if (bsfp4_status e = check_workspace(ws, ws_bytes, bsfp4_int8_quantize_gemm_workspace_size(M, N, K))) return e;
  if (M == 0) return ok();
  if (bsfp4_status e = check_apart({{D, M * N * 2, "D"}},
                                   {{x, M * K * 2, "x"}, {B, N * K, "B"}, {sb, N * 4, "sb"}, {bias, N * 2, "bias"}}))
    return e;
  if (bsfp4_status e = check_device()) return e;
  if (bsfp4::int8_fused_quant_ok(M, N, K))
    return launched(bsfp4::launch_int8_fused_quant_gemm(x, B, sb, bias, D, M, N, K, as_stream(stream)),
                    "bsfp4_int8_quantize_gemm launch");
  int8_t* q = static_cast<int8_t*>(ws);
  float* s = reinterpret_cast<float*>(q + round256((size_t)M * K));
  void* rest = reinterpret_cast<uint8_t*>(s) + round256((size_t)M * sizeof(float));
  hipError_t e = bsfp4::launch_int8_quant(x, M, K, q, s, as_stream(stream));
  if (e == hipSuccess) e = bsfp4::launch_int8_gemm(q, s, B, sb, bias, D, M, N, K, rest, as_stream(stream));
  return launched(e, "bsfp4_int8_quantize_gemm launch");
}

size_t bsfp4_int8_gated_ffn_workspace_size(int64_t M, int64_t I, int64_t K) {
  if (M <= 0 || I <= 0 || K <= 0) return 0;
  return bsfp4::int8_gated_workspace(M, I, K);
}

bsfp4_status bsfp4_int8_gated_ffn(const int8_t* A, const float* sa, const int8_t* W, const float* sw, int act,
                                  uint16_t* h, int64_t M, int64_t I, int64_t K, void* ws, size_t ws_bytes,
                                  void* stream) {
  if (bsfp4_status e = check_act(act)) return e;
  if (bsfp4_status e = check_rows_cols("M", M, "I", I, 8, "K", K, 16)) return e;
  if (bsfp4_status e = check_int8_k(K)) return e;
  if (M > 0) {
    REQUIRE_PTR(A);
    REQUIRE_SCALAR_PTR(sa);
    REQUIRE_PTR(h);
  }
  REQUIRE_PTR(W);
  REQUIRE_PTR(sw);
  if (bsfp4_status e = check_workspace(ws, ws_bytes, bsfp4_int8_gated_ffn_workspace_size(M, I, K))) return e;
  if (M == 0) return ok();
  if (bsfp4_status e = check_apart({{h, M * I * 2, "h"}},
                                   {{A, M * K, "A"}, {sa, M * 4, "sa"}, {W, 2 * I * K, "W"}, {sw, I * 8, "sw"}}))
    return e;
  if (bsfp4_status e = check_device()) return e;
  return launched(bsfp4::launch_int8_gated(A, sa, W, sw, act, h, M, I, K, ws, as_stream(stream)),
                  "bsfp4_int8_gated_ffn launch");
}

// ------------------------------------------------------------------ gated feed-forward, bf16

static bsfp4_status check_gated(int act, int64_t M, int64_t I, int64_t H) {
  if (bsfp4_status e = check_act(act)) return e;
  if (bsfp4_status e = check_rows_cols("M", M, "I", I, 8, "H", H, 8)) return e;
  if (2 * H >= kTileRowBytes || 4 * I >= kTileRowBytes)
    return fail(BSFP4_ERR_SHAPE, "need H < 2^22 and I < 2^21 (H=%lld I=%lld)", (long long)H, (long long)I);
  if (M > ((int64_t)1 << 40) / H) return fail(BSFP4_ERR_SHAPE, "M * H exceeds 2^40");
  return BSFP4_OK;
}

size_t bsfp4_gated_ffn_workspace_size(int64_t M, int64_t I, int64_t H) {
  if (M <= 0 || I <= 0 || H <= 0) return 0;
  return bsfp4::gated_ffn_workspace(M, I, H);
}

bsfp4_status bsfp4_gated_ffn(const uint16_t* x, const uint16_t* W, int act, uint16_t* h, float* gate_up, int64_t M,
                             int64_t I, int64_t H, void* ws, size_t ws_bytes, void* stream) {
  if (bsfp4_status e = check_gated(act, M, I, H)) return e;
  if (M > 0) {
    REQUIRE_PTR(x);
    REQUIRE_PTR(h);
  }
  REQUIRE_PTR(W);
  if (gate_up != nullptr && !aligned(gate_up, 16)) return fail(BSFP4_ERR_ALIGNMENT, "gate_up is not 16-byte aligned");
  if (bsfp4_status e = check_workspace(ws, ws_bytes, bsfp4_gated_ffn_workspace_size(M, I, H))) return e;
  if (M == 0) return ok();
  if (bsfp4_status e = check_apart({{h, M * I * 2, "h"}, {gate_up, M * I * 8, "gate_up"}},
                                   {{x, M * H * 2, "x"}, {W, 4 * I * H, "W"}}))
    return e;
  if (bsfp4_status e = check_device()) return e;
  return launched(bsfp4::launch_gated_ffn(x, W, act, h, gate_up, M, I, H, ws, as_stream(stream)),
                  "bsfp4_gated_ffn launch");
}

size_t bsfp4_gated_ffn_backward_workspace_size(int64_t M, int64_t I, int64_t H) {
  if (M < 0 || I <= 0 || H <= 0) return 0;
  return bsfp4::gated_ffn_bwd_workspace(M, I, H);
}

bsfp4_status bsfp4_gated_ffn_backward(const uint16_t* dh, const uint16_t* x, const uint16_t* W,
                                      const float* gate_up, int act, uint16_t* dx, uint16_t* dW, int64_t M,
                                      int64_t I, int64_t H, void* ws, size_t ws_bytes, void* stream) {
  if (bsfp4_status e = check_gated(act, M, I, H)) return e;
  if (M > 0) {
    REQUIRE_PTR(dh);
    REQUIRE_PTR(gate_up);
    if (dx != nullptr) REQUIRE_PTR(W);
    if (dW != nullptr) REQUIRE_PTR(x);
  }
  if (dx == nullptr && dW == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "dx and dW are both NULL");
  if (dx != nullptr && !aligned(dx, 16)) return fail(BSFP4_ERR_ALIGNMENT, "dx is not 16-byte aligned");
  if (dW != nullptr && !aligned(dW, 16)) return fail(BSFP4_ERR_ALIGNMENT, "dW is not 16-byte aligned");
  if (bsfp4_status e = check_workspace(ws, ws_bytes, bsfp4_gated_ffn_backward_workspace_size(M, I, H))) return e;
  if (M == 0 && dW == nullptr) return ok();
  // dh and gate_up are read whole before the products write; x is read for dW, W for dx
  if (bsfp4_status e = check_apart({{dx, M * H * 2, "dx"}, {dW, 4 * I * H, "dW"}},
                                   {{dW == nullptr ? nullptr : x, M * H * 2, "x"},
                                    {M == 0 || dx == nullptr ? nullptr : W, 4 * I * H, "W"}}))
    return e;
  if (bsfp4_status e = check_device()) return e;
  return launched(bsfp4::launch_gated_ffn_bwd(dh, x, W, gate_up, act, M == 0 ? nullptr : dx, dW, M, I, H, ws,
                                              as_stream(stream)),
                  "bsfp4_gated_ffn_backward launch");
}

// ------------------------------------------------------------------ block norms

namespace {

bsfp4_status check_block_norm(const bsfp4_block_norm_args* a) {
  if (a == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "args is NULL");
  if (a->T < 0 || a->H <= 0 || a->groups <= 0)
    return fail(BSFP4_ERR_SHAPE, "need T >= 0, H > 0, groups > 0 (T=%lld H=%lld groups=%lld)", (long long)a->T,
                (long long)a->H, (long long)a->groups);
  if (a->H % 8) return fail(BSFP4_ERR_SHAPE, "H=%lld is not a multiple of 8", (long long)a->H);
  if (a->H > bsfp4::kBlockNormMaxH)
    return fail(BSFP4_ERR_SHAPE, "H=%lld exceeds %lld", (long long)a->H, (long long)bsfp4::kBlockNormMaxH);
  if (bsfp4_status e = check_row_count(a->T, a->H)) return e;
  if (a->groups > INT32_MAX) return fail(BSFP4_ERR_SHAPE, "dimensions must fit in 31 bits");
  if (a->T % a->groups)
    return fail(BSFP4_ERR_SHAPE, "T=%lld is not a multiple of groups=%lld", (long long)a->T, (long long)a->groups);
  if (!(a->eps > 0.0 && a->eps < 1e30)) return fail(BSFP4_ERR_INVALID_ARG, "eps must be positive and finite");
  // (no rows: the row tensors may be NULL whatever the vectors are)
  if (a->T > 0 && a->x == nullptr && (a->w_post != nullptr || a->gate != nullptr))
    return fail(BSFP4_ERR_INVALID_ARG, "without x there is no w_post and no gate");
  if (a->T > 0 && a->x == nullptr && a->w_pre == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "neither x nor w_pre is given");
  if (a->gate == nullptr && a->groups != 1) return fail(BSFP4_ERR_SHAPE, "groups must be 1 without a gate");
  const struct {
    const void* p;
    const char* name;
  } ptrs[] = {{a->x, "x"},           {a->residual, "residual"}, {a->w_post, "w_post"},     {a->w_pre, "w_pre"},
              {a->gate, "gate"},     {a->res_out, "res_out"},   {a->z, "z"},               {a->q, "q"},
              {a->dres_out, "dres_out"}, {a->dz, "dz"},         {a->dx, "dx"},             {a->dres, "dres"},
              {a->dw_post, "dw_post"},   {a->dw_pre, "dw_pre"}, {a->dgate, "dgate"}};
  for (const auto& q : ptrs)
    if (!aligned(q.p, 16)) return fail(BSFP4_ERR_ALIGNMENT, "%s is not 16-byte aligned", q.name);
  if (!aligned(a->s, 4)) return fail(BSFP4_ERR_ALIGNMENT, "s is not 4-byte aligned");
  return BSFP4_OK;
}

bsfp4::BlockNormArgs norm_args(const bsfp4_block_norm_args* a) {
  bsfp4::BlockNormArgs p{};
  p.x = a->x;
  p.residual = a->residual;
  p.w_post = a->w_post;
  p.w_pre = a->w_pre;
  p.gate = a->gate;
  p.scale = (float)a->scale;
  p.eps = a->eps;
  p.inv_h = 1.0 / (double)a->H;
  p.T = a->T;
  p.groups = a->groups;
  p.group_rows = a->T / a->groups;
  p.H = (int)a->H;
  return p;
}

#define REQUIRE_FIELD(f) \
  if (a->f == nullptr) return fail(BSFP4_ERR_INVALID_ARG, #f " is NULL")

}  // namespace

bsfp4_status bsfp4_block_norm(const bsfp4_block_norm_args* a, void* stream) {
  if (bsfp4_status e = check_block_norm(a)) return e;
  if ((a->q == nullptr) != (a->s == nullptr)) return fail(BSFP4_ERR_INVALID_ARG, "q and s go together");
  if (a->z != nullptr && a->q != nullptr) return fail(BSFP4_ERR_INVALID_ARG, "z and q are both given");
  if (a->w_pre == nullptr && (a->z != nullptr || a->q != nullptr))
    return fail(BSFP4_ERR_INVALID_ARG, "z or q without w_pre");
  if (a->T == 0) return ok();
  REQUIRE_FIELD(residual);
  if (a->x != nullptr) REQUIRE_FIELD(res_out);
  if (a->w_pre != nullptr && a->z == nullptr && a->q == nullptr)
    return fail(BSFP4_ERR_INVALID_ARG, "w_pre without z or q");
  const int64_t n = a->T * a->H, vec = 2 * a->H;
  if (bsfp4_status e = check_apart({{a->x == nullptr ? nullptr : a->res_out, 2 * n, "res_out", true},
                                    {a->z, 2 * n, "z", true},
                                    {a->q, n, "q"},
                                    {a->s, 4 * a->T, "s"}},
                                   {{a->x, 2 * n, "x", true},
                                    {a->residual, 2 * n, "residual", true},
                                    {a->w_post, vec, "w_post"},
                                    {a->w_pre, vec, "w_pre"},
                                    {a->gate, vec * a->groups, "gate"}}))
    return e;
  if (bsfp4_status e = check_device()) return e;
  bsfp4::BlockNormArgs p = norm_args(a);
  p.res_out = a->res_out;
  p.z = a->z;
  p.q = a->q;
  p.s = a->s;
  return launched(bsfp4::launch_block_norm(p, as_stream(stream)), "bsfp4_block_norm launch");
}

size_t bsfp4_block_norm_backward_workspace_size(int64_t T, int64_t H, int64_t groups) {
  if (T < 0 || H <= 0 || groups <= 0 || T % groups) return 0;
  return bsfp4::block_norm_bwd_workspace(T, H, groups);
}

bsfp4_status bsfp4_block_norm_backward(const bsfp4_block_norm_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (bsfp4_status e = check_block_norm(a)) return e;
  if (a->w_pre == nullptr && a->dz != nullptr) return fail(BSFP4_ERR_INVALID_ARG, "dz without w_pre");
  if (a->T > 0) {
    if (a->w_pre != nullptr) {
      REQUIRE_FIELD(res_out);
      REQUIRE_FIELD(dz);
    } else {
      REQUIRE_FIELD(dres_out);
    }
    if (a->x != nullptr) REQUIRE_FIELD(dx);
    REQUIRE_FIELD(dres);
  }
  if (a->w_post != nullptr) REQUIRE_FIELD(dw_post);
  if (a->w_pre != nullptr) REQUIRE_FIELD(dw_pre);
  if (a->gate != nullptr) REQUIRE_FIELD(dgate);
  if (bsfp4_status e = check_workspace(ws, ws_bytes, bsfp4_block_norm_backward_workspace_size(a->T, a->H, a->groups)))
    return e;
  const int64_t n = 2 * a->T * a->H, vec = 2 * a->H;
  const bool pre = a->w_pre != nullptr;
  if (bsfp4_status e = check_apart({{a->x == nullptr ? nullptr : a->dx, n, "dx", true},
                                    {a->dres, n, "dres", true},
                                    {a->w_post == nullptr ? nullptr : a->dw_post, 2 * vec, "dw_post"},
                                    {pre ? a->dw_pre : nullptr, 2 * vec, "dw_pre"},
                                    {a->gate == nullptr ? nullptr : a->dgate, 2 * vec * a->groups, "dgate"}},
                                   {{a->x, n, "x", true},
                                    {pre ? a->res_out : nullptr, n, "res_out", true},
                                    {a->dres_out, n, "dres_out", true},
                                    {a->dz, n, "dz", true},
                                    {a->w_post, vec, "w_post"},
                                    {a->w_pre, vec, "w_pre"},
                                    {a->gate, vec * a->groups, "gate"}}))
    return e;
  if (bsfp4_status e = check_device()) return e;
  bsfp4::BlockNormArgs p = norm_args(a);
  p.res = a->res_out;
  p.dres_out = a->dres_out;
  p.dz = a->dz;
  p.dx = a->dx;
  p.dres = a->dres;
  p.dw_post = a->dw_post;
  p.dw_pre = a->dw_pre;
  p.dgate = a->dgate;
  return launched(bsfp4::launch_block_norm_bwd(p, static_cast<float*>(ws), as_stream(stream)),
                  "bsfp4_block_norm_backward launch");
}

// ------------------------------------------------------------------ E2M1 conversion

bsfp4_status bsfp4_e2m1_convert(int mode, const void* in, const uint8_t* scale_codes, int64_t pairs,
                                uint8_t* codes, void* stream) {
  if (mode != BSFP4_CVT_F32 && mode != BSFP4_CVT_BF16_E8M0 && mode != BSFP4_CVT_F32_E8M0)
    return fail(BSFP4_ERR_INVALID_ARG, "unknown conversion mode %d", mode);
  if (pairs < 0 || pairs % 4)
    return fail(BSFP4_ERR_SHAPE, "pairs must be >= 0 and a multiple of 4 (got %lld)", (long long)pairs);
  if (mode == BSFP4_CVT_F32) {
    if (scale_codes != nullptr) return fail(BSFP4_ERR_INVALID_ARG, "BSFP4_CVT_F32 takes no scale codes");
  }
  if (pairs == 0) return ok();
  REQUIRE_PTR(in);
  REQUIRE_PTR(codes);
  if (mode != BSFP4_CVT_F32) REQUIRE_PTR(scale_codes);
  if (bsfp4_status s = check_device()) return s;
  return launched(bsfp4::launch_e2m1_convert(mode, in, scale_codes, pairs, codes, as_stream(stream)),
                  "bsfp4_e2m1_convert launch");
}

// ------------------------------------------------------------------ peak probes

namespace {
int64_t mfma_flops(int kind) {
  return (kind == 2 || kind == 3 || kind == 6) ? 2LL * 32 * 32 * 64 : 2LL * 32 * 32 * 16;
}
// kinds 6 and 7 rotate four operand pairs: iters is a multiple of 4
bool probe_args_ok(int kind, int iters) {
  return kind >= 0 && kind <= 7 && iters > 0 && iters <= (1 << 24) && (kind < 6 || iters % 4 == 0);
}
}  // namespace

int64_t bsfp4_probe_mfma_flops(int kind, int iters) {
  if (!probe_args_ok(kind, iters)) return 0;
  // 8 MFMAs per iteration per wave, 4 waves per workgroup
  return bsfp4::probe_mfma_grid() * 4 * (int64_t)iters * 8 * mfma_flops(kind);
}

bsfp4_status bsfp4_probe_mfma(int kind, int iters, void* stream) {
  if (kind < 0 || kind > 7) return fail(BSFP4_ERR_INVALID_ARG, "unknown MFMA probe kind %d", kind);
  if (!probe_args_ok(kind, iters))
    return fail(BSFP4_ERR_SHAPE, "iters must be in [1, 2^24] and a multiple of 4 for kinds 6 and 7 (got %d)", iters);
  if (bsfp4_status s = check_device()) return s;
  return launched(bsfp4::launch_probe_mfma(kind, iters, as_stream(stream)), "bsfp4_probe_mfma launch");
}

bsfp4_status bsfp4_probe_read(const void* buf, int64_t bytes, void* stream) {
  if (bytes <= 0 || bytes % 16) return fail(BSFP4_ERR_SHAPE, "bytes must be a positive multiple of 16");
  REQUIRE_PTR(buf);
  if (bsfp4_status s = check_device()) return s;
  return launched(bsfp4::launch_probe_read(buf, bytes, as_stream(stream)), "bsfp4_probe_read launch");
}

// ------------------------------------------------------------------ scale layouts

size_t fp4_scales_swizzled_size(int64_t rows, int64_t kblocks) {
  if (rows < 0 || kblocks <= 0) return 0;
  return (size_t)((rows + 127) / 128 * 128) * (size_t)((kblocks + 3) / 4 * 4);
}

static bsfp4_status check_scale_layout(int layout, const void* a, const void* b, int64_t rows, int64_t kblocks,
                                       const void* swz) {
  if (layout != BSFP4_SF_128X4 && layout != BSFP4_SF_128X4_M8)
    return fail(BSFP4_ERR_INVALID_ARG, "unknown scale layout %d", layout);
  if (rows < 0 || kblocks <= 0)
    return fail(BSFP4_ERR_SHAPE, "need rows >= 0 and kblocks > 0 (rows=%lld kblocks=%lld)", (long long)rows,
                (long long)kblocks);
  if (rows > INT32_MAX || kblocks > INT32_MAX || fp4_scales_swizzled_size(rows, kblocks) >= ((size_t)1 << 31))
    return fail(BSFP4_ERR_SHAPE, "padded scale buffer must stay below 2^31 bytes");
  if (rows == 0) return ok();
  if (a == nullptr || b == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "a scale pointer is NULL");
  if (!aligned(swz, 4)) return fail(BSFP4_ERR_ALIGNMENT, "the swizzled buffer is not 4-byte aligned");
  return ok();
}

bsfp4_status fp4_scales_swizzle(int layout, const uint8_t* sf, int64_t rows, int64_t kblocks, uint8_t* swz,
                                void* stream) {
  if (bsfp4_status s = check_scale_layout(layout, sf, swz, rows, kblocks, swz)) return s;
  if (rows == 0) return ok();
  if (bsfp4_status s = check_device()) return s;
  return launched(bsfp4::launch_scale_layout(layout, true, sf, swz, rows, kblocks, as_stream(stream)),
                  "fp4_scales_swizzle launch");
}

bsfp4_status fp4_scales_unswizzle(int layout, const uint8_t* swz, int64_t rows, int64_t kblocks, uint8_t* sf,
                                  void* stream) {
  if (bsfp4_status s = check_scale_layout(layout, swz, sf, rows, kblocks, swz)) return s;
  if (rows == 0) return ok();
  if (bsfp4_status s = check_device()) return s;
  return launched(bsfp4::launch_scale_layout(layout, false, swz, sf, rows, kblocks, as_stream(stream)),
                  "fp4_scales_unswizzle launch");
}

// ------------------------------------------------------------------ MoE

size_t fp4_moe_prep_workspace_size(int64_t T, int64_t topk, int64_t E) {
  (void)T;
  (void)topk;
  (void)E;
  return 0;
}

bsfp4_status fp4_moe_prep(const int32_t* topk_ids, int64_t T, int64_t topk, int64_t E,
                          int32_t* expert_offsets, int32_t* sorted_ids, int32_t* sorted_tokens, void* ws,
                          size_t ws_bytes, void* stream) {
  (void)ws;
  (void)ws_bytes;
  if (T < 0 || topk <= 0 || E <= 0 || E > bsfp4::kMaxExperts)
    return fail(BSFP4_ERR_SHAPE, "need T >= 0, topk > 0, 0 < E <= %lld (T=%lld topk=%lld E=%lld)",
                (long long)bsfp4::kMaxExperts, (long long)T, (long long)topk, (long long)E);
  if (T * topk > INT32_MAX) return fail(BSFP4_ERR_SHAPE, "T*topk must fit in 31 bits");
  if (T > 0) {
    REQUIRE_PTR(topk_ids);
    if (sorted_ids == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "sorted_ids is NULL");
    if (!aligned(sorted_ids, 4)) return fail(BSFP4_ERR_ALIGNMENT, "sorted_ids is not 4-byte aligned");
    if (sorted_tokens != nullptr && !aligned(sorted_tokens, 4))
      return fail(BSFP4_ERR_ALIGNMENT, "sorted_tokens is not 4-byte aligned");
  }
  if (expert_offsets == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "expert_offsets is NULL");
  if (!aligned(expert_offsets, 4)) return fail(BSFP4_ERR_ALIGNMENT, "expert_offsets is not 4-byte aligned");
  if (bsfp4_status s = check_device()) return s;
  return launched(bsfp4::launch_moe_prep(topk_ids, T, topk, E, expert_offsets, sorted_ids, sorted_tokens,
                                         as_stream(stream)),
                  "fp4_moe_prep launch");
}

size_t mxfp4_moe_grouped_gemm_workspace_size(int64_t rows, int64_t E, int64_t N, int64_t K, int epilogue,
                                             int64_t num_tokens) {
  (void)E;
  (void)K;
  (void)num_tokens;
  if (epilogue == BSFP4_MOE_WEIGHTED_COMBINE && rows > 0 && N > 0)
    return (size_t)rows * (size_t)N * sizeof(float);
  return 0;
}

bsfp4_status mxfp4_moe_grouped_gemm(const uint8_t* Aq, const uint8_t* Asf, int64_t a_rows_total,
                                    const int32_t* a_row_index, const int32_t* expert_offsets, int64_t E,
                                    int64_t rows, const uint8_t* W, const uint8_t* Wsf, int64_t N, int64_t K,
                                    int epilogue, const bsfp4_moe_epilogue_args* ep, void* ws, size_t ws_bytes,
                                    void* stream) {
  if (epilogue != BSFP4_MOE_STORE_BF16 && epilogue != BSFP4_MOE_SILU_MUL_QUANT &&
      epilogue != BSFP4_MOE_WEIGHTED_COMBINE)
    return fail(BSFP4_ERR_INVALID_ARG, "unknown epilogue %d", epilogue);
  if (ep == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "ep is NULL");
  if (rows < 0 || a_rows_total < 0 || E <= 0 || E > bsfp4::kMaxExperts || N <= 0 || K <= 0)
    return fail(BSFP4_ERR_SHAPE, "need rows >= 0, a_rows_total >= 0, 0 < E <= %lld, N > 0, K > 0",
                (long long)bsfp4::kMaxExperts);
  if (a_row_index == nullptr && a_rows_total != rows)
    return fail(BSFP4_ERR_SHAPE, "without a_row_index, a_rows_total (%lld) must equal rows (%lld)",
                (long long)a_rows_total, (long long)rows);
  if (K % 32) return fail(BSFP4_ERR_SHAPE, "K=%lld is not a multiple of 32", (long long)K);
  if (N % 32) return fail(BSFP4_ERR_SHAPE, "N=%lld is not a multiple of 32", (long long)N);
  if (epilogue == BSFP4_MOE_SILU_MUL_QUANT && N % 64)
    return fail(BSFP4_ERR_SHAPE, "SILU_MUL_QUANT needs N %% 64 == 0 (got N=%lld)", (long long)N);
  if (rows > INT32_MAX || a_rows_total > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
    return fail(BSFP4_ERR_SHAPE, "dimensions must fit in 31 bits");
  if (a_rows_total * (K / 2) >= kLim31 || N * (K / 2) >= kLim31)
    return fail(BSFP4_ERR_SHAPE, "Aq (a_rows_total*K/2=%lld) and one expert's W (N*K/2=%lld) must stay below 2^31 bytes",
                (long long)(a_rows_total * (K / 2)), (long long)(N * (K / 2)));
  REQUIRE_PTR(W);
  REQUIRE_PTR(Wsf);
  REQUIRE_PTR(expert_offsets);
  if (a_row_index != nullptr && !aligned(a_row_index, 4))
    return fail(BSFP4_ERR_ALIGNMENT, "a_row_index is not 4-byte aligned");
  if (rows > 0) {
    REQUIRE_PTR(Aq);
    REQUIRE_PTR(Asf);
    if (epilogue == BSFP4_MOE_STORE_BF16) {
      if (ep->out == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "ep.out is NULL");
      if (!aligned(ep->out, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ep.out is not 16-byte aligned");
    } else if (epilogue == BSFP4_MOE_SILU_MUL_QUANT) {
      if (ep->out_q == nullptr || ep->out_sf == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "ep.out_q/out_sf is NULL");
      if (!aligned(ep->out_q, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ep.out_q is not 16-byte aligned");
    }
  }
  const int64_t T = ep->num_tokens;
  if (epilogue == BSFP4_MOE_WEIGHTED_COMBINE) {
    if (T <= 0 || ep->topk <= 0 || T * ep->topk != rows)
      return fail(BSFP4_ERR_SHAPE, "WEIGHTED_COMBINE needs num_tokens*topk == rows (T=%lld topk=%lld rows=%lld)",
                  (long long)T, (long long)ep->topk, (long long)rows);
    if (ep->out == nullptr || ep->sorted_ids == nullptr || ep->topk_weights == nullptr)
      return fail(BSFP4_ERR_INVALID_ARG, "ep.out / sorted_ids / topk_weights is NULL");
    if (!aligned(ep->out, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ep.out is not 16-byte aligned");
    const size_t need = mxfp4_moe_grouped_gemm_workspace_size(rows, E, N, K, epilogue, T);
    if (ws == nullptr || ws_bytes < need)
      return fail(BSFP4_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws == nullptr ? 0 : ws_bytes, need);
    if (!aligned(ws, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ws is not 16-byte aligned");
  }
  if (rows == 0) return ok();
  if (bsfp4_status s = check_device()) return s;
  const hipStream_t st = as_stream(stream);
  if (epilogue == BSFP4_MOE_WEIGHTED_COMBINE) {
    float* y = static_cast<float*>(ws);
    hipError_t e = bsfp4::launch_mxfp4_grouped(Aq, Asf, a_row_index, a_rows_total, expert_offsets, E, rows, W, Wsf,
                                               N, K, bsfp4::kEpiCombine, nullptr, nullptr, nullptr, ep->sorted_ids, y,
                                               st);
    if (e == hipSuccess)
      e = bsfp4::launch_topk_sum(y, ep->topk_weights, static_cast<uint16_t*>(ep->out), T, ep->topk, N, st);
    return launched(e, "mxfp4_moe_grouped_gemm launch");
  }
  return launched(bsfp4::launch_mxfp4_grouped(Aq, Asf, a_row_index, a_rows_total, expert_offsets, E, rows, W, Wsf,
                                              N, K,
                                              epilogue == BSFP4_MOE_STORE_BF16 ? bsfp4::kEpiStore : bsfp4::kEpiSilu,
                                              static_cast<uint16_t*>(ep->out), ep->out_q, ep->out_sf, nullptr,
                                              nullptr, st),
                  "mxfp4_moe_grouped_gemm launch");
}

// ------------------------------------------------------------------ quantise + GEMM

namespace {
int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }
}  // namespace

size_t nvfp4_quantize_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 32 || N % 32) return 0;
  if (bsfp4::nvfp4_fused_quant_gemm_ok(M, N, K)) return 0;
  return (size_t)(round16(M * (K / 2)) + round16(M * (K / 16))) + bsfp4::nvfp4_gemm_workspace(M, N, K);
}

bsfp4_status nvfp4_quantize_gemm(const uint16_t* x, const float* gs, const uint8_t* B, const uint8_t* SFB,
                                 const float* alpha, uint16_t* D, int64_t M, int64_t N, int64_t K, void* ws,
                                 size_t ws_bytes, void* stream) {
  if (M < 0 || N <= 0 || K <= 0)
    return fail(BSFP4_ERR_SHAPE, "need M >= 0, N > 0, K > 0 (M=%lld N=%lld K=%lld)", (long long)M, (long long)N,
                (long long)K);
  if (K % 32) return fail(BSFP4_ERR_SHAPE, "K=%lld is not a multiple of 32", (long long)K);
  if (N % 32) return fail(BSFP4_ERR_SHAPE, "N=%lld is not a multiple of 32", (long long)N);
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return fail(BSFP4_ERR_SHAPE, "dimensions must fit in 31 bits");
  REQUIRE_SCALAR_PTR(gs);
  REQUIRE_PTR(B);
  REQUIRE_PTR(SFB);
  if (alpha != nullptr && !aligned(alpha, 4)) return fail(BSFP4_ERR_ALIGNMENT, "alpha is not 4-byte aligned");
  if (M > 0) {
    REQUIRE_PTR(x);
    REQUIRE_PTR(D);
  }
  const size_t need = nvfp4_quantize_gemm_workspace_size(M, N, K);
  if (need > 0) {
    if (ws == nullptr || ws_bytes < need)
      return fail(BSFP4_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws == nullptr ? 0 : ws_bytes, need);
    if (!aligned(ws, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ws is not 16-byte aligned");
  }
  if (M == 0) return ok();
  if (bsfp4_status s = check_device()) return s;
  const hipStream_t st = as_stream(stream);
  if (need == 0)
    return launched(bsfp4::launch_nvfp4_fused_quant_gemm(x, gs, B, SFB, alpha, D, M, N, K, st),
                    "nvfp4_quantize_gemm launch");
  uint8_t* q = static_cast<uint8_t*>(ws);
  uint8_t* sf = q + round16(M * (K / 2));
  uint8_t* gws = sf + round16(M * (K / 16));
  const size_t gws_bytes = ws_bytes - (size_t)(gws - q);
  hipError_t e = bsfp4::launch_quantize(0, x, M, K, gs, nullptr, M, q, sf, st);
  if (e == hipSuccess) e = bsfp4::launch_nvfp4_gemm(q, sf, B, SFB, alpha, D, M, N, K, gws, gws_bytes, st);
  return launched(e, "nvfp4_quantize_gemm launch");
}

// ------------------------------------------------------------------ NVFP4 MoE

bsfp4_status nvfp4_experts_quantize(const uint16_t* x, int64_t rows_in, int64_t K, const int32_t* row_map,
                                    const int32_t* expert_offsets, int64_t E, const float* gs_experts,
                                    int64_t rows_out, uint8_t* q, uint8_t* sf, void* stream) {
  if (rows_in < 0 || rows_out < 0 || K <= 0)
    return fail(BSFP4_ERR_SHAPE, "need rows >= 0 and K > 0 (rows_in=%lld rows_out=%lld K=%lld)",
                (long long)rows_in, (long long)rows_out, (long long)K);
  if (K % 16) return fail(BSFP4_ERR_SHAPE, "K=%lld is not a multiple of 16", (long long)K);
  if (E <= 0 || E > bsfp4::kMaxExperts)
    return fail(BSFP4_ERR_SHAPE, "need 0 < E <= %lld (E=%lld)", (long long)bsfp4::kMaxExperts, (long long)E);
  if (row_map == nullptr && rows_out != rows_in)
    return fail(BSFP4_ERR_SHAPE, "without row_map rows_out (%lld) must equal rows_in (%lld)",
                (long long)rows_out, (long long)rows_in);
  REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(gs_experts);
  if (!aligned(expert_offsets, 4) || !aligned(gs_experts, 4))
    return fail(BSFP4_ERR_ALIGNMENT, "expert_offsets / gs_experts are not 4-byte aligned");
  if (rows_out == 0) return ok();
  if (rows_in > 0) REQUIRE_PTR(x);
  if (row_map != nullptr && !aligned(row_map, 4)) return fail(BSFP4_ERR_ALIGNMENT, "row_map is not 4-byte aligned");
  REQUIRE_PTR(q);
  if (sf == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "sf is NULL");
  if (bsfp4_status s = check_device()) return s;
  return launched(bsfp4::launch_nvfp4_experts_quant(x, rows_in, K, row_map, expert_offsets, E, gs_experts, rows_out,
                                                    q, sf, as_stream(stream)),
                  "nvfp4_experts_quantize launch");
}

size_t nvfp4_moe_grouped_gemm_workspace_size(int64_t rows, int64_t E, int64_t N, int64_t K, int epilogue,
                                             int64_t num_tokens) {
  (void)E;
  (void)K;
  (void)num_tokens;
  if (epilogue == BSFP4_MOE_WEIGHTED_COMBINE && rows > 0 && N > 0)
    return (size_t)rows * (size_t)N * sizeof(float);
  return 0;
}

bsfp4_status nvfp4_moe_grouped_gemm(const uint8_t* Aq, const uint8_t* Asf, const int32_t* expert_offsets,
                                    int64_t E, int64_t rows, const uint8_t* W, const uint8_t* Wsf,
                                    const float* alpha_experts, int64_t N, int64_t K, int epilogue,
                                    const bsfp4_moe_epilogue_args* ep, void* ws, size_t ws_bytes, void* stream) {
  if (epilogue != BSFP4_MOE_STORE_BF16 && epilogue != BSFP4_MOE_SILU_MUL_QUANT &&
      epilogue != BSFP4_MOE_WEIGHTED_COMBINE)
    return fail(BSFP4_ERR_INVALID_ARG, "unknown epilogue %d", epilogue);
  if (ep == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "ep is NULL");
  if (rows < 0 || E <= 0 || E > bsfp4::kMaxExperts || N <= 0 || K <= 0)
    return fail(BSFP4_ERR_SHAPE, "need rows >= 0, 0 < E <= %lld, N > 0, K > 0", (long long)bsfp4::kMaxExperts);
  if (K % 32) return fail(BSFP4_ERR_SHAPE, "K=%lld is not a multiple of 32", (long long)K);
  if (N % 32) return fail(BSFP4_ERR_SHAPE, "N=%lld is not a multiple of 32", (long long)N);
  if (epilogue == BSFP4_MOE_SILU_MUL_QUANT && N % 64)
    return fail(BSFP4_ERR_SHAPE, "SILU_MUL_QUANT needs N %% 64 == 0 (got N=%lld)", (long long)N);
  if (rows > INT32_MAX || N * (K / 2) >= ((int64_t)1 << 31))
    return fail(BSFP4_ERR_SHAPE, "rows must fit in 31 bits and one expert's N*K/2 bytes below 2^31");
  REQUIRE_PTR(W);
  REQUIRE_PTR(Wsf);
  REQUIRE_PTR(expert_offsets);
  if (!aligned(expert_offsets, 4)) return fail(BSFP4_ERR_ALIGNMENT, "expert_offsets is not 4-byte aligned");
  if (alpha_experts != nullptr && !aligned(alpha_experts, 4))
    return fail(BSFP4_ERR_ALIGNMENT, "alpha_experts is not 4-byte aligned");
  if (rows > 0) {
    REQUIRE_PTR(Aq);
    REQUIRE_PTR(Asf);
    if (epilogue == BSFP4_MOE_STORE_BF16) {
      if (ep->out == nullptr) return fail(BSFP4_ERR_INVALID_ARG, "ep.out is NULL");
      if (!aligned(ep->out, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ep.out is not 16-byte aligned");
    } else if (epilogue == BSFP4_MOE_SILU_MUL_QUANT) {
      if (ep->out_q == nullptr || ep->out_sf == nullptr || ep->out_gs == nullptr)
        return fail(BSFP4_ERR_INVALID_ARG, "ep.out_q / out_sf / out_gs is NULL");
      if (!aligned(ep->out_q, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ep.out_q is not 16-byte aligned");
      if (!aligned(ep->out_sf, 2)) return fail(BSFP4_ERR_ALIGNMENT, "ep.out_sf is not 2-byte aligned");
      if (!aligned(ep->out_gs, 4)) return fail(BSFP4_ERR_ALIGNMENT, "ep.out_gs is not 4-byte aligned");
    }
  }
  const int64_t T = ep->num_tokens;
  if (epilogue == BSFP4_MOE_WEIGHTED_COMBINE) {
    if (T <= 0 || ep->topk <= 0 || T * ep->topk != rows)
      return fail(BSFP4_ERR_SHAPE, "WEIGHTED_COMBINE needs num_tokens*topk == rows (T=%lld topk=%lld rows=%lld)",
                  (long long)T, (long long)ep->topk, (long long)rows);
    if (ep->out == nullptr || ep->sorted_ids == nullptr || ep->topk_weights == nullptr)
      return fail(BSFP4_ERR_INVALID_ARG, "ep.out / sorted_ids / topk_weights is NULL");
    if (!aligned(ep->out, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ep.out is not 16-byte aligned");
    const size_t need = nvfp4_moe_grouped_gemm_workspace_size(rows, E, N, K, epilogue, T);
    if (ws == nullptr || ws_bytes < need)
      return fail(BSFP4_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws == nullptr ? 0 : ws_bytes, need);
    if (!aligned(ws, 16)) return fail(BSFP4_ERR_ALIGNMENT, "ws is not 16-byte aligned");
  }
  if (rows == 0) return ok();
  if (bsfp4_status s = check_device()) return s;
  const hipStream_t st = as_stream(stream);
  if (epilogue == BSFP4_MOE_WEIGHTED_COMBINE) {
    float* y = static_cast<float*>(ws);
    hipError_t e = bsfp4::launch_nvfp4_grouped(Aq, Asf, expert_offsets, E, rows, W, Wsf, alpha_experts, N, K,
                                               bsfp4::kEpiCombine, nullptr, nullptr, nullptr, nullptr,
                                               ep->sorted_ids, y, st);
    if (e == hipSuccess)
      e = bsfp4::launch_topk_sum(y, ep->topk_weights, static_cast<uint16_t*>(ep->out), T, ep->topk, N, st);
    return launched(e, "nvfp4_moe_grouped_gemm launch");
  }
  return launched(bsfp4::launch_nvfp4_grouped(Aq, Asf, expert_offsets, E, rows, W, Wsf, alpha_experts, N, K,
                                              epilogue == BSFP4_MOE_STORE_BF16 ? bsfp4::kEpiStore : bsfp4::kEpiSilu,
                                              static_cast<uint16_t*>(ep->out), ep->out_q, ep->out_sf, ep->out_gs,
                                              nullptr, nullptr, st),
                  "nvfp4_moe_grouped_gemm launch");
}

}  // extern "C"
