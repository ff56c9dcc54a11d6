// C entry points of the products of microscaled 4-bit matrices: argument
// checks, then the kernels of fp4_gemm.cu and fp4_matvec.cu.
#include "fp4.cuh"
#include "fp4_products.h"
#include "internal.h"

namespace kq {
namespace {

constexpr int64_t kMatvecMaxN = int64_t(1) << 24;   // column slices are a grid dimension

// The checks that the three products share; name is the caller's.
kronq_status check_product(const char* name, int fmt, int64_t T, int64_t m, int64_t n, const void* x, const void* wc,
                           const void* ws, const float* wg, const void* y, int ydt, int64_t ldy) {
  const auto who = [name] { return std::string(name); };
  if (!fp4_fmt_ok(fmt)) return fail(KRONQ_ERR_INVALID_ARG, who() + ": bad format");
  if (ydt != KRONQ_BF16 && ydt != KRONQ_F32) return fail(KRONQ_ERR_INVALID_ARG, who() + ": bad dtype");
  if (T < 0 || T > kFp4MaxDim || m <= 0 || m > kFp4MaxDim || n <= 0 || n > kFp4MaxDim)
    return fail(KRONQ_ERR_INVALID_ARG, who() + ": sizes out of range");
  if (ldy < m || ldy > kFp4MaxStride) return fail(KRONQ_ERR_INVALID_ARG, who() + ": row stride of y out of range");
  if (!wc || !ws || (T > 0 && (!x || !y))) return fail(KRONQ_ERR_INVALID_ARG, who() + ": NULL pointer");
  if ((fmt == KRONQ_NVFP4) != (wg != nullptr))
    return fail(KRONQ_ERR_INVALID_ARG, who() + ": tensor scales go with NVFP4 and with it only");
  if (!aligned(wc, 16) || !aligned(ws, 16) || !aligned(wg, 4) || !aligned(y, ydt == KRONQ_BF16 ? 2 : 4))
    return fail(KRONQ_ERR_INVALID_ARG, who() + ": misaligned pointer");
  return KRONQ_OK;
}

kronq_status check_tokens(const char* name, int fmt, int64_t T, const void* xc, const void* xs, const float* xg) {
  const auto who = [name] { return std::string(name); };
  if (T > 0 && !xs) return fail(KRONQ_ERR_INVALID_ARG, who() + ": NULL pointer");
  if ((fmt == KRONQ_NVFP4) != (xg != nullptr))
    return fail(KRONQ_ERR_INVALID_ARG, who() + ": tensor scales go with NVFP4 and with it only");
  if (!aligned(xc, 16) || !aligned(xs, 16) || !aligned(xg, 4))
    return fail(KRONQ_ERR_INVALID_ARG, who() + ": misaligned pointer");
  return KRONQ_OK;
}

}  // namespace

int fp4_sms(int* dev) {
  static std::atomic<int> known[kMaxDevices];
  int d = 0, v = 148;
  if (cudaGetDevice(&d) != cudaSuccess) d = -1;
  if (dev) *dev = d;
  if (d < 0 || d >= kMaxDevices) return sm_count();
  v = known[d].load(std::memory_order_relaxed);
  if (v == 0) {
    v = sm_count();
    known[d].store(v, std::memory_order_relaxed);
  }
  return v;
}

cudaError_t fp4_allow_smem(const void* fn, int bytes, int dev, std::atomic<bool>* done) {
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = allow_smem(fn, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace kq

using namespace kq;

extern "C" {

size_t kronq_fp4_matmul_workspace_bytes(int64_t T, int64_t m, int64_t n, kronq_fp4_format fmt) {
  if (!fp4_fmt_ok(fmt) || T <= 0 || T > kFp4MaxDim || m <= 0 || m > kFp4MaxDim || n <= 0 || n > kFp4MaxDim) return 0;
  return fp4_gemm_workspace(T, m, n);
}

kronq_status kronq_fp4_matmul(const uint8_t* xc, const uint8_t* xs, const float* xg, const uint8_t* wc,
                              const uint8_t* ws, const float* wg, kronq_fp4_format fmt, int64_t T, int64_t m,
                              int64_t n, void* y, kronq_dtype ydt, int64_t ldy, void* workspace, size_t ws_bytes,
                              kronq_stream_t s) {
  return fp4_entry([&]() -> kronq_status {
    kronq_status r = check_product("fp4_matmul", fmt, T, m, n, xc, wc, ws, wg, y, ydt, ldy);
    if (r == KRONQ_OK) r = check_tokens("fp4_matmul", fmt, T, xc, xs, xg);
    if (r != KRONQ_OK || T == 0) return r;
    const size_t need = fp4_gemm_workspace(T, m, n);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256)))
      return fail(KRONQ_ERR_INVALID_ARG, "fp4_matmul: workspace too small or not 256-byte aligned");
    Fp4Gemm g{xc, xs, xg, wc, ws, wg, T, m, n, y, ydt == KRONQ_BF16, ldy, nullptr, 1, workspace};
    return fp4_gemm(g, fmt, as_stream(s));
  });
}

size_t kronq_fp4_matvec_workspace_bytes(int64_t T, int64_t m, int64_t n, kronq_fp4_format fmt) {
  if (!fp4_fmt_ok(fmt) || T <= 0 || T > KRONQ_FP4_MATVEC_MAX_TOKENS || m <= 0 || m > kFp4MaxDim || n <= 0 ||
      n > kMatvecMaxN)
    return 0;
  return fp4_matvec_workspace(T, m, n);
}

kronq_status kronq_fp4_matvec(const void* x, kronq_dtype xdt, int64_t ldx, const uint8_t* wc, const uint8_t* ws,
                              const float* wg, kronq_fp4_format fmt, int64_t T, int64_t m, int64_t n, void* y,
                              kronq_dtype ydt, int64_t ldy, void* workspace, size_t ws_bytes, kronq_stream_t s) {
  return fp4_entry([&]() -> kronq_status {
    kronq_status r = check_product("fp4_matvec", fmt, T, m, n, x, wc, ws, wg, y, ydt, ldy);
    if (r != KRONQ_OK) return r;
    if (xdt != KRONQ_BF16 && xdt != KRONQ_F32) return fail(KRONQ_ERR_INVALID_ARG, "fp4_matvec: bad dtype");
    if (T > KRONQ_FP4_MATVEC_MAX_TOKENS)
      return fail(KRONQ_ERR_UNSUPPORTED, "fp4_matvec: more than KRONQ_FP4_MATVEC_MAX_TOKENS tokens");
    if (n > kMatvecMaxN) return fail(KRONQ_ERR_UNSUPPORTED, "fp4_matvec: row too long");
    if (ldx < n || ldx > kFp4MaxStride) return fail(KRONQ_ERR_INVALID_ARG, "fp4_matvec: row stride of x out of range");
    if (!aligned(x, xdt == KRONQ_BF16 ? 2 : 4)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_matvec: misaligned pointer");
    if (T == 0) return KRONQ_OK;
    const size_t need = fp4_matvec_workspace(T, m, n);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256)))
      return fail(KRONQ_ERR_INVALID_ARG, "fp4_matvec: workspace too small or not 256-byte aligned");
    Fp4Matvec v{x, xdt == KRONQ_F32, ldx, wc, ws, wg, T, m, n, y, ydt == KRONQ_BF16, ldy, workspace};
    return fp4_matvec(v, fmt, as_stream(s));
  });
}

kronq_status kronq_fp4_grouped_matmul(const uint8_t* xc, const uint8_t* xs, const float* xg, const int* offsets,
                                      int64_t E, const uint8_t* wc, const uint8_t* ws, const float* wg,
                                      kronq_fp4_format fmt, int64_t T, int64_t m, int64_t n, void* y,
                                      kronq_dtype ydt, int64_t ldy, kronq_stream_t s) {
  return fp4_entry([&]() -> kronq_status {
    kronq_status r = check_product("fp4_grouped_matmul", fmt, T, m, n, xc, wc, ws, wg, y, ydt, ldy);
    if (r == KRONQ_OK) r = check_tokens("fp4_grouped_matmul", fmt, T, xc, xs, xg);
    if (r != KRONQ_OK) return r;
    if (E <= 0 || E > KRONQ_FP4_MAX_EXPERTS)
      return fail(KRONQ_ERR_INVALID_ARG, "fp4_grouped_matmul: expert count out of range");
    if (E * m > kFp4MaxDim) return fail(KRONQ_ERR_INVALID_ARG, "fp4_grouped_matmul: sizes out of range");
    if (!offsets) return fail(KRONQ_ERR_INVALID_ARG, "fp4_grouped_matmul: NULL pointer");
    if (!aligned(offsets, 4)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_grouped_matmul: misaligned pointer");
    if (T == 0) return KRONQ_OK;
    Fp4Gemm g{xc, xs, xg, wc, ws, wg, T, m, n, y, ydt == KRONQ_BF16, ldy, offsets, E, nullptr};
    return fp4_gemm(g, fmt, as_stream(s));
  });
}

}  // extern "C"
