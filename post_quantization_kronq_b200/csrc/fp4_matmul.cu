// Products of microscaled 4-bit matrices: y = A W^T with both operands
// quantised, with full-precision tokens (a few rows), and grouped by expert.
//
// First form: one 64 x 64 tile of y per CTA, both operands dequantised into
// shared memory 32 columns at a time (E2M1 value times block scale, exact in
// float32), float32 accumulation.
#include "fp4.cuh"
#include "fp4_gemm.h"
#include "internal.h"

namespace kq {
namespace {

constexpr int TT = 64, TM = 64, TK = 32;

struct SimpleArgs {
  const uint8_t *xc, *xs;   // quantised tokens, or
  const void* x;            // full-precision tokens
  int x_bf16;
  int64_t ldx;
  const float *xg, *wg;
  const uint8_t *wc, *ws;
  int64_t T, m, n, ldc, lds;
  void* y;
  int y_bf16;
  int64_t ldy;
  const int* offsets;       // grouped: E + 1
  int E;
};

template <int FMT>
__device__ __forceinline__ float fp4_at(const uint8_t* codes, const uint8_t* scales, int64_t r, int64_t k, int64_t ldc,
                                        int64_t lds) {
  const uint32_t b = codes[r * ldc + (k >> 1)];
  const float2 v = e2m1x2_float2(b);
  return ((k & 1) ? v.y : v.x) * fp4_scale_value<FMT>(scales[r * lds + k / (FMT == KRONQ_MXFP4 ? 32 : 16)]);
}

template <int FMT>
__global__ void __launch_bounds__(256) fp4_simple_kernel(const SimpleArgs a) {
  __shared__ float xs[TK][TT + 1], wsm[TK][TM + 1];
  const int e = blockIdx.z;
  int64_t t_lo = 0, t_hi = a.T;
  if (a.offsets) {
    int64_t lo = 0;
    for (int i = 0; i <= e; ++i) lo = max(lo, min((int64_t)max(a.offsets[i], 0), a.T));
    t_lo = lo;
    t_hi = max(lo, min((int64_t)max(a.offsets[e + 1], 0), a.T));
  }
  const int64_t t0 = t_lo + (int64_t)blockIdx.y * TT, m0 = (int64_t)blockIdx.x * TM;
  if (t0 >= t_hi) return;
  const uint8_t* wc = a.wc + (int64_t)e * a.m * a.ldc;
  const uint8_t* wsc = a.ws + (int64_t)e * a.m * a.lds;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < a.n; k0 += TK) {
    for (int i = threadIdx.x; i < TT * TK; i += 256) {
      const int r = i / TK, k = i % TK;
      float v = 0.f;
      if (t0 + r < t_hi && k0 + k < a.n) {
        if (a.x) v = a.x_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.x)[(t0 + r) * a.ldx + k0 + k])
                              : static_cast<const float*>(a.x)[(t0 + r) * a.ldx + k0 + k];
        else v = fp4_at<FMT>(a.xc, a.xs, t0 + r, k0 + k, a.ldc, a.lds);
      }
      xs[k][r] = v;
      wsm[k][r] = (m0 + r < a.m && k0 + k < a.n) ? fp4_at<FMT>(wc, wsc, m0 + r, k0 + k, a.ldc, a.lds) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[k][ty * 4 + i], wsm[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + ty * 4 + i, r = m0 + tx + 16 * j;
      if (t >= t_hi || r >= a.m) continue;
      float v = acc[i][j];
      if (a.xg) v *= *a.xg;
      if (a.wg) v *= a.wg[e];
      if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[t * a.ldy + r] = __float2bfloat16_rn(v);
      else static_cast<float*>(a.y)[t * a.ldy + r] = v;
    }
}

kronq_status simple(const SimpleArgs& a, int fmt, cudaStream_t st) {
  dim3 grid((unsigned)ceil_div(a.m, TM), (unsigned)ceil_div(a.T, TT), (unsigned)a.E);
  if (fmt == KRONQ_MXFP4) fp4_simple_kernel<KRONQ_MXFP4><<<grid, 256, 0, st>>>(a);
  else fp4_simple_kernel<KRONQ_NVFP4><<<grid, 256, 0, st>>>(a);
  KQ_LAUNCH_CHECK("fp4_simple_kernel");
  return KRONQ_OK;
}

// The checks that the three products share; name is the caller's.
kronq_status check_product(const char* name, int fmt, int64_t T, int64_t m, int64_t n, const void* x, const void* wc,
                           const void* ws, const float* wg, const void* y, int ydt, int64_t ldy) {
  const std::string who(name);
  if (!fp4_fmt_ok(fmt)) return fail(KRONQ_ERR_INVALID_ARG, who + ": bad format");
  if (ydt != KRONQ_BF16 && ydt != KRONQ_F32) return fail(KRONQ_ERR_INVALID_ARG, who + ": bad dtype");
  if (T < 0 || T > kFp4MaxDim || m <= 0 || m > kFp4MaxDim || n <= 0 || n > kFp4MaxDim)
    return fail(KRONQ_ERR_INVALID_ARG, who + ": sizes out of range");
  if (ldy < m) return fail(KRONQ_ERR_INVALID_ARG, who + ": row stride of y below m");
  if (!wc || !ws || (T > 0 && (!x || !y))) return fail(KRONQ_ERR_INVALID_ARG, who + ": NULL pointer");
  if ((fmt == KRONQ_NVFP4) != (wg != nullptr))
    return fail(KRONQ_ERR_INVALID_ARG, who + ": tensor scales go with NVFP4 and with it only");
  if (!aligned(wc, 16) || !aligned(ws, 16) || !aligned(wg, 4) || !aligned(y, ydt == KRONQ_BF16 ? 2 : 4))
    return fail(KRONQ_ERR_INVALID_ARG, who + ": misaligned pointer");
  return KRONQ_OK;
}

kronq_status check_tokens(const char* name, int fmt, int64_t T, const void* xc, const void* xs, const float* xg) {
  const std::string who(name);
  if (T > 0 && !xs) return fail(KRONQ_ERR_INVALID_ARG, who + ": NULL pointer");
  if ((fmt == KRONQ_NVFP4) != (xg != nullptr))
    return fail(KRONQ_ERR_INVALID_ARG, who + ": tensor scales go with NVFP4 and with it only");
  if (!aligned(xc, 16) || !aligned(xs, 16) || !aligned(xg, 4))
    return fail(KRONQ_ERR_INVALID_ARG, who + ": misaligned pointer");
  return KRONQ_OK;
}

}  // namespace
}  // namespace kq

using namespace kq;

extern "C" {

size_t kronq_fp4_matmul_workspace_bytes(int64_t T, int64_t m, int64_t n, kronq_fp4_format fmt) {
  return 0;
}

kronq_status kronq_fp4_matmul(const uint8_t* xc, const uint8_t* xs, const float* xg, const uint8_t* wc,
                              const uint8_t* ws, const float* wg, kronq_fp4_format fmt, int64_t T, int64_t m,
                              int64_t n, void* y, kronq_dtype ydt, int64_t ldy, void* workspace, size_t ws_bytes,
                              kronq_stream_t s) {
  kronq_status r = check_product("fp4_matmul", fmt, T, m, n, xc, wc, ws, wg, y, ydt, ldy);
  if (r == KRONQ_OK) r = check_tokens("fp4_matmul", fmt, T, xc, xs, xg);
  if (r != KRONQ_OK || T == 0) return r;
  Fp4Gemm g{xc, xs, xg, wc, ws, wg, T, m, n, y, ydt == KRONQ_BF16, ldy, nullptr, 1};
  return fp4_gemm(g, fmt, as_stream(s));
}

size_t kronq_fp4_matvec_workspace_bytes(int64_t T, int64_t m, int64_t n, kronq_fp4_format fmt) {
  return 0;
}

kronq_status kronq_fp4_matvec(const void* x, kronq_dtype xdt, int64_t ldx, const uint8_t* wc, const uint8_t* ws,
                              const float* wg, kronq_fp4_format fmt, int64_t T, int64_t m, int64_t n, void* y,
                              kronq_dtype ydt, int64_t ldy, void* workspace, size_t ws_bytes, kronq_stream_t s) {
  kronq_status r = check_product("fp4_matvec", fmt, T, m, n, x, wc, ws, wg, y, ydt, ldy);
  if (r != KRONQ_OK) return r;
  if (xdt != KRONQ_BF16 && xdt != KRONQ_F32) return fail(KRONQ_ERR_INVALID_ARG, "fp4_matvec: bad dtype");
  if (T > KRONQ_FP4_MATVEC_MAX_TOKENS)
    return fail(KRONQ_ERR_UNSUPPORTED, "fp4_matvec: more than KRONQ_FP4_MATVEC_MAX_TOKENS tokens");
  if (ldx < n) return fail(KRONQ_ERR_INVALID_ARG, "fp4_matvec: row stride of x below n");
  if (!aligned(x, xdt == KRONQ_BF16 ? 2 : 4)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_matvec: misaligned pointer");
  if (T == 0) return KRONQ_OK;
  SimpleArgs a{};
  a.x = x; a.x_bf16 = xdt == KRONQ_BF16; a.ldx = ldx; a.wc = wc; a.ws = ws; a.wg = wg;
  a.T = T; a.m = m; a.n = n; a.ldc = fp4_code_row(n); a.lds = fp4_scale_row(fmt, n);
  a.y = y; a.y_bf16 = ydt == KRONQ_BF16; a.ldy = ldy; a.E = 1;
  return simple(a, fmt, as_stream(s));
}

kronq_status kronq_fp4_grouped_matmul(const uint8_t* xc, const uint8_t* xs, const float* xg, const int* offsets,
                                      int64_t E, const uint8_t* wc, const uint8_t* ws, const float* wg,
                                      kronq_fp4_format fmt, int64_t T, int64_t m, int64_t n, void* y,
                                      kronq_dtype ydt, int64_t ldy, kronq_stream_t s) {
  kronq_status r = check_product("fp4_grouped_matmul", fmt, T, m, n, xc, wc, ws, wg, y, ydt, ldy);
  if (r == KRONQ_OK) r = check_tokens("fp4_grouped_matmul", fmt, T, xc, xs, xg);
  if (r != KRONQ_OK) return r;
  if (E <= 0 || E > KRONQ_FP4_MAX_EXPERTS)
    return fail(KRONQ_ERR_INVALID_ARG, "fp4_grouped_matmul: expert count out of range");
  if (E * m > kFp4MaxDim) return fail(KRONQ_ERR_INVALID_ARG, "fp4_grouped_matmul: sizes out of range");
  if (!offsets) return fail(KRONQ_ERR_INVALID_ARG, "fp4_grouped_matmul: NULL pointer");
  if (!aligned(offsets, 4)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_grouped_matmul: misaligned pointer");
  if (T == 0) return KRONQ_OK;
  Fp4Gemm g{xc, xs, xg, wc, ws, wg, T, m, n, y, ydt == KRONQ_BF16, ldy, offsets, E};
  return fp4_gemm(g, fmt, as_stream(s));
}

}  // extern "C"
