// Launchers of the products of microscaled 4-bit matrices (fp4_gemm.cu,
// fp4_matvec.cu); the arguments are those of the C entry points, checked.
#pragma once

#include "internal.h"

namespace kq {

struct Fp4Gemm {
  const uint8_t *xc, *xs;
  const float* xg;
  const uint8_t *wc, *ws;
  const float* wg;
  int64_t T, m, n;
  void* y;
  bool y_bf16;
  int64_t ldy;
  const int* offsets;   // grouped: E + 1 bounds on the device, else NULL
  int64_t E;
  void* workspace;      // plain: fp4_gemm_workspace bytes
};
size_t fp4_gemm_workspace(int64_t T, int64_t m, int64_t n);
kronq_status fp4_gemm(const Fp4Gemm& g, int fmt, cudaStream_t s);

struct Fp4Matvec {
  const void* x;
  bool x_f32;
  int64_t ldx;
  const uint8_t *wc, *ws;
  const float* wg;
  int64_t T, m, n;
  void* y;
  bool y_bf16;
  int64_t ldy;
  void* workspace;      // fp4_matvec_workspace bytes
};
size_t fp4_matvec_workspace(int64_t T, int64_t m, int64_t n);
kronq_status fp4_matvec(const Fp4Matvec& v, int fmt, cudaStream_t s);

cudaError_t status_fetch_fp4(int* out, cudaStream_t s);

}  // namespace kq
