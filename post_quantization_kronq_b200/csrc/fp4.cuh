// The microscaled 4-bit formats' layout and device conversions, shared by the
// quantiser, its inverse and the products.
//
// A quantised matrix (rows x n, blocks along n) is two byte arrays:
//   codes   rows x code_row_bytes(n): two E2M1 codes a byte, the even element
//           in the low half;
//   scales  rows x scale_row_bytes(fmt, n): one byte per block of 32 (MXFP4,
//           E8M0) or 16 (NVFP4, E4M3) elements.
// Both row lengths are rounded up to 16 bytes (what TMA and 16-byte loads
// need), the padding is zero.  NVFP4 has one float32 scale per tensor on top.
#pragma once

#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"

namespace kq {

inline bool fp4_fmt_ok(int fmt) { return fmt == KRONQ_MXFP4 || fmt == KRONQ_NVFP4; }
inline int fp4_block(int fmt) { return fmt == KRONQ_MXFP4 ? 32 : 16; }
inline int64_t fp4_code_row(int64_t n) { return ceil_div(ceil_div(n, 2), 16) * 16; }
inline int64_t fp4_scale_row(int fmt, int64_t n) { return ceil_div(ceil_div(n, fp4_block(fmt)), 16) * 16; }

// Largest row and column counts of the 4-bit calls (coordinates of the tensor
// maps and tile indices are 32-bit), and the largest row stride (offsets stay
// within 64 bits).
constexpr int64_t kFp4MaxDim = int64_t(1) << 30;
constexpr int64_t kFp4MaxStride = int64_t(1) << 32;

// Number of SMs of the current device, and a kernel's dynamic shared memory
// limit raised on it, each asked of the runtime once per device (a decoded
// token's calls are shorter than the questions).  `done` is the kernel's own
// array of kMaxDevices flags.
constexpr int kMaxDevices = 64;
int fp4_sms(int* dev);
cudaError_t fp4_allow_smem(const void* fn, int bytes, int dev, std::atomic<bool>* done);

// Runs a C entry point's body; no exception (out of host memory, in building
// an error message) passes the C boundary.
template <typename F>
kronq_status fp4_entry(F body) {
  try {
    return body();
  } catch (...) {
    return KRONQ_ERR_CUDA;
  }
}

// A call's second kernel need not wait to be launched until the first has
// ended: it may begin when every block of the first has left or let it in, and
// then waits for the first's end, its writes included, before it touches
// memory.  The quantiser's first pass lets the second in early (0.3 us of 5.5
// for 16 x 4096, nothing from 500 x 4096 on).  The products do not: they leave
// few SMs with room, all of a join's blocks gather on those, and it got up to
// 1 us slower.
__device__ __forceinline__ void fp4_let_next_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void fp4_await_first() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t fp4_launch_second(void (*fn)(P...), unsigned grid, unsigned threads, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

// Value of an E8M0 byte (255 is NaN) and of an E4M3 byte (0x7F is NaN).
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  // 2^-127 (b = 0) is a float32 subnormal
  return b == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(b ? b << 23 : 0x00400000u);
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(b));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}
template <int FMT>
__device__ __forceinline__ float fp4_scale_value(uint32_t b) {
  return FMT == KRONQ_MXFP4 ? e8m0_value(b) : e4m3_value(b);
}

// Sum of `count` partial sums `stride` apart, in order, eight loads at a time.
__device__ __forceinline__ float fp4_join(const float* part, int64_t stride, int count) {
  float v = 0.f;
  for (int s = 0; s < count; s += 8) {
    float p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = s + k < count ? part[(s + k) * stride] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s + k < count) v += p[k];
  }
  return v;
}

// Two E2M1 codes (a byte, the first in the low half) as a pair of halves.
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
  return h;
}
__device__ __forceinline__ float2 e2m1x2_float2(uint32_t byte) {
  const uint32_t h = e2m1x2_f16x2(byte);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace kq
