// Microscaled 4-bit floating point: the quantiser and its inverse.
//
// MXFP4: blocks of 32, scale 2^E with E = floor(log2 amax) - 2 clamped to
// [-127, 127] (the OCP microscaling rule; the largest E2M1 exponent is 2),
// q = RN_e2m1(x / 2^E), saturating at 6.  NVFP4: blocks of 16,
// s = RN_e4m3(amax / (6 g)) saturating at 448, q = RN_e2m1(x / (s g)), with
// g = RN_f32(max|x| / (448 * 6)) or the caller's.  All roundings are to
// nearest, ties to even, and every decision is that of the exact quotient:
//   - MXFP4's x 2^-E is exact in float32 (it can only underflow far below the
//     first rounding border), so the conversion instruction rounds it;
//   - NVFP4's x / (s g) is never formed.  The borders b of E2M1 have at most
//     3 significant bits and s at most 4, so b s is exact in float32 and
//     x > b s g (x >= b s g where the tie goes up) is decided by comparing x
//     with b s g rounded down (up) by one directed product.  For bf16 x the
//     borders are rounded on to bf16 in the same direction and two elements
//     are compared per instruction; the code is the count of borders passed.
//   - the E4M3 scale is taken from a float32 quotient (off by at most one
//     code) and corrected by the same comparison of amax with 6 g times the
//     two neighbouring midpoints.
//
// One thread per 16 elements (8 bytes of codes, 32 or 64 bytes of input),
// lane pairs share an MXFP4 block.  Bound by HBM: the input once (twice when
// the tensor scale is computed), codes, scales and the optional dequantised
// values once.
#include "fp4.cuh"
#include "internal.h"

namespace kq {
namespace {

constexpr int QT = 256;               // threads per block
constexpr int MAX_PARTIALS = 1184;    // 8 blocks on each of 148 SMs

// ---------------------------------------------------------------- amax
// Largest finite |x| of a rows x n tensor as one partial per block (float
// bits; non-negative floats order like their bits).
__device__ __forceinline__ uint32_t finite_abs_bits(uint32_t bits) {
  const uint32_t a = bits & 0x7FFFFFFFu;
  return a < 0x7F800000u ? a : 0u;
}

template <bool BF16>
__global__ void __launch_bounds__(QT)
    fp4_amax_kernel(const void* x, int64_t rows, int64_t n, int64_t ldx, int vec, uint32_t* partial) {
  uint32_t best = 0;
  constexpr int E = BF16 ? 8 : 4;  // elements of a 16-byte load
  const int64_t per = vec ? (n + E - 1) / E : n;
  const int64_t total = rows * per;
  const int64_t stride = (int64_t)gridDim.x * QT;
  int64_t i = (int64_t)blockIdx.x * QT + threadIdx.x;
  int64_t r = i / per, c = i - r * per;
  const int64_t dr = stride / per, dc = stride - dr * per;
#pragma unroll 4
  for (; i < total; i += stride) {
    if (vec && (c + 1) * E <= n) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const char*>(x) + (r * ldx + c * E) * (BF16 ? 2 : 4));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (BF16) {
          best = max(best, finite_abs_bits(u[q] << 16));
          best = max(best, finite_abs_bits(u[q] & 0xFFFF0000u));
        } else {
          best = max(best, finite_abs_bits(u[q]));
        }
      }
    } else {
      const int64_t c0 = vec ? c * E : c, c1 = vec ? n : c + 1;
      for (int64_t j = c0; j < c1; ++j) {
        const int64_t at = r * ldx + j;
        best = max(best, finite_abs_bits(BF16 ? (uint32_t)static_cast<const uint16_t*>(x)[at] << 16
                                              : static_cast<const uint32_t*>(x)[at]));
      }
    }
    r += dr;
    c += dc;
    if (c >= per) { c -= per; ++r; }
  }
  best = __reduce_max_sync(0xffffffffu, best);
  __shared__ uint32_t red[QT / 32];
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < QT / 32; ++w) best = max(best, red[w]);
    partial[blockIdx.x] = best;
  }
}

// ---------------------------------------------------------------- quantise
struct QuantArgs {
  const void* x;
  int64_t rows, n, ldx;
  uint8_t* codes;
  uint8_t* scales;
  int64_t ldc, lds;       // row bytes
  float* gscale;          // NVFP4: in (given) or out
  const uint32_t* partial;  // amax partials, or NULL when gscale is given
  int npartial;
  void* deq;              // dequantised values in x's type, or NULL
  int64_t ldd;
  int vec_in, vec_out;      // rows are 32-byte aligned
  uintptr_t x_lo, x_hi;     // first byte of x, one behind its last
};

// RN_e4m3(amax / (6 g)), ties to even, at most 448: the byte.
__device__ __forceinline__ uint32_t nv_scale(float amax, float g) {
  const float t = __fdiv_rn(__fmul_rn(amax, 1.f / 6.f), g);
  uint16_t p;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(0.f), "f"(t));
  uint32_t c = p & 0xFFu;
  if (c > 126u) c = 126u;   // t overflowed to infinity
  const float v = e4m3_value(c);
  if (c < 126u) {
    const float mid = __fmul_rn(3.f, __fadd_rn(v, e4m3_value(c + 1)));   // 6 (v + v') / 2, exact
    const bool up = (c & 1u) ? amax >= __fmul_ru(mid, g) : amax > __fmul_rd(mid, g);
    if (up) return c + 1;
  }
  if (c > 0u) {
    const float mid = __fmul_rn(3.f, __fadd_rn(v, e4m3_value(c - 1)));
    const bool down = (c & 1u) ? amax <= __fmul_rd(mid, g) : amax < __fmul_ru(mid, g);
    if (down) return c - 1;
  }
  return c;
}

// E2M1's rounding borders; a tie at an odd index (counted from 0) goes up.
__device__ __forceinline__ float border(int i) {
  constexpr float b[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.f};
  return b[i];
}

// The smallest float32 whose magnitude passes border i under s and g.
__device__ __forceinline__ float pass_f32(int i, float s, float g) {
  const float t = __fmul_rn(border(i), s);  // exact
  if (i & 1) return __fmul_ru(t, g);
  return __uint_as_float(__float_as_uint(__fmul_rd(t, g)) + 1u);   // the next float above
}
// The same among bf16 values, twice in a word.
__device__ __forceinline__ uint32_t pass_bf16x2(int i, float s, float g) {
  const float t = __fmul_rn(border(i), s);
  uint32_t u;
  if (i & 1) u = (__float_as_uint(__fmul_ru(t, g)) + 0xFFFFu) >> 16;
  else u = (__float_as_uint(__fmul_rd(t, g)) >> 16) + 1u;
  return u | (u << 16);
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 32-byte global loads and stores (whole sectors a lane).
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 16 elements of a row from column j0 (bf16: pairs in w[0..7], f32: w[0..15]);
// columns from n on are zero.  Rows that are not 32-byte aligned are read as
// the 16-byte words around the elements and shifted into place; the words
// stay inside x's first to last element, next to which single elements are
// read instead.
template <bool BF16>
__device__ __forceinline__ void load16(const QuantArgs& a, int64_t r, int64_t j0, uint32_t (&w)[BF16 ? 8 : 16]) {
  constexpr int NW = BF16 ? 8 : 16;
  const char* p = static_cast<const char*>(a.x) + (r * a.ldx + j0) * (BF16 ? 2 : 4);
  if (a.vec_in && j0 + 16 <= a.n) {
    load32(p, w);
    if (!BF16) load32(p + 32, w + (BF16 ? 0 : 8));
    return;
  }
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15);
  if (j0 + 16 <= a.n && lo >= a.x_lo && lo + NW * 4 + 16 <= a.x_hi) {
    uint32_t c[NW + 4];
#pragma unroll
    for (int q = 0; q < NW / 4 + 1; ++q) {
      const uint4 v = reinterpret_cast<const uint4*>(lo)[q];
      c[4 * q] = v.x; c[4 * q + 1] = v.y; c[4 * q + 2] = v.z; c[4 * q + 3] = v.w;
    }
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
    if (off & 8) {
#pragma unroll
      for (int q = 0; q < NW + 2; ++q) c[q] = c[q + 2];
    }
    if (off & 4) {
#pragma unroll
      for (int q = 0; q < NW + 1; ++q) c[q] = c[q + 1];
    }
#pragma unroll
    for (int q = 0; q < NW; ++q) w[q] = BF16 ? __funnelshift_r(c[q], c[q + 1], 8 * (off & 2)) : c[q];
    return;
  }
#pragma unroll
  for (int q = 0; q < NW; ++q) {
    if (BF16) {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
      const uint32_t e0 = j0 + 2 * q < a.n ? h[2 * q] : 0u;
      const uint32_t e1 = j0 + 2 * q + 1 < a.n ? h[2 * q + 1] : 0u;
      w[q] = e0 | (e1 << 16);
    } else {
      w[q] = j0 + q < a.n ? reinterpret_cast<const uint32_t*>(p)[q] : 0u;
    }
  }
}

// A warp's 32 runs of up to 16 values, each to its place in a row: `at` the
// element offset, `count` the elements (0 for a lane without any).  Aligned
// rows take 32-byte stores.  Others go through shared memory, so that a store
// instruction writes two runs' neighbouring elements, not one of each lane's.
struct RunSmem {
  float v[32 * 17];
  int64_t at[32];
  int count[32];
};
template <bool BF16>
__device__ __forceinline__ void store_runs(void* out, int64_t at, int count, bool vec, const float (&v)[16], RunSmem& sm,
                                           int lane) {
  const bool whole = vec && count == 16;
  if (whole) {
    if (BF16) {
      uint32_t u[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) u[q] = as_u32(__floats2bfloat162_rn(v[2 * q], v[2 * q + 1]));
      store32(static_cast<__nv_bfloat16*>(out) + at, u);
    } else {
      uint32_t u[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) u[q] = __float_as_uint(v[q]);
      store32(static_cast<float*>(out) + at, u);
      store32(static_cast<float*>(out) + at + 8, u + 8);
    }
  }
  if (__all_sync(0xffffffffu, whole || count == 0)) return;
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 16; ++q) sm.v[lane * 17 + q] = v[q];
  sm.at[lane] = at;
  sm.count[lane] = whole ? 0 : count;
  __syncwarp();
  const int e = lane & 15;
#pragma unroll 4
  for (int k = 0; k < 16; ++k) {
    const int u = 2 * k + (lane >> 4);
    if (e < sm.count[u]) {
      const float f = sm.v[u * 17 + e];
      if (BF16) static_cast<__nv_bfloat16*>(out)[sm.at[u] + e] = __float2bfloat16_rn(f);
      else static_cast<float*>(out)[sm.at[u] + e] = f;
    }
  }
  __syncwarp();
}

// Values of 16 codes under a scale (and the tensor scale), with float32's roundings.
template <int FMT>
__device__ __forceinline__ void values16(uint32_t lo, uint32_t hi, float s, float g, float (&v)[16]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float2 d = e2m1x2_float2(((q < 4 ? lo : hi) >> (8 * (q & 3))) & 0xFFu);
    v[2 * q] = __fmul_rn(d.x, s);
    v[2 * q + 1] = __fmul_rn(d.y, s);
    if (FMT == KRONQ_NVFP4) {
      v[2 * q] = __fmul_rn(v[2 * q], g);
      v[2 * q + 1] = __fmul_rn(v[2 * q + 1], g);
    }
  }
}

template <int FMT, bool BF16>
__global__ void __launch_bounds__(QT, 4) fp4_quantize_kernel(const QuantArgs a) {
  __shared__ RunSmem runs[QT / 32];
  float g = 1.f;
  bool g_bad = false;
  if (FMT == KRONQ_NVFP4) {
    if (a.partial) {
      __shared__ uint32_t red[QT / 32];
      uint32_t best = 0;
      for (int i = threadIdx.x; i < a.npartial; i += QT) best = max(best, a.partial[i]);
      best = __reduce_max_sync(0xffffffffu, best);
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = best;
      __syncthreads();
      best = red[0];
#pragma unroll
      for (int w = 1; w < QT / 32; ++w) best = max(best, red[w]);
      if (best) g = fmaxf(__fdiv_rn(__uint_as_float(best), 2688.f), 1.17549435e-38f);
      if (blockIdx.x == 0 && threadIdx.x == 0) *a.gscale = g;
    } else {
      g = *a.gscale;
      g_bad = !(g >= 1.17549435e-38f && g <= 3.40282347e38f);
    }
  }
  // units of 16 columns; the scale row's padding is covered too
  const int64_t per = a.lds * (FMT == KRONQ_MXFP4 ? 2 : 1);
  const int64_t total = a.rows * per;
  const int64_t stride = (int64_t)gridDim.x * QT;
  const int64_t first = (int64_t)blockIdx.x * QT;
  int64_t i = first + threadIdx.x;
  int64_t r = i / per, c = i - r * per;
  const int64_t dr = stride / per, dc = stride - dr * per;
  // per is even for MXFP4, so a lane pair always holds one block; every warp
  // runs the same number of steps (total is a multiple of 16, lanes beyond it
  // only take part in the pair exchange)
  for (int64_t base = first + (threadIdx.x & ~31); base < total; base += stride) {
    const bool live = i < total;
    const int64_t j0 = c * 16;
    uint32_t w[BF16 ? 8 : 16];
    if (live && j0 < a.n) {
      load16<BF16>(a, r, j0, w);
    } else {
#pragma unroll
      for (int q = 0; q < (BF16 ? 8 : 16); ++q) w[q] = 0u;
    }
    // block maximum; a NaN stays NaN
    float amax;
    if (BF16) {
      __nv_bfloat162 m2 = __habs2(as_bf162(w[0]));
#pragma unroll
      for (int q = 1; q < 8; ++q) m2 = __hmax2_nan(m2, __habs2(as_bf162(w[q])));
      const uint32_t u = as_u32(m2);
      amax = max_nan(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    } else {
      amax = fabsf(__uint_as_float(w[0]));
#pragma unroll
      for (int q = 1; q < 16; ++q) amax = max_nan(amax, fabsf(__uint_as_float(w[BF16 ? 0 : q])));
    }
    if (FMT == KRONQ_MXFP4) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const bool bad = g_bad || !(amax <= 3.40282347e38f);
    uint32_t sbyte;
    uint64_t packed = 0;
    if (FMT == KRONQ_MXFP4) {
      const int e = (int)(__float_as_uint(amax) >> 23) - 127 - 2;
      sbyte = bad ? 255u : (uint32_t)(max(e, -127) + 127);
      // 2^-E: the exponent field 254 - sbyte (sbyte <= 252, so it is normal)
      const float inv = bad ? 0.f : __uint_as_float((254u - sbyte) << 23);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float lo, hi;
        if (BF16) {
          lo = __uint_as_float(w[q] << 16);
          hi = __uint_as_float(w[q] & 0xFFFF0000u);
        } else {
          lo = __uint_as_float(w[BF16 ? 0 : 2 * q]);
          hi = __uint_as_float(w[BF16 ? 0 : 2 * q + 1]);
        }
        uint32_t b;
        asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
            : "=r"(b) : "f"(__fmul_rn(hi, inv)), "f"(__fmul_rn(lo, inv)));
        packed |= (uint64_t)b << (8 * q);
      }
    } else {
      sbyte = bad ? 0x7Fu : nv_scale(amax, g);
      const float s = e4m3_value(sbyte);
      const bool none = bad || sbyte == 0u;   // no border is passed
      if (BF16) {
        uint32_t cnt[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) cnt[q] = 0x43004300u;   // 128: the count ends up in the low bits
#pragma unroll
        for (int b = 0; b < 7; ++b) {
          const __nv_bfloat162 t2 = as_bf162(none ? 0x7FFF7FFFu : pass_bf16x2(b, s, g));
#pragma unroll
          for (int q = 0; q < 8; ++q)
            cnt[q] = as_u32(__hadd2(as_bf162(cnt[q]), __hge2(__habs2(as_bf162(w[q])), t2)));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t nib = (cnt[q] & 0x00070007u) | ((w[q] >> 12) & 0x00080008u);
          packed |= (uint64_t)((nib | (nib >> 12)) & 0xFFu) << (8 * q);
        }
      } else {
        float t[7];
#pragma unroll
        for (int b = 0; b < 7; ++b) t[b] = none ? __uint_as_float(0x7FC00000u) : pass_f32(b, s, g);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const uint32_t bits = w[BF16 ? 0 : q];
          const float v = fabsf(__uint_as_float(bits));
          // three steps of a binary search among the seven borders
          const bool c2 = v >= t[3];
          const bool c1 = v >= (c2 ? t[5] : t[1]);
          const float lo = c2 ? t[4] : t[0], hi = c2 ? t[6] : t[2];
          const bool c0 = v >= (c1 ? hi : lo);
          const uint32_t nib = (c2 ? 4u : 0u) | (c1 ? 2u : 0u) | (c0 ? 1u : 0u) | ((bits >> 28) & 8u);
          packed |= (uint64_t)nib << (4 * q);
        }
      }
    }
    if (bad) packed = 0;
    if (live) {
      if (FMT == KRONQ_NVFP4) a.scales[r * a.lds + c] = j0 < a.n ? (uint8_t)sbyte : (uint8_t)0;
      else if ((c & 1) == 0) a.scales[r * a.lds + (c >> 1)] = j0 < a.n ? (uint8_t)sbyte : (uint8_t)0;
      if (j0 + 16 > a.n && j0 < a.n)   // the sign of a padding zero is +
        packed &= (1ull << (4 * (a.n - j0))) - 1ull;
      if (c * 8 < a.ldc) *reinterpret_cast<uint64_t*>(a.codes + r * a.ldc + c * 8) = packed;
    }
    if (a.deq) {
      float v[16];
      values16<FMT>((uint32_t)packed, (uint32_t)(packed >> 32), fp4_scale_value<FMT>(sbyte), g, v);
      const int count = live && j0 < a.n ? (int)min((int64_t)16, a.n - j0) : 0;
      store_runs<BF16>(a.deq, r * a.ldd + j0, count, a.vec_out, v, runs[threadIdx.x >> 5], threadIdx.x & 31);
    }
    i += stride;
    r += dr;
    c += dc;
    if (c >= per) { c -= per; ++r; }
  }
}

// ---------------------------------------------------------------- dequantise
struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, n, ldc, lds;
  const float* gscale;
  void* out;
  int64_t ldo;
  int vec_out;
};

// Each warp step takes UNROLL runs of 16 codes a lane, so that enough loads
// are in flight: a run reads only 9 bytes for the 32 or 64 that it writes.
constexpr int UNROLL = 4;

template <int FMT, bool BF16>
__global__ void __launch_bounds__(QT) fp4_dequantize_kernel(const DequantArgs a) {
  __shared__ RunSmem runs[QT / 32];
  const float g = FMT == KRONQ_NVFP4 ? *a.gscale : 1.f;
  const int64_t per = (a.n + 15) / 16;
  const int64_t total = a.rows * per;
  const int lane = threadIdx.x & 31;
  const int64_t stride = (int64_t)gridDim.x * QT * UNROLL;
  const int64_t dr = stride / per, dc = stride - dr * per;   // a step of the grid
  int64_t base = (int64_t)blockIdx.x * QT * UNROLL + (int64_t)(threadIdx.x >> 5) * 32 * UNROLL;
  int64_t r = (base + lane) / per, c = base + lane - r * per;
  const int64_t ur = 32 / per, uc = 32 - ur * per;           // from run to run
  for (; base < total; base += stride) {
    uint2 w[UNROLL];
    uint32_t sb[UNROLL];
    int64_t at[UNROLL];
    int count[UNROLL];
    int64_t rr = r, cc = c;
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const bool live = base + 32 * k + lane < total;
      w[k] = make_uint2(0, 0);
      sb[k] = 0;
      if (live) {
        w[k] = *reinterpret_cast<const uint2*>(a.codes + rr * a.ldc + cc * 8);
        sb[k] = a.scales[rr * a.lds + (FMT == KRONQ_MXFP4 ? (cc >> 1) : cc)];
      }
      at[k] = rr * a.ldo + cc * 16;
      count[k] = live ? (int)min((int64_t)16, a.n - cc * 16) : 0;
      rr += ur;
      cc += uc;
      if (cc >= per) { cc -= per; ++rr; }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      float v[16];
      values16<FMT>(w[k].x, w[k].y, fp4_scale_value<FMT>(sb[k]), g, v);
      store_runs<BF16>(a.out, at[k], count[k], a.vec_out, v, runs[threadIdx.x >> 5], lane);
    }
    r += dr;
    c += dc;
    if (c >= per) { c -= per; ++r; }
  }
}

// Blocks for `total` units of one thread each: at most as many as run at once
// (per_sm: the kernel's registers allow that many).
unsigned quant_grid(int64_t total, int per_sm) {
  const int64_t want = ceil_div(total, QT), cap = per_sm * (int64_t)sm_count();
  return (unsigned)(want < 1 ? 1 : want < cap ? want : cap);
}

}  // namespace
}  // namespace kq

using namespace kq;

extern "C" {

int64_t kronq_fp4_code_row_bytes(int64_t n) { return n <= 0 || n > kFp4MaxDim ? 0 : fp4_code_row(n); }

int64_t kronq_fp4_scale_row_bytes(kronq_fp4_format fmt, int64_t n) {
  return n <= 0 || n > kFp4MaxDim || !fp4_fmt_ok(fmt) ? 0 : fp4_scale_row(fmt, n);
}

size_t kronq_fp4_quantize_workspace_bytes(int64_t rows, int64_t n, kronq_fp4_format fmt) {
  if (rows <= 0 || n <= 0 || fmt != KRONQ_NVFP4) return 0;
  return ((MAX_PARTIALS * sizeof(uint32_t) + 255) / 256) * 256;
}

kronq_status kronq_fp4_quantize(const void* x, kronq_dtype dt, int64_t rows, int64_t n, int64_t ldx,
                                kronq_fp4_format fmt, uint8_t* codes, uint8_t* scales, float* gscale,
                                int gscale_given, void* deq, int64_t ldd, void* workspace, size_t ws_bytes,
                                kronq_stream_t s) {
  if (!fp4_fmt_ok(fmt)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: bad format");
  if (dt != KRONQ_BF16 && dt != KRONQ_F32) return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: bad dtype");
  if (rows < 0 || rows > kFp4MaxDim || n <= 0 || n > kFp4MaxDim)
    return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: sizes out of range");
  if (ldx < n || (deq && ldd < n)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: row stride below n");
  if (rows > 0 && (!x || !codes || !scales)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: NULL pointer");
  if (fmt == KRONQ_NVFP4 && !gscale) return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: NVFP4 needs gscale");
  if (fmt == KRONQ_MXFP4 && gscale) return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: MXFP4 has no tensor scale");
  if (!aligned(codes, 16) || !aligned(scales, 16))
    return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: codes and scales must be 16-byte aligned");
  const int esize = dt == KRONQ_BF16 ? 2 : 4;
  if (!aligned(x, esize) || (deq && !aligned(deq, esize)) || (gscale && !aligned(gscale, 4)))
    return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: misaligned pointer");
  const bool compute = fmt == KRONQ_NVFP4 && !gscale_given;
  if (compute && rows > 0 &&
      (!workspace || ws_bytes < kronq_fp4_quantize_workspace_bytes(rows, n, fmt) || !aligned(workspace, 256)))
    return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: workspace too small or not 256-byte aligned");
  if (rows == 0 && !compute) return KRONQ_OK;
  cudaStream_t st = as_stream(s);
  QuantArgs a;
  a.x = x; a.rows = rows; a.n = n; a.ldx = ldx;
  a.codes = codes; a.scales = scales;
  a.ldc = fp4_code_row(n); a.lds = fp4_scale_row(fmt, n);
  a.gscale = gscale;
  a.partial = nullptr; a.npartial = 0;
  a.deq = deq; a.ldd = ldd;
  a.vec_in = aligned(x, 32) && (ldx * esize) % 32 == 0;
  a.vec_out = deq && aligned(deq, 32) && (ldd * esize) % 32 == 0;
  a.x_lo = reinterpret_cast<uintptr_t>(x);
  a.x_hi = a.x_lo + (size_t)(rows > 0 ? (rows - 1) * ldx + n : 0) * esize;
  if (compute) {
    uint32_t* partial = rows > 0 ? static_cast<uint32_t*>(workspace) : reinterpret_cast<uint32_t*>(gscale);
    a.partial = partial;
    if (rows > 0) {
      const int64_t units = rows * (a.vec_in ? ceil_div(n, 16 / esize) : n);
      unsigned grid = quant_grid(ceil_div(units, 4), 6);   // four loads in flight a thread
      if (grid > (unsigned)MAX_PARTIALS) grid = MAX_PARTIALS;
      if (dt == KRONQ_BF16) fp4_amax_kernel<true><<<grid, QT, 0, st>>>(x, rows, n, ldx, a.vec_in, partial);
      else fp4_amax_kernel<false><<<grid, QT, 0, st>>>(x, rows, n, ldx, a.vec_in, partial);
      KQ_LAUNCH_CHECK("fp4_amax_kernel");
      a.npartial = (int)grid;
    }
  }
  const unsigned grid = quant_grid(rows * a.lds * (fmt == KRONQ_MXFP4 ? 2 : 1), 4);
  if (fmt == KRONQ_MXFP4) {
    if (dt == KRONQ_BF16) fp4_quantize_kernel<KRONQ_MXFP4, true><<<grid, QT, 0, st>>>(a);
    else fp4_quantize_kernel<KRONQ_MXFP4, false><<<grid, QT, 0, st>>>(a);
  } else {
    if (dt == KRONQ_BF16) fp4_quantize_kernel<KRONQ_NVFP4, true><<<grid, QT, 0, st>>>(a);
    else fp4_quantize_kernel<KRONQ_NVFP4, false><<<grid, QT, 0, st>>>(a);
  }
  KQ_LAUNCH_CHECK("fp4_quantize_kernel");
  return KRONQ_OK;
}

kronq_status kronq_fp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* gscale,
                                  kronq_fp4_format fmt, int64_t rows, int64_t n, void* out, kronq_dtype dt,
                                  int64_t ldo, kronq_stream_t s) {
  if (!fp4_fmt_ok(fmt)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: bad format");
  if (dt != KRONQ_BF16 && dt != KRONQ_F32) return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: bad dtype");
  if (rows < 0 || rows > kFp4MaxDim || n <= 0 || n > kFp4MaxDim)
    return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: sizes out of range");
  if (ldo < n) return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: row stride below n");
  if (rows > 0 && (!codes || !scales || !out)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: NULL pointer");
  if ((fmt == KRONQ_NVFP4) != (gscale != nullptr))
    return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: gscale goes with NVFP4 and with it only");
  const int esize = dt == KRONQ_BF16 ? 2 : 4;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, esize) || (gscale && !aligned(gscale, 4)))
    return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: misaligned pointer");
  if (rows == 0) return KRONQ_OK;
  DequantArgs a;
  a.codes = codes; a.scales = scales; a.rows = rows; a.n = n;
  a.ldc = fp4_code_row(n); a.lds = fp4_scale_row(fmt, n);
  a.gscale = gscale; a.out = out; a.ldo = ldo;
  a.vec_out = aligned(out, 32) && (ldo * esize) % 32 == 0;
  const unsigned grid = quant_grid(ceil_div(rows * ceil_div(n, 16), UNROLL), 3);
  cudaStream_t st = as_stream(s);
  if (fmt == KRONQ_MXFP4) {
    if (dt == KRONQ_BF16) fp4_dequantize_kernel<KRONQ_MXFP4, true><<<grid, QT, 0, st>>>(a);
    else fp4_dequantize_kernel<KRONQ_MXFP4, false><<<grid, QT, 0, st>>>(a);
  } else {
    if (dt == KRONQ_BF16) fp4_dequantize_kernel<KRONQ_NVFP4, true><<<grid, QT, 0, st>>>(a);
    else fp4_dequantize_kernel<KRONQ_NVFP4, false><<<grid, QT, 0, st>>>(a);
  }
  KQ_LAUNCH_CHECK("fp4_dequantize_kernel");
  return KRONQ_OK;
}

}  // extern "C"
