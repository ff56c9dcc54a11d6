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
// Large tensors work out per CTA, for every scale byte, the amax that reaches
// it and a reciprocal that gives bf16's exact decisions by the conversion
// instruction (checked at the borders; NvTable).
//
// One thread per 16 elements (8 bytes of codes, 32 or 64 bytes of input),
// lane pairs share an MXFP4 block.  Bound by HBM: the input once (twice when
// the tensor scale is computed), codes, scales and the optional dequantised
// values once.  Measured, with dequantised values: 16384 x 8192 bf16 to MXFP4
// 104 us (0.89 of the measured HBM rate), 8192 x 8192 bf16 to NVFP4 under a
// given scale 60 us (0.78; 82 us when every block compares its borders),
// 11008 x 4096 float32 to NVFP4 98 us, 26 of them the pass for the tensor
// scale; 28672 x 8192 NVFP4 back to bf16 103 us (0.89).
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"

namespace kq {
namespace {

constexpr int QT = 256;               // threads per block
constexpr int MAX_PARTIALS = 1024;    // partial maxima, at most one per block

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
  int table;                // NVFP4: borders and reciprocals of every scale are worked out first
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

// What NVFP4's rounding takes from a scale's byte, for all of them at once (a
// CTA works out both in about a microsecond, which pays from two blocks a
// thread on): the smallest amax that reaches the byte, and for bf16 input a
// reciprocal r of scale g for which RN_e2m1(x r) in float32 is the exact
// decision for every bf16 x.  RN_e2m1(x r) does not decrease in x, so it is
// enough that it is right on both sides of the seven borders; 0 where none of
// the neighbouring floats does that (the borders are compared then).  For
// float32 input the reciprocal is just the rounded one: x r is off by at most
// 3 units in its last place (three roundings of 2^-24 relative), and a block
// with an x r within 8 units of a value of three significant bits, as the
// borders are, compares with the borders.
struct NvTable {
  float reach[128];
  float recip[128];
};
__device__ __forceinline__ uint32_t e2m1_code(float x) {
  uint32_t b;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(b) : "f"(0.f), "f"(x));
  return b & 15u;
}
template <bool BF16>
__device__ __forceinline__ void fill_table(NvTable& tab, float g, int c) {
  const float v = e4m3_value(min(c, 126));
  if (c == 0) {
    tab.reach[0] = 0.f;
  } else if (c == 127) {
    tab.reach[127] = __uint_as_float(0x7F800000u);
  } else {   // a tie at an even byte's lower midpoint reaches it
    const float mid = __fmul_rn(3.f, __fadd_rn(v, e4m3_value(c - 1)));
    tab.reach[c] = (c & 1) ? __uint_as_float(__float_as_uint(__fmul_rd(mid, g)) + 1u) : __fmul_ru(mid, g);
  }
  if (BF16) {
    float found = 0.f;
    if (c > 0 && c < 127) {
      const float r0 = __fdiv_rn(1.f, __fmul_rn(v, g));
      for (int k = 0; k < 5 && found == 0.f; ++k) {   // r0, then one and two steps down and up
        const float r = __uint_as_float(__float_as_uint(r0) + (k & 1 ? -((k + 1) >> 1) : k >> 1));
        bool right = true;
        for (int i = 0; i < 7; ++i) {
          const uint32_t pass = pass_bf16x2(i, v, g) << 16;
          right &= e2m1_code(__uint_as_float(pass) * r) > (uint32_t)i &&
                   e2m1_code(__uint_as_float(pass - 0x10000u) * r) <= (uint32_t)i;
        }
        if (right) found = r;
      }
    }
    tab.recip[c] = found;
  } else {
    tab.recip[c] = c > 0 && c < 127 ? __fdiv_rn(1.f, __fmul_rn(v, g)) : 0.f;
  }
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
// rows take 32-byte stores.  In others a lane's stores are the 16-byte words
// of memory that end in its run: it takes what the first of them needs from
// the lane before, where that holds the run before in the row.  Elements that
// no such word covers are stored one by one.
template <bool BF16, bool VEC>
__device__ __forceinline__ void store_runs(void* out, int64_t at, int count, const float (&v)[16], int lane) {
  constexpr int NW = BF16 ? 8 : 16, ES = BF16 ? 2 : 4;
  uint32_t c[NW + 5];   // the four words before the run, the run
#pragma unroll
  for (int q = 0; q < NW; ++q)
    c[4 + q] = BF16 ? as_u32(__floats2bfloat162_rn(v[2 * (q % 8)], v[2 * (q % 8) + 1])) : __float_as_uint(v[q]);
  const uintptr_t addr = reinterpret_cast<uintptr_t>(out) + at * ES;
  const bool whole = count == 16;
  if (VEC) {
    if (whole) {
      store32(reinterpret_cast<void*>(addr), c + 4);
      if (!BF16) store32(reinterpret_cast<void*>(addr + 32), c + (BF16 ? 4 : 12));
    } else if (count > 0) {
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        if (q < count) {
          if (BF16) reinterpret_cast<__nv_bfloat16*>(addr)[q] = __float2bfloat16_rn(v[q]);
          else reinterpret_cast<float*>(addr)[q] = v[q];
        }
      }
    }
    return;
  }
  const uintptr_t before = __shfl_up_sync(0xffffffffu, (unsigned long long)addr, 1);
  const int before_whole = __shfl_up_sync(0xffffffffu, (int)whole, 1);
  const bool joins = lane > 0 && whole && before_whole && before + NW * 4 == addr;
  const int next_joins = __shfl_down_sync(0xffffffffu, (int)joins, 1);
#pragma unroll
  for (int q = 0; q < 4; ++q) c[q] = __shfl_up_sync(0xffffffffu, c[NW + q], 1);
  c[NW + 4] = 0;
  const int off = (int)(addr & 15);
  int lo = 0, hi = count;      // elements stored one by one: up to lo, and from hi on
  if (whole) {
    uint32_t w[NW + 5];
#pragma unroll
    for (int q = 0; q < NW + 5; ++q) w[q] = c[q];
    // the words begin 16 - off bytes into c
    const int skip = 16 - off;
    if (skip & 16) {
#pragma unroll
      for (int q = 0; q < NW + 1; ++q) w[q] = w[q + 4];
    }
    if (skip & 8) {
#pragma unroll
      for (int q = 0; q < NW + 3; ++q) w[q] = w[q + 2];
    }
    if (skip & 4) {
#pragma unroll
      for (int q = 0; q < NW + 1; ++q) w[q] = w[q + 1];
    }
    if (BF16) {
#pragma unroll
      for (int q = 0; q < NW; ++q) w[q] = __funnelshift_r(w[q], w[q + 1], 8 * (skip & 2));
    }
    uint4* o = reinterpret_cast<uint4*>(addr - off);
    const bool head = off == 0 || joins;
    if (head) o[0] = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
    for (int q = 1; q < NW / 4; ++q) o[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    lo = head ? 0 : skip / ES;
    hi = next_joins && lane < 31 ? 16 : 16 - off / ES;
    count = 16;
  } else {
    hi = 0;
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    if (q < count && (q < lo || q >= hi)) {
      if (BF16) reinterpret_cast<__nv_bfloat16*>(addr)[q] = __float2bfloat16_rn(v[q]);
      else reinterpret_cast<float*>(addr)[q] = v[q];
    }
  }
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

// Largest magnitude of 16 elements; a NaN stays NaN.
template <bool BF16>
__device__ __forceinline__ float block_max(const uint32_t (&w)[BF16 ? 8 : 16]) {
  if (BF16) {
    __nv_bfloat162 m2 = __habs2(as_bf162(w[0]));
#pragma unroll
    for (int q = 1; q < 8; ++q) m2 = __hmax2_nan(m2, __habs2(as_bf162(w[q])));
    const uint32_t u = as_u32(m2);
    return max_nan(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
  float m = fabsf(__uint_as_float(w[0]));
#pragma unroll
  for (int q = 1; q < 16; ++q) m = max_nan(m, fabsf(__uint_as_float(w[BF16 ? 0 : q])));
  return m;
}

// Largest finite |x| as one partial per block (float bits; non-negative floats
// order like their bits).  A warp takes AMAX_RUNS runs of 32 x 16 elements at
// a time, so that their loads are in flight together.
constexpr int AMAX_RUNS = 2;
template <bool BF16>
__global__ void __launch_bounds__(QT, 4) fp4_amax_kernel(const QuantArgs a, uint32_t* partial) {
  constexpr int NW = BF16 ? 8 : 16;
  constexpr int RUNS = BF16 ? 2 * AMAX_RUNS : AMAX_RUNS;
  fp4_let_next_in();
  float best = 0.f;
  const int64_t per = (a.n + 15) / 16, total = a.rows * per;
  const int lane = threadIdx.x & 31;
  const int64_t stride = (int64_t)gridDim.x * QT * RUNS;
  const int64_t dr = stride / per, dc = stride - dr * per, ur = 32 / per, uc = 32 - ur * per;
  int64_t base = (int64_t)blockIdx.x * QT * RUNS + (int64_t)(threadIdx.x >> 5) * 32 * RUNS;
  int64_t r = (base + lane) / per, c = base + lane - r * per;
  for (; base < total; base += stride) {
    uint32_t w[RUNS][NW];
    int64_t rr = r, cc = c;
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      if (base + 32 * k + lane < total) {
        load16<BF16>(a, rr, cc * 16, w[k]);
      } else {
#pragma unroll
        for (int q = 0; q < NW; ++q) w[k][q] = 0u;
      }
      rr += ur;
      cc += uc;
      if (cc >= per) { cc -= per; ++rr; }
    }
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const float m = block_max<BF16>(w[k]);
      if (m <= 3.40282347e38f) {
        best = fmaxf(best, m);
      } else {   // the block's finite values
#pragma unroll
        for (int q = 0; q < NW; ++q) {
          const float hi = fabsf(__uint_as_float(BF16 ? w[k][q] & 0xFFFF0000u : w[k][q]));
          const float lo = BF16 ? fabsf(__uint_as_float(w[k][q] << 16)) : 0.f;
          if (hi <= 3.40282347e38f) best = fmaxf(best, hi);
          if (lo <= 3.40282347e38f) best = fmaxf(best, lo);
        }
      }
    }
    r += dr;
    c += dc;
    if (c >= per) { c -= per; ++r; }
  }
  uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(best));
  __shared__ uint32_t red[QT / 32];
  if (lane == 0) red[threadIdx.x >> 5] = bits;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int q = 1; q < QT / 32; ++q) bits = max(bits, red[q]);
    partial[blockIdx.x] = bits;
  }
}

template <int FMT, bool BF16>
__global__ void __launch_bounds__(QT, 4) fp4_quantize_kernel(const QuantArgs a) {
  __shared__ NvTable tab;
  float g = 1.f, inv6g = 0.f;
  bool g_bad = false;
  if (FMT == KRONQ_NVFP4) {
    if (a.partial) {
      fp4_await_first();
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
  // (the quotients stay normal for these g)
  const bool table = FMT == KRONQ_NVFP4 && a.table && g >= 0x1p-100f && g <= 0x1p100f;
  if (FMT == KRONQ_NVFP4 && table) {
    inv6g = __fdiv_rn(1.f, __fmul_rn(6.f, g));
    if (threadIdx.x < 128) fill_table<BF16>(tab, g, threadIdx.x);
    __syncthreads();
  }
  // units of 16 columns; the scale row's padding is covered too
  const int64_t per = a.lds * (FMT == KRONQ_MXFP4 ? 2 : 1);
  const int64_t total = a.rows * per;
  const int64_t stride = (int64_t)gridDim.x * QT;
  const int64_t first = (int64_t)blockIdx.x * QT;
  // from the last units to the first: what the pass for the tensor scale read
  // last is still in L2
  const int64_t warp0 = first + (threadIdx.x & ~31);
  const int64_t steps = warp0 < total ? (total - warp0 + stride - 1) / stride : 0;
  int64_t i = first + threadIdx.x + (steps - 1) * stride;
  int64_t r = i / per, c = i - r * per;
  const int64_t dr = stride / per, dc = stride - dr * per;
  // per is even for MXFP4, so a lane pair always holds one block; every warp
  // runs the same number of steps (total is a multiple of 16, lanes beyond it
  // only take part in the pair exchange)
  for (int64_t n = 0; n < steps; ++n) {
    const bool live = i < total;
    const int64_t j0 = c * 16;
    uint32_t w[BF16 ? 8 : 16];
    if (live && j0 < a.n) {
      load16<BF16>(a, r, j0, w);
    } else {
#pragma unroll
      for (int q = 0; q < (BF16 ? 8 : 16); ++q) w[q] = 0u;
    }
    float amax = block_max<BF16>(w);
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
      if (bad) {
        sbyte = 0x7Fu;
      } else if (table) {   // a quotient that is off by one byte at most, then the exact borders
        uint16_t p;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(0.f), "f"(amax * inv6g));
        sbyte = min(p & 0xFFu, 126u);
        if (amax < tab.reach[sbyte]) --sbyte;
        else if (amax >= tab.reach[sbyte + 1]) ++sbyte;
      } else {
        sbyte = nv_scale(amax, g);
      }
      const float s = e4m3_value(sbyte);
      const bool none = bad || sbyte == 0u;   // no border is passed
      float recip = table && !bad ? tab.recip[sbyte] : 0.f;
      if (!BF16) {
        bool near = false;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const uint32_t y = __float_as_uint(__fmul_rn(__uint_as_float(w[BF16 ? 0 : q]), recip));
          near |= ((y + 8u) & 0x1FFFFFu) <= 16u;
        }
        if (near) recip = 0.f;   // (zeros count as near: blocks with exact zeros are compared too)
      }
      if (!BF16 && recip != 0.f) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t b;
          asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
              : "=r"(b)
              : "f"(__fmul_rn(__uint_as_float(w[BF16 ? 0 : 2 * q + 1]), recip)),
                "f"(__fmul_rn(__uint_as_float(w[BF16 ? 0 : 2 * q]), recip)));
          packed |= (uint64_t)b << (8 * q);
        }
      } else if (BF16 && recip != 0.f) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t b;
          asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
              : "=r"(b)
              : "f"(__uint_as_float(w[q] & 0xFFFF0000u) * recip), "f"(__uint_as_float(w[q] << 16) * recip));
          packed |= (uint64_t)b << (8 * q);
        }
      } else if (BF16) {
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
      if (a.vec_out) store_runs<BF16, true>(a.deq, r * a.ldd + j0, count, v, threadIdx.x & 31);
      else store_runs<BF16, false>(a.deq, r * a.ldd + j0, count, v, threadIdx.x & 31);
    }
    i -= stride;
    r -= dr;
    c -= dc;
    if (c < 0) { c += per; --r; }
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
};

// Each warp step takes UNROLL runs of 16 codes a lane, so that enough loads
// are in flight: a run reads only 9 bytes for the 32 or 64 that it writes.
// Where DQ_RUNS would leave SMs without a block, or with one where another's
// stores would have covered its waits, one run: 100 x 4095 NVFP4 to float32
// 5.2 -> 2.8 us, 1000 x 4095 8.0 -> 7.3, but 28672 x 8192 to bf16 104 -> 132.
constexpr int DQ_RUNS = 4;

template <int FMT, bool BF16, bool VEC, int UNROLL>
__global__ void __launch_bounds__(QT, UNROLL == 1 ? 4 : 3) fp4_dequantize_kernel(const DequantArgs a) {
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
      store_runs<BF16, VEC>(a.out, at[k], count[k], v, lane);
    }
    r += dr;
    c += dc;
    if (c >= per) { c -= per; ++r; }
  }
}

// Blocks for `total` units of one thread each: at most as many as run at once
// (per_sm: the kernel's registers allow that many).
unsigned quant_grid(int64_t total, int per_sm) {
  const int64_t want = ceil_div(total, QT), cap = std::min<int64_t>(per_sm * (int64_t)fp4_sms(nullptr), MAX_PARTIALS);
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
  return fp4_entry([&]() -> kronq_status {
    if (!fp4_fmt_ok(fmt)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: bad format");
    if (dt != KRONQ_BF16 && dt != KRONQ_F32) return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: bad dtype");
    if (rows < 0 || rows > kFp4MaxDim || n <= 0 || n > kFp4MaxDim)
      return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: sizes out of range");
    if (ldx < n || ldx > kFp4MaxStride || (deq && (ldd < n || ldd > kFp4MaxStride)))
      return fail(KRONQ_ERR_INVALID_ARG, "fp4_quantize: row stride out of range");
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
        const unsigned grid = quant_grid(ceil_div(rows * ceil_div(n, 16), dt == KRONQ_BF16 ? 2 * AMAX_RUNS : AMAX_RUNS), 4);
        if (dt == KRONQ_BF16) fp4_amax_kernel<true><<<grid, QT, 0, st>>>(a, partial);
        else fp4_amax_kernel<false><<<grid, QT, 0, st>>>(a, partial);
        KQ_LAUNCH_CHECK("fp4_amax_kernel");
        a.npartial = (int)grid;
      }
    }
    const int64_t units = rows * a.lds * (fmt == KRONQ_MXFP4 ? 2 : 1);
    const unsigned grid = quant_grid(units, 4);
    a.table = units >= 2 * (int64_t)grid * QT;
    if (a.npartial) {
      const cudaError_t e = dt == KRONQ_BF16 ? fp4_launch_second(fp4_quantize_kernel<KRONQ_NVFP4, true>, grid, QT, st, a)
                                             : fp4_launch_second(fp4_quantize_kernel<KRONQ_NVFP4, false>, grid, QT, st, a);
      count_launch();
      if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail(e, "fp4_quantize_kernel");
      }
      return KRONQ_OK;
    }
    if (fmt == KRONQ_MXFP4) {
      if (dt == KRONQ_BF16) fp4_quantize_kernel<KRONQ_MXFP4, true><<<grid, QT, 0, st>>>(a);
      else fp4_quantize_kernel<KRONQ_MXFP4, false><<<grid, QT, 0, st>>>(a);
    } else {
      if (dt == KRONQ_BF16) fp4_quantize_kernel<KRONQ_NVFP4, true><<<grid, QT, 0, st>>>(a);
      else fp4_quantize_kernel<KRONQ_NVFP4, false><<<grid, QT, 0, st>>>(a);
    }
    KQ_LAUNCH_CHECK("fp4_quantize_kernel");
    return KRONQ_OK;
  });
}

kronq_status kronq_fp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* gscale,
                                  kronq_fp4_format fmt, int64_t rows, int64_t n, void* out, kronq_dtype dt,
                                  int64_t ldo, kronq_stream_t s) {
  return fp4_entry([&]() -> kronq_status {
    if (!fp4_fmt_ok(fmt)) return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: bad format");
    if (dt != KRONQ_BF16 && dt != KRONQ_F32) return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: bad dtype");
    if (rows < 0 || rows > kFp4MaxDim || n <= 0 || n > kFp4MaxDim)
      return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: sizes out of range");
    if (ldo < n || ldo > kFp4MaxStride) return fail(KRONQ_ERR_INVALID_ARG, "fp4_dequantize: row stride out of range");
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
    const int vec_out = aligned(out, 32) && (ldo * esize) % 32 == 0;   // rows are 32-byte aligned
    // aligned bf16 rows leave a block the least to store (2048 x 2048: 3.9 us
    // with DQ_RUNS, 4.2 with one)
    const int64_t runs = rows * ceil_div(n, 16);
    const bool one = runs < (dt == KRONQ_BF16 && vec_out ? 1 : 2) * (int64_t)fp4_sms(nullptr) * QT * DQ_RUNS;
    const unsigned grid = quant_grid(one ? runs : ceil_div(runs, DQ_RUNS), 6);
    cudaStream_t st = as_stream(s);
    using K = void (*)(const DequantArgs);
#define FP4_DQ(F, B) \
  fp4_dequantize_kernel<F, B, false, DQ_RUNS>, fp4_dequantize_kernel<F, B, false, 1>, \
  fp4_dequantize_kernel<F, B, true, DQ_RUNS>, fp4_dequantize_kernel<F, B, true, 1>
    static const K kernels[16] = {FP4_DQ(KRONQ_MXFP4, false), FP4_DQ(KRONQ_MXFP4, true), FP4_DQ(KRONQ_NVFP4, false),
                                  FP4_DQ(KRONQ_NVFP4, true)};
#undef FP4_DQ
    kernels[8 * (fmt == KRONQ_NVFP4) + 4 * (dt == KRONQ_BF16) + 2 * vec_out + one]<<<grid, QT, 0, st>>>(a);
    KQ_LAUNCH_CHECK("fp4_dequantize_kernel");
    return KRONQ_OK;
  });
}

}  // extern "C"
