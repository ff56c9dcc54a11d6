// Product of a few full-precision tokens with microscaled 4-bit weights
// (single-token decode): y[t, r] = g sum_k x[t, k] W[r, k], at most 16 tokens.
//
// Bound by HBM: each weight is 4 bits plus its share of a scale and is used
// once per token.  Eight warps of a CTA split the columns in interleaved spans
// of 128 (lane t of a row's four takes 16 bytes of codes, 32 weights); a warp
// works on 16 rows at a time.  A slice of few spans (many tokens fill the
// shared memory) gives the spare warps other rows.  Each warp copies its spans
// into a ring of its own in shared memory with cp.async, RING - 1 pairs ahead
// and on into its next rows: loads into registers this far ahead share the
// warp's few scoreboards, and a wait for the first became one for the last
// (61 us against 41 us for 28672 x 8192 NVFP4 and one token).  The products
// run on mma.sync (m16n8k16, fp16 in, float32 out), rows on the M side, tokens
// on the N side: one weight load serves 8 tokens at the price of one.
//
// Measured: 28672 x 8192 NVFP4 with one bf16 token 38 us (0.53 of the measured
// HBM rate), eight 52 us, 16 float32 ones 108 us; 8192 x 28672 MXFP4 with five
// float32 tokens 58 us; 4096 x 4096 NVFP4 with one 7.3 us.  Above a stream of the
// weights alone (29 us) it is bound by its instructions, 172 a warp and span.
//
// Both operands are exact in fp16, or nearly so.  A weight is E2M1 times its
// block scale, at most 6 significant bits: one conversion and one
// multiplication for two weights (E8M0 scales are taken times 2^12, good for
// 2^-35 .. 2^1).  A token's span of 128 columns is scaled by a power of two
// that brings its largest magnitude to [2^14, 2^15): bf16 values down to
// 2^-31 of it are exact; a float32 value down to 2^-28 of it is two parts of 11
// bits (2^-23 off at most; 2^-22 in the lowest binade, where the second is
// subnormal: a third part would cost half as much again).  The sum over a span
// is scaled back when it joins the float32 sum of the row.  What this does not
// cover is computed in float32, one weight and token at a time: a token's span
// with a wider range within its 128 columns, infinities or NaN, and a block whose
// E8M0 scale is beyond the range, unless it holds zeros alone (the quantiser's own
// scale for those is the lowest).  The mma sees zeros there, so that neither the
// other tokens of a call nor the other rows of a tile are summed in another order.
// 28672 x 8192: a bf16 token whose spans are all wide 140 us alone and 214 us among
// five; one MXFP4 block of zeros in a hundred 45 us against 40.
//
// The order of k inside an mma is free as long as weights and tokens agree:
// lane t of a span holds k = 32 t + 8 j + {0..7} as word j.  Tokens are staged
// in shared memory in that order, 16-byte pieces placed so that a warp reads
// without bank conflicts.
#include <algorithm>

#include "fp4.cuh"
#include "fp4_products.h"
#include "internal.h"

namespace kq {
namespace {

constexpr int VT = 256, VW = VT / 32;
constexpr int SPAN = 128;                 // columns of one step of a warp
constexpr int PAIR = 2;                   // neighbouring spans of a step: independent chains of mma
constexpr int RING = 3;                   // steps of a warp in shared memory
constexpr int RSLOT = 16 * SPAN / 2 + 16 * 8;   // codes of 16 rows, up to 8 scale bytes of each
constexpr int RBYTES = VW * RING * PAIR * RSLOT;
constexpr int CTAS = 2;                   // on an SM
constexpr int XSMEM = 40 * 1024;          // shared memory of each for tokens

struct VecArgs {
  const void* x;
  int64_t ldx;
  const uint8_t *wc, *ws;
  const float* wg;
  int T;
  int64_t m, n, ldc, lds;
  int kslice;             // columns of a slice, a multiple of SPAN (grid.y slices)
  int wk;                 // warps that split a slice's columns (1, 2, 4 or 8); the others take other rows
  int xrow;               // bytes of a token's part in shared memory
  int vec;                // 4-element loads of x
  void* y;
  int y_bf16;
  int64_t ldy;
  float* part;            // partial sums [slice][T][m], or NULL
};

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The eight codes of a word as four pairs of halves, in order.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ float x_at(const VecArgs& a, bool f32, int64_t at) {
  return f32 ? static_cast<const float*>(a.x)[at]
             : __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.x)[at] << 16);
}

// E8M0 scales that the fp16 path takes, and their power of two.
constexpr uint32_t kMxLow = 127 - 35, kMxHigh = 127 + 1;
constexpr int kMxShift = 12;

template <int FMT, bool XF32, int NT>
struct Vec {
  static constexpr int PARTS = XF32 ? 2 : 1;
  static constexpr int BPL = FMT == KRONQ_NVFP4 ? 2 : 1;   // scale blocks of a lane's 32 columns
  // spans of a step that are multiplied together, so that four chains of mma are
  // in flight and the registers suffice (16 float32 tokens, 28672 x 8192 MXFP4: 142 us
  // with both spans together, 131 with one; NVFP4 109 and 111)
  static constexpr int AT_ONCE = NT * PARTS >= 4 ? 1 : PAIR;

  struct Load {
    uint4 w[2];
    uint32_t s[2];
  };
  // What a lane copies of a row tile: 16 bytes of codes of rows g and g + 8,
  // and four scale bytes of one row (NVFP4: lane / 2, MXFP4: lane, of the
  // first 16); pointers to the span that is copied next.
  struct Rows {
    const uint8_t *c[2], *s;
  };
  static __device__ __forceinline__ Rows rows(const VecArgs& a, int64_t tile, int64_t k, int lane) {
    Rows p;
#pragma unroll
    for (int h = 0; h < 2; ++h)   // rows beyond m read the last one: their results are not stored
      p.c[h] = a.wc + min(tile * 16 + (lane >> 2) + 8 * h, a.m - 1) * a.ldc + (k >> 1) + 16 * (lane & 3);
    const int row = BPL == 2 ? lane >> 1 : lane & 15;
    p.s = a.ws + min(tile * 16 + row, a.m - 1) * a.lds + k / (32 / BPL) + (BPL == 2 ? 4 * (lane & 1) : 0);
    return p;
  }
  // A pair of whole spans into a ring slot.
  static __device__ __forceinline__ void copy_whole(const Rows& p, uint32_t slot, int lane) {
    const uint32_t code = slot + 16 * lane, scale = slot + 1024 + 4 * lane;
    asm volatile(
        "cp.async.cg.shared.global [%0], [%1], 16;\n\tcp.async.cg.shared.global [%0 + 512], [%2], 16;\n\t"
        "cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16;\n\tcp.async.cg.shared.global [%0 + %5], [%2 + %4], 16;" ::"r"(code),
        "l"(p.c[0]), "l"(p.c[1]), "n"(RSLOT), "n"(SPAN / 2), "n"(RSLOT + 512)
        : "memory");
    if (BPL == 2 || lane < 16)
      asm volatile(
          "cp.async.ca.shared.global [%0], [%1], 4;\n\tcp.async.ca.shared.global [%0 + %2], [%1 + %3], 4;" ::"r"(scale),
          "l"(p.s), "n"(RSLOT), "n"(4 * BPL)
          : "memory");
  }
  // The pair of spans into a ring slot: zeros where the lane's codes do not lie
  // within the row, and for a second span beyond the slice (`left`: columns
  // from the lane's first on of the row, of the slice; a copy of nothing names
  // the first row).
  static __device__ __forceinline__ void copy(const VecArgs& a, const Rows& p, int row_left, int slice_left, uint32_t slot,
                                              int lane) {
#pragma unroll
    for (int s = 0; s < PAIR; ++s) {
      const bool there = s * SPAN < slice_left, in = there && s * SPAN < row_left;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + s * RSLOT + 512 * h + 16 * lane),
                     "l"(in ? p.c[h] + s * (SPAN / 2) : a.wc), "r"(in ? 16 : 0)
                     : "memory");
      if (BPL == 2 || lane < 16)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(slot + s * RSLOT + 1024 + 4 * lane),
                     "l"(there ? p.s + s * (4 * BPL) : a.ws), "r"(there ? 4 : 0)
                     : "memory");
    }
  }
  static __device__ __forceinline__ Load take(const uint8_t* slot, int lane) {
    Load v;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v.w[h] = *reinterpret_cast<const uint4*>(slot + 512 * h + 16 * lane);
      const uint8_t* s = slot + 1024 + (g + 8 * h) * (4 * BPL) + t * BPL;
      v.s[h] = BPL == 2 ? (uint32_t)*reinterpret_cast<const uint16_t*>(s) : (uint32_t)*s;
    }
    return v;
  }

  // Whether fp16 does not take an E8M0 scale, and whether that matters: it does
  // not for zeros (a block of zeros has the lowest scale), except under NaN.
  static __device__ __forceinline__ bool beyond(uint32_t byte) { return byte < kMxLow || byte > kMxHigh; }
  static __device__ __forceinline__ bool counts(uint32_t byte, const uint4& w) {
    return ((w.x | w.y | w.z | w.w) & 0x77777777u) != 0 || byte == 255u;
  }

  // Multipliers of the lane's blocks, of which `left` columns are there (the
  // others count as zero, and so does a block that fp16 does not take); true
  // where there is one of those.
  template <bool WHOLE>
  static __device__ __forceinline__ bool multipliers(const Load& v, int left, uint32_t (&mul)[2][BPL]) {
    bool odd = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (FMT == KRONQ_NVFP4) {
        uint32_t two = v.s[h], f;
        if (!WHOLE && left < 32) two = left <= 0 ? 0u : left <= 16 ? two & 0xFFu : two;
        asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(f) : "r"(two));
        mul[h][0] = __byte_perm(f, f, 0x1010);
        mul[h][BPL - 1] = __byte_perm(f, f, 0x3232);
      } else {
        const bool in = WHOLE || left > 0, off = beyond(v.s[h]);
        odd |= in && off;
        // fp16 2^(byte - 127 + 12), subnormal below 2^-14
        const int e = (int)v.s[h] - 127 + kMxShift + 15;
        const uint32_t one = e >= 1 ? (uint32_t)e << 10 : 1024u >> (1 - e);
        mul[h][0] = in && !off ? one | (one << 16) : 0u;
      }
    }
    return odd;
  }

  // acc += the products of a step's spans in `slot`; left: columns of the slice from the
  // lane's first on (WHOLE: both spans are there); xs: its first piece of the tokens there (row stride of a token
  // and part a.xrow); fac: the factors of the lane's two tokens there; xnext,
  // fnext: offsets of the second span's; apart: the tokens of each span that
  // fp16 does not cover, a bit each.
  //
  // What fp16 does not cover is zero in the mma and added behind it, token by
  // token and block by block, so that a sum's order does not depend on the
  // other tokens and rows.
  template <bool WHOLE>
  static __device__ __forceinline__ void step(const VecArgs& a, const uint8_t* slot, int left, const uint8_t* const (&xs)[NT], int xnext, const float* fac, int fnext,
                                              uint32_t apart0, uint32_t apart1, int64_t kend, int lane, float (&acc)[NT][4]) {
    bool odd = false;
    // no token left for the mma (looked at for few tokens, where it is likely: one
    // token whose spans are all wide 166 -> 142 us, but 16 float32 ones 119 -> 125)
    const bool none = NT == 1 && (apart0 & apart1) == (1u << a.T) - 1u;
#pragma unroll
    for (int s0 = 0; s0 < PAIR && !none; s0 += AT_ONCE) {
      Load v[AT_ONCE];
      uint32_t mul[AT_ONCE][2][BPL];
#pragma unroll
      for (int s = 0; s < AT_ONCE; ++s) {
        v[s] = take(slot + (s0 + s) * RSLOT, lane);
        odd |= multipliers<WHOLE>(v[s], left - (s0 + s) * SPAN, mul[s]);
      }
      float sum[AT_ONCE][NT][PARTS][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int s = 0; s < AT_ONCE; ++s) {
          uint32_t p[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            codes_f16(j == 0 ? v[s].w[h].x : j == 1 ? v[s].w[h].y : j == 2 ? v[s].w[h].z : v[s].w[h].w, p[h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[h][i] = mul_f16x2(p[h][i], mul[s][h][BPL == 2 ? j >> 1 : 0]);
          }
          // registers: rows g, g + 8 at the first k pair, then at the second
          const uint32_t a0[4] = {p[0][0], p[1][0], p[0][1], p[1][1]};
          const uint32_t a1[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
              const uint4 x = *reinterpret_cast<const uint4*>(xs[nt] + (s0 + s) * xnext + q * a.xrow + j * 64);
              mma_16816(sum[s][nt][q], a0, x.x, x.y);
              mma_16816(sum[s][nt][q], a1, x.z, x.w);
            }
        }
      }
#pragma unroll
      for (int s = 0; s < AT_ONCE; ++s)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 f = *reinterpret_cast<const float2*>(fac + (s0 + s) * fnext + 8 * nt);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float w = sum[s][nt][0][e];
            if (XF32) w = fmaf(sum[s][nt][PARTS - 1][e], 0x1p-11f, w);
            acc[nt][e] = fmaf(w, (e & 1) ? f.y : f.x, acc[nt][e]);
          }
        }
    }
    if ((apart0 | apart1) != 0 || (FMT == KRONQ_MXFP4 && __any_sync(0xffffffffu, odd))) {
#pragma unroll 1
      for (int s = 0; s < PAIR; ++s) singly(a, slot + s * RSLOT, left - s * SPAN, kend, s ? apart1 : apart0, lane, acc);
    }
  }

  // A span's products that fp16 does not cover, in float32 from the tokens as
  // given: all of the tokens in `apart`, and every token's with blocks whose
  // scale is beyond its range.
  static __device__ __forceinline__ void singly(const VecArgs& a, const uint8_t* slot, int left, int64_t kend, uint32_t apart, int lane, float (&acc)[NT][4]) {
    const Load v = take(slot, lane);
    const int t = lane & 3;
    uint32_t who[2];   // lanes with such a block, of the rows g and g + 8
#pragma unroll
    for (int h = 0; h < 2; ++h) who[h] = __ballot_sync(0xffffffffu, FMT == KRONQ_MXFP4 && left > 0 && beyond(v.s[h]) && counts(v.s[h], v.w[h]));
    if (!(apart | who[0] | who[1])) return;
#pragma unroll 1
    for (int tk = 0; tk < a.T; ++tk) {
      const bool all = (apart >> tk) & 1u;
      if (!all && !(who[0] | who[1])) continue;
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (all || (who[h] >> lane & 1u)) {
          // 4 * 2^126 and more is beyond float32: a block under the highest scales is summed at an eighth
          const bool high = FMT == KRONQ_MXFP4 && v.s[h] >= 253u && v.s[h] != 255u;
          const uint32_t w[4] = {v.w[h].x, v.w[h].y, v.w[h].z, v.w[h].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float sc = fp4_scale_value<FMT>(BPL == 2 ? (v.s[h] >> (8 * (j >> 1))) & 0xFFu : high ? v.s[h] - 3u : v.s[h]);
            const int64_t at = tk * a.ldx + kend - left + 8 * j;
#pragma unroll 1
            for (int i = 0; i < 8; i += 2) {
              const float2 d = e2m1x2_float2((w[j] >> (4 * i)) & 0xFFu);
              if (8 * j + i < left) s[h] = fmaf(d.x * sc, x_at(a, XF32, at + i), s[h]);
              if (8 * j + i + 1 < left) s[h] = fmaf(d.y * sc, x_at(a, XF32, at + i + 1), s[h]);
            }
          }
          if (high) s[h] *= 8.f;
        }
        s[h] += __shfl_xor_sync(0xffffffffu, s[h], 1);
        s[h] += __shfl_xor_sync(0xffffffffu, s[h], 2);
      }
      // who >> (lane & 28): the four lanes of a row
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (tk == 8 * nt + 2 * t + (e & 1) && (all || (who[e >> 1] >> (lane & 28) & 15u))) acc[nt][e] += s[e >> 1];
    }
  }
};

// Byte offset of column k (of a slice) in a token's row: spans of 256 bytes,
// piece j of lane t at 64 j + 16 t.
__device__ __forceinline__ int x_offset(int k) {
  const int t = (k >> 5) & 3, j = (k >> 3) & 3;
  return (k / SPAN) * 256 + j * 64 + t * 16 + (k & 7) * 2;
}

// One span of a token into shared memory (a warp, a lane per four columns):
// scaled to fp16 parts; its factor, or false where fp16 does not cover it.
template <int FMT, bool XF32>
__device__ __forceinline__ bool stage_span(const float (&f)[4], uint8_t* dst, int xrow, float& factor) {
  uint32_t big = 0, small = 0xFFFFFFFFu;     // magnitudes as bits; zeros are no smallest
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t b = __float_as_uint(f[c]) & 0x7FFFFFFFu;
    big = max(big, b);
    small = min(small, b - 1u);
  }
  big = __reduce_max_sync(0xffffffffu, big);
  small = __reduce_min_sync(0xffffffffu, small);
  const int e = (int)(big >> 23) - 127;      // [2^e, 2^(e+1)) holds the largest
  // the range that fp16 parts cover, away from the ends of float32's
  constexpr int kRange = XF32 ? 28 : 31;
  const bool covered = big == 0 || (e >= -90 && e < 128 && (int)((small + 1u) >> 23) - 127 >= e - kRange);
  const float up = covered && big ? __uint_as_float((uint32_t)(14 - e + 127) << 23) : 0.f;
  factor = covered && big ? __uint_as_float((uint32_t)(e - 14 - (FMT == KRONQ_MXFP4 ? kMxShift : 0) + 127) << 23) : 0.f;
  float r[4];
  __half h[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float s = covered ? f[c] * up : 0.f;
    h[c] = __float2half_rn(s);
    r[c] = (s - __half2float(h[c])) * 2048.f;
  }
  *reinterpret_cast<uint2*>(dst) =
      make_uint2((uint32_t)__half_as_ushort(h[0]) | ((uint32_t)__half_as_ushort(h[1]) << 16),
                 (uint32_t)__half_as_ushort(h[2]) | ((uint32_t)__half_as_ushort(h[3]) << 16));
  if (XF32) {
#pragma unroll
    for (int c = 0; c < 4; ++c) h[c] = __float2half_rn(r[c]);
    *reinterpret_cast<uint2*>(dst + xrow) =
        make_uint2((uint32_t)__half_as_ushort(h[0]) | ((uint32_t)__half_as_ushort(h[1]) << 16),
                   (uint32_t)__half_as_ushort(h[2]) | ((uint32_t)__half_as_ushort(h[3]) << 16));
  }
  return covered;
}

template <int FMT, bool XF32, int NT>
__global__ void __launch_bounds__(VT, CTAS) fp4_matvec_kernel(const __grid_constant__ VecArgs a) {
  using V = Vec<FMT, XF32, NT>;
  // the warps' rings, the tokens' parts, then per span the factors of 8 NT
  // tokens and a bit for each token that is computed in float32 there
  extern __shared__ __align__(16) uint8_t xsm[];
  __shared__ float red[2][VW][16 * 8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t k0 = (int64_t)blockIdx.y * a.kslice;
  const int cols = (int)min((int64_t)a.kslice, a.n - k0);
  const int spans = (cols + SPAN - 1) / SPAN;
  const int wk = a.wk, wr = VW / wk;                        // warps along the columns, along the rows
  const int kw = warp & (wk - 1), rw = warp / wk;
  const int64_t tiles = (a.m + 15) / 16, hop = (int64_t)gridDim.x * wr;
  uint8_t* ring = xsm + warp * (RING * PAIR * RSLOT);
  uint8_t* xpart = xsm + RBYTES;
  float* fac = reinterpret_cast<float*>(xpart + (int64_t)a.T * V::PARTS * a.xrow);
  uint32_t* apart = reinterpret_cast<uint32_t*>(fac + spans * 8 * NT);

  // the copies' position: RING - 1 steps ahead of the arithmetic's
  const int whole = cols / SPAN;                            // spans without a ragged end
  const int hop_k = wk * PAIR;                              // spans from a warp's step to its next
  int64_t ctile = (int64_t)blockIdx.x * wr + rw;
  int cspan = kw * PAIR;
  uint32_t cslot = smem_u32(ring);
  typename V::Rows at = V::rows(a, ctile, k0 + cspan * SPAN, lane);
  const int row_left = (int)min(a.ldc * 2 - k0 - 32 * t, (int64_t)1 << 30);
  auto copy_next = [&]() {
    if (ctile < tiles && cspan < spans) {
      if (cspan + PAIR <= whole) V::copy_whole(at, cslot, lane);
      else V::copy(a, at, row_left - cspan * SPAN, (spans - cspan) * SPAN, cslot, lane);
      cspan += hop_k;
#pragma unroll
      for (int h = 0; h < 2; ++h) at.c[h] += hop_k * (SPAN / 2);
      at.s += hop_k * (4 * V::BPL);
      if (cspan >= spans) {
        cspan = kw * PAIR;
        ctile += hop;
        if (ctile < tiles) at = V::rows(a, ctile, k0 + cspan * SPAN, lane);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    cslot += PAIR * RSLOT;
    if (cslot == smem_u32(ring) + RING * PAIR * RSLOT) cslot = smem_u32(ring);
  };
#pragma unroll 1
  for (int i = 0; i < RING - 1; ++i) copy_next();

  for (int i = threadIdx.x; i < spans * (8 * NT + 1); i += VT) fac[i] = 0.f;   // and apart
  __syncthreads();
  // a warp per span and token, four of them in flight
  for (int u0 = warp; u0 < spans * a.T; u0 += 4 * VW) {
    float f[4][4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int u = min(u0 + w * VW, spans * a.T - 1), sp = u / a.T;
      const int k = sp * SPAN + 4 * lane;
      const int64_t src = (u - sp * a.T) * a.ldx + k0 + k;
      if (a.vec && k + 4 <= cols) {
        if (XF32) {
          const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + src);
          f[w][0] = q.x; f[w][1] = q.y; f[w][2] = q.z; f[w][3] = q.w;
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.x) + src);
          f[w][0] = __uint_as_float(q.x << 16); f[w][1] = __uint_as_float(q.x & 0xFFFF0000u);
          f[w][2] = __uint_as_float(q.y << 16); f[w][3] = __uint_as_float(q.y & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) f[w][c] = k + c < cols ? x_at(a, XF32, src + c) : 0.f;
      }
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int u = u0 + w * VW, sp = u / a.T, tk = u - sp * a.T;
      if (u < spans * a.T) {
        float factor;
        const bool covered = stage_span<FMT, XF32>(
            f[w], xpart + (int64_t)tk * V::PARTS * a.xrow + x_offset(sp * SPAN + 4 * lane), a.xrow, factor);
        if (lane == 0) {
          fac[sp * 8 * NT + tk] = factor;
          if (!covered) atomicOr(&apart[sp], 1u << tk);
        }
      }
    }
  }
  __syncthreads();

  // columns of the mma beyond T read the last token: their sums are not stored
  const uint8_t* xs[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xs[nt] = xpart + (int64_t)min(8 * nt + g, a.T - 1) * V::PARTS * a.xrow + 16 * t;

  const float wg = !a.part && a.wg ? *a.wg : 1.f;
  int buf = 0;
  const uint8_t* held = ring;
  for (int64_t tile0 = (int64_t)blockIdx.x * wr; tile0 < tiles; tile0 += hop, buf ^= 1) {
    float acc[NT][4] = {};
    if (tile0 + rw < tiles) {
#pragma unroll 1
      for (int sp = kw * PAIR; sp < spans; sp += hop_k) {
        asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
        __syncwarp();   // the other lanes' copies are in, and they are done with the slot that is copied to next
        copy_next();
        const uint8_t* xp[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) xp[nt] = xs[nt] + sp * 256;
        const float* fp = fac + sp * 8 * NT + 2 * t;
        const int left = cols - sp * SPAN - 32 * t;
        if (sp + PAIR <= whole) {
          V::template step<true>(a, held, left, xp, 256, fp, 8 * NT, apart[sp], apart[sp + 1], k0 + cols, lane, acc);
        } else {
          // a second span beyond the last has zero weights: any tokens do
          const int has = sp + 1 < spans ? 1 : 0;
          V::template step<false>(a, held, left, xp, has * 256, fp, has * 8 * NT, apart[sp], has ? apart[sp + 1] : 0u,
                                  k0 + cols, lane, acc);
        }
        held += PAIR * RSLOT;
        if (held == ring + RING * PAIR * RSLOT) held = ring;
      }
    }
    float* out = red[buf][warp];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)   // token-major: [token][row]
        out[(8 * nt + 2 * t + (e & 1)) * 16 + g + 8 * (e >> 1)] = acc[nt][e];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * a.T * wr; i += VT) {
      const int part = i / (16 * a.T), in = i - part * 16 * a.T;
      float v = red[buf][part * wk][in];
      for (int w = 1; w < wk; ++w) v += red[buf][part * wk + w][in];
      const int64_t r = (tile0 + part) * 16 + (in & 15), tk = in >> 4;
      if (r < a.m) {
        if (a.part) {
          a.part[((int64_t)blockIdx.y * a.T + tk) * a.m + r] = v;
        } else {
          v = __fmul_rn(v, wg);
          if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[tk * a.ldy + r] = __float2bfloat16_rn(v);
          else static_cast<float*>(a.y)[tk * a.ldy + r] = v;
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// y = the slices' partial sums in order, scaled.
__global__ void __launch_bounds__(256) fp4_matvec_join_kernel(const VecArgs a, int slices) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, total = (int64_t)a.T * a.m;
  fp4_await_first();
  if (i >= total) return;
  const float v = __fmul_rn(fp4_join(a.part + i, total, slices), a.wg ? *a.wg : 1.f);
  const int64_t tk = i / a.m, r = i - tk * a.m;
  if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[tk * a.ldy + r] = __float2bfloat16_rn(v);
  else static_cast<float*>(a.y)[tk * a.ldy + r] = v;
}

// Shared memory of a span's factors and its float32 tokens.
int span_bytes(int64_t T) { return (T > 8 ? 17 : 9) * 4; }

// Columns of a slice: as many as leave room for the tokens' parts, fewer
// where there are not enough row tiles for the SMs.
int64_t slice_columns(int64_t T, int64_t m, int64_t n, bool x_f32) {
  const int64_t bytes = T * (x_f32 ? 4 : 2) * SPAN + span_bytes(T);
  const int64_t spans = ceil_div(n, SPAN);
  int64_t slices = ceil_div(spans, XSMEM / bytes);
  const int64_t tiles = ceil_div(m, 16);
  while (tiles * slices < 148 && ceil_div(spans, 2 * slices) * SPAN >= 4096) slices *= 2;
  return ceil_div(spans, slices) * SPAN;
}

template <int FMT, bool XF32>
kronq_status launch_vec(const VecArgs& a, dim3 grid, int smem, int dev, cudaStream_t st) {
  static std::atomic<bool> done[2][kMaxDevices];
  void (*fn)(const VecArgs) = a.T > 8 ? fp4_matvec_kernel<FMT, XF32, 2> : fp4_matvec_kernel<FMT, XF32, 1>;
  // one limit for every call, so that calls of other threads do not lower it
  cudaError_t e = fp4_allow_smem(reinterpret_cast<const void*>(fn), RBYTES + XSMEM + 4 * 1024, dev, done[a.T > 8]);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(fp4 matvec)");
  fn<<<grid, VT, smem, st>>>(a);
  KQ_LAUNCH_CHECK("fp4_matvec_kernel");
  return KRONQ_OK;
}

}  // namespace

// Partial sums for either token type.
size_t fp4_matvec_workspace(int64_t T, int64_t m, int64_t n) {
  const int64_t slices = std::max(ceil_div(n, slice_columns(T, m, n, false)), ceil_div(n, slice_columns(T, m, n, true)));
  return slices > 1 ? (size_t)(ceil_div(slices * T * m * 4, 256) * 256) : 0;
}

kronq_status fp4_matvec(const Fp4Matvec& v, int fmt, cudaStream_t st) {
  const int64_t kslice = slice_columns(v.T, v.m, v.n, v.x_f32), slices = ceil_div(v.n, kslice);
  VecArgs a;
  a.x = v.x; a.ldx = v.ldx; a.wc = v.wc; a.ws = v.ws; a.wg = v.wg;
  a.T = (int)v.T; a.m = v.m; a.n = v.n;
  a.ldc = fp4_code_row(v.n); a.lds = fp4_scale_row(fmt, v.n);
  a.kslice = (int)kslice;
  a.xrow = (int)kslice * 2 + 64;   // a token's row is shifted by half of the banks against its neighbour's
  const int esize = v.x_f32 ? 4 : 2;
  a.vec = aligned(v.x, 4 * esize) && v.ldx % 4 == 0;
  a.y = v.y; a.y_bf16 = v.y_bf16; a.ldy = v.ldy;
  a.part = slices > 1 ? static_cast<float*>(v.workspace) : nullptr;
  // Warps along the columns: all eight, unless that leaves a warp fewer than
  // four steps of a row tile between two joins of the warps' sums and there are
  // rows enough to keep two rounds of CTAs busy.
  const int64_t pairs = ceil_div(kslice, SPAN * PAIR), tiles = ceil_div(v.m, 16);
  a.wk = VW;
  while (a.wk > 1 && (a.wk > pairs || (pairs < 4 * a.wk && tiles * (a.wk / 2) / VW * slices >= 2 * CTAS * 148)))
    a.wk /= 2;
  const int64_t groups = ceil_div(tiles, VW / a.wk);   // row tiles that a CTA takes at once
  int dev = 0;
  int64_t gx = CTAS * (int64_t)fp4_sms(&dev) / slices;
  if (gx < 1) gx = 1;
  if (gx > groups) gx = groups;
  const dim3 grid((unsigned)gx, (unsigned)slices);
  const int smem = RBYTES + (int)(v.T * (v.x_f32 ? 2 : 1)) * a.xrow + (int)(kslice / SPAN) * span_bytes(v.T);
  kronq_status r;
  if (fmt == KRONQ_MXFP4) r = v.x_f32 ? launch_vec<KRONQ_MXFP4, true>(a, grid, smem, dev, st) : launch_vec<KRONQ_MXFP4, false>(a, grid, smem, dev, st);
  else r = v.x_f32 ? launch_vec<KRONQ_NVFP4, true>(a, grid, smem, dev, st) : launch_vec<KRONQ_NVFP4, false>(a, grid, smem, dev, st);
  if (r != KRONQ_OK || slices == 1) return r;
  const cudaError_t e = fp4_launch_second(fp4_matvec_join_kernel, (unsigned)ceil_div(v.T * v.m, 256), 256, st, a, (int)slices);
  count_launch();
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_fail(e, "fp4_matvec_join_kernel");
  }
  return KRONQ_OK;
}

}  // namespace kq
