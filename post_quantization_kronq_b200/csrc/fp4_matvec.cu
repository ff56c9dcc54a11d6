// Product of a few full-precision tokens with microscaled 4-bit weights
// (single-token decode): y[t, r] = g sum_k x[t, k] W[r, k], at most 16 tokens.
//
// Bound by HBM: each weight is 4 bits plus its share of a scale and is used
// once per token.  A CTA of eight warps owns 16 rows at a time, the warps
// split the columns in interleaved spans of 128 (lane t of a row's four loads
// 16 bytes of codes, 32 weights), four spans in flight ahead of the
// arithmetic.  The products run on mma.sync (m16n8k16, bf16 in, float32
// out), rows on the M side, tokens on the N side: one weight load serves 8
// tokens at the price of one.
//
// Weights in bf16 are exact.  A code's bits seem, shifted to the sign and the
// lowest exponent and highest mantissa bits of bf16, are the value times
// 2^-126 (0.5 as a subnormal); one multiplication by scale * 2^118 gives
// value * scale * 2^-8, at most 6 significant bits.  The sums carry 2^-8 to
// their end.  An E8M0 scale outside 2^-119 .. 2^9 takes a second
// multiplication instead.  float32 tokens are three bf16 parts of 8 bits,
// the second and third scaled by 2^8 and 2^16 against underflow, with a sum
// each: all 24 bits take part.
//
// The order of k inside an mma is free as long as weights and tokens agree:
// lane t of a span holds k = 32 t + 8 j + {0..7} as word j, whose pairs
// (i, i + 4) are the halves of one register.  Tokens are staged in shared
// memory in that order, 16-byte pieces placed so that a warp reads without
// bank conflicts.
#include <algorithm>

#include "fp4.cuh"
#include "fp4_products.h"
#include "internal.h"

namespace kq {
namespace {

constexpr int VT = 256, VW = VT / 32;
constexpr int SPAN = 128;                 // columns of one step of a warp
constexpr int BATCH = 4;                  // steps in flight
constexpr int XSMEM = 80 * 1024;          // most shared memory for tokens: two CTAs on an SM

struct VecArgs {
  const void* x;
  int64_t ldx;
  const uint8_t *wc, *ws;
  const float* wg;
  int T;
  int64_t m, n, ldc, lds;
  int kslice;             // columns of a slice, a multiple of SPAN (grid.y slices)
  int xrow;               // bytes of a token's part in shared memory
  int vec;                // 16-byte loads of x
  void* y;
  int y_bf16;
  int64_t ldy;
  float* part;            // partial sums [slice][T][m] (times 2^-8), or NULL
};

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Codes i and i + 4 of a word as bf16 halves, times 2^-126.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  constexpr int up = 12 - 4 * I, mag = 6 - 4 * I;
  const uint32_t s = (up ? w << up : w) & 0x80008000u;
  const uint32_t e = (mag >= 0 ? w << (mag >= 0 ? mag : 0) : w >> (mag < 0 ? -mag : 0)) & 0x01C001C0u;
  return s | e;
}

// Twice in a word: bf16 of an E4M3 scale times 2^118, of an E8M0 one times
// 2^118 (wide: times 2^-8 for the second multiplication by 2^126).
__device__ __forceinline__ uint32_t dup_bf16(float f) {
  const uint32_t u = __float_as_uint(f) >> 16;   // exact: at most 4 significant bits (NaN keeps its top bits)
  return u | (u << 16);
}

template <int FMT, bool XF32, int NT>
struct Vec {
  static constexpr int PARTS = XF32 ? 3 : 1;
  static constexpr int BPL = FMT == KRONQ_NVFP4 ? 2 : 1;   // scale blocks of a lane's 32 columns

  struct Load {
    uint4 w[2];
    uint32_t s[2];
  };

  // Span `sp` of rows r0 + g and r0 + g + 8: codes beyond the row read as
  // zeros, scales beyond it are masked in use.
  static __device__ __forceinline__ void load(const VecArgs& a, int64_t r0, int64_t k, int g, Load& v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = min(r0 + g + 8 * h, a.m - 1);
      if ((k >> 1) < a.ldc) {
        v.w[h] = __ldcs(reinterpret_cast<const uint4*>(a.wc + r * a.ldc + (k >> 1)));
        const uint8_t* s = a.ws + r * a.lds + k / (32 / BPL);
        v.s[h] = BPL == 2 ? (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(s)) : (uint32_t)__ldg(s);
      } else {
        v.w[h] = make_uint4(0, 0, 0, 0);
        v.s[h] = 0;
      }
    }
  }

  static __device__ __forceinline__ void word(const uint32_t (&w)[2], const uint32_t (&mul)[2], bool wide,
                                              const uint4 (&x)[NT][PARTS], float (&acc)[NT][PARTS][4]) {
    uint32_t p[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      p[h][0] = code_pair<0>(w[h]);
      p[h][1] = code_pair<1>(w[h]);
      p[h][2] = code_pair<2>(w[h]);
      p[h][3] = code_pair<3>(w[h]);
      if (FMT == KRONQ_MXFP4 && wide) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[h][i] = mul_bf16x2(p[h][i], 0x7E807E80u);   // 2^126
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) p[h][i] = mul_bf16x2(p[h][i], mul[h]);
    }
    // registers: rows g, g + 8 at the first k pair, then at the second
    const uint32_t a0[4] = {p[0][0], p[1][0], p[0][1], p[1][1]};
    const uint32_t a1[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        mma_16816(acc[nt][q], a0, x[nt][q].x, x[nt][q].y);
        mma_16816(acc[nt][q], a1, x[nt][q].z, x[nt][q].w);
      }
  }

  static __device__ __forceinline__ void step(const VecArgs& a, const Load& v, int64_t k, const uint8_t* xs, int g,
                                              float (&acc)[NT][PARTS][4]) {
    // multipliers of the lane's blocks; blocks at or beyond n count as zero
    uint32_t mul[2][BPL];
    bool wide = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (FMT == KRONQ_NVFP4) {
#pragma unroll
        for (int b = 0; b < BPL; ++b) {
          const uint32_t byte = k + 16 * b < a.n ? (v.s[h] >> (8 * b)) & 0xFFu : 0u;
          mul[h][b] = dup_bf16(e4m3_value(byte) * 0x1p118f);
        }
      } else {
        const bool in = k < a.n;
        wide |= in && (v.s[h] < 8u || v.s[h] > 136u);
        mul[h][0] = in ? dup_bf16(__uint_as_float((v.s[h] + 118u) << 23)) : 0u;
      }
    }
    if (FMT == KRONQ_MXFP4) {
      wide = __any_sync(0xffffffffu, wide);
      if (wide) {   // plain scales, the sums without their 2^-8
#pragma unroll
        for (int h = 0; h < 2; ++h) mul[h][0] = k < a.n ? dup_bf16(e8m0_value(v.s[h])) : 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][q][e] *= 256.f;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 x[NT][PARTS];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
          x[nt][q] = 8 * nt + g < a.T
                         ? *reinterpret_cast<const uint4*>(xs + ((8 * nt + g) * PARTS + q) * a.xrow + j * 64)
                         : make_uint4(0, 0, 0, 0);
      const uint32_t w[2] = {j == 0 ? v.w[0].x : j == 1 ? v.w[0].y : j == 2 ? v.w[0].z : v.w[0].w,
                             j == 0 ? v.w[1].x : j == 1 ? v.w[1].y : j == 2 ? v.w[1].z : v.w[1].w};
      const uint32_t mj[2] = {mul[0][BPL == 2 ? j >> 1 : 0], mul[1][BPL == 2 ? j >> 1 : 0]};
      word(w, mj, wide, x, acc);
    }
    if (FMT == KRONQ_MXFP4 && wide) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][q][e] *= 0x1p-8f;
    }
  }
};

// Byte offset of the eight columns from k on (of a slice) in a token's row:
// spans of 256 bytes, piece j of lane t at 64 j + 16 t.
__device__ __forceinline__ int x_offset(int k) {
  const int t = (k >> 5) & 3, j = (k >> 3) & 3;
  return (k / SPAN) * 256 + j * 64 + t * 16;
}

template <int FMT, bool XF32, int NT>
__global__ void __launch_bounds__(VT, 2) fp4_matvec_kernel(const VecArgs a) {
  using V = Vec<FMT, XF32, NT>;
  extern __shared__ __align__(16) uint8_t xs[];
  __shared__ float red[2][VW][16 * 8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t k0 = (int64_t)blockIdx.y * a.kslice;
  const int cols = (int)min((int64_t)a.kslice, a.n - k0);
  const int spans = (cols + SPAN - 1) / SPAN;
  const int nb = (spans + VW * BATCH - 1) / (VW * BATCH);   // batches of a row tile
  const int64_t tiles = (a.m + 15) / 16;

  // the first batch of weights starts before the tokens are staged; each of
  // its places is refilled for the next batch as soon as it is used
  typename V::Load held[BATCH];
  int64_t tile = blockIdx.x;
  auto fetch = [&](int64_t tl, int b, int i) {
    const int sp = (b * BATCH + i) * VW + warp;
    if (tl < tiles && sp < spans) V::load(a, tl * 16, k0 + sp * SPAN + 32 * t, g, held[i]);
  };
#pragma unroll
  for (int i = 0; i < BATCH; ++i) fetch(tile, 0, i);

  const int padded = spans * SPAN;
  for (int tk = 0; tk < a.T; ++tk) {
    uint8_t* row = xs + (int64_t)tk * V::PARTS * a.xrow;
    for (int k = 8 * threadIdx.x; k < padded; k += 8 * VT) {
      float f[8];
      if (XF32) {
        const float* src = static_cast<const float*>(a.x) + tk * a.ldx + k0 + k;
        if (a.vec && k + 8 <= cols) {
          const float4 u = reinterpret_cast<const float4*>(src)[0], v = reinterpret_cast<const float4*>(src)[1];
          f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
          f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c] = k + c < cols ? src[c] : 0.f;
        }
      } else {
        const uint16_t* src = static_cast<const uint16_t*>(a.x) + tk * a.ldx + k0 + k;
        if (a.vec && k + 8 <= cols) {
          const uint4 u = *reinterpret_cast<const uint4*>(src);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c] = __uint_as_float((c & 1) ? w[c >> 1] & 0xFFFF0000u : w[c >> 1] << 16);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c] = k + c < cols ? __uint_as_float((uint32_t)src[c] << 16) : 0.f;
        }
      }
      const int at = x_offset(k);
#pragma unroll
      for (int q = 0; q < V::PARTS; ++q) {
        uint32_t h[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          // the top 8 bits, then the exact remainder scaled to its place; an
          // infinity or a NaN stays in the first part
          h[c] = __float_as_uint(f[c]) >> 16;
          if (XF32) {
            if (q == 0 && (h[c] & 0x7F80u) == 0x7F80u) {
              if (f[c] != f[c]) h[c] |= 0x40u;
              f[c] = 0.f;
            } else {
              f[c] = (f[c] - __uint_as_float(h[c] << 16)) * 256.f;
            }
          }
        }
        // register i of the piece: codes i (low half) and i + 4 (high half)
        *reinterpret_cast<uint4*>(row + q * a.xrow + at) =
            make_uint4(h[0] | (h[4] << 16), h[1] | (h[5] << 16), h[2] | (h[6] << 16), h[3] | (h[7] << 16));
      }
    }
  }
  __syncthreads();

  const float scale = 256.f, wg = !a.part && a.wg ? *a.wg : 1.f;
  int buf = 0;
  for (; tile < tiles; tile += gridDim.x, buf ^= 1) {
    float acc[NT][V::PARTS][4] = {};
    for (int b = 0; b < nb; ++b) {
      const int64_t tl = b + 1 < nb ? tile : tile + gridDim.x;
      const int bn = b + 1 < nb ? b + 1 : 0;
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int sp = (b * BATCH + i) * VW + warp;
        if (sp < spans) V::step(a, held[i], k0 + sp * SPAN + 32 * t, xs + sp * 256 + 16 * t, g, acc);
        fetch(tl, bn, i);
      }
    }
    float* out = red[buf][warp];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = acc[nt][0][e];
        if (XF32) v = fmaf(acc[nt][V::PARTS - 1][e], 0x1p-16f, fmaf(acc[nt][V::PARTS / 2][e], 0x1p-8f, v));
        // token-major: [token][row]
        out[(8 * nt + 2 * t + (e & 1)) * 16 + g + 8 * (e >> 1)] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * a.T; i += VT) {
      float v = red[buf][0][i];
#pragma unroll
      for (int w = 1; w < VW; ++w) v += red[buf][w][i];
      const int64_t r = tile * 16 + (i & 15), tk = i >> 4;
      if (r < a.m) {
        if (a.part) {
          a.part[((int64_t)blockIdx.y * a.T + tk) * a.m + r] = v;
        } else {
          v = __fmul_rn(__fmul_rn(v, scale), wg);
          if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[tk * a.ldy + r] = __float2bfloat16_rn(v);
          else static_cast<float*>(a.y)[tk * a.ldy + r] = v;
        }
      }
    }
  }
}

// y = the slices' partial sums in order, scaled.
__global__ void __launch_bounds__(256) fp4_matvec_join_kernel(const VecArgs a, int slices) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, total = (int64_t)a.T * a.m;
  if (i >= total) return;
  float v = 0.f;
  for (int s = 0; s < slices; ++s) v += a.part[s * total + i];
  v = __fmul_rn(__fmul_rn(v, 256.f), a.wg ? *a.wg : 1.f);
  const int64_t tk = i / a.m, r = i - tk * a.m;
  if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[tk * a.ldy + r] = __float2bfloat16_rn(v);
  else static_cast<float*>(a.y)[tk * a.ldy + r] = v;
}

// Columns of a slice: as many as leave room for the tokens' parts, fewer
// where there are not enough row tiles for the SMs.
int64_t slice_columns(int64_t T, int64_t m, int64_t n, bool x_f32) {
  const int64_t bytes = T * (x_f32 ? 6 : 2);
  int64_t most = XSMEM / bytes / SPAN * SPAN;
  const int64_t spans = ceil_div(n, SPAN);
  int64_t slices = ceil_div(spans * SPAN, most);
  const int64_t tiles = ceil_div(m, 16);
  while (tiles * slices < 148 && ceil_div(spans, 2 * slices) * SPAN >= 4096) slices *= 2;
  return ceil_div(spans, slices) * SPAN;
}

template <int FMT, bool XF32>
kronq_status launch_vec(const VecArgs& a, dim3 grid, int smem, cudaStream_t st) {
  void (*fn)(const VecArgs) = a.T > 8 ? fp4_matvec_kernel<FMT, XF32, 2> : fp4_matvec_kernel<FMT, XF32, 1>;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), smem);
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
  a.vec = aligned(v.x, 16) && (v.ldx * esize) % 16 == 0;
  a.y = v.y; a.y_bf16 = v.y_bf16; a.ldy = v.ldy;
  a.part = slices > 1 ? static_cast<float*>(v.workspace) : nullptr;
  const int64_t tiles = ceil_div(v.m, 16);
  int64_t gx = 2 * (int64_t)sm_count() / slices;
  if (gx < 1) gx = 1;
  if (gx > tiles) gx = tiles;
  const dim3 grid((unsigned)gx, (unsigned)slices);
  const int smem = (int)(v.T * (v.x_f32 ? 3 : 1)) * a.xrow;
  kronq_status r;
  if (fmt == KRONQ_MXFP4) r = v.x_f32 ? launch_vec<KRONQ_MXFP4, true>(a, grid, smem, st) : launch_vec<KRONQ_MXFP4, false>(a, grid, smem, st);
  else r = v.x_f32 ? launch_vec<KRONQ_NVFP4, true>(a, grid, smem, st) : launch_vec<KRONQ_NVFP4, false>(a, grid, smem, st);
  if (r != KRONQ_OK || slices == 1) return r;
  fp4_matvec_join_kernel<<<(unsigned)ceil_div(v.T * v.m, 256), 256, 0, st>>>(a, (int)slices);
  KQ_LAUNCH_CHECK("fp4_matvec_join_kernel");
  return KRONQ_OK;
}

}  // namespace kq
