// Product of two microscaled 4-bit matrices on the tensor cores, plain or
// grouped by expert: y[t, r] = gx gw sum_k X[t, k] W[r, k].
//
// tcgen05 multiplies E2M1 operands with their block scales (kind::mxf4nvf4
// with four E4M3 scales per 64 columns, kind::mxf4 with two E8M0 ones) at four
// times the bf16 rate; accumulation is float32 in TMEM, the tensor scales
// multiply the sums.  The weights are the M side: a pair of SMs
// (cta_group::2) owns 256 rows of W and up to 256 tokens (N, a multiple of
// 64, so few tokens cost few columns), 128 rows and half of the tokens' codes
// in each CTA.  Per 256-column chunk a CTA stages 128 bytes of codes of each
// of its rows by TMA (128-byte swizzle).
//
// Scales: the tensor core wants, for 128 rows and 4 scale bytes, 32 lanes x 4
// words with row r in lane r % 32, word r / 32.  The user's layout is row by
// row, so loader warps read 16 bytes of four rows 32 apart, transpose the
// 4 x 4 words in registers and store 16-byte rows of four such 512-byte atoms;
// tcgen05.cp spreads an atom over TMEM, one loader group ahead of its MMAs.
// They work in groups of two such pieces (32 bytes of scales of a row), four
// groups in flight in registers and two or four in shared memory, because a
// load, its way to the barrier and the copy take longer than the MMAs of a few
// chunks.  A tile of 256 x 256 leaves 256 of the 512 TMEM columns for scales;
// the eight epilogue warps drain the accumulator into registers first and
// release it before they store.
//
// Bound by the 1 kW power cap for long runs of large products (back to back for
// seconds 2048 x 28672 x 8192 NVFP4 246 us, 3.9 PFLOP/s at 1.48 GHz, and 8192 x 8192
// x 28672 MXFP4 779 us, 4.9 PFLOP/s at 1.24 GHz, 0.82 of the tensor rate at that
// clock; 209 and 723 us before the clock falls), by the supply of operands and
// scales at full clocks, by HBM for few tokens (16 tokens, 8192 x 28672 NVFP4
// 32 us, 0.62 of the measured rate with the columns split), by latency below that
// (100 x 1000 x 4095 9 us in four parts).
//
// The loaders of both CTAs arrive at the even CTA's barrier, whose MMA thread
// copies the scales of both.  Each loader's stores go behind a proxy fence (the
// copies read by the async proxy) and a release at cluster scope that is
// restricted to the CTA's own shared memory, and the MMA thread acquires at the
// same scope.  An unrestricted release also waits for the loader's global loads in
// flight (1500 - 2200 cycles), and from a warp without any, which hands the
// arrivals on, it still made products 20 - 35 % slower.  The epilogue's
// arrival orders reads of TMEM alone: the tcgen05 fences around it do that.
//
// Warps: 0 TMA, 1 MMA (one lane of the even CTA), 2-7 scales, 8-15 epilogue.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp4.cuh"
#include "fp4_products.h"
#include "internal.h"

namespace kq {
namespace {

constexpr int GM = 256, GH = 128, GN = 256;   // rows of W per pair, per CTA; most tokens per tile
constexpr int NG = 64;                        // granularity of a tile's tokens
constexpr int CK = 256;                       // columns per chunk: 128 bytes of codes
constexpr int WBOX = GH * 128;                // 16 KB
constexpr int XROWS = NG / 2;                 // token rows of one TMA box
constexpr int XBOX = XROWS * 128;             // 4 KB
constexpr int STAGE = WBOX + GH * 128;        // 32 KB
constexpr int PIECE = 3 * 2048;               // 16 scale bytes of 128 + 256 rows, as atoms
constexpr int SLOT = 2 * PIECE;               // a loader group
constexpr int AHEAD = 4;                      // groups in a loader's registers
// Stages of codes and slots of scales: a group is two chunks of NVFP4, whose
// MMAs take about as long as a slot's turn, and four of MXFP4.
constexpr int stages(int fmt) { return fmt == KRONQ_NVFP4 ? 5 : 6; }
constexpr int slots(int fmt) { return fmt == KRONQ_NVFP4 ? 4 : 2; }
constexpr int GROUP_INTS = 2 * (KRONQ_FP4_MAX_EXPERTS + 1);
constexpr int LOADERS = 6, EPI = 8;           // warps
constexpr int THREADS = 32 * (2 + LOADERS + EPI);
constexpr int smem_bytes(int fmt) { return stages(fmt) * STAGE + slots(fmt) * SLOT + 256 + GROUP_INTS * 4 + 1024; }
constexpr uint32_t SF_COL = GN;               // TMEM columns of the scales: two groups of 96

struct GemmArgs {
  const uint8_t *xs, *ws;
  const float *xg, *wg;
  const int* offsets;     // grouped: E + 1 bounds, else NULL
  int E;
  int64_t T, m, lds;
  int kb;                 // scale bytes of a row that are data
  int nchunks, tiles_m;
  int splits, per_split;  // chunks of a split
  void* y;
  int64_t ldy;
  int y_pairs;            // bf16 rows are 4-byte aligned
  float* part;            // split partial sums [split][T][m], or NULL
};

// Tile u of the persistent loop.
struct Tile {
  int e;            // expert
  int64_t m0;       // first row within the expert
  int64_t t0, t1;   // tokens
  int cols;         // N: tokens rounded up to NG
  int c0, c1;       // chunks
  int split;
};

// Group bounds and first tiles, and the walk over tiles: up to eight token
// tiles of a group run next to each other on the same rows of W, so that W
// comes from L2 after its first reader.
struct Walk {
  const int* bound;
  const int* first;
  int ntiles;

  __device__ __forceinline__ bool get(const GemmArgs& a, int u, Tile& t) const {
    if (u >= ntiles) return false;
    t.split = u % a.splits;
    u /= a.splits;
    int e = 0;
    int64_t lo = 0, hi = a.T;
    if (a.offsets) {
      int l = 0, h = a.E - 1;   // the last group whose first tile is <= u
      while (l < h) {
        const int mid = (l + h + 1) >> 1;
        if (first[mid] <= u) l = mid; else h = mid - 1;
      }
      e = l;
      u -= first[e];
      lo = bound[e];
      hi = bound[e + 1];
    }
    const int tn = (int)((hi - lo + GN - 1) / GN);
    const int band = 8 * a.tiles_m;
    const int b = u / band, in = u - b * band;
    const int width = min(8, tn - 8 * b);
    const int i = in / width, j = 8 * b + (in - i * width);
    t.e = e;
    t.m0 = (int64_t)i * GM;
    t.t0 = lo + (int64_t)j * GN;
    t.t1 = min(hi, t.t0 + GN);
    t.cols = ((int)(t.t1 - t.t0) + NG - 1) / NG * NG;
    t.c0 = t.split * a.per_split;
    t.c1 = min(a.nchunks, t.c0 + a.per_split);
    return true;
  }
};

// Bounds as documented (each at least its predecessor, within [0, T]) and the
// number of tiles before each group, by one warp.
__device__ void group_walk(const GemmArgs& a, int* bound, int* first, int lane) {
  int top = 0;
  for (int i0 = 0; i0 <= a.E; i0 += 32) {
    const int i = i0 + lane;
    int v = i <= a.E ? (int)min((int64_t)max(a.offsets[i], 0), a.T) : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, p);
    }
    v = max(v, top);
    if (i <= a.E) bound[i] = v;
    top = __shfl_sync(0xffffffffu, v, 31);
  }
  __syncwarp();
  int sum = 0;
  for (int i0 = 0; i0 < a.E; i0 += 32) {
    const int i = i0 + lane;
    const int own = i < a.E ? (bound[i + 1] - bound[i] + GN - 1) / GN * a.tiles_m : 0;
    int v = own;
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += p;
    }
    if (i < a.E) first[i] = sum + v - own;
    sum += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) first[a.E] = sum;
}

// A 512-byte scale atom to four TMEM columns, where `go` is not 0; lo, hi:
// words of its descriptor.
__device__ __forceinline__ void copy_atom(uint32_t tcol, uint32_t lo, uint32_t hi, uint32_t go) {
  asm volatile(
      "{\n\t.reg .b64 d;\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b64 d, {%1, %2};\n\t"
      "@p tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(tcol),
      "r"(lo), "r"(hi), "r"(go)
      : "memory");
}

// One lane of a converged warp, in the form from which the compiler knows that
// a single thread issues (a test of the lane number costs tens of cycles per
// tcgen05 instruction).
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Arrival at a barrier of the pair's even CTA.  Relaxed: what it announces is
// ordered by a fence before it and one behind the wait, lighter ones than a
// release and an acquire of all memory.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_remote(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// This CTA's shared memory to the pair's other CTA, and the other side.
__device__ __forceinline__ void fence_release_smem() {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
__device__ __forceinline__ void fence_acquire_smem() {
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

// D (+)= A B for the pair; alo, blo, hi: words of the operands' descriptors.
template <int FMT>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint32_t alo, uint32_t blo, uint32_t hi, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (FMT == KRONQ_NVFP4)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %7, 0;\n\tmov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %4, [%5], [%6], p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %7, 0;\n\tmov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %4, [%5], [%6], p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: E2M1 operands (both K-major), scale type E4M3 (0) or
// E8M0 (1), M 256; id selects the first scale byte of a word (MXFP4: 0 or 2).
template <int FMT>
__device__ __forceinline__ uint32_t fp4_idesc(int cols, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) |
         ((FMT == KRONQ_MXFP4 ? 1u : 0u) << 23) | ((uint32_t)(GM >> 4) << 24) | (id << 29);
}

// Waits for a barrier's phase.  The first try is the common case and costs one
// instruction; the bounded wait (which records a time-out) and the look at the
// CTA's abort flag come only after it fails.
__device__ __forceinline__ bool await(uint32_t bar, uint32_t parity, volatile int* abort_s) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*abort_s) return false;
  if (mbar_wait(bar, parity)) return true;
  *abort_s = 1;
  return false;
}

// The same at a barrier that mbar_arrive_remote arrives at.
__device__ __forceinline__ bool await_remote(uint32_t bar, uint32_t parity, volatile int* abort_s) {
  while (!mbar_try_wait_remote(bar, parity))
    if (!await(bar, parity, abort_s)) return false;
  return true;
}

// Bytes of word j of a 16-byte piece of which `valid` bytes are data.
__device__ __forceinline__ uint32_t tail_mask(int valid, int j) {
  const int left = valid - 4 * j;
  return left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
}

// Both tensor scales as factors of a sum: their product and 1, unless the
// product leaves float32's normal range.
__device__ __forceinline__ float2 tensor_scales(const GemmArgs& a, int e) {
  const float xg = a.xg ? *a.xg : 1.f, wg = a.wg ? a.wg[e] : 1.f, both = __fmul_rn(xg, wg);
  return both >= 1.17549435e-38f && both <= 3.40282347e38f ? make_float2(both, 1.f) : make_float2(xg, wg);
}

template <int FMT, bool BF16, bool PART>
__global__ void __launch_bounds__(THREADS, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX,
                    const __grid_constant__ CUtensorMap mXfull, const GemmArgs a) {
  constexpr int CPP = FMT == KRONQ_NVFP4 ? 1 : 2;   // chunks per 16-byte scale piece
  constexpr int STAGES = stages(FMT), SLOTS = slots(FMT);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sfmem = smem + STAGES * STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sfmem + SLOTS * SLOT);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
  const uint32_t sffull0 = empty0 + 8 * STAGES, sfempty0 = sffull0 + 8 * SLOTS;
  const uint32_t accfull = sfempty0 + 8 * SLOTS, accempty = accfull + 8, done = accempty + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 2 * SLOTS + 3);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* bound = reinterpret_cast<int*>(sfmem + SLOTS * SLOT + 256);
  int* first = bound + KRONQ_FP4_MAX_EXPERTS + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cl_rank();
  const int pair = (int)blockIdx.x >> 1, npairs = (int)gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < SLOTS; ++b) {
      mbar_init(sffull0 + 8 * b, 2 * LOADERS);
      mbar_init(sfempty0 + 8 * b, 1);
    }
    mbar_init(accfull, 1);
    mbar_init(accempty, 2 * EPI);
    mbar_init(done, 1);
    *abort_s = 0;
    fence_mbar_init();
    prefetch_tmap(&mW);
    prefetch_tmap(&mX);
    prefetch_tmap(&mXfull);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  if (warp == 2 && a.offsets) group_walk(a, bound, first, lane);
  tc_fence_before();
  cl_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk walk;
  walk.bound = bound;
  walk.first = first;
  walk.ntiles = a.offsets ? first[a.E] : a.tiles_m * (int)((a.T + GN - 1) / GN) * a.splits;
  Tile t;

  if (warp == 0) {
    if (elect_lane()) {
      const uint32_t full_lead = cl_map(full0, 0);
      uint32_t s = 0, ph = 0;
      bool ok = true;
      for (int u = pair; ok && walk.get(a, u, t); u += npairs) {
        const int rw = (int)((int64_t)t.e * a.m + t.m0) + GH * (int)rank;
        const int boxes = t.cols / NG;
        const int rx = (int)t.t0 + (t.cols / 2) * (int)rank;
        for (int c = t.c0; c < t.c1; ++c) {
          ok = await(empty0 + 8 * s, ph ^ 1, abort_s);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2u * (uint32_t)(WBOX + boxes * XBOX));
          const uint32_t st = smem_u32(smem) + s * STAGE, fb = full_lead + 8 * s;
          tma_load_2d_pair(st, &mW, fb, c * (CK / 2), rw);
          if (boxes == GN / NG) {
            tma_load_2d_pair(st + WBOX, &mXfull, fb, c * (CK / 2), rx);
          } else {
            for (int b = 0; b < boxes; ++b)
              tma_load_2d_pair(st + WBOX + b * XBOX, &mX, fb, c * (CK / 2), rx + b * XROWS);
          }
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_lane()) {
      // This thread's own instructions take about as long as the MMAs, so the
      // loop runs over whole loader groups without a branch for each chunk,
      // counters advance by increments and descriptors by adding to their low
      // words.  A group's scales go to TMEM while the group before is
      // multiplied, chunk by chunk, into the other of two buffers (copies and
      // MMAs of one thread run in the order of their issue, so a copy does not
      // overtake the MMAs that still read its buffer).
      constexpr int CH = 2 * CPP;             // chunks of a group
      constexpr uint32_t kCols = 48 / CPP;    // TMEM columns of a chunk's scales
      uint32_t s = 0, ph = 0;                 // stage of codes
      uint32_t slot = 0, sph = 0;             // slot of scales
      uint32_t buf = 0;                       // TMEM buffer of the group that is multiplied
      int done_tiles = 0;
      bool ok = true, issued = false;
      const uint32_t stage0 = (smem_u32(smem) >> 4) | (1u << 16);
      const uint32_t atom0 = (smem_u32(sfmem) >> 4) | (128u >> 4 << 16);
      constexpr uint32_t kAtomHi = (128 >> 4) | (1u << 14);                 // no swizzle, 8-row groups of 128 bytes
      constexpr uint32_t kCodeHi = (1024 >> 4) | (1u << 14) | (2u << 29);   // 128-byte swizzle
      // scales of chunk i of the group in `slot`
      auto copy_scales = [&](int i, uint32_t to, uint32_t two) {
        const uint32_t atom = atom0 + slot * (SLOT >> 4) + (i / CPP) * (PIECE >> 4) + (CPP == 1 ? 0 : (i & 1) * 64);
        const uint32_t sf = tmem + SF_COL + to * 96 + i * kCols;
#pragma unroll
        for (int j = 0; j < 4 / CPP; ++j) {
          copy_atom(sf + 4 * j, atom + 32 * j, kAtomHi, 1u);
          copy_atom(sf + kCols / 3 + 8 * j, atom + 128 + 32 * j, kAtomHi, 1u);
          copy_atom(sf + kCols / 3 + 4 + 8 * j, atom + 256 + 32 * j, kAtomHi, two);
        }
      };
      auto scales_done = [&]() {
        mma_commit_pair_mc(sfempty0 + 8 * slot, 0x3);
        if (++slot == SLOTS) { slot = 0; sph ^= 1; }
      };
      for (int u = pair; ok && walk.get(a, u, t); u += npairs, ++done_tiles) {
        const int count = t.c1 - t.c0;
        const uint32_t two = t.cols > GH ? 1u : 0u;
        const uint32_t idesc = fp4_idesc<FMT>(t.cols, 0);
        ok = await_remote(sffull0 + 8 * slot, sph, abort_s);
        if (!ok) break;
        fence_acquire_smem();
        tc_fence_after();
        issued = true;
#pragma unroll
        for (int i = 0; i < CH; ++i) copy_scales(i, buf, two);
        scales_done();
        if (done_tiles > 0) ok = await_remote(accempty, (done_tiles - 1) & 1, abort_s);
        tc_fence_after();
        for (int lc = 0; ok && lc < count; lc += CH) {
          const bool more = lc + CH < count;
          if (more) {
            ok = await_remote(sffull0 + 8 * slot, sph, abort_s);
            if (!ok) break;
            fence_acquire_smem();
            tc_fence_after();
          }
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            if (lc + i < count) {
              if (more) copy_scales(i, buf ^ 1, two);
              ok = ok && await(full0 + 8 * s, ph, abort_s);
              if (!ok) break;
              tc_fence_after();
              const uint32_t sf = tmem + SF_COL + buf * 96 + i * kCols;
              const uint32_t wlo = stage0 + s * (STAGE >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const int j = kk / CPP;
                const uint32_t id = CPP == 1 ? 0u : 2u * (kk & 1);
                mma_fp4_pair<FMT>(tmem, wlo + 2 * kk, wlo + (WBOX >> 4) + 2 * kk, kCodeHi,
                                  idesc | (id << 4) | (id << 29), sf + 4 * j, sf + kCols / 3 + 8 * j,
                                  i + kk > 0 || lc > 0 ? 1u : 0u);
              }
              mma_commit_pair_mc(empty0 + 8 * s, 0x3);
              if (++s == STAGES) { s = 0; ph ^= 1; }
            }
          }
          if (ok && more) scales_done();
          buf ^= 1;
        }
        if (ok) mma_commit_pair_mc(accfull, 0x3);
      }
      if (issued) {
        mma_commit_pair_mc(done, 0x1);
        mbar_wait(done, 0);
      }
    }
    __syncwarp();
  } else if (warp < 2 + LOADERS) {
    // Two warps load the scales of the CTA's rows of W, four those of the
    // tile's tokens.  A group is two pieces of a unit (32 bytes of a row's
    // scales, a sector): lane (p, i) holds piece p of rows i, i + 32, i + 64
    // and i + 96.  AHEAD groups are in flight in registers.
    const int part = (warp - 2) >> 1;                        // W, tokens 0 - 127, tokens 128 - 255
    const int p = lane >> 4, i = 16 * (warp & 1) + (lane & 15);
    const uint32_t lead = cl_map(sffull0, 0);
    const int lds = (int)a.lds;
    int u = pair, c = 0;                                     // the walk's unit and next chunk
    bool more = walk.get(a, u, t);
    if (more) c = t.c0;
    const uint8_t* base = nullptr;                           // the unit's first row
    int last = 0;                                            // rows beyond it read it: their results are not stored
    auto enter = [&]() {
      if (part == 0) {
        const int64_t r0 = (int64_t)t.e * a.m + t.m0 + GH * (int64_t)rank, rem = (int64_t)a.E * a.m - 1 - r0;
        last = (int)min((int64_t)GH, max(rem, (int64_t)0));
        base = a.ws + (rem < 0 ? r0 + rem : r0) * a.lds;
      } else {
        const int64_t r0 = t.t0 + GH * (part - 1), rem = a.T - 1 - r0;
        last = (int)min((int64_t)GH, max(rem, (int64_t)0));
        base = a.xs + (rem < 0 ? r0 + rem : r0) * a.lds;
      }
    };
    if (more) enter();
    uint4 v[AHEAD][4];
    // data bytes of the lane's piece (may be below 0 or above 16); nothing to
    // store for a part that the tile lacks; no more groups
    constexpr int NOTHING = -(1 << 30), END = NOTHING - 1;
    int valid[AHEAD];
    auto issue = [&](uint4 (&w)[4]) -> int {
      if (!more) return END;
      const int byte = 16 * (c / CPP + p);
      int n = NOTHING;
      if (part < 2 || t.cols > GH) {
        n = a.kb - byte;
        const int at = min(byte, lds - 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = __ldg(reinterpret_cast<const uint4*>(base + (min(i + 32 * q, last) * lds + at)));
      }
      c += 2 * CPP;
      if (c >= t.c1) {
        u += npairs;
        more = walk.get(a, u, t);
        if (more) {
          c = t.c0;
          enter();
        }
      }
      return n;
    };
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) valid[d] = issue(v[d]);
    uint32_t slot = 0, sph = 0;
    for (bool ok = true; ok;) {
#pragma unroll
      for (int d = 0; d < AHEAD; ++d) {
        if (!ok) break;
        ok = valid[d] != END;
        if (!ok) break;
        ok = __all_sync(0xffffffffu, await(sfempty0 + 8 * slot, sph ^ 1, abort_s));
        if (!ok) break;
        uint4(&w)[4] = v[d];
        if (valid[d] != NOTHING) {
          if (valid[d] < 16) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              w[q].x &= tail_mask(valid[d], 0);
              w[q].y &= tail_mask(valid[d], 1);
              w[q].z &= tail_mask(valid[d], 2);
              w[q].w &= tail_mask(valid[d], 3);
            }
          }
          uint4* o = reinterpret_cast<uint4*>(sfmem + slot * SLOT + p * PIECE + part * 2048 + i * 16);
          o[0] = make_uint4(w[0].x, w[1].x, w[2].x, w[3].x);
          o[32] = make_uint4(w[0].y, w[1].y, w[2].y, w[3].y);
          o[64] = make_uint4(w[0].z, w[1].z, w[2].z, w[3].z);
          o[96] = make_uint4(w[0].w, w[1].w, w[2].w, w[3].w);
          fence_proxy_async_smem();
        }
        __syncwarp();
        fence_release_smem();
        if (lane == 0) mbar_arrive_remote(lead + 8 * slot);
        if (++slot == SLOTS) { slot = 0; sph ^= 1; }
        valid[d] = issue(w);
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2 - LOADERS) >> 2;
    const uint32_t lead = cl_map(accempty, 0);
    int done_tiles = 0;
    for (int u = pair; walk.get(a, u, t); u += npairs, ++done_tiles) {
      int good = 1;
      if (lane == 0) good = await(accfull, done_tiles & 1, abort_s) ? 1 : 0;
      if (!__shfl_sync(0xffffffffu, good, 0)) break;
      tc_fence_after();
      const int64_t r = t.m0 + GH * (int64_t)rank + q * 32 + lane;
      const float2 scale = PART ? make_float2(1.f, 1.f) : tensor_scales(a, t.e);
      const float xg = scale.x, wg = scale.y;
      const bool one = wg == 1.f;
      const int groups = t.cols / 64;    // 32-column groups of this warp: half, half + 2, ...
      const int64_t ld = PART ? a.m : a.ldy;
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
      if (BF16) {
        uint32_t pk[4][16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g < groups) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(acc + (uint32_t)(2 * g + half) * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float lo = __fmul_rn(__uint_as_float(v[2 * e]), xg), hi = __fmul_rn(__uint_as_float(v[2 * e + 1]), xg);
              if (!one) lo = __fmul_rn(lo, wg), hi = __fmul_rn(hi, wg);
              const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
              pk[g][e] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead);
        uint16_t* y = static_cast<uint16_t*>(a.y);
        const bool rows32 = t.m0 + GH * (int64_t)rank + q * 32 + 32 <= a.m;   // the warp's rows are all there
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g < groups) {
            const int64_t tk = t.t0 + (2 * g + half) * 32;
            if (a.y_pairs && rows32 && tk + 32 <= t.t1) {
              // neighbouring lanes exchange halves: an even lane stores two rows
              // of the first token of a pair, an odd lane those of the second
              const uint32_t pick = (lane & 1) ? 0x3276u : 0x5410u;
              uint16_t* o = y + (tk + (lane & 1)) * ld + (r & ~int64_t(1));
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, pk[g][e], 1);
                *reinterpret_cast<uint32_t*>(o) = __byte_perm(pk[g][e], other, pick);
                o += 2 * ld;
              }
            } else {
              uint16_t* o = y + tk * ld + r;
              const int left = (int)min(t.t1 - tk, (int64_t)32);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                if (r < a.m && 2 * e < left) o[0] = (uint16_t)(pk[g][e] & 0xFFFFu);
                if (r < a.m && 2 * e + 1 < left) o[ld] = (uint16_t)(pk[g][e] >> 16);
                o += 2 * ld;
              }
            }
          }
        }
      } else {
        float* y = PART ? a.part + (int64_t)t.split * a.T * a.m : static_cast<float*>(a.y);
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(acc + (uint32_t)(2 * g + half) * 32, v);
          tmem_wait_ld();
          const int64_t tk = t.t0 + (2 * g + half) * 32;
          const int left = (int)min(t.t1 - tk, (int64_t)32);
          float* o = y + tk * ld + r;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (r < a.m && e < left) {
              const float f = PART ? __uint_as_float(v[e]) : __fmul_rn(__uint_as_float(v[e]), xg);
              *o = one ? f : __fmul_rn(f, wg);
            }
            o += ld;
          }
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead);
      }
    }
  }
  if (*abort_s) {   // copies in flight land within microseconds; leave after a millisecond
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 1000000ull) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  cl_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// y = the splits' partial sums in order, scaled.
__global__ void __launch_bounds__(256) fp4_join_kernel(const GemmArgs a, int bf16) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, total = a.T * a.m;
  fp4_await_first();
  if (i >= total) return;
  const float2 scale = tensor_scales(a, 0);
  const float v = __fmul_rn(__fmul_rn(fp4_join(a.part + i, total, a.splits), scale.x), scale.y);
  const int64_t t = i / a.m, r = i - t * a.m;
  if (bf16) static_cast<__nv_bfloat16*>(a.y)[t * a.ldy + r] = __float2bfloat16_rn(v);
  else static_cast<float*>(a.y)[t * a.ldy + r] = v;
}

// Chunks of a split.  The columns are split where the tiles would leave at
// least half of the pairs of SMs idle, into at most one part for each pair, as
// the sum of three times decides: a chunk of a part 0.3 us (0.22 - 0.35
// measured), the kernel that joins the parts 2.2 us, and the partial sums'
// way to memory and back at 4.5 TB/s (256 tokens, 4096 x 4096 NVFP4: 14 us
// whole, 18 in four parts; 100 tokens, 1000 x 4095: 11.0 and 9.0).
constexpr int64_t kSplitPairs = 74;
int64_t split_chunks(int64_t T, int64_t m, int64_t n) {
  const int64_t chunks = ceil_div(n, CK), tiles = ceil_div(m, GM) * ceil_div(T, GN);
  if (2 * tiles > kSplitPairs) return chunks;
  int64_t best = chunks, best_ns = 300 * chunks;
  for (int64_t parts = 2; parts <= kSplitPairs / tiles; ++parts) {
    const int64_t per = ceil_div(ceil_div(chunks, parts), 4) * 4;   // whole loader groups
    const int64_t ns = 300 * per + 2200 + ceil_div(chunks, per) * T * m * 8 / 4500;
    if (per < chunks && ns < best_ns) best = per, best_ns = ns;
  }
  return best;
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const GemmArgs);

// Most pairs of the kernel that run at once on the current device (a property
// of the device, asked for once per kernel), 0 on error.
int active_pairs(Kernel fn, int which, int smem) {
  static std::atomic<int> known[kMaxDevices][6];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int v = known[dev][which].load(std::memory_order_relaxed);
  if (v > 0) return v;
  if (allow_smem(reinterpret_cast<const void*>(fn), smem) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(2 * (sm_count() / 2)));
  if (cudaOccupancyMaxActiveClusters(&v, reinterpret_cast<const void*>(fn), &cfg) != cudaSuccess || v < 1) {
    cudaGetLastError();
    return 0;
  }
  known[dev][which].store(v, std::memory_order_relaxed);
  return v;
}

}  // namespace

cudaError_t status_fetch_fp4(int* out, cudaStream_t s) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  const int zero = 0;
  e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(s);
  *out = v;
  return e;
}

size_t fp4_gemm_workspace(int64_t T, int64_t m, int64_t n) {
  const int64_t splits = ceil_div(ceil_div(n, CK), split_chunks(T, m, n));
  return splits > 1 ? (size_t)(ceil_div(splits * T * m * 4, 256) * 256) : 0;
}

kronq_status fp4_gemm(const Fp4Gemm& g, int fmt, cudaStream_t s) {
  const int64_t tiles_m = ceil_div(g.m, GM), tiles_t = ceil_div(g.T, GN) + (g.offsets ? g.E : 0);
  if (g.n > (int64_t(1) << 24)) return fail(KRONQ_ERR_UNSUPPORTED, "fp4 product: row too long");
  if (tiles_m * tiles_t > (int64_t(1) << 30)) return fail(KRONQ_ERR_UNSUPPORTED, "fp4 product: more than 2^30 tiles");
  CUtensorMap mw, mx, mxf;
  const int64_t ldc = fp4_code_row(g.n), bytes = ceil_div(g.n, 2);
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!tma_map_2d(&mw, u8, 1, g.wc, bytes, (g.offsets ? g.E : 1) * g.m, ldc, 128, GH) ||
      !tma_map_2d(&mx, u8, 1, g.xc, bytes, g.T, ldc, 128, XROWS) ||
      (g.T > GN - NG && !tma_map_2d(&mxf, u8, 1, g.xc, bytes, g.T, ldc, 128, GH)))
    return fail(KRONQ_ERR_CUDA, "cuTensorMapEncodeTiled failed (fp4 product)");
  if (g.T <= GN - NG) mxf = mx;   // no tile of GN tokens
  GemmArgs a;
  a.xs = g.xs; a.ws = g.ws; a.xg = g.xg; a.wg = g.wg;
  a.offsets = g.offsets;
  a.E = g.offsets ? (int)g.E : 1;
  a.T = g.T; a.m = g.m;
  a.lds = fp4_scale_row(fmt, g.n);
  a.kb = (int)ceil_div(g.n, fp4_block(fmt));
  a.nchunks = (int)ceil_div(g.n, CK);
  a.tiles_m = (int)tiles_m;
  a.per_split = g.offsets ? a.nchunks : (int)split_chunks(g.T, g.m, g.n);
  a.splits = (int)ceil_div(a.nchunks, a.per_split);
  a.y = g.y; a.ldy = g.ldy;
  a.y_pairs = g.y_bf16 && aligned(g.y, 4) && g.ldy % 2 == 0;
  a.part = a.splits > 1 ? static_cast<float*>(g.workspace) : nullptr;
  static const Kernel kernels[6] = {fp4_gemm_kernel<KRONQ_MXFP4, false, false>, fp4_gemm_kernel<KRONQ_MXFP4, true, false>,
                                    fp4_gemm_kernel<KRONQ_MXFP4, false, true>, fp4_gemm_kernel<KRONQ_NVFP4, false, false>,
                                    fp4_gemm_kernel<KRONQ_NVFP4, true, false>, fp4_gemm_kernel<KRONQ_NVFP4, false, true>};
  const int which = 3 * (fmt == KRONQ_NVFP4) + (a.part ? 2 : g.y_bf16 ? 1 : 0);
  const int smem = smem_bytes(fmt), pairs = active_pairs(kernels[which], which, smem);
  if (pairs < 1) return fail(KRONQ_ERR_CUDA, "fp4 product: no pair of SMs can run the kernel");
  const int64_t most = tiles_m * tiles_t * a.splits;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(2 * (most < pairs ? most : pairs)));
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernels[which], mw, mx, mxf, a);
  count_launch();
  if (e != cudaSuccess) {
    cudaGetLastError();   // the next launch's check is not to find this one's error
    return cuda_fail(e, "fp4_gemm_kernel");
  }
  if (a.part) {
    e = fp4_launch_second(fp4_join_kernel, (unsigned)ceil_div(g.T * g.m, 256), 256, s, a, g.y_bf16);
    count_launch();
    if (e != cudaSuccess) {
      cudaGetLastError();
      return cuda_fail(e, "fp4_join_kernel");
    }
  }
  return KRONQ_OK;
}

}  // namespace kq
