// Product of int8 operands with a scale a row of each (gemm_int8_run):
//
//   C[m, n] = sa[m] sb[n] S[m, n] (+ bias[n]) (+ source[m, n]),  S[m, n] = sum over k of a[m, k] b[n, k]
//
// S is exact: 16 x 16 x 64 int8 MFMAs add to int32, K is cut where that could overflow, and pieces are added
// in 64 bits.  So every kernel here gives the same bits, whatever the shape of the rest of C, and the
// scales cost nothing before the epilogue.
#include "../../include/gemm_ops.h"
#include "ops_int8.h"

namespace dg {
namespace {

typedef i32x4 __attribute__((aligned(4))) i32x4_any;

__device__ __forceinline__ f32x4 floats(const i32x4 &v) {
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

// ---- few rows ---------------------------------------------------------------------------------

// Up to 16 FM rows of A: what counts is to read B once at the memory's rate.  A workgroup takes 16 GN
// rows of B (columns of C); its eight waves take every eighth k-block (of its piece of K) straight
// into registers, and their sums meet in LDS.
template <int FM, int GN>
__global__ void __launch_bounds__(512) few_kernel(const Int8Args a) {
  constexpr int WAVES = 8;
  constexpr int AHEAD = FM * GN > 2 ? 2 : 4;   // k-blocks of a wave whose loads are in flight together
  __shared__ int part[WAVES][FM][GN][16][17];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r16 = lane & 15, g4 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * GN);
  const auto ra = make_rsrc(a.A, a.M * a.lda);
  const int64_t rows_b = a.N - n0 < 16 * GN ? a.N - n0 : 16 * GN;
  const auto rb = make_rsrc(a.B + n0 * a.ldb, rows_b * a.ldb);
  const int split = blockIdx.y;
  const int32_t kb1 = (int32_t)((int64_t)a.kb * (split + 1) / a.splits);
  i32x4 acc[FM][GN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < GN; ++g) acc[f][g] = i32x4{0, 0, 0, 0};
  // past K an operand reads as zeros
  auto take = [&](i32x4 (&q)[2], auto r, uint32_t row, uint32_t ld, uint32_t k) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t o = k + h * 16 < (uint32_t)a.kbytes ? row * ld + k + h * 16 : kOOB;
      q[h] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
    }
  };
  for (int32_t kb0 = (int32_t)((int64_t)a.kb * split / a.splits) + wave; kb0 < kb1;
       kb0 += WAVES * AHEAD) {
    i32x4 b[AHEAD][GN][2], x[AHEAD][FM][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int32_t kb = kb0 + WAVES * u;
      // past the last k-block too
      const uint32_t k = kb < kb1 ? (uint32_t)kb * 128 + g4 * 32 : (uint32_t)a.kbytes;
#pragma unroll
      for (int g = 0; g < GN; ++g) take(b[u][g], rb, g * 16 + r16, (uint32_t)a.ldb, k);
#pragma unroll
      for (int f = 0; f < FM; ++f) take(x[u][f], ra, f * 16 + r16, (uint32_t)a.lda, k);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
          for (int g = 0; g < GN; ++g)
            acc[f][g] = mfma_int8(b[u][g][h], x[u][f][h], acc[f][g]);
  }
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < GN; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][f][g][r16][g4 * 4 + e] = acc[f][g][e];
  __syncthreads();
  for (int i = threadIdx.x; i < FM * GN * 64; i += WAVES * 64) {
    const int f = i / (64 * GN), g = i / 64 % GN, m16 = i / 4 % 16, q = i % 4;
    const int64_t m = f * 16 + m16, n = n0 + g * 16 + q * 4;
    if (m >= a.M || n >= a.N) continue;
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += part[w][f][g][m16][q * 4 + e];
    if (a.splits == 1) {
      finish_four(a, m, n, floats(v));
      continue;
    }
    int *const p = (int *)a.partials + ((int64_t)split * a.M + m) * a.N + n;
    if (n + 4 <= a.N) {
      *(i32x4_any *)p = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) p[e] = v[e];
    }
  }
}

// The sums of `splits` pieces, `pitch` apart, in 64 bits; `n` of the four are there.
__device__ __forceinline__ f32x4 joined(const int *p, int64_t pitch, int splits, int64_t n) {
  int64_t v[4] = {0, 0, 0, 0};
  for (int s = 0; s < splits; s += 8) {
    i32x4 q[8];   // loads in flight together
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      q[u] = i32x4{0, 0, 0, 0};
      if (s + u >= splits) continue;
      const int *const x = p + (s + u) * pitch;
      if (n >= 4) {
        q[u] = *(const i32x4_any *)x;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < n) q[u][e] = x[e];
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += q[u][e];
  }
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

// Adds the pieces of few rows, then the epilogue.
__global__ void __launch_bounds__(256) join_kernel(const Int8Args a) {
  const int64_t per_row = (a.N + 3) / 4, all = a.M * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per_row, n = i % per_row * 4;
    finish_four(a, m, n,
                joined((const int *)a.partials + m * a.N + n, a.M * a.N, a.splits, a.N - n));
  }
}

// ---- tiles through LDS ------------------------------------------------------------------------

// Where tile t of the order lies: strips of eight rows of tiles, walked down first.
__device__ __forceinline__ void tile_corner(const Int8Args &a, int32_t t, int bm, int bn,
                                            int64_t &m0, int64_t &n0) {
  const int32_t strip = t / (8 * a.nt), in = t % (8 * a.nt);
  const int32_t high = a.mt - strip * 8 < 8 ? a.mt - strip * 8 : 8;
  m0 = (int64_t)(strip * 8 + in % high) * bm;
  n0 = (int64_t)(in / high) * bn;
}
// The place of workgroup i of n, so that those of one XCD (i mod 8) are neighbours.
__device__ __forceinline__ int32_t place(int32_t i, int32_t n) {
  const int32_t per = n / 8, more = n % 8, x = i % 8;
  return x * per + (x < more ? x : more) + i / 8;
}

// KG groups of WGM x WGN waves own a BM x BN tile of C, each for every KG-th k-block; their sums meet
// in LDS.  Each group has a ring of S stages in LDS: the k-block that is multiplied, and S - 1 that are on
// their way (loads that write LDS directly, rows swizzled in 16-byte chunks).  One barrier a step: behind
// it every wave's loads of this step have landed, and its reads of the step before are done, whose
// stage the next loads go to.
//
// The first a.whole tiles have a workgroup each; the k-blocks of the others are cut into a.splits
// pieces, whose sums join_tiles_kernel adds.
template <int BM, int BN, int WGM, int WGN, int KG, int S>
__global__ void __launch_bounds__(KG *WGM *WGN * 64) tile_kernel(const Int8Args a) {
  constexpr int NW = WGM * WGN, WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;   // 1 KiB loads (8 rows) a wave and stage
  constexpr int STAGE = (BM + BN) * 128;
  static_assert(LA * 8 * NW == BM && LB * 8 * NW == BN, "whole loads");
  static_assert((S - 2) * (LA + LB) <= 63, "vmcnt");
  static_assert(KG * S * STAGE <= 160 * 1024, "LDS");
  __shared__ __align__(1024) char smem_[KG * S * STAGE];
  const int wave_ = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int group = wave_ / NW, wave = wave_ % NW;
  lds_t *const smem = (lds_t *)smem_ + group * S * STAGE;

  const int32_t i = blockIdx.x, cut = a.mt * a.nt - a.whole;   // tiles whose K is cut
  int32_t t, piece = -1, kb0 = 0, kb1 = a.kb;   // piece: of the partial sums
  if (i < a.whole) {
    t = place(i, a.whole);
  } else {
    const int32_t split = (i - a.whole) / cut, at = place((i - a.whole) % cut, cut);
    t = a.whole + at;
    if (a.splits > 1) {
      piece = split * cut + at;
      kb0 = (int32_t)((int64_t)a.kb * split / a.splits);
      kb1 = (int32_t)((int64_t)a.kb * (split + 1) / a.splits);
    }
  }
  int64_t m0, n0;
  tile_corner(a, t, BM, BN, m0, n0);

  // producer
  const int32_t rows_a = (int32_t)(a.M - m0 < BM ? a.M - m0 : BM);
  const int32_t rows_b = (int32_t)(a.N - n0 < BN ? a.N - n0 : BN);
  const auto ra = make_rsrc(a.A + m0 * a.lda, (int64_t)rows_a * a.lda);
  const auto rb = make_rsrc(a.B + n0 * a.ldb, (int64_t)rows_b * a.ldb);
  const uint32_t row0 = wave * 8 + lane / 8;
  const uint32_t chunk = ((lane % 8) ^ ((row0 >> 1) & 7)) * 16;
  const uint32_t voa = row0 * (uint32_t)a.lda + chunk, vob = row0 * (uint32_t)a.ldb + chunk;
  const uint32_t kend =
      (uint32_t)(kb1 * 128 < a.kbytes ? kb1 * 128 : a.kbytes);   // a piece ends inside K
  // (a step past the end loads zeros: as many loads are in flight in every step)
  auto load_stage = [&](int32_t kb, int s) {
    const uint32_t k = (uint32_t)kb * 128;
    const bool past = k + chunk >= kend;
    lds_t *const to = smem + s * STAGE + wave * 1024;
    // rows past the edge lie past the range of the buffer: their lanes read zeros
    const uint32_t oa = past ? kOOB : voa + k, ob = past ? kOOB : vob + k;
#pragma unroll
    for (int j = 0; j < LA; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to + j * NW * 1024, 16,
                                               oa + (uint32_t)(j * NW * 8) * (uint32_t)a.lda, 0, 0,
                                               0);
#pragma unroll
    for (int j = 0; j < LB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, to + BM * 128 + j * NW * 1024, 16,
                                               ob + (uint32_t)(j * NW * 8) * (uint32_t)a.ldb, 0, 0,
                                               0);
  };

  // consumer
  const int wm = wave / WGN, wn = wave % WGN, r16 = lane & 15, g4 = lane >> 4;
  const uint32_t x = (r16 >> 1) & 7;
  // a lane's two chunks of a row are g4 and g4 + 4, in A and B alike: reads of neighbours cost an
  // LDS pass more
  const uint32_t ck[2] = {(g4 ^ x) * 16, ((g4 + 4) ^ x) * 16};
  const uint32_t arow = (wm * WM + r16) * 128, brow = BM * 128 + (wn * WN + r16) * 128;
  typedef const i32x4 __attribute__((address_space(3))) *frag;

  i32x4 acc[FM][FN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < FN; ++g) acc[f][g] = i32x4{0, 0, 0, 0};
  // a wave wholly past the edge only loads
  const bool inside = m0 + wm * WM < a.M && n0 + wn * WN < a.N;

#pragma unroll
  for (int s = 0; s < S - 1; ++s) load_stage(kb0 + group + s * KG, s);
  int s = 0;
  for (int32_t kb = kb0 + group; kb < kb1 + group; kb += KG) {   // as often in every group
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * (LA + LB))
                 : "memory");
    load_stage(kb + (S - 1) * KG, s == 0 ? S - 1 : s - 1);
    const lds_t *const st = smem + s * STAGE;
    s = s == S - 1 ? 0 : s + 1;
    if (!inside || kb >= kb1) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 b[FN];
#pragma unroll
      for (int g = 0; g < FN; ++g) b[g] = *(frag)(st + brow + ck[h] + g * 2048);
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        const i32x4 af = *(frag)(st + arow + ck[h] + f * 2048);
#pragma unroll
        for (int g = 0; g < FN; ++g) acc[f][g] = mfma_int8(b[g], af, acc[f][g]);
      }
    }
  }
  // no load is on its way into LDS that the sums below, or the next workgroup, use
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // each group gives away the sums of the rows of blocks that the other one writes
  constexpr int OWN = FM / KG;
  static_assert(KG == 1 || (KG == 2 && OWN * KG == FM && NW * OWN * FN * 1024 <= S * STAGE), "");
  if constexpr (KG == 2) {
    typedef i32x4 __attribute__((address_space(3))) *i4p;
    lds_t *const area = (lds_t *)smem_ + wave * (OWN * FN * 1024) + lane * 16;
#pragma unroll
    for (int f = 0; f < OWN; ++f)
#pragma unroll
      for (int g = 0; g < FN; ++g)
        *(i4p)(area + (group ^ 1) * S * STAGE + (f * FN + g) * 1024) =
            group ? acc[f][g] : acc[f + OWN][g];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int f = 0; f < OWN; ++f)
#pragma unroll
      for (int g = 0; g < FN; ++g)
        acc[f][g] = (group ? acc[f + OWN][g] : acc[f][g]) +
                    *(i4p)(area + group * S * STAGE + (f * FN + g) * 1024);
  }
  const int ml0 = wm * WM + group * OWN * 16 + r16, nl0 = wn * WN + g4 * 4;
  if (piece >= 0 || a.N < 4) {
#pragma unroll
    for (int f = 0; f < OWN; ++f) {
      const int ml = ml0 + f * 16;
      if (m0 + ml >= a.M) continue;
#pragma unroll
      for (int g = 0; g < FN; ++g) {
        const int nl = nl0 + g * 16;
        if (n0 + nl >= a.N) continue;
        if (piece >= 0)
          *(i32x4 *)((int *)a.partials + (int64_t)piece * (BM * BN) + ml * BN + nl) = acc[f][g];
        else
          finish_four(a, m0 + ml, n0 + nl, floats(acc[f][g]));
      }
    }
    return;
  }
  f32x4 bias[FN], sb[FN];
#pragma unroll
  for (int g = 0; g < FN; ++g) {
    bias[g] = bias_four(a, n0 + nl0 + g * 16);
    sb[g] = vector_four(a, a.sb, n0 + nl0 + g * 16);
  }
  float sa[OWN];
#pragma unroll
  for (int f = 0; f < OWN; ++f) {
    const int64_t m = m0 + ml0 + f * 16;
    sa[f] = a.sa[m < a.M ? m : a.M - 1];
  }
  with_source(a, [&](auto src_c) {
    constexpr int SRC = decltype(src_c)::value, STEP = OWN < 2 ? 1 : 2;
#pragma unroll
    for (int f0 = 0; f0 < OWN; f0 += STEP) {
      u32x4 src[STEP][FN];
      if constexpr (SRC != SRC_NONE) {
#pragma unroll
        for (int f = 0; f < STEP; ++f)
#pragma unroll
          for (int g = 0; g < FN; ++g)
            src[f][g] = source_at<SRC>(a, m0 + ml0 + (f0 + f) * 16, n0 + nl0 + g * 16);
      }
#pragma unroll
      for (int f = 0; f < STEP; ++f)
#pragma unroll
        for (int g = 0; g < FN; ++g) {
          const int64_t m = m0 + ml0 + (f0 + f) * 16, n = n0 + nl0 + g * 16;
          if (m >= a.M || n >= a.N) continue;
          f32x4 v = floats(acc[f0 + f][g]);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = scaled(v[e], sa[f0 + f], sb[g][e], bias[g][e]);
          if constexpr (SRC != SRC_NONE) v += source_four<SRC>(a, n, src[f][g]);
          put_four(a, m, n, v);
        }
    }
  });
}

// Adds the pieces of the tiles whose K is cut, then the epilogue.  1024 elements of a tile a workgroup.
template <int BM, int BN>
__global__ void __launch_bounds__(256) join_tiles_kernel(const Int8Args a) {
  constexpr int QUADS = BN / 4, GROUPS = BM * BN / 1024;
  const int32_t cut = a.mt * a.nt - a.whole, at = blockIdx.x / GROUPS;
  const int i = blockIdx.x % GROUPS * 256 + threadIdx.x;
  const int ml = i / QUADS, nl = i % QUADS * 4;
  int64_t m0, n0;
  tile_corner(a, a.whole + at, BM, BN, m0, n0);
  const int64_t m = m0 + ml, n = n0 + nl;
  if (m >= a.M || n >= a.N) return;
  finish_four(a, m, n,
              joined((const int *)a.partials + (int64_t)at * (BM * BN) + ml * BN + nl,
                     (int64_t)cut * (BM * BN), a.splits, 4));
}

// ---- choice -----------------------------------------------------------------------------------

constexpr int kCUs = 256;

enum { PLAN_FEW, PLAN_128 };
struct Int8Plan {
  int kind, splits;
  int32_t bm, bn, mt, nt, whole;   // whole: the tiles whose K is not cut
};

Int8Plan plan_of(const gemm_int8_desc &d) {
  const int64_t kb = (d.K + 127) / 128;
  const int64_t least = kb > kMostBlocks ? (kb + kMostBlocks - 1) / kMostBlocks : 1;   // of pieces
  if (d.M <= 64) {
    const int cols = 16;
    const int64_t nt = (d.N + cols - 1) / cols;
    int64_t splits = nt < 128 ? 256 / nt : 1;
    if (splits > kb / 16) splits = kb / 16;
    if (splits < least) splits = least;
    return {PLAN_FEW, splits > 1 ? (int)splits : 1, 0, 0, 1, (int32_t)nt, 0};
  }
  const int64_t mt = (d.M + 127) / 128, nt = (d.N + 127) / 128, t = mt * nt;
  int64_t splits = least;
  if (t < kCUs / 2 && kb >= 16) splits = kCUs / t;
  if (splits > kb / 8) splits = kb / 8;
  if (splits < least) splits = least;
  return {PLAN_128, (int)splits, 128, 128, (int32_t)mt, (int32_t)nt,
          (int32_t)(splits > 1 ? 0 : t)};
}

template <int FM, int GN>
void launch_few(const Int8Args &a, hipStream_t s) {
  const dim3 grid((uint32_t)a.nt, (uint32_t)a.splits);
  hipLaunchKernelGGL((few_kernel<FM, GN>), grid, dim3(512), 0, s, a);
}
template <int BM, int BN, int WGM, int WGN, int KG, int S>
void launch_tiles(const Int8Args &a, hipStream_t s) {
  const dim3 grid((uint32_t)(a.whole + (a.mt * a.nt - a.whole) * a.splits));
  hipLaunchKernelGGL((tile_kernel<BM, BN, WGM, WGN, KG, S>), grid, dim3(KG * WGM * WGN * 64), 0, s,
                     a);
  if (a.splits > 1)
    hipLaunchKernelGGL((join_tiles_kernel<BM, BN>),
                       dim3((uint32_t)((a.mt * a.nt - a.whole) * (BM * BN / 1024))), dim3(256), 0,
                       s, a);
}

int check(const gemm_int8_desc *d) {
  if (!d || d->M < 0 || d->N < 0 || d->K < 0) return GEMM_ERR_INVALID_ARG;
  if ((d->dtype_c != GEMM_BF16 && d->dtype_c != GEMM_F32) ||
      (d->dtype_source != GEMM_BF16 && d->dtype_source != GEMM_F32))
    return GEMM_ERR_INVALID_ARG;
  if (d->lda < d->K || d->ldb < d->K || d->lda % 16 || d->ldb % 16) return GEMM_ERR_INVALID_ARG;
  // offsets inside a tile of 256 rows (of A, B or C) stay under 31 bits, work-items under 2^32
  if (d->lda > (1 << 22) || d->ldb > (1 << 22)) return GEMM_ERR_UNSUPPORTED;
  if (d->M > (1ll << 31) || d->N > (1ll << 22)) return GEMM_ERR_UNSUPPORTED;
  if (((d->M + 127) / 128) * ((d->N + 127) / 128) > (1ll << 22)) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

size_t workspace_of(const gemm_int8_desc &d, const Int8Plan &p) {
  if (p.splits <= 1) return 0;
  return (size_t)p.splits * sizeof(int) *
         (p.kind == PLAN_FEW ? (size_t)d.M * (size_t)d.N
                             : (size_t)(p.mt * p.nt - p.whole) * (size_t)(p.bm * p.bn));
}

}  // namespace
}  // namespace dg

extern "C" int gemm_int8_workspace(const gemm_int8_desc *d, size_t *bytes) {
  const int st = dg::check(d);
  if (st != GEMM_OK) return st;
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  *bytes = 0;
  if (d->M == 0 || d->N == 0) return GEMM_OK;
  *bytes = dg::workspace_of(*d, dg::plan_of(*d));
  return GEMM_OK;
}

extern "C" int gemm_int8_run(const gemm_int8_desc *d, const void *A, const float *scale_a,
                             const void *B, const float *scale_b, void *C, const float *bias,
                             const void *source, void *workspace, size_t workspace_bytes,
                             void *stream) {
  using namespace dg;
  const int st = check(d);
  if (st != GEMM_OK) return st;
  if (d->M == 0 || d->N == 0) return GEMM_OK;
  if (!C || !scale_a || !scale_b || (d->K > 0 && (!A || !B))) return GEMM_ERR_INVALID_ARG;
  const uintptr_t out = d->dtype_c == GEMM_BF16 ? 1 : 3, in = d->dtype_source == GEMM_BF16 ? 1 : 3;
  if (((uintptr_t)A & 15) || ((uintptr_t)B & 15) || ((uintptr_t)scale_a & 3) ||
      ((uintptr_t)scale_b & 3) || ((uintptr_t)bias & 3) || ((uintptr_t)C & out) ||
      ((uintptr_t)source & in) || ((uintptr_t)workspace & 15))
    return GEMM_ERR_ALIGNMENT;
  // an element of the source is read before that of C is written, by the same lane; any other overlap would
  // be read by one workgroup and written by another
  const uintptr_t c0 = (uintptr_t)C, c1 = c0 + (uintptr_t)(d->M * d->N) * (out + 1);
  const auto apart = [&](const void *p, int64_t n, uintptr_t es) {
    const uintptr_t p0 = (uintptr_t)p;
    return !p || p0 >= c1 || p0 + (uintptr_t)n * es <= c0;
  };
  if (!(source == C && d->dtype_source == d->dtype_c) && !apart(source, d->M * d->N, in + 1))
    return GEMM_ERR_INVALID_ARG;
  if (!apart(bias, d->N, 4) || !apart(scale_a, d->M, 4) || !apart(scale_b, d->N, 4) ||
      !apart(A, (d->M - 1) * d->lda + d->K, 1) || !apart(B, (d->N - 1) * d->ldb + d->K, 1))
    return GEMM_ERR_INVALID_ARG;
  const Int8Plan p = plan_of(*d);
  const size_t need = workspace_of(*d, p);
  if (need && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
  Int8Args a{};
  a.A = (const char *)A;
  a.B = (const char *)B;
  a.sa = scale_a;
  a.sb = scale_b;
  a.C = (char *)C;
  a.bias = bias;
  a.source = (const char *)source;
  a.partials = (float *)workspace;
  a.M = d->M;
  a.N = d->N;
  a.lda = d->lda;
  a.ldb = d->ldb;
  a.kbytes = (int32_t)((d->K + 15) / 16 * 16);
  a.kb = (int32_t)((d->K + 127) / 128);
  a.mt = p.mt;
  a.nt = p.nt;
  a.splits = p.splits;
  a.whole = p.whole;
  a.out_bf16 = d->dtype_c == GEMM_BF16;
  a.src_bf16 = d->dtype_source == GEMM_BF16;
  a.plain_rows = !source && (d->N * (a.out_bf16 ? 2 : 4)) % 16 == 0 && !((uintptr_t)C & 15);
  hipStream_t s = (hipStream_t)stream;
  if (p.kind == PLAN_FEW) {
    if (d->M <= 16)
      launch_few<1, 1>(a, s);
    else if (d->M <= 32)
      launch_few<2, 1>(a, s);
    else
      launch_few<4, 1>(a, s);
    if (p.splits > 1) {
      const int64_t need_wg = (d->M * ((d->N + 3) / 4) + 255) / 256;
      hipLaunchKernelGGL(join_kernel, dim3((uint32_t)(need_wg < 8 * kCUs ? need_wg : 8 * kCUs)),
                         dim3(256), 0, s, a);
    }
  } else {
    launch_tiles<128, 128, 2, 2, 2, 2>(a, s);
  }
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}
