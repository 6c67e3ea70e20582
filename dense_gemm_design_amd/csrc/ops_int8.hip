// Product of int8 operands with a scale a row of each (gemm_int8_run):
//
//   C[m, n] = sa[m] sb[n] S[m, n] (+ bias[n]) (+ source[m, n]),  S[m, n] = sum over k of a[m, k] b[n, k]
//
// S is exact: 16 x 16 x 64 int8 MFMAs add to int32, K is cut where that could overflow, and pieces are added
// in 64 bits.  So every kernel here gives the same bits, whatever the shape of the rest of C, and the
// scales cost nothing before the epilogue.
#include "../../include/gemm_ops.h"
#include "int8_plan.h"
#include "ops_int8.h"

namespace dg {
namespace {

typedef i32x4 __attribute__((aligned(4))) i32x4_any;

__device__ __forceinline__ f32x4 floats(const i32x4 &v) {
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

// ---- few rows ---------------------------------------------------------------------------------

// Up to 16 FM rows of A: what counts is to read B once at the memory's rate.  A workgroup takes 16 rows
// of B (columns of C); its eight waves take every eighth k-block (of its piece of K) straight into
// registers, and their sums meet in LDS.  1 x 4096 x 4096 takes 5.5 us (5.9 with the scales loaded
// last, 7.4 with 32 columns a workgroup), 1 x 16384 x 16384 54 us, 5.0 TB/s.
template <int FM>
__global__ void __launch_bounds__(512) few_kernel(const Int8Args a) {
  constexpr int WAVES = 8, AHEAD = 4;   // AHEAD: k-blocks of a wave whose loads are in flight together
  __shared__ int part[WAVES][FM][16][17];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r16 = lane & 15, g4 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const auto ra = make_rsrc(a.A, a.M * a.lda);
  const int64_t rows_b = a.N - n0 < 16 ? a.N - n0 : 16;
  const auto rb = make_rsrc(a.B + n0 * a.ldb, rows_b * a.ldb);
  const int split = blockIdx.y;
  const int32_t kb1 = (int32_t)((int64_t)a.kb * (split + 1) / a.splits);
  // the four columns of one row that a lane finishes; what they take besides the sums is loaded first
  const int64_t m = threadIdx.x / 64 * 16 + lane / 4, n = n0 + lane % 4 * 4;
  const bool mine = threadIdx.x < FM * 64 && m < a.M && n < a.N;
  Extras extras;
  if (mine && a.splits == 1) extras = extras_of(a, m, n);
  i32x4 acc[FM];
#pragma unroll
  for (int f = 0; f < FM; ++f) acc[f] = i32x4{0, 0, 0, 0};
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
    i32x4 b[AHEAD][2], x[AHEAD][FM][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int32_t kb = kb0 + WAVES * u;
      // past the last k-block too
      const uint32_t k = kb < kb1 ? (uint32_t)kb * 128 + g4 * 32 : (uint32_t)a.kbytes;
      take(b[u], rb, r16, (uint32_t)a.ldb, k);
#pragma unroll
      for (int f = 0; f < FM; ++f) take(x[u][f], ra, f * 16 + r16, (uint32_t)a.lda, k);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < FM; ++f) acc[f] = mfma_int8(b[u][h], x[u][f][h], acc[f]);
  }
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][f][r16][g4 * 4 + e] = acc[f][e];
  __syncthreads();
  if (!mine) return;
  const int f = threadIdx.x / 64, m16 = lane / 4, q = lane % 4;
  i32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < WAVES; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += part[w][f][m16][q * 4 + e];
  if (a.splits == 1) {
    finish_four(a, m, n, floats(v), extras);
    return;
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

// ---- pieces of K ------------------------------------------------------------------------------

// Adds the `splits` pieces of four sums, `pitch` apart, in 64 bits; `n` of the four are there, none where it is
// not positive.  PARTS lanes of the workgroup, 256 apart, take every PARTS-th piece each; the first has the
// result.  One trip to other XCDs' results for eight pieces takes 2 to 3 us: 40 x 320 x 32896, 24 pieces, in one
// part 16.0 us, in four 13.0.
template <int PARTS>
__device__ __forceinline__ f32x4 joined(const int *p, int64_t pitch, int splits, int64_t n) {
  const int part = PARTS > 1 ? threadIdx.x >> 8 : 0;
  int64_t v[4] = {0, 0, 0, 0};
  for (int s = part; s < splits; s += 8 * PARTS) {
    i32x4 q[8];   // loads in flight together
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      q[u] = i32x4{0, 0, 0, 0};
      if (s + u * PARTS >= splits) continue;
      const int *const x = p + (s + u * PARTS) * pitch;
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
  if constexpr (PARTS > 1) {
    __shared__ int64_t more[PARTS - 1][4][256];
    const int at = threadIdx.x & 255;
    __syncthreads();   // those of the round before are read
    if (part > 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) more[part - 1][e][at] = v[e];
    }
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int k = 0; k < PARTS - 1; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += more[k][e][at];
    }
  }
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
constexpr int kPartsFrom = 9;   // pieces from which on four parts add them

// Adds the pieces of few rows, then the epilogue.
template <int PARTS>
__global__ void __launch_bounds__(256 * PARTS) join_kernel(const Int8Args a) {
  const int64_t per_row = (a.N + 3) / 4, all = a.M * per_row;
  for (int64_t i0 = (int64_t)blockIdx.x * 256; i0 < all; i0 += (int64_t)gridDim.x * 256) {
    const int64_t i = i0 + (threadIdx.x & 255);
    const bool there = i < all;
    const int64_t m = there ? i / per_row : 0, n = there ? i % per_row * 4 : 0;
    const Extras x = extras_of(a, m, n);
    const f32x4 sum = joined<PARTS>((const int *)a.partials + m * a.N + n, a.M * a.N, a.splits,
                                    there ? a.N - n : 0);
    if (there && threadIdx.x < 256) finish_four(a, m, n, sum, x);
  }
}

// ---- tiles through LDS ------------------------------------------------------------------------

// Where tile t of the order lies: strips of eight rows of tiles, walked down first.
__device__ __forceinline__ void tile_corner(const Int8Args &a, int32_t t, int bm, int bn,
                                            int64_t &m0, int64_t &n0) {
  const int32_t strip = t / (8 * a.nt), in = t % (8 * a.nt);
  const int32_t high = a.mt - strip * 8 < 8 ? a.mt - strip * 8 : 8;
  m0 = (int64_t)(strip * 8 + in % high) * bm;
  n0 = a.n_first + (int64_t)(in / high) * bn;
}
// The place of workgroup i of n, so that those of one XCD (i mod 8) are neighbours.
__device__ __forceinline__ int32_t place(int32_t i, int32_t n) {
  const int32_t per = n / 8, more = n % 8, x = i % 8;
  return x * per + (x < more ? x : more) + i / 8;
}

// Scales and bias of a lane's FM x FN quads, quad (f, g) at row m + 16 f and column n + 16 g.
template <int FM, int FN>
struct Scales {
  f32x4 bias[FN], sb[FN];
  float sa[FM];
  __device__ __forceinline__ void load(const Int8Args &a, int64_t m, int64_t n) {
    if (a.N < 4) return;
#pragma unroll
    for (int g = 0; g < FN; ++g) {
      bias[g] = bias_four(a, n + g * 16);
      sb[g] = vector_four(a, a.sb, n + g * 16);
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = a.sa[m + f * 16 < a.M ? m + f * 16 : a.M - 1];
  }
};

// Writes a lane's quads of sums, at row ml0 + 16 f and column nl0 + 16 g of the tile at (m0, n0): as they are
// to its piece of the partial sums, or finished to C.
template <int BM, int BN, int FM, int FN, class Get>
__device__ __forceinline__ void write_blocks(const Int8Args &a, int32_t piece, int64_t m0, int64_t n0,
                                             int ml0, int nl0, const Scales<FM, FN> &x, Get get) {
  if (piece >= 0 || a.N < 4) {
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      const int ml = ml0 + f * 16;
#pragma unroll
      for (int g = 0; g < FN; ++g) {
        const int nl = nl0 + g * 16;
        const i32x4 v = get(f, g);
        if (m0 + ml >= a.M || n0 + nl >= a.N) continue;
        if (piece >= 0)
          *(i32x4 *)((int *)a.partials + (int64_t)piece * (BM * BN) + ml * BN + nl) = v;
        else
          finish_four(a, m0 + ml, n0 + nl, floats(v));
      }
    }
    return;
  }
  with_source(a, [&](auto src_c) {
    constexpr int SRC = decltype(src_c)::value, STEP = FM < 2 ? 1 : 2;
#pragma unroll
    for (int f0 = 0; f0 < FM; f0 += STEP) {
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
          f32x4 v = floats(get(f0 + f, g));
          if (m >= a.M || n >= a.N) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = scaled(v[e], x.sa[f0 + f], x.sb[g][e], x.bias[g][e]);
          if constexpr (SRC != SRC_NONE) v += source_four<SRC>(a, n, src[f][g]);
          put_four(a, m, n, v);
        }
    }
  });
}

// KG groups of WGM x WGN waves own a BM x BN tile of C, each for every KG-th k-block; their sums meet
// in LDS.  A ring of S stages in LDS holds the KG k-blocks that are multiplied, and S - KG that are on their
// way (loads that write LDS directly, by all waves, rows swizzled in 16-byte chunks).  One barrier a step:
// behind it every wave's loads of this step's blocks have landed, and its reads of the step before are done,
// whose stages the next loads go to.
//
// The first a.whole tiles have a workgroup each; the k-blocks of the others are cut into a.splits
// pieces, whose sums join_tiles_kernel adds.  Bound by the way to the caches: 64 x 14336 x 4096 takes 12.8 us,
// 4.7 TB/s, 256 x 4096 x 4096 11.5, 32 bytes a clock and CU.
template <int BM, int BN, int WGM, int WGN, int KG, int S>
__global__ void __launch_bounds__(KG *WGM *WGN * 64) tile_kernel(const Int8Args a) {
  constexpr int NW = WGM * WGN, WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  constexpr int ALL = KG * NW;                           // waves
  constexpr int LA = BM / 8 / ALL, LB = BN / 8 / ALL;    // 1 KiB loads (8 rows) a wave and stage
  constexpr int STAGE = (BM + BN) * 128, AHEAD = S - KG;
  static_assert(LA * 8 * ALL == BM && LB * 8 * ALL == BN, "whole loads");
  static_assert(AHEAD >= KG && (AHEAD - KG) * (LA + LB) <= 63, "vmcnt");
  static_assert(S * STAGE <= 160 * 1024, "LDS");
  __shared__ __align__(1024) char smem_[S * STAGE];
  lds_t *const smem = (lds_t *)smem_;
  const int wave_ = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int group = wave_ / NW, wave = wave_ % NW;

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
  const uint32_t row0 = wave_ * 8 + lane / 8;
  const uint32_t chunk = ((lane % 8) ^ ((row0 >> 1) & 7)) * 16;
  const uint32_t voa = row0 * (uint32_t)a.lda + chunk, vob = row0 * (uint32_t)a.ldb + chunk;
  const uint32_t kend =
      (uint32_t)(kb1 * 128 < a.kbytes ? kb1 * 128 : a.kbytes);   // a piece ends inside K
  uint32_t kload = (uint32_t)kb0 * 128;   // of the next block to load
  int sload = 0;                          // and its stage
  // (a block past the end loads zeros: as many loads are in flight in every step)
  auto load_next = [&] {
    const bool past = kload + chunk >= kend;
    lds_t *const to = smem + sload * STAGE + wave_ * 1024;
    // rows past the edge lie past the range of the buffer: their lanes read zeros
    const uint32_t oa = past ? kOOB : voa + kload, ob = past ? kOOB : vob + kload;
#pragma unroll
    for (int j = 0; j < LA; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to + j * ALL * 1024, 16,
                                               oa + (uint32_t)(j * ALL * 8) * (uint32_t)a.lda, 0, 0,
                                               0);
#pragma unroll
    for (int j = 0; j < LB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, to + BM * 128 + j * ALL * 1024, 16,
                                               ob + (uint32_t)(j * ALL * 8) * (uint32_t)a.ldb, 0, 0,
                                               0);
    kload += 128;
    sload = sload == S - 1 ? 0 : sload + 1;
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

  // what the end takes besides the sums, ahead of everything: 188 x 108 x 1316 5.5 us, 5.8 with it
  // at the end; 64 x 14336 x 4096 12.8, 13.2
  constexpr int OWN = FM / KG;
  const int ml0 = wm * WM + group * OWN * 16 + r16, nl0 = wn * WN + g4 * 4;
  Scales<OWN, FN> scales;
  if (piece < 0) scales.load(a, m0 + ml0, n0 + nl0);

#pragma unroll
  for (int j = 0; j < AHEAD; ++j) load_next();
  int s = group;
  for (int32_t kb = kb0 + group; kb < kb1 + group; kb += KG) {   // as often in every group
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((AHEAD - KG) * (LA + LB))
                 : "memory");
#pragma unroll
    for (int j = 0; j < KG; ++j) load_next();
    const lds_t *const st = smem + s * STAGE;
    s = s + KG >= S ? s + KG - S : s + KG;
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
  constexpr int HALF = NW * OWN * FN * 1024;
  static_assert(KG == 1 || (KG == 2 && OWN * KG == FM && 2 * HALF <= S * STAGE), "");
  if constexpr (KG == 2) {
    typedef i32x4 __attribute__((address_space(3))) *i4p;
    lds_t *const area = smem + wave * (OWN * FN * 1024) + lane * 16;
#pragma unroll
    for (int f = 0; f < OWN; ++f)
#pragma unroll
      for (int g = 0; g < FN; ++g)
        *(i4p)(area + (group ^ 1) * HALF + (f * FN + g) * 1024) =
            group ? acc[f][g] : acc[f + OWN][g];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int f = 0; f < OWN; ++f)
#pragma unroll
      for (int g = 0; g < FN; ++g)
        acc[f][g] = (group ? acc[f + OWN][g] : acc[f][g]) +
                    *(i4p)(area + group * HALF + (f * FN + g) * 1024);
  }
  write_blocks<BM, BN, OWN, FN>(a, piece, m0, n0, ml0, nl0, scales,
                                [&](int f, int g) { return acc[f][g]; });
}

// Tiles of BM x BN, four waves of half of their rows and columns, each alone on its SIMD, the instruction
// stream laid out by hand as in the wide kernel (ops_int8_wide.hip): in each slot behind a block's two MFMAs
// goes a share of what the next steps need.  A ring of S stages in LDS: behind the handshake of step c the
// next step's loads have landed and this step's fragments are all read, so that step c + S may be loaded to
// their stage.  A workgroup stays for one item (a tile, or a piece of one's K)
// after the other, and the loads run ahead into the next.
struct Item {
  int64_t m0, n0;
  int32_t kb0, kb1, piece;
};
// Item `round` of worker b; false if there is none.
__device__ __forceinline__ bool item_at(const Int8Args &a, int32_t b, int32_t round, int bm, int bn,
                                        Item &w) {
  const int32_t cut = a.mt * a.nt - a.whole, all = a.whole + cut * a.splits, first = round * kCUs;
  if (first + b >= all) return false;
  const int32_t i = first + place(b, all - first < kCUs ? all - first : kCUs);
  int32_t t = i;
  w.piece = -1;
  w.kb0 = 0;
  w.kb1 = a.kb;
  if (i >= a.whole) {
    const int32_t split = (i - a.whole) / cut, at = (i - a.whole) % cut;
    t = a.whole + at;
    w.piece = a.splits > 1 ? split * cut + at : -1;
    w.kb0 = (int32_t)((int64_t)a.kb * split / a.splits);
    w.kb1 = (int32_t)((int64_t)a.kb * (split + 1) / a.splits);
  }
  tile_corner(a, t, bm, bn, w.m0, w.n0);
  return true;
}

// SHIFTED: rows that do not start at multiples of 128 bytes.  A k-block's 128 bytes of such a row lie in two of
// memory's lines, and loading both for every block took 1000 x 4104 x 8201 from 40 to 52 us.  So a stage holds
// a line of each row instead, chunk c of a k-block at the place that it has anyway, and a lane reads it from
// this stage or, where its row starts `off` chunks behind a line and c + off > 7, from the next.  All rows of
// a lane start alike: they are 16 apart.  An item has a line more than k-blocks, so a step goes by
// behind it without a product.
template <int BM, int BN, int S, bool SHIFTED>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
pipe_kernel(const Int8Args a) {
  constexpr int NW = 4, WM = BM / 2, WN = BN / 2, FM = WM / 16, FN = WN / 16, NM = FM * FN;
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW, L = LA + LB;
  constexpr int STAGE = (BM + BN) * 128;
  constexpr int MORE = SHIFTED ? 1 : 0;   // stages that a step reads besides its own
  static_assert(S * STAGE <= 160 * 1024 && (S - 2) * L <= 63, "");
  __shared__ __align__(1024) char smem_[S * STAGE];
  lds_t *const smem = (lds_t *)smem_;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / 2, wn = wave % 2, r16 = lane & 15, g4 = lane >> 4;

  // ---- producer: the k-block to load next, its stage, and where its item lies
  int32_t pround = 0, pk = 0, pend = 0;
  int pstage = 0;
  __amdgpu_buffer_rsrc_t ra = uniform_rsrc(a.A, 0), rb = ra;
  const uint32_t row0 = wave * 8 + lane / 8;
  const uint32_t spot = (lane % 8) ^ ((row0 >> 1) & 7);   // a chunk of the k-block
  // where the line's chunk that goes there lies, from the line's k-block on: one before it where a row starts
  // behind it, which is no chunk of the row, or the one of the block before
  const auto chunk_at = [&](const char *base, int64_t ld) {
    const uint32_t off = SHIFTED ? (uint32_t)((uintptr_t)base + row0 * ld) >> 4 & 7 : 0;
    return (int32_t)((spot + off) % 8 - off) * 16;
  };
  const int32_t chunk_a = chunk_at(a.A, a.lda), chunk_b = chunk_at(a.B, a.ldb);
  const uint32_t stepa = NW * 8 * (uint32_t)a.lda, stepb = NW * 8 * (uint32_t)a.ldb;
  const uint32_t oa = row0 * (uint32_t)a.lda + chunk_a, ob = row0 * (uint32_t)a.ldb + chunk_b;
  auto producer_item = [&] {
    Item w;
    if (item_at(a, blockIdx.x, pround, BM, BN, w)) {
      const int32_t rows_a = (int32_t)(a.M - w.m0 < BM ? a.M - w.m0 : BM);
      const int32_t rows_b = (int32_t)(a.N - w.n0 < BN ? a.N - w.n0 : BN);
      pk = w.kb0;
      pend = w.kb1 + MORE;
      ra = uniform_rsrc(a.A + w.m0 * a.lda, rows_a * a.lda);
      rb = uniform_rsrc(a.B + w.n0 * a.ldb, rows_b * a.ldb);
    } else {   // empty ranges read as zeros
      pk = 0;
      pend = 1 << 30;
      ra = uniform_rsrc(a.A, 0);
      rb = ra;   // (in the order of the other branch, or both are kept in memory)
    }
  };
  uint32_t la, lb;
  lds_t *to;
  auto begin = [&] {
    const uint32_t k = (uint32_t)pk * 128;
    la = (int32_t)k + chunk_a >= a.kbytes ? kOOB : oa + k;
    lb = (int32_t)k + chunk_b >= a.kbytes ? kOOB : ob + k;
    to = smem + pstage * STAGE + wave * 1024;
  };
  // load J of the k-block: eight rows of A or of B.  A row past the tile's edge lies past its
  // buffer's range and reads as zeros.
  auto load = [&](auto j_c) {
    constexpr int J = decltype(j_c)::value;
    if constexpr (J < LA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to + J * NW * 1024, 16, la + J * stepa, 0, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, to + BM * 128 + (J - LA) * NW * 1024, 16,
                                               lb + (J - LA) * stepb, 0, 0, 0);
  };
  auto end = [&] {
    pstage = pstage == S - 1 ? 0 : pstage + 1;
    if (++pk == pend) {
      ++pround;
      producer_item();
    }
  };

  // ---- consumer
  const uint32_t x = (r16 >> 1) & 7;
  const uint32_t ck[2] = {(g4 ^ x) * 16, ((g4 + 4) ^ x) * 16};
  const uint32_t arow = (wm * WM + r16) * 128, brow = BM * 128 + (wn * WN + r16) * 128;
  typedef const i32x4 __attribute__((address_space(3))) *frag;
  // the rows of a lane in A and B whose chunk of a half is in the next stage
  const auto is_next = [&](const char *base, int64_t ld, int h) {
    return SHIFTED && g4 + 4 * h + ((uint32_t)((uintptr_t)base + r16 * ld) >> 4 & 7) > 7;
  };
  const bool next_a[2] = {is_next(a.A, a.lda, 0), is_next(a.A, a.lda, 1)};
  const bool next_b[2] = {is_next(a.B, a.ldb, 0), is_next(a.B, a.ldb, 1)};
  i32x4 fa[2][FM], fb[2][FN], acc[FM][FN];
  const lds_t *at_a[2], *at_b[2];   // of the lane's first row, in each half
  auto stage_of = [&](auto half_c, int stage, int after) {
    constexpr int H = decltype(half_c)::value;
    const lds_t *const st = smem + stage * STAGE, *const more = smem + after * STAGE;
    at_a[H] = (SHIFTED && next_a[H] ? more : st) + arow + ck[H];
    at_b[H] = (SHIFTED && next_b[H] ? more : st) + brow + ck[H];
  };
  // fragment E of a half: B's first
  auto read = [&](auto half_c, auto e_c) {
    constexpr int H = decltype(half_c)::value, E = decltype(e_c)::value;
    if constexpr (E < FN)
      fb[H][E] = *(frag)(at_b[H] + E * 2048);
    else
      fa[H][E - FN] = *(frag)(at_a[H] + (E - FN) * 2048);
  };
  const auto after = [](int stage) { return stage == S - 1 ? 0 : stage + 1; };
  using FIRST_HALF = std::integral_constant<int, 0>;
  using OTHER_HALF = std::integral_constant<int, 1>;
  producer_item();
#pragma unroll
  for (int s = 0; s < S; ++s) {
    begin();
    [&]<int... J>(std::integer_sequence<int, J...>) {
      (load(std::integral_constant<int, J>()), ...);
    }(std::make_integer_sequence<int, L>());
    end();
  }
  constexpr int LEFT = (S - 1 - MORE) * L < 63 ? (S - 1 - MORE) * L : 63;
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(LEFT) : "memory");
  int stage = 0;   // of the step
  auto read_first_half = [&] {
    stage_of(FIRST_HALF(), stage, after(stage));
    [&]<int... E>(std::integer_sequence<int, E...>) {
      (read(FIRST_HALF(), std::integral_constant<int, E>()), ...);
    }(std::make_integer_sequence<int, FM + FN>());
  };
  read_first_half();

  auto handshake = [&] {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2 - MORE) * L) : "memory");
    begin();
  };
  auto kstep = [&](auto first_c) {
    const int next = after(stage);
    stage_of(OTHER_HALF(), stage, next);
    stage_of(FIRST_HALF(), next, after(next));
    stage = next;
    // what was moved or made ready between steps is two wait states old before an MFMA reads it
    asm volatile("s_nop 1" ::: "memory");
    int8_step<FM, FN, L>(
        [&](auto half_c, auto f_c, auto g_c) {
          constexpr int H = decltype(half_c)::value, f = decltype(f_c)::value, g = decltype(g_c)::value;
          if constexpr (decltype(first_c)::value && H == 0)
            mfma_int8_zero(acc[f][g], fb[H][g], fa[H][f]);
          else
            mfma_int8_inplace(acc[f][g], fb[H][g], fa[H][f]);
        },
        read, handshake, load);
    end();
  };
  Item w;
  for (int32_t round = 0; item_at(a, blockIdx.x, round, BM, BN, w); ++round) {
    kstep(std::true_type());
    for (int32_t kb = w.kb0 + 1; kb < w.kb1; ++kb) kstep(std::false_type());
    mfma_wait_states();
    if constexpr (SHIFTED) {
      handshake();
      [&]<int... J>(std::integer_sequence<int, J...>) {
        (load(std::integral_constant<int, J>()), ...);
      }(std::make_integer_sequence<int, L>());
      end();
      stage = after(stage);
      read_first_half();
    }
    Scales<FM, FN> scales;
    if (w.piece < 0) scales.load(a, w.m0 + wm * WM + r16, w.n0 + wn * WN + g4 * 4);
    write_blocks<BM, BN, FM, FN>(a, w.piece, w.m0, w.n0, wm * WM + r16, wn * WN + g4 * 4, scales,
                                 [&](int f, int g) {
                                   return i32x4{acc_read(acc[f][g][0]), acc_read(acc[f][g][1]),
                                                acc_read(acc[f][g][2]), acc_read(acc[f][g][3])};
                                 });
  }
  wait_vmcnt<0>();   // no load is on its way into LDS that the workgroup no longer has
}

// Adds the pieces of the tiles whose K is cut, then the epilogue.  1024 elements of a tile a workgroup.
template <int PARTS>
__global__ void __launch_bounds__(256 * PARTS) join_tiles_kernel(const Int8Args a) {
  const int32_t size = a.bm * a.bn, quads = a.bn / 4, groups = size / 1024;
  const int32_t cut = a.mt * a.nt - a.whole, at = blockIdx.x / groups;
  const int32_t i = blockIdx.x % groups * 256 + (threadIdx.x & 255);
  const int32_t ml = i / quads, nl = i % quads * 4;
  int64_t m0, n0;
  tile_corner(a, a.whole + at, a.bm, a.bn, m0, n0);
  const bool there = m0 + ml < a.M && n0 + nl < a.N;
  const int64_t m = there ? m0 + ml : 0, n = there ? n0 + nl : 0;
  const Extras x = extras_of(a, m, n);
  const f32x4 sum = joined<PARTS>((const int *)a.partials + (int64_t)at * size + ml * a.bn + nl,
                                  (int64_t)cut * size, a.splits, there ? 4 : 0);
  if (there && threadIdx.x < 256) finish_four(a, m, n, sum, x);
}

// ---- choice -----------------------------------------------------------------------------------

template <int BM, int BN, int WGM, int WGN, int KG, int S>
void launch_tiles(const Int8Args &a, hipStream_t s) {
  const dim3 grid((uint32_t)(a.whole + (a.mt * a.nt - a.whole) * a.splits));
  hipLaunchKernelGGL((tile_kernel<BM, BN, WGM, WGN, KG, S>), grid, dim3(KG * WGM * WGN * 64), 0, s,
                     a);
}
template <int BM, int BN, int S>
void launch_pipe(const Int8Args &a, hipStream_t s) {
  const int64_t items = a.whole + (int64_t)(a.mt * a.nt - a.whole) * a.splits;
  const dim3 grid((uint32_t)(items < kCUs ? items : kCUs));
  if (((uintptr_t)a.A | (uintptr_t)a.B | (uintptr_t)a.lda | (uintptr_t)a.ldb) % 128)
    hipLaunchKernelGGL((pipe_kernel<BM, BN, S, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((pipe_kernel<BM, BN, S, false>), grid, dim3(256), 0, s, a);
}
void (*const kLaunchTiles[])(const Int8Args &, hipStream_t) = {   // in the order of kTiles
    launch_tiles<64, 64, 2, 2, 2, 8>,
    launch_pipe<64, 128, 5>,
    launch_pipe<128, 128, 4>,
    launch_pipe<128, 192, 4>,
    launch_pipe<192, 128, 4>,
    launch_pipe<192, 192, 3>,
    launch_pipe<128, 256, 3>,
    launch_pipe<256, 128, 3>,
};
static_assert(sizeof(kLaunchTiles) / sizeof(kLaunchTiles[0]) == kKinds, "");

template <int FM>
void launch_few(const Int8Args &a, hipStream_t s) {
  hipLaunchKernelGGL(few_kernel<FM>, dim3((uint32_t)a.nt, (uint32_t)a.splits), dim3(512), 0, s, a);
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
  // K that is cut everywhere: those of the kernel that adds the pieces, 256 for 1024 elements of whole tiles
  const int64_t tiles = ((d->M + 63) / 64) * ((d->N + 63) / 64);
  if (tiles > (1ll << (d->K > 128ll * kMostBlocks ? 19 : 22))) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

size_t workspace_of(const gemm_int8_desc &d, const Int8Plan &p) {
  if (p.splits <= 1) return 0;
  const size_t one = p.tiles < 0 ? (size_t)d.M * (size_t)d.N
                                 : (size_t)(p.mt * p.nt - p.whole) *
                                       (size_t)(kTiles[p.tiles].bm * kTiles[p.tiles].bn);
  return (size_t)p.splits * sizeof(int) * one;
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
  a.out_bf16 = d->dtype_c == GEMM_BF16;
  a.src_bf16 = d->dtype_source == GEMM_BF16;
  a.plain_rows = !source && d->N % 4 == 0 && !((uintptr_t)C & (a.out_bf16 ? 7 : 15));
  hipStream_t s = (hipStream_t)stream;
  if (p.wide > 0) {
    a.mt = (int32_t)((d->M + kWide - 1) / kWide);
    a.nt = p.wide;
    if (launch_int8_wide(a, s) != hipSuccess) return GEMM_ERR_HIP;
    if (p.tiles == -2) return GEMM_OK;
  }
  a.n_first = (int64_t)p.wide * kWide;
  a.mt = p.mt;
  a.nt = p.nt;
  a.splits = p.splits;
  a.whole = p.whole;
  if (p.tiles < 0) {
    if (d->M <= 16)
      launch_few<1>(a, s);
    else
      launch_few<2>(a, s);
  } else {
    a.bm = kTiles[p.tiles].bm;
    a.bn = kTiles[p.tiles].bn;
    kLaunchTiles[p.tiles](a, s);
  }
  if (hipGetLastError() != hipSuccess) return GEMM_ERR_HIP;
  if (p.splits > 1) {
    const int64_t few = (d->M * ((d->N + 3) / 4) + 255) / 256;
    const bool parts = p.splits >= kPartsFrom;
    const auto join = p.tiles < 0 ? (parts ? join_kernel<4> : join_kernel<1>)
                                  : (parts ? join_tiles_kernel<4> : join_tiles_kernel<1>);
    const int64_t groups = p.tiles < 0 ? (few < 8 * kCUs ? few : 8 * kCUs)
                                       : (int64_t)(p.mt * p.nt - p.whole) * (a.bm * a.bn / 1024);
    hipLaunchKernelGGL(join, dim3((uint32_t)groups), dim3(parts ? 1024 : 256), 0, s, a);
    if (hipGetLastError() != hipSuccess) return GEMM_ERR_HIP;
  }
  return GEMM_OK;
}
