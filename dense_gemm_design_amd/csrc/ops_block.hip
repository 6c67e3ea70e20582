// Product of e4m3 operands with a scale per block of 128 (gemm_block_run):
//
//   C[m, n] = sum over kb of sa[m, kb] sb[n, kb] P_kb[m, n] (+ bias[n]) (+ source[m, n]),
//   P_kb[m, n] = sum over the 128 k of block kb of a[m, k] b[n, k]
//
// with sb per row of B, or per 128 rows.  P_kb leaves the matrix unit and is added to accumulators
// in registers: one vector instruction a value (two where B has row scales), beside the next block's
// MFMAs.  One of the scales gives its power of two to the matrix unit, so that neither sa sb nor P sa nor
// P sb leaves the range of fp32 where the term does not (ops_block.h).  With sa sb formed first, as it
// was, 8192^3 took 518 us (now 535), 4096 x 14336 x 4096 with row scales 298 (312), 2048 x 4096 x 8192 77 (80).
//
// What the matrix unit rounds.  The e4m3 MFMAs align the products of eight neighbouring k to the
// largest of them and keep 13 binary places below its leading one; all other sums in them, and all
// sums of the bf16 forms, keep 24.  (Seen by adding one product 2^-e as large as another: e4m3 loses
// it from e = 14 within eight k, from e = 24 otherwise.)  On normal data that is 1.5e-5 of C.  So
//  * a bf16 C, whose own rounding is 2^-8, takes one 16 x 16 x 128 e4m3 MFMA a block of k -- and
//    where all scales are powers of two, gives it their exponents as operands and lets it
//    accumulate by itself;
//  * an fp32 C takes four 16 x 16 x 32 bf16 MFMAs a block, at half the rate, on the codes converted
//    in registers, which is exact; so does a bf16 C that the caller wants exact, and so do products of few
//    rows, which wait for memory anyway.
#include "../../include/gemm_ops.h"
#include "ops_block.h"

namespace dg {
namespace {

constexpr int kTile = 128;   // rows and columns of the smaller tiles

// ---- tiles through LDS ------------------------------------------------------------------------

// Where tile t of the order lies: strips of eight rows of tiles, walked down first.
__device__ __forceinline__ void tile_corner(const BlockArgs &a, int32_t t, int bm, int bn,
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
// in LDS.  A ring of two stages a group in LDS holds the k-block that is multiplied and the next one
// on its way (loads that write LDS directly, rows swizzled in 16-byte chunks as in the plain product's
// kernels).  The scales of a stage's block travel with it.
//
// The first a.whole tiles have a workgroup each; the k-blocks of the others are cut into a.splits
// pieces, whose sums join_tiles_kernel adds.
enum { MODE_FMA, MODE_POW2, MODE_EXACT };
template <int BM, int BN, int WGM, int WGN, int KG, bool ROWB, int MODE>
__global__ void __launch_bounds__(KG *WGM *WGN * 64, 2) block_kernel(const BlockArgs a) {
  constexpr int NW = WGM * WGN, WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;   // 1 KiB loads (8 rows) a wave and stage
  constexpr int SCALES = (BM + BN) * 4, STAGE = (BM + BN) * 128 + SCALES;
  static_assert(BM % 64 == 0 && BN % 64 == 0 && (BM + BN) / 64 == NW, "one scale load a wave");
  __shared__ __align__(1024) char smem_[KG * 2 * STAGE];
  const int wave_ = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int group = wave_ / NW, wave = wave_ % NW;
  lds_t *const smem = (lds_t *)smem_ + group * 2 * STAGE;

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
  // the wave's 64 scales of a stage: of A's rows, or of B's
  const bool scales_a = wave < BM / 64;
  const int32_t sfirst = (scales_a ? wave : wave - BM / 64) * 64;
  const float *const sbase = scales_a ? a.sa + m0 : a.sb + (ROWB ? n0 : n0 / 128);
  const int64_t spitch = scales_a ? a.lsa : a.lsb;
  const int32_t scount = scales_a ? rows_a : ROWB ? rows_b : (rows_b + 127) / 128;
  const uint32_t svo = (uint32_t)(scales_a || ROWB ? sfirst + lane : (sfirst + lane) / 128) * 4;

  auto load_stage = [&](int32_t kb, int s) {
    const uint32_t k = (uint32_t)kb * 128;
    const bool past = k + chunk >= (uint32_t)a.kbytes;
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
    const auto rs = make_rsrc((const char *)(sbase + kb * spitch),
                              (int64_t)scount * 4);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, smem + s * STAGE + (BM + BN) * 128 + wave * 256,
                                             4, svo, 0, 0, 0);
  };

  // consumer
  const int wm = wave / WGN, wn = wave % WGN, r16 = lane & 15, g4 = lane >> 4;
  const uint32_t x = (r16 >> 1) & 7;
  // a lane's two chunks of a row are g4 and g4 + 4, in A and B alike: reads of neighbours cost an
  // LDS pass more
  const uint32_t c0 = (g4 ^ x) * 16, c1 = ((g4 + 4) ^ x) * 16;
  const uint32_t arow = (wm * WM + r16) * 128, brow = BM * 128 + (wn * WN + r16) * 128;
  const uint32_t sarow = (BM + BN) * 128 + (wm * WM + r16) * 4;
  const uint32_t sbrow = (BM + BN) * 128 + (BM + wn * WN) * 4;

  f32x4 acc[FM][FN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < FN; ++g) acc[f][g] = f32x4{0, 0, 0, 0};
  // a wave wholly past the edge only loads
  const bool inside = m0 + wm * WM < a.M && n0 + wn * WN < a.N;

  if (kb0 + group < kb1) load_stage(kb0 + group, 0);
  int s = 1;
  for (int32_t kb = kb0 + group; kb < kb1 + group; kb += KG) {   // as often in every group
    s ^= 1;
    // this wave's loads of the stage have landed and its reads of the other stage are done; after
    // the barrier that holds for every wave
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (kb + KG < kb1) load_stage(kb + KG, s ^ 1);
    if (!inside || kb >= kb1) continue;
    const lds_t *const st = smem + s * STAGE;
    typedef const float __attribute__((address_space(3))) *fp;
    typedef const f32x4 __attribute__((address_space(3))) *f4p;
    i32x8 b[FN];
#pragma unroll
    for (int g = 0; g < FN; ++g)
      b[g] = lds_frag<DT_FP8>(st + brow + c0 + g * 2048, st + brow + c1 + g * 2048);
    if constexpr (MODE == MODE_POW2) {
      int eb[FN];
#pragma unroll
      for (int g = 0; g < FN; ++g) eb[g] = exponent_of(*(fp)(st + sbrow + (g * 16 + r16) * 4));
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        const i32x8 af = lds_frag<DT_FP8>(st + arow + c0 + f * 2048, st + arow + c1 + f * 2048);
        const int ea = exponent_of(*(fp)(st + sarow + f * 64));
#pragma unroll
        for (int g = 0; g < FN; ++g) acc[f][g] = mfma_block_scaled(b[g], af, acc[f][g], eb[g], ea);
      }
    } else {
      // the scale of which a power of two goes to the matrix unit: B's tile's, or A's rows'
      f32x4 sb[FN];
      if constexpr (ROWB) {
#pragma unroll
        for (int g = 0; g < FN; ++g) sb[g] = *(f4p)(st + sbrow + (g * 16 + g4 * 4) * 4);
      }
      const TileScale tile(__float_as_int(ROWB ? 1.0f : *(fp)(st + sbrow)));
      using Frag = std::conditional_t<MODE == MODE_EXACT, BlockBf16, i32x8>;
      auto frag = [](const i32x8 &q, float power) {
        if constexpr (MODE == MODE_EXACT)
          return widen(q, power);
        else
          return q;
      };
      Frag bf[FN];
#pragma unroll
      for (int g = 0; g < FN; ++g) bf[g] = frag(b[g], ROWB ? 1.0f : tile.power());
      f32x4 p[2][FN];
      float sa[2];   // ROWB: what is left of A's scale; else A's times what is left of B's
#pragma unroll
      for (int f = 0; f <= FM; ++f) {
        Frag af;
        int byte = 127;
        if (f < FM) {
          const float s = *(fp)(st + sarow + f * 64);
          if constexpr (ROWB) {
            byte = scale_byte(s, 0);
            sa[f & 1] = scale_rest(s, byte);
          } else {
            sa[f & 1] = tile.times(s);
          }
          af = frag(lds_frag<DT_FP8>(st + arow + c0 + f * 2048, st + arow + c1 + f * 2048),
                    power_of(byte));
        }
#pragma unroll
        for (int g = 0; g < FN; ++g) {
          if (f < FM) {
            if constexpr (MODE == MODE_EXACT)
              p[f & 1][g] = mfma_block(bf[g], af);
            else if constexpr (ROWB)
              p[f & 1][g] = mfma_block_a(bf[g], af, byte);
            else
              p[f & 1][g] = mfma_block_b(bf[g], af, tile.bytes);
          }
          if (f > 0) {
            const float sf = sa[(f - 1) & 1];
            f32x4 &c = acc[f - 1][g];
            const f32x4 q = p[(f - 1) & 1][g];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = fmaf(ROWB ? q[e] * sb[g][e] : q[e], sf, c[e]);
          }
        }
      }
    }
  }

  // each group gives away the sums of the rows of blocks that the other one writes
  constexpr int OWN = FM / KG;
  static_assert(KG == 1 || (KG == 2 && OWN * KG == FM && NW * OWN * FN * 1024 <= 2 * STAGE), "");
  if constexpr (KG == 2) {
    typedef f32x4 __attribute__((address_space(3))) *f4p;
    lds_t *const area = (lds_t *)smem_ + wave * (OWN * FN * 1024) + lane * 16;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // all stages are read
#pragma unroll
    for (int f = 0; f < OWN; ++f)
#pragma unroll
      for (int g = 0; g < FN; ++g)
        *(f4p)(area + (group ^ 1) * 2 * STAGE + (f * FN + g) * 1024) =
            group ? acc[f][g] : acc[f + OWN][g];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int f = 0; f < OWN; ++f)
#pragma unroll
      for (int g = 0; g < FN; ++g)
        acc[f][g] = (group ? acc[f + OWN][g] : acc[f][g]) +
                    *(f4p)(area + group * 2 * STAGE + (f * FN + g) * 1024);
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
          *(f32x4 *)(a.partials + (int64_t)piece * (BM * BN) + ml * BN + nl) = acc[f][g];
        else
          store_four(a, m0 + ml, n0 + nl, acc[f][g]);
      }
    }
    return;
  }
  f32x4 bias[FN];
#pragma unroll
  for (int g = 0; g < FN; ++g) bias[g] = bias_four(a, n0 + nl0 + g * 16);
  with_source(a, [&](auto src_c) {
    constexpr int SRC = decltype(src_c)::value;
#pragma unroll
    for (int f0 = 0; f0 < OWN; f0 += 2) {
      u32x4 src[2][FN];
      if constexpr (SRC != SRC_NONE) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int g = 0; g < FN; ++g)
            src[f][g] = source_at<SRC>(a, m0 + ml0 + (f0 + f) * 16, n0 + nl0 + g * 16);
      }
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int g = 0; g < FN; ++g) {
          const int64_t m = m0 + ml0 + (f0 + f) * 16, n = n0 + nl0 + g * 16;
          if (m >= a.M || n >= a.N) continue;
          f32x4 v = acc[f0 + f][g];
          if (a.bias) v += bias[g];
          if constexpr (SRC != SRC_NONE) v += source_four<SRC>(a, n, src[f][g]);
          put_four(a, m, n, v);
        }
    }
  });
}

// Adds the pieces of the tiles whose K is cut, in order, then the epilogue.  Eight rows of a tile a
// workgroup.
__global__ void __launch_bounds__(256) join_tiles_kernel(const BlockArgs a) {
  constexpr int B = kTile;
  const int32_t cut = a.mt * a.nt - a.whole, at = blockIdx.x / (B / 8);
  const int ml = blockIdx.x % (B / 8) * 8 + threadIdx.x / 32, nl = threadIdx.x % 32 * 4;
  int64_t m0, n0;
  tile_corner(a, a.whole + at, B, B, m0, n0);
  const int64_t m = m0 + ml, n = n0 + nl;
  if (m >= a.M || n >= a.N) return;
  const bool ahead = a.N >= 4;   // the extras are loaded before the pieces
  with_source(a, [&](auto src_c) {
    constexpr int SRC = decltype(src_c)::value;
    u32x4 src;
    f32x4 bias = {0, 0, 0, 0}, v = {0, 0, 0, 0};
    if (ahead) {
      bias = bias_four(a, n);
      if constexpr (SRC != SRC_NONE) src = source_at<SRC>(a, m, n);
    }
    for (int s = 0; s < a.splits; s += 8) {
      f32x4 q[8];   // loads in flight together
#pragma unroll
      for (int u = 0; u < 8; ++u)
        q[u] = s + u < a.splits
                   ? *(const f32x4 *)(a.partials + (int64_t)((s + u) * cut + at) * (B * B) + ml * B + nl)
                   : f32x4{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 8; ++u) v += q[u];
    }
    if (!ahead) {
      store_four(a, m, n, v);
      return;
    }
    if (a.bias) v += bias;
    if constexpr (SRC != SRC_NONE) v += source_four<SRC>(a, n, src);
    put_four(a, m, n, v);
  });
}

// Adds the splits' sums of few rows in order, then the epilogue.
__global__ void __launch_bounds__(256) join_kernel(const BlockArgs a) {
  const int64_t per_row = (a.N + 3) / 4, all = a.M * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per_row, n = i % per_row * 4;
    f32x4 v = {0, 0, 0, 0};
    for (int s = 0; s < a.splits; s += 4) {
      f32x4 q[4];   // loads in flight together
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float *p = a.partials + ((int64_t)(s + u) * a.M + m) * a.N + n;
        q[u] = f32x4{0, 0, 0, 0};
        if (s + u >= a.splits) continue;
        if (n + 4 <= a.N) {
          q[u] = __builtin_bit_cast(f32x4, *(const u32x4_any *)p);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) q[u][e] = p[e];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) v += q[u];
    }
    store_four(a, m, n, v);
  }
}

// ---- few rows ---------------------------------------------------------------------------------

// Up to 16 FM rows of A: what counts is to read B once at the memory's rate.  A workgroup takes 16 GN
// rows of B (columns of C); its eight waves take every eighth k-block (of its piece of K) straight
// into registers, and their sums meet in LDS.  1 x 4096 x 4096 takes 5.9 us on the GPU, 6.7 with
// sixteen waves; 1 x 16384 x 16384 52.6 us, 5.1 TB/s.
template <int FM, int GN, bool ROWB>
__global__ void __launch_bounds__(512) few_kernel(const BlockArgs a) {
  constexpr int WAVES = 8;
  constexpr int AHEAD = FM * GN > 2 ? 2 : 4;   // k-blocks of a wave whose loads are in flight together
  __shared__ float part[WAVES][FM][GN][16][17];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r16 = lane & 15, g4 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * GN);
  const auto ra = make_rsrc(a.A, a.M * a.lda);
  const int64_t rows_b = a.N - n0 < 16 * GN ? a.N - n0 : 16 * GN;
  const auto rb = make_rsrc(a.B + n0 * a.ldb, rows_b * a.ldb);
  const int split = blockIdx.y;
  const int32_t kb1 = (int32_t)((int64_t)a.kb * (split + 1) / a.splits);
  f32x4 acc[FM][GN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < GN; ++g) acc[f][g] = f32x4{0, 0, 0, 0};
  // past K an operand reads as zeros
  auto take = [&](auto r, uint32_t row, uint32_t ld, uint32_t k) {
    const uint32_t o0 = k < (uint32_t)a.kbytes ? row * ld + k : kOOB;
    const uint32_t o1 = k + 16 < (uint32_t)a.kbytes ? row * ld + k + 16 : kOOB;
    const i32x4 lo = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o0, 0, 0));
    const i32x4 hi = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o1, 0, 0));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  for (int32_t kb0 = (int32_t)((int64_t)a.kb * split / a.splits) + wave; kb0 < kb1;
       kb0 += WAVES * AHEAD) {
    i32x8 b[AHEAD][GN], x[AHEAD][FM];
    float s[AHEAD][FM];
    f32x4 sb[AHEAD][GN];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int32_t kb = kb0 + WAVES * u;
      const bool in = kb < kb1;   // past the last k-block too
      const uint32_t k = in ? (uint32_t)kb * 128 + g4 * 32 : (uint32_t)a.kbytes;
#pragma unroll
      for (int g = 0; g < GN; ++g) b[u][g] = take(rb, g * 16 + r16, (uint32_t)a.ldb, k);
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        const int64_t m = f * 16 + r16;
        x[u][f] = take(ra, (uint32_t)m, (uint32_t)a.lda, k);
        s[u][f] = in && m < a.M ? a.sa[kb * a.lsa + m] : 0.0f;
      }
#pragma unroll
      for (int g = 0; g < GN; ++g) {
        if constexpr (ROWB) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t n = n0 + g * 16 + g4 * 4 + e;
            sb[u][g][e] = in && n < a.N ? a.sb[kb * a.lsb + n] : 0.0f;
          }
        } else {
          const float z = in ? a.sb[kb * a.lsb + n0 / 128] : 0.0f;
          sb[u][g] = f32x4{z, z, z, z};
        }
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      BlockBf16 wide[GN];
#pragma unroll
      for (int g = 0; g < GN; ++g) wide[g] = widen(b[u][g], 1.0f);
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        const int byte = scale_byte(s[u][f], 0);
        const float rest = scale_rest(s[u][f], byte);
        const BlockBf16 w = widen(x[u][f], power_of(byte));
#pragma unroll
        for (int g = 0; g < GN; ++g) {
          const f32x4 p = mfma_block(wide[g], w);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[f][g][e] = fmaf(p[e] * sb[u][g][e], rest, acc[f][g][e]);
        }
      }
    }
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
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += part[w][f][g][m16][q * 4 + e];
    if (a.splits > 1)
      partial_four(a, split, m, n, v);
    else
      store_four(a, m, n, v);
  }
}

// ---- choice -----------------------------------------------------------------------------------

constexpr int kCUs = 256;

enum { PLAN_FEW, PLAN_128, PLAN_CUT, PLAN_256, PLAN_WIDE };
struct BlockPlan {
  int kind, splits;
  int32_t mt, nt, whole;   // whole: the tiles whose K is not cut
};

int few_columns(const gemm_block_desc &d) { return d.M > 16 && d.N > 16 * kCUs ? 32 : 16; }

BlockPlan plan_of(const gemm_block_desc &d) {
  const int64_t kb = (d.K + 127) / 128;
  if (d.M <= 32) {
    // 32 columns a workgroup where there are more rows of A to read beside them than one block's and
    // columns enough (32 x 16384 x 16384 79 us, 103 on 16; 32 x 4096 x 4096 11.7, 9.5); K in pieces where
    // there are few columns and much of it
    const int cols = few_columns(d);
    const int64_t nt = (d.N + cols - 1) / cols;
    int64_t splits = nt < 128 ? 256 / nt : 1;
    if (splits > kb / 16) splits = kb / 16;
    return {PLAN_FEW, splits > 1 ? (int)splits : 1, 1, (int32_t)nt, 0};
  }
  const bool bf16_mfma = d.dtype_c == GEMM_F32 || d.exact;
  if (!bf16_mfma && kb && d.N >= 4) {   // (the wide tiles' quads want four columns)
    // Tiles of 256 x 256 (wide with powers of two, eight waves otherwise) or, for fp32 scales of 128 x
    // 128 blocks, wide ones of 192 x 256, whose round over the CUs takes 0.74 as long: 8192^3 560 us on
    // six rounds of them, 514 on four of 256; 4096 x 14336 x 4096 236 us on five, 271 on four.  (0.62 to 0.73
    // over eleven shapes: 2048 x 16384 x 4096 takes 151 us by this rule, 142 on the other side.)
    const auto rounds = [&](int rows) {
      return (((d.M + rows - 1) / rows) * ((d.N + 255) / 256) + kCUs - 1) / kCUs;
    };
    const bool fp32_tiles = !d.pow2 && d.block_b == GEMM_BLOCK_TILE;
    const bool narrow = fp32_tiles && 0.74 * rounds(wide_rows(false)) < rounds(256);
    const int rows = narrow ? wide_rows(false) : 256;
    const int64_t mt = (d.M + rows - 1) / rows, nt = (d.N + 255) / 256;
    if (mt * nt >= kCUs)
      return {d.pow2 || narrow ? PLAN_WIDE : PLAN_256, 1, (int32_t)mt, (int32_t)nt, (int32_t)(mt * nt)};
  }
  // Tiles of 128 x 128 (codes as bf16 leave no registers for larger sub-tiles).  Either
  // PLAN_128, two workgroups a CU, a tile each: a k-block takes c1 us for one of them alone, c2 for two.
  // Or PLAN_CUT, one of twice the waves a CU, which takes two k-blocks in c us, and a round of tiles
  // 1.5 us more, in which it only writes: as many tiles as fill rounds of all CUs are taken whole, and K
  // is cut for the rest, which costs 8 bytes an element and piece to write and read, and a launch.  What
  // is less by this estimate.  (us on PLAN_128 and PLAN_CUT, fp32: 4096 x 14336 x 4096 448, 506; 2048 x
  // 4096 x 8192 130, 135; 2048 x 2048 x 8192 79, 67; 1000 x 4104 x 8201 133, 90.  bf16, fp32 scales: 77,
  // 90 and 56, 47 for the two in the middle; powers of two: 66, 80 and 48, 39.)
  const int64_t mt = (d.M + kTile - 1) / kTile, nt = (d.N + kTile - 1) / kTile;
  const int64_t t = mt * nt, rest = t % kCUs;
  const double c1 = bf16_mfma ? 1.3 : d.pow2 ? 0.75 : 0.9;
  const double c2 = bf16_mfma ? 2.1 : d.pow2 ? 1.05 : 1.27;
  const double c = bf16_mfma ? 2.33 : d.pow2 ? 1.22 : 1.45;
  const int64_t last = t % (2 * kCUs);
  const double pairs =
      (double)kb * ((double)(t / (2 * kCUs)) * c2 + (last > kCUs ? c2 : last ? c1 : 0.0));
  int splits = 1;
  double least = 0.0;
  for (int s = 1; s <= 64 && (s == 1 || (rest && s * 2 <= kb && rest * s <= 8 * kCUs)); ++s) {
    const int64_t steps = ((kb + s - 1) / s + 1) / 2, rounds = (rest * s + kCUs - 1) / kCUs;
    double us = (double)rounds * ((double)steps * c + 1.5);
    if (s > 1) us += 3.0 + (double)(rest * s) * (kTile * kTile) * 1e-6;
    if (s == 1 || us < least) {
      least = us;
      splits = s;
    }
  }
  if (pairs <= (double)(t / kCUs) * ((double)((kb + 1) / 2) * c + 1.5) + least)
    return {PLAN_128, 1, (int32_t)mt, (int32_t)nt, (int32_t)t};
  return {PLAN_CUT, splits, (int32_t)mt, (int32_t)nt, (int32_t)(t - rest)};
}

template <int BM, int BN, int WGM, int WGN, int KG, int MODE>
void launch_tiles(const BlockArgs &a, bool rowb, hipStream_t s) {
  const dim3 grid((uint32_t)(a.whole + (a.mt * a.nt - a.whole) * a.splits)),
      block(KG * WGM * WGN * 64);
  if (rowb)
    hipLaunchKernelGGL((block_kernel<BM, BN, WGM, WGN, KG, true, MODE>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((block_kernel<BM, BN, WGM, WGN, KG, false, MODE>), grid, block, 0, s, a);
}
template <int KG>
void launch_small(const BlockArgs &a, bool rowb, const gemm_block_desc &d, hipStream_t s) {
  if (d.dtype_c == GEMM_F32 || d.exact)
    launch_tiles<kTile, kTile, 2, 2, KG, MODE_EXACT>(a, rowb, s);
  else if (d.pow2)
    launch_tiles<kTile, kTile, 2, 2, KG, MODE_POW2>(a, rowb, s);
  else
    launch_tiles<kTile, kTile, 2, 2, KG, MODE_FMA>(a, rowb, s);
}
template <int FM, int GN>
void launch_few(const BlockArgs &a, bool rowb, hipStream_t s) {
  const dim3 grid((uint32_t)a.nt, (uint32_t)a.splits), block(512);
  if (rowb)
    hipLaunchKernelGGL((few_kernel<FM, GN, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((few_kernel<FM, GN, false>), grid, block, 0, s, a);
}

int check(const gemm_block_desc *d) {
  if (!d || d->M < 0 || d->N < 0 || d->K < 0) return GEMM_ERR_INVALID_ARG;
  if (d->block_b != GEMM_BLOCK_ROW && d->block_b != GEMM_BLOCK_TILE) return GEMM_ERR_INVALID_ARG;
  if ((d->dtype_c != GEMM_BF16 && d->dtype_c != GEMM_F32) ||
      (d->dtype_source != GEMM_BF16 && d->dtype_source != GEMM_F32))
    return GEMM_ERR_INVALID_ARG;
  if (d->lda < d->K || d->ldb < d->K || d->lda % 16 || d->ldb % 16) return GEMM_ERR_INVALID_ARG;
  if (d->K > 128) {
    if (d->scale_lda < d->M) return GEMM_ERR_INVALID_ARG;
    if (d->scale_ldb < (d->block_b == GEMM_BLOCK_ROW ? d->N : (d->N + 127) / 128))
      return GEMM_ERR_INVALID_ARG;
  }
  // offsets inside a tile of 256 rows (of A, B or C) stay under 31 bits, work-items under 2^32
  if (d->lda > (1 << 22) || d->ldb > (1 << 22)) return GEMM_ERR_UNSUPPORTED;
  if (d->M > (1ll << 31) || d->N > (1ll << 22)) return GEMM_ERR_UNSUPPORTED;
  if (((d->M + 127) / 128) * ((d->N + 127) / 128) > (1ll << 22)) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

}  // namespace
}  // namespace dg

extern "C" int gemm_block_workspace(const gemm_block_desc *d, size_t *bytes) {
  const int st = dg::check(d);
  if (st != GEMM_OK) return st;
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  *bytes = 0;
  if (d->M == 0 || d->N == 0) return GEMM_OK;
  const dg::BlockPlan p = dg::plan_of(*d);
  if (p.splits > 1)
    *bytes = (size_t)p.splits * sizeof(float) *
             (p.kind == dg::PLAN_FEW ? (size_t)d->M * (size_t)d->N
                                     : (size_t)(p.mt * p.nt - p.whole) * (dg::kTile * dg::kTile));
  return GEMM_OK;
}

extern "C" int gemm_block_run(const gemm_block_desc *d, const void *A, const float *scale_a,
                              const void *B, const float *scale_b, void *C, const float *bias,
                              const void *source, void *workspace, size_t workspace_bytes,
                              void *stream) {
  using namespace dg;
  const int st = check(d);
  if (st != GEMM_OK) return st;
  if (d->M == 0 || d->N == 0) return GEMM_OK;
  if (!C || (d->K > 0 && (!A || !B || !scale_a || !scale_b))) return GEMM_ERR_INVALID_ARG;
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
  if (!(bias == C && d->M == 1 && d->dtype_c == GEMM_F32) && !apart(bias, d->N, 4))
    return GEMM_ERR_INVALID_ARG;
  const BlockPlan p = plan_of(*d);
  size_t need = 0;
  gemm_block_workspace(d, &need);
  if (need && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
  BlockArgs a{};
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
  a.lsa = d->scale_lda;
  a.lsb = d->scale_ldb;
  a.kbytes = (int32_t)((d->K + 15) / 16 * 16);
  a.kb = (int32_t)((d->K + 127) / 128);
  a.mt = p.mt;
  a.nt = p.nt;
  a.splits = p.splits;
  a.whole = p.whole;
  a.out_bf16 = d->dtype_c == GEMM_BF16;
  a.src_bf16 = d->dtype_source == GEMM_BF16;
  a.plain_rows = !source && (d->N * (a.out_bf16 ? 2 : 4)) % 16 == 0 && !((uintptr_t)C & 15);
  const bool rowb = d->block_b == GEMM_BLOCK_ROW;
  hipStream_t s = (hipStream_t)stream;
  if (p.kind == PLAN_FEW) {
    if (d->M <= 16)
      launch_few<1, 1>(a, rowb, s);
    else if (few_columns(*d) == 16)
      launch_few<2, 1>(a, rowb, s);
    else
      launch_few<2, 2>(a, rowb, s);
  } else if (p.kind == PLAN_256) {
    launch_tiles<256, 256, 2, 4, 1, MODE_FMA>(a, rowb, s);
  } else if (p.kind == PLAN_WIDE) {
    if (launch_block_wide(a, rowb, d->pow2 != 0, s) != hipSuccess) return GEMM_ERR_HIP;
  } else if (p.kind == PLAN_128) {
    launch_small<1>(a, rowb, *d, s);
  } else {
    launch_small<2>(a, rowb, *d, s);
  }
  if (hipGetLastError() != hipSuccess) return GEMM_ERR_HIP;
  if (p.splits > 1 && p.kind != PLAN_FEW) {
    hipLaunchKernelGGL(join_tiles_kernel, dim3((uint32_t)((p.mt * p.nt - p.whole) * (kTile / 8))),
                       dim3(256), 0, s, a);
    if (hipGetLastError() != hipSuccess) return GEMM_ERR_HIP;
  } else if (p.splits > 1) {
    const int64_t need_wg = (d->M * ((d->N + 3) / 4) + 255) / 256;
    hipLaunchKernelGGL(join_kernel, dim3((uint32_t)(need_wg < 8 * kCUs ? need_wg : 8 * kCUs)),
                       dim3(256), 0, s, a);
    if (hipGetLastError() != hipSuccess) return GEMM_ERR_HIP;
  }
  return GEMM_OK;
}
