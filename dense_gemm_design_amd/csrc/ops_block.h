// The block-scaled product's arguments, epilogue and operand conversions, shared by its translation
// units: ops_block.hip (tiles of 128 x 128 and less, the choice of kernel, the C ABI) and
// ops_block_wide.hip (large tiles).
#pragma once
#include "gemm_kernel.h"

namespace dg {

struct BlockArgs {
  const char *A, *B;
  const float *sa, *sb;
  char *C;
  const float *bias;
  const char *source;
  float *partials;          // splits > 1: [split][M][N] of few rows, [split][tile][128][128] of tiles
  int64_t M, N;
  int64_t lda, ldb, lsa, lsb;
  int32_t kbytes;           // K rounded up to 16: what is read of a row
  int32_t kb;               // blocks of 128 along K
  int32_t mt, nt;           // tiles
  int32_t splits, whole;    // pieces of K; the tiles in front that are not cut
  int32_t out_bf16, src_bf16;
  int32_t plain_rows;       // no source, and rows of C in whole, aligned 16 bytes
};

// ---- epilogue ---------------------------------------------------------------------------------

typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;

// Bias, source, rounding and store of four neighbouring outputs n .. n + 3 of row m; where N ends
// among them, one by one.
__device__ __forceinline__ void store_four(const BlockArgs &a, int64_t m, int64_t n, f32x4 v) {
  const int64_t at = m * a.N + n;
  if (n + 4 <= a.N) {
    if (a.bias) v += __builtin_bit_cast(f32x4, *(const u32x4_any *)(a.bias + n));
    if (a.source) {
      if (a.src_bf16) {
        const u32x2 s = *(const u32x2_any *)(a.source + at * 2);
        v += f32x4{__uint_as_float(s[0] << 16), __uint_as_float(s[0] & 0xFFFF0000u),
                   __uint_as_float(s[1] << 16), __uint_as_float(s[1] & 0xFFFF0000u)};
      } else {
        v += __builtin_bit_cast(f32x4, *(const u32x4_any *)(a.source + at * 4));
      }
    }
    if (a.out_bf16)
      *(u32x2_any *)(a.C + at * 2) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else
      *(u32x4_any *)(a.C + at * 4) = __builtin_bit_cast(u32x4, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) break;
    float z = v[i];
    if (a.bias) z += a.bias[n + i];
    if (a.source)
      z += a.src_bf16 ? __uint_as_float((uint32_t)((const uint16_t *)a.source)[at + i] << 16)
                      : ((const float *)a.source)[at + i];
    if (a.out_bf16)
      ((uint16_t *)a.C)[at + i] = (uint16_t)pack_bf16x2(z, 0.0f);
    else
      ((float *)a.C)[at + i] = z;
  }
}

// The same in three steps, for kernels whose threads have many outputs: the extras are loaded for several
// of them before the first is used (one after the other, each waited for a trip to memory: 8026 x
// 5184 x 192 with an fp32 source took 157 us, 74 to 79 so).  N >= 4; what lies past M or N is loaded from inside,
// a quad that N ends in from the row's last four.
__device__ __forceinline__ int64_t quad_inside(const BlockArgs &a, int64_t n) {
  return n + 4 <= a.N ? n : a.N - 4;
}
// SRC: what the source holds, known when compiled: where two kinds of loads meet, one is waited for.
enum { SRC_NONE, SRC_BF16, SRC_F32 };
template <int SRC>
__device__ __forceinline__ u32x4 source_at(const BlockArgs &a, int64_t m, int64_t n) {
  const int64_t at = (m < a.M ? m : a.M - 1) * a.N + quad_inside(a, n);
  if constexpr (SRC == SRC_BF16) {
    const u32x2 s = *(const u32x2_any *)(a.source + at * 2);
    return u32x4{s[0], s[1], 0, 0};
  } else {
    return *(const u32x4_any *)(a.source + at * 4);
  }
}
// the extras of n .. n + 3, of which quad_inside() loaded x
__device__ __forceinline__ f32x4 from_inside(const BlockArgs &a, int64_t n, u32x4 x) {
  f32x4 v = __builtin_bit_cast(f32x4, x);
  const int64_t by = n - quad_inside(a, n);
  if (by == 1) v = f32x4{v[1], v[2], v[3], 0.0f};
  if (by == 2) v = f32x4{v[2], v[3], 0.0f, 0.0f};
  if (by == 3) v = f32x4{v[3], 0.0f, 0.0f, 0.0f};
  return v;
}
template <int SRC>
__device__ __forceinline__ f32x4 source_four(const BlockArgs &a, int64_t n, u32x4 s) {
  if constexpr (SRC == SRC_BF16)
    s = u32x4{s[0] << 16, s[0] & 0xFFFF0000u, s[1] << 16, s[1] & 0xFFFF0000u};
  return from_inside(a, n, s);
}
template <class F>
__device__ __forceinline__ void with_source(const BlockArgs &a, F f) {
  if (!a.source)
    f(std::integral_constant<int, SRC_NONE>());
  else if (a.src_bf16)
    f(std::integral_constant<int, SRC_BF16>());
  else
    f(std::integral_constant<int, SRC_F32>());
}
__device__ __forceinline__ f32x4 bias_four(const BlockArgs &a, int64_t n) {
  if (!a.bias) return f32x4{0, 0, 0, 0};
  return from_inside(a, n, *(const u32x4_any *)(a.bias + quad_inside(a, n)));
}
__device__ __forceinline__ void put_four(const BlockArgs &a, int64_t m, int64_t n, const f32x4 &v) {
  const int64_t at = m * a.N + n;
  if (n + 4 <= a.N) {
    if (a.out_bf16)
      *(u32x2_any *)(a.C + at * 2) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else
      *(u32x4_any *)(a.C + at * 4) = __builtin_bit_cast(u32x4, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) break;
    if (a.out_bf16)
      ((uint16_t *)a.C)[at + i] = (uint16_t)pack_bf16x2(v[i], 0.0f);
    else
      ((float *)a.C)[at + i] = v[i];
  }
}

__device__ __forceinline__ void partial_four(const BlockArgs &a, int split, int64_t m, int64_t n,
                                             f32x4 v) {
  float *p = a.partials + ((int64_t)split * a.M + m) * a.N + n;
  if (n + 4 <= a.N) {
    *(u32x4_any *)p = __builtin_bit_cast(u32x4, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) p[i] = v[i];
}

// The exponent byte of a power of two, in every byte-position the MFMA may be told to read: byte 0.
__device__ __forceinline__ int exponent_of(float s) { return (int)(__float_as_uint(s) >> 23); }

__device__ __forceinline__ f32x4 mfma_block_scaled(const i32x8 &b, const i32x8 &a, const f32x4 &c,
                                                   int eb, int ea) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, 0, eb, 0, ea);
}

// ---- fp32 scales of any size ------------------------------------------------------------------
//
// A term is P sa sb, where P, a block's sum, is zero or between 2^-18 and 2^25.  sa sb alone may pass
// the largest number (and 0 inf is NaN) or fall under the smallest normal one, and so may P times
// either scale, where the term itself does neither.  So one scale gives a power of two to the matrix
// unit, which applies it to P without rounding, s = 2^h m with h between -100 and 100, and what is left
// stays in range:
//  * B scaled by tiles: sb = 2^h m, m from 1/2 to 1, and the term is (2^h P) (sa m);
//  * B scaled by rows: sa = 2^h m, m from 1 to 2, and the term is ((2^h P) sb) m.
// Where h is at its bound, m is outside these.  Then sa m may still pass the largest number, and is cut
// to it: 2^h is 2^100, and the term zero if P is, and itself past the largest number if not.  (Whatever
// else leaves the range then does so in terms that leave it.)
__device__ __forceinline__ int scale_byte(float s, int more) {   // h + 127, the MFMA's e8m0
  const int e = (int)(__float_as_uint(s) >> 23 & 255) + more;
  return e < 27 ? 27 : e > 227 ? 227 : e;
}
__device__ __forceinline__ float scale_rest(float s, int byte) {   // m, exact
  return s * __uint_as_float((uint32_t)(254 - byte) << 23);
}
__device__ __forceinline__ float power_of(int byte) { return __uint_as_float((uint32_t)byte << 23); }

struct TileScale {   // of B, the same in all lanes: the work on it is the scalar unit's
  uint32_t bytes;    // of B's power, and 1, for the MFMA to pick from
  float rest, most;
  __device__ __forceinline__ explicit TileScale(int bits) {
    const float s = __int_as_float(__builtin_amdgcn_readfirstlane(bits));
    const int byte = scale_byte(s, 1);
    bytes = (uint32_t)byte | 127u << 8;
    rest = scale_rest(s, byte);
    const bool large = byte == 227 && fabsf(s) < __builtin_inff();
    most = large ? 0x1.fffffep127f : __builtin_inff();
  }
  __device__ __forceinline__ float power() const { return power_of(bytes & 255); }
  __device__ __forceinline__ float times(float sa) const {   // a NaN stays
    return __builtin_elementwise_maximum(__builtin_elementwise_minimum(sa * rest, most), -most);
  }
};

// 2^(byte - 127) P, the byte that of a's scale, or TileScale's of b's
__device__ __forceinline__ f32x4 mfma_block_a(const i32x8 &b, const i32x8 &a, int byte) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0, 0, 0, 0}, 0, 0, 0, 127, 0,
                                                          byte);
}
__device__ __forceinline__ f32x4 mfma_block_b(const i32x8 &b, const i32x8 &a, uint32_t bytes) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0, 0, 0, 0}, 0, 0, 0,
                                                          (int)bytes, 1, (int)bytes);
}

// The codes of a fragment, times a power of two, as bf16, eight a vector.
struct BlockBf16 {
  bf16x8 v[4];
};
__device__ __forceinline__ BlockBf16 widen(const i32x8 &q, float power) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  BlockBf16 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * j], power, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * j], power, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * j + 1], power, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * j + 1], power, true);
    r.v[j] = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  return r;
}
__device__ __forceinline__ f32x4 mfma_block(const BlockBf16 &b, const BlockBf16 &a) {
  f32x4 p = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[j], a.v[j], p, 0, 0, 0);
  return p;
}

// Large tiles of a bf16 C (ops_block_wide.hip), wide_rows() x 256: a.mt x a.nt of them, K > 0 and not
// split.  All scales are powers of two, or B's are of 128 x 128 blocks.
constexpr int wide_rows(bool pow2) { return pow2 ? 256 : 192; }
hipError_t launch_block_wide(const BlockArgs &a, bool rowb, bool pow2, hipStream_t s);

}  // namespace dg
