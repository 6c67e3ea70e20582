// The int8 product's arguments and epilogue, shared by its translation units: ops_int8.hip (few rows, tiles,
// the choice of kernel, the C ABI) and ops_int8_wide.hip (large tiles).
#pragma once
#include "ops_block.h"

namespace dg {

// The arguments are the block-scaled product's: sa and sb hold one scale a row, partials are int32.
using Int8Args = BlockArgs;

__device__ __forceinline__ i32x4 mfma_int8(const i32x4 &b, const i32x4 &a, const i32x4 &c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0);
}

// A sum, as a float, times both scales, plus the bias.  In this order nothing is lost on the way: the sum is a
// whole number, so that times A's scale it has no less than the scale's own places, and it passes the
// largest number only if that scale is over 2^90 (sums are under 2^37), where B's scale comes first.
constexpr float kLargeScale = 0x1p90f;
__device__ __forceinline__ float scaled(float sum, float sa, float sb, float bias) {
  const bool large = fabsf(sa) > kLargeScale;
  return fmaf(sum * (large ? sb : sa), large ? sa : sb, bias);
}

// Four floats of a vector of N at n .. n + 3; what lies past N is anything.
__device__ __forceinline__ f32x4 vector_four(const Int8Args &a, const float *p, int64_t n) {
  if (a.N >= 4) return from_inside(a, n, *(const u32x4_any *)(p + quad_inside(a, n)));
  f32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) v[i] = p[n + i];
  return v;
}

// From the sums of four neighbouring outputs n .. n + 3 of row m to C, one after the other.
__device__ __forceinline__ void finish_four(const Int8Args &a, int64_t m, int64_t n, f32x4 sum) {
  const float sa = a.sa[m];
  const f32x4 sb = vector_four(a, a.sb, n);
  f32x4 v = {0, 0, 0, 0};
  if (a.bias) v = vector_four(a, a.bias, n);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = scaled(sum[i], sa, sb[i], v[i]);
  if (a.source) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= a.N) break;
      const int64_t at = m * a.N + n + i;
      v[i] += a.src_bf16 ? __uint_as_float((uint32_t)((const uint16_t *)a.source)[at] << 16)
                         : ((const float *)a.source)[at];
    }
  }
  put_four(a, m, n, v);
}

// Sums stay in int32 up to this many blocks of 128 along K (128^2 K < 2^31); past it K is cut.
constexpr int32_t kMostBlocks = 1023;

}  // namespace dg
