// The int8 product's arguments and epilogue, shared by its translation units: ops_int8.hip (few rows, tiles,
// the choice of kernel, the C ABI) and ops_int8_wide.hip (large tiles).
#pragma once
#include "ops_block.h"

namespace dg {

// The block-scaled product's arguments, where sa and sb hold one scale a row and partials are int32.
struct Int8Args : BlockArgs {
  int64_t n_first;   // the column that the tiles start at
  int32_t bm, bn;    // of the tiles whose K is cut
};

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

// Stores four neighbouring outputs past the caches: for tiles that all CUs write at the same time.
__device__ __forceinline__ void put_four_once(const Int8Args &a, int64_t m, int64_t n, const f32x4 &v) {
  const int64_t at = m * a.N + n;
  if (n + 4 > a.N)
    put_four(a, m, n, v);
  else if (a.out_bf16)
    __builtin_nontemporal_store(u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])},
                                (u32x2_any *)(a.C + at * 2));
  else
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), (u32x4_any *)(a.C + at * 4));
}

// What four neighbouring outputs n .. n + 3 of row m take besides their sums.
struct Extras {
  float sa;
  f32x4 sb, bias, source;
};
__device__ __forceinline__ Extras extras_of(const Int8Args &a, int64_t m, int64_t n) {
  Extras x{a.sa[m], vector_four(a, a.sb, n), {0, 0, 0, 0}, {0, 0, 0, 0}};
  if (a.bias) x.bias = vector_four(a, a.bias, n);
  if (a.source) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= a.N) break;
      const int64_t at = m * a.N + n + i;
      x.source[i] = a.src_bf16 ? __uint_as_float((uint32_t)((const uint16_t *)a.source)[at] << 16)
                               : ((const float *)a.source)[at];
    }
  }
  return x;
}
// From their sums to C.
__device__ __forceinline__ void finish_four(const Int8Args &a, int64_t m, int64_t n, const f32x4 &sum,
                                            const Extras &x) {
  f32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = scaled(sum[i], x.sa, x.sb[i], x.bias[i]);
    if (a.source) v[i] += x.source[i];
  }
  put_four(a, m, n, v);
}
__device__ __forceinline__ void finish_four(const Int8Args &a, int64_t m, int64_t n, const f32x4 &sum) {
  finish_four(a, m, n, sum, extras_of(a, m, n));
}

// ---- streams of instructions laid out by hand --------------------------------------------------

// The accumulators stay in accumulation registers, named as both source and destination: given the builtin, the
// compiler moves them in and out around every MFMA.  It does not see the latency of these: an MFMA that adds to
// what the one before it wrote may follow at once, anything else that reads it waits (mfma_wait_states).
__device__ __forceinline__ void mfma_int8_inplace(i32x4 &c, const i32x4 &b, const i32x4 &a) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}
__device__ __forceinline__ void mfma_int8_zero(i32x4 &c, const i32x4 &b, const i32x4 &a) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, 0" : "=a"(c) : "v"(b), "v"(a));
}
// keeps the accumulator where it is until here
__device__ __forceinline__ int acc_read(int x) {
  int y;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(y) : "a"(x));
  return y;
}

// A buffer of `bytes` from `base` on.  Both are the same in all lanes, which is said here: where the compiler does
// not see it, it makes a loop of every access.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void *base, int64_t bytes) {
  const uint64_t p = (uint64_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)p);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(p >> 32));
  const int32_t n = bytes <= 0 ? 0 : bytes > 0x7FFFFFF0ll ? 0x7FFFFFF0 : (int32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc((void *)((uint64_t)hi << 32 | lo), (short)0,
                                           __builtin_amdgcn_readfirstlane(n), 0x00020000);
}

// One step of a wave with FM x FN blocks of 16 x 16: a k-block of 128, its first 64 k in all blocks and then its
// other 64, so that each half's fragments are read from LDS beside the other half's MFMAs, in the registers that
// were last used half a step ago.  `mfma(half, f, g)` is called for every block in each half; between the first
// half's go read(1, ...) of this step and the handshake (behind it the next step's loads have landed and
// this step's stage is free), between the second half's read(0, ...) of the next step and the L loads.
//
template <int FM, int FN, int L, class Mfma, class Read, class Shake, class Load>
__device__ __forceinline__ void int8_step(Mfma mfma, Read read, Shake handshake, Load load) {
  constexpr int NM = FM * FN, NF = FM + FN;
  constexpr int HS = NM * 5 / 8, RE = NM / 2, LS = HS + 1, LE = 2 * NM - NM / 16;
  [&]<int... I>(std::integer_sequence<int, I...>) {
    (
        [&] {
          constexpr int i = I % NM, half = I / NM;
          mfma(std::integral_constant<int, half>(), std::integral_constant<int, i / FN>(),
               std::integral_constant<int, i % FN>());
          constexpr int lo = ops_before(i, NF, 0, RE), hi = ops_before(i + 1, NF, 0, RE);
          [&]<int... E>(std::integer_sequence<int, E...>) {
            (read(std::integral_constant<int, 1 - half>(), std::integral_constant<int, lo + E>()), ...);
          }(std::make_integer_sequence<int, hi - lo>());
          if constexpr (half == 0 && i == HS) handshake();
          if constexpr (I >= LS) {
            constexpr int plo = ops_before(I, L, LS, LE), phi = ops_before(I + 1, L, LS, LE);
            [&]<int... J>(std::integer_sequence<int, J...>) {
              (load(std::integral_constant<int, plo + J>()), ...);
            }(std::make_integer_sequence<int, phi - plo>());
          }
          __builtin_amdgcn_sched_barrier(0);
        }(),
        ...);
  }(std::make_integer_sequence<int, 2 * NM>());
}

// Tiles of 256 x 256 (ops_int8_wide.hip): a.mt x a.nt of them from column zero on, N >= 4, K > 0 and not
// split.
hipError_t launch_int8_wide(const Int8Args &a, hipStream_t s);

}  // namespace dg
