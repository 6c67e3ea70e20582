// Device helpers shared by the operators around the product (ops_*.hip): eight-element vectors of
// bf16 or fp32 at any element alignment, and sums over waves and workgroups.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
// 16- and 8-byte accesses at an address that is only known to be aligned to an element: the
// hardware takes them, so rows of odd length need no path of their own but their last few elements
typedef u32x4_t __attribute__((aligned(2))) u32x4_any;
typedef u32x2_t __attribute__((aligned(2))) u32x2_any;

struct bf16_t {
  uint16_t bits;
};

__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ float float_of(uint32_t v) { return __builtin_bit_cast(float, v); }

// round to nearest even, lo in the low half (one v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const bf16_t *p) {
  return float_of((uint32_t)p->bits << 16);
}
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16_t *p, float v) {
  p->bits = (uint16_t)bf16_pair(v, 0.0f);
}

// Eight elements as they lie in memory.  at(i) gives them as fp32.
template <class T>
struct Vec8;
template <>
struct Vec8<bf16_t> {
  u32x4_t w;
  __device__ __forceinline__ float at(int i) const {
    return float_of((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void load(const bf16_t *p) { w = *(const u32x4_any *)p; }
  // a value that is not read again soon: the caches keep others instead
  __device__ __forceinline__ void load_once(const bf16_t *p) {
    w = __builtin_nontemporal_load((const u32x4_any *)p);
  }
  __device__ __forceinline__ void zero() { w = u32x4_t{0, 0, 0, 0}; }
  // the first n < 8 elements, zeros behind them
  __device__ __forceinline__ void load_some(const bf16_t *p, int n) {
    zero();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i / 2] |= (uint32_t)p[i].bits << (16 * (i & 1));
  }
};
template <>
struct Vec8<float> {
  u32x4_t lo, hi;
  __device__ __forceinline__ float at(int i) const {
    return float_of(i < 4 ? lo[i & 3] : hi[i & 3]);
  }
  __device__ __forceinline__ void load(const float *p) {
    lo = *(const u32x4_any *)p;
    hi = *(const u32x4_any *)(p + 4);
  }
  __device__ __forceinline__ void load_once(const float *p) {
    lo = __builtin_nontemporal_load((const u32x4_any *)p);
    hi = __builtin_nontemporal_load((const u32x4_any *)(p + 4));
  }
  __device__ __forceinline__ void zero() { lo = hi = u32x4_t{0, 0, 0, 0}; }
  __device__ __forceinline__ void load_some(const float *p, int n) {
    zero();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if (i < 4)
          lo[i & 3] = bits_of(p[i]);
        else
          hi[i & 3] = bits_of(p[i]);
      }
  }
};

// n >= 8 loads the whole vector, n <= 0 nothing
template <class T>
__device__ __forceinline__ void load8(Vec8<T> &v, const T *p, int64_t n) {
  if (n >= 8)
    v.load(p);
  else if (n > 0)
    v.load_some(p, (int)n);
  else
    v.zero();
}

__device__ __forceinline__ void store8_full(float *p, const float (&v)[8]) {
  *(u32x4_any *)p = u32x4_t{bits_of(v[0]), bits_of(v[1]), bits_of(v[2]), bits_of(v[3])};
  *(u32x4_any *)(p + 4) = u32x4_t{bits_of(v[4]), bits_of(v[5]), bits_of(v[6]), bits_of(v[7])};
}
__device__ __forceinline__ void store8_full(bf16_t *p, const float (&v)[8]) {
  *(u32x4_any *)p = u32x4_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                            bf16_pair(v[6], v[7])};
}
__device__ __forceinline__ void store8_once(float *p, const float (&v)[8]) {
  __builtin_nontemporal_store(
      u32x4_t{bits_of(v[0]), bits_of(v[1]), bits_of(v[2]), bits_of(v[3])}, (u32x4_any *)p);
  __builtin_nontemporal_store(
      u32x4_t{bits_of(v[4]), bits_of(v[5]), bits_of(v[6]), bits_of(v[7])}, (u32x4_any *)(p + 4));
}
__device__ __forceinline__ void store8_once(bf16_t *p, const float (&v)[8]) {
  __builtin_nontemporal_store(u32x4_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                      bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])},
                              (u32x4_any *)p);
}
template <class T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8], int64_t n) {
  if (n >= 8) {
    store8_full(p, v);
  } else if (n > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store1(p + i, v[i]);
  }
}

// Sum over the 64 lanes of a wave, in every lane, always in the same order.
template <class F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
// fp32: within rows of 16 lanes by rotation, then pairs of rows and halves swapped -- vector
// instructions only, where a shuffle goes through LDS
template <>
__device__ __forceinline__ float wave_sum(float v) {
#define DG_ROR(n) \
  v += float_of((uint32_t)__builtin_amdgcn_update_dpp(0, (int)bits_of(v), 0x120 + n, 0xF, 0xF, false))
  DG_ROR(8);
  DG_ROR(4);
  DG_ROR(2);
  DG_ROR(1);
#undef DG_ROR
  const auto p = __builtin_amdgcn_permlane16_swap(bits_of(v), bits_of(v), false, false);
  v = float_of(p[0]) + float_of(p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(bits_of(v), bits_of(v), false, false);
  return float_of(q[0]) + float_of(q[1]);
}

// Sums of N values over the WAVES waves of a workgroup.  `slot` is the LDS of one sum; a caller
// alternates between two, so that a wave that is ahead writes the next sum's slot while others
// still read this one's (one barrier a sum).
template <int WAVES, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*slot)[N], int wave, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (WAVES > 1) {
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slot[wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = slot[0][i];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) s += slot[w][i];
      v[i] = s;
    }
  }
}

}  // namespace dg
