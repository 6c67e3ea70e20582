// Block quantisation to e4m3 (gemm_block_quantize): codes q and one fp32 scale s per block of 128
// (1 x 128 of a row, or 128 x 128), x ~ s q, of x, of its transpose, or of both from one read.
//
//   s = max(amax / 448, 2^-126), or the next power of two that is not below it;  q = e4m3(x / s)
//
// One workgroup takes one 128 x 128 tile: it holds whole blocks of every kind, so the maxima of
// rows, columns and the tile come from one read, kept in registers as it was loaded (a thread has
// an 8 x 8 corner: 16-byte loads, and eight rows that make eight bytes of a transposed row).  The
// transposed codes go through 16 KB of LDS to leave as whole 128-byte lines.
//
// Rounding: the code is that of the exact quotient x / s, and x * (1 / s) in fp32 is within 2^-22 of
// that, which matters next to a border between two codes.
//  * A power of two divides exactly.
//  * fp32 x: the product is converted twice, moved down and up by 2^-21; only where the two codes
//    differ (one vector of eight in 10^4 lanes) is the quotient's side of the border found exactly.
//  * bf16 x: quotients on a border are common (0.3 % of values), but 448 x / amax of 8-bit mantissas
//    is either on a border or 2^-13 away, so the rounding of s alone decides: the reciprocal is moved
//    by 2^-15 to the side that s was rounded from, and the product rounded to 17 bits, which puts
//    those on the border exactly there where s is exact.  (8192 x 4096, both sides: 73 us by the
//    fp32 way, where nearly every wave met a border, 27 us with powers of two.)
//
// Bound by memory: reads each element once and writes each code once.
#include "../../include/gemm_ops.h"
#include "ops_common.h"

namespace dg {
namespace {

struct QuantArgs {
  const void *x;
  int64_t rows, cols, stride;
  uint8_t *codes, *codes_t;
  float *scales, *scales_t;
  int64_t pitch, pitch_t, spitch, spitch_t;
  int32_t col_tiles;
};

// Largest over the 16 lanes of a DPP row, in each of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
#define DG_ROR(n) \
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xF, 0xF, false))
  DG_ROR(8);
  DG_ROR(4);
  DG_ROR(2);
  DG_ROR(1);
#undef DG_ROR
  return v;
}

// The scale of a block from the bits of its largest magnitude (NaN and infinity order above every
// number, so they carry through the integer maxima).
template <bool POW2>
__device__ __forceinline__ float scale_of(uint32_t amax) {
  if (amax >= 0x7F800000u) return float_of(0x7FC00000u);
  if constexpr (POW2) {
    // amax = 1.f * 2^E and 448 = 1.75 * 2^8: the power is 2^(E - 8), one more if 1.f > 1.75
    const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u);
    return float_of((uint32_t)max(e, 1) << 23);
  } else {
    // the quotient rounded to nearest: one step of correction makes amax * (1 / 448) exact
    const float a = float_of(amax), y = 1.0f / 448.0f;
    const float q = a * y;
    return fmaxf(fmaf(fmaf(-448.0f, q, a), y, q), 0x1p-126f);
  }
}

// How elements are divided by a scale of a block whose largest magnitude has the bits amax.
template <class T, bool POW2>
struct Divide;
template <class T>
struct Divide<T, true> {
  float r;
  __device__ __forceinline__ Divide(float s, uint32_t)
      : r(s == s ? float_of(0x7F000000u - bits_of(s)) : s) {}   // exact: 2^-e, and NaN for NaN
  __device__ __forceinline__ float operator()(float x) const { return x * r; }
};
template <>
struct Divide<bf16_t, false> {
  float r;
  __device__ __forceinline__ Divide(float s, uint32_t amax) {
    const float e = fmaf(-448.0f, s, float_of(amax));   // exact; s = 2^-126 divides exactly
    r = __builtin_amdgcn_rcpf(s);
    if (s > 0x1p-126f) r *= e > 0.0f ? 1.0f + 0x1p-15f : e < 0.0f ? 1.0f - 0x1p-15f : 1.0f;
  }
  __device__ __forceinline__ float operator()(float x) const {
    return float_of((bits_of(x * r) + 0x40u) & ~0x7Fu);
  }
};
template <>
struct Divide<float, false> {
  float s, lo, hi;
  __device__ __forceinline__ Divide(float scale, uint32_t) : s(scale) {
    const float r = __builtin_amdgcn_rcpf(s);
    lo = r * (1.0f - 0x1p-21f);
    hi = r * (1.0f + 0x1p-21f);
  }
};

__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// A float on the same side of every border between two codes as x / s: the quotient cut towards
// zero, its last bit set if anything was cut (borders have that bit clear).
__device__ __noinline__ float sticky_quotient(float x, float s) {
  float q = x * (1.0f / s);
  q = fmaf(fmaf(-q, s, x), 1.0f / s, q);   // less than one step off
  if (q == 0.0f || q != q) return q;
  const double r = (double)x - (double)q * (double)s;  // the product has 48 bits: r's sign is exact
  if (r == 0.0) return q;
  uint32_t u = bits_of(q);
  if ((r > 0.0) != (q > 0.0f)) --u;
  return float_of(u | 1u);
}

// Eight codes: element i is x(i) divided by d.
template <class T, bool POW2, class GetX>
__device__ __forceinline__ u32x2_t codes8(GetX x, const Divide<T, POW2> &d) {
  u32x2_t lo;
  if constexpr (POW2 || sizeof(T) == 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      lo[h] = cvt4(d(x(4 * h)), d(x(4 * h + 1)), d(x(4 * h + 2)), d(x(4 * h + 3)));
  } else {
    u32x2_t hi;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lo[h] = cvt4(x(4 * h) * d.lo, x(4 * h + 1) * d.lo, x(4 * h + 2) * d.lo, x(4 * h + 3) * d.lo);
      hi[h] = cvt4(x(4 * h) * d.hi, x(4 * h + 1) * d.hi, x(4 * h + 2) * d.hi, x(4 * h + 3) * d.hi);
    }
    if (((lo[0] ^ hi[0]) | (lo[1] ^ hi[1])) != 0) {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = sticky_quotient(x(i), d.s);
      lo[0] = cvt4(q[0], q[1], q[2], q[3]);
      lo[1] = cvt4(q[4], q[5], q[6], q[7]);
    }
  }
  return lo;
}

// The bytes of the first n of eight codes: what lies past the matrix is stored as zeros, also in
// a block whose scale is NaN.
__device__ __forceinline__ u32x2_t first_bytes(u32x2_t c, int64_t n) {
  if (n >= 8) return c;
  const uint64_t keep = n <= 0 ? 0 : ~0ull >> (64 - 8 * n);
  return u32x2_t{c[0] & (uint32_t)keep, c[1] & (uint32_t)(keep >> 32)};
}

enum { SIDE_ROWS = 1, SIDE_COLS = 2 };

template <class T, int SIDES, bool TILE, bool POW2>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a) {
  __shared__ uint32_t cmax[4][128];
  __shared__ __align__(16) uint8_t turned[(SIDES & SIDE_COLS) ? 128 * 128 : 16];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int cg = tid & 15, rg = tid >> 4;
  const int64_t ct = blockIdx.x % (uint32_t)a.col_tiles, rt = blockIdx.x / (uint32_t)a.col_tiles;
  const int64_t c0 = ct * 128 + cg * 8, r0 = rt * 128 + rg * 8;
  const int64_t nc = a.cols - c0, nr = a.rows - r0;   // elements of the corner inside x

  Vec8<T> v[8];
#pragma unroll
  for (int p = 0; p < 8; ++p)
    load8(v[p], (const T *)a.x + (r0 + p) * a.stride + c0, p < nr ? nc : 0);

  uint32_t rmax[8], kmax[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) rmax[j] = kmax[j] = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = bits_of(v[p].at(j)) & 0x7FFFFFFFu;
      rmax[p] = max(rmax[p], u);
      kmax[j] = max(kmax[j], u);
    }

  if constexpr (TILE) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) m = max(m, rmax[p]);
    m = row16_max(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    if (lane == 0) cmax[0][wave] = m;
    __syncthreads();
    m = max(max(cmax[0][0], cmax[0][1]), max(cmax[0][2], cmax[0][3]));
    const float s = scale_of<POW2>(m);
    const Divide<T, POW2> d(s, m);
    if (tid == 0) {
      if (SIDES & SIDE_ROWS) a.scales[ct * a.spitch + rt] = s;
      if (SIDES & SIDE_COLS) a.scales_t[rt * a.spitch_t + ct] = s;
    }
    u32x2_t c[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      c[p] = codes8<T, POW2>([&](int i) { return v[p].at(i); }, d);
      c[p] = p < nr ? first_bytes(c[p], nc) : u32x2_t{0, 0};
      if ((SIDES & SIDE_ROWS) && p < nr && c0 < a.pitch)
        *(u32x2_t *)(a.codes + (r0 + p) * a.pitch + c0) = c[p];
    }
    if constexpr ((SIDES & SIDE_COLS) != 0) {
      // 8 x 8 bytes turned in registers: byte j of the eight rows is one row of the transpose
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int h = j >> 2, b = j & 3;
        const uint32_t sel = 0x0C0C0400u + 0x0101u * b;   // byte b of each of two words
        u32x2_t t;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t lo = __builtin_amdgcn_perm(c[4 * q + 1][h], c[4 * q][h], sel);
          const uint32_t hi = __builtin_amdgcn_perm(c[4 * q + 3][h], c[4 * q + 2][h], sel);
          t[q] = lo | (hi << 16);
        }
        *(u32x2_t *)&turned[(cg * 8 + j) * 128 + (((rg >> 1) ^ (cg & 7)) << 4) + (rg & 1) * 8] = t;
      }
    }
  } else {
    if constexpr ((SIDES & SIDE_COLS) != 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        kmax[j] = max(kmax[j], (uint32_t)__shfl_xor((int)kmax[j], 16, 64));
        kmax[j] = max(kmax[j], (uint32_t)__shfl_xor((int)kmax[j], 32, 64));
      }
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) cmax[wave][cg * 8 + j] = kmax[j];
      }
    }
    if constexpr ((SIDES & SIDE_ROWS) != 0) {
      float own = 0.0f;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const uint32_t m = row16_max(rmax[p]);
        const float s = scale_of<POW2>(m);
        own = cg == p ? s : own;
        const u32x2_t c = codes8<T, POW2>([&](int i) { return v[p].at(i); }, Divide<T, POW2>(s, m));
        if (p < nr && c0 < a.pitch)
          *(u32x2_t *)(a.codes + (r0 + p) * a.pitch + c0) = first_bytes(c, nc);
      }
      if (cg < 8 && cg < nr) a.scales[ct * a.spitch + r0 + cg] = own;
    }
    if constexpr ((SIDES & SIDE_COLS) != 0) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = cg * 8 + j;
        const uint32_t m =
            max(max(cmax[0][col], cmax[1][col]), max(cmax[2][col], cmax[3][col]));
        const float s = scale_of<POW2>(m);
        if (tid < 16 && j < nc) a.scales_t[rt * a.spitch_t + c0 + j] = s;
        const u32x2_t c = codes8<T, POW2>([&](int i) { return v[i].at(j); }, Divide<T, POW2>(s, m));
        *(u32x2_t *)&turned[col * 128 + (((rg >> 1) ^ (cg & 7)) << 4) + (rg & 1) * 8] =
            first_bytes(c, nr);
      }
    }
  }
  if constexpr ((SIDES & SIDE_COLS) != 0) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = i * 32 + (tid >> 3), chunk = tid & 7;
      const u32x4_t w = *(const u32x4_t *)&turned[col * 128 + ((chunk ^ ((col >> 3) & 7)) << 4)];
      const int64_t row_t = ct * 128 + col, at = rt * 128 + chunk * 16;
      if (row_t < a.cols && at < a.pitch_t) *(u32x4_t *)(a.codes_t + row_t * a.pitch_t + at) = w;
    }
  }
}

template <class T, int SIDES, bool TILE>
void launch_pow2(const QuantArgs &a, uint32_t grid, bool pow2, hipStream_t s) {
  if (pow2)
    hipLaunchKernelGGL((quantize_kernel<T, SIDES, TILE, true>), dim3(grid), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((quantize_kernel<T, SIDES, TILE, false>), dim3(grid), dim3(256), 0, s, a);
}
template <class T, int SIDES>
void launch_block(const QuantArgs &a, uint32_t grid, bool tile, bool pow2, hipStream_t s) {
  if (tile)
    launch_pow2<T, SIDES, true>(a, grid, pow2, s);
  else
    launch_pow2<T, SIDES, false>(a, grid, pow2, s);
}
template <class T>
void launch_sides(const QuantArgs &a, uint32_t grid, bool tile, bool pow2, hipStream_t s) {
  if (a.codes && a.codes_t)
    launch_block<T, SIDE_ROWS | SIDE_COLS>(a, grid, tile, pow2, s);
  else if (a.codes)
    launch_block<T, SIDE_ROWS>(a, grid, tile, pow2, s);
  else
    launch_block<T, SIDE_COLS>(a, grid, tile, pow2, s);
}

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace
}  // namespace dg

extern "C" int gemm_block_quantize(const void *x, int dtype, int64_t rows, int64_t cols,
                                   int64_t stride, int block, int pow2, void *codes,
                                   int64_t pitch, float *scales, int64_t scale_pitch,
                                   void *codes_t, int64_t pitch_t, float *scales_t,
                                   int64_t scale_pitch_t, void *stream) {
  using namespace dg;
  if (rows < 0 || cols < 0 || (dtype != GEMM_BF16 && dtype != GEMM_F32)) return GEMM_ERR_INVALID_ARG;
  if (block != GEMM_BLOCK_ROW && block != GEMM_BLOCK_TILE) return GEMM_ERR_INVALID_ARG;
  if (!codes && !codes_t) return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_OK;
  const int64_t rt = (rows + 127) / 128, ct = (cols + 127) / 128;
  const bool tile = block == GEMM_BLOCK_TILE;
  if (!x || (codes && !scales) || (codes_t && !scales_t)) return GEMM_ERR_INVALID_ARG;
  if (stride < 0 || (rows > 1 && stride < cols && stride != 0)) return GEMM_ERR_INVALID_ARG;
  if (codes && (pitch < cols || pitch % 16 || pitch >= cols + 16 ||
                (ct > 1 && scale_pitch < (tile ? rt : rows))))
    return GEMM_ERR_INVALID_ARG;
  if (codes_t && (pitch_t < rows || pitch_t % 16 || pitch_t >= rows + 16 ||
                  (rt > 1 && scale_pitch_t < (tile ? ct : cols))))
    return GEMM_ERR_INVALID_ARG;
  if (rt > 0xFFFFFF / ct) return GEMM_ERR_UNSUPPORTED;   // 2^32 work-items
  if (!aligned(x, dtype == GEMM_BF16 ? 2 : 4) || !aligned(codes, 16) || !aligned(codes_t, 16) ||
      !aligned(scales, 4) || !aligned(scales_t, 4))
    return GEMM_ERR_ALIGNMENT;
  QuantArgs a{x, rows, cols, stride, (uint8_t *)codes, (uint8_t *)codes_t, scales, scales_t,
              pitch, pitch_t, scale_pitch, scale_pitch_t, (int32_t)ct};
  const uint32_t grid = (uint32_t)(rt * ct);
  if (dtype == GEMM_BF16)
    launch_sides<bf16_t>(a, grid, tile, pow2 != 0, (hipStream_t)stream);
  else
    launch_sides<float>(a, grid, tile, pow2 != 0, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}
