// Quantisation to int8 with one fp32 scale a row (gemm_int8_quantize), of x, of its transpose (a scale
// a column of x), or of both:
//
//   s = max(amax / 127, 2^-120),  q = the exact quotient x / s rounded to even
//
// Rounding: t = x r + 1.5 2^23 with r near 1 / s leaves an integer next to x / s in t's last bits.  Which one
// matters next to a border between two, k + 1/2.
//  * rest = x - q s is exact in fp32 (a multiple of the smaller of x's and s's last places, at most s / 2
//    and a little in size), so |rest| against s / 2 says whether q is the nearest integer, and where it is a
//    tie.  fp32 x: four instructions a value; what is not right yet, one in some thousands, is mended
//    behind a branch.  (2^-120 as the smallest scale keeps every rest a normal multiple of 2^-149.)
//  * bf16 x: 127 x / amax of 8-bit mantissas is either on a border, which is common enough (x = amax / 2)
//    that most waves would take that branch, or 2^-16 of itself away from it.  So the rounding of s alone
//    decides: r is moved by 2^-18 to the side that s was rounded from.  One instruction a value; where s is
//    exact, a border is a tie, and the values go the other way.  (8192 x 4096, both sides: the second kernel
//    takes 28 us, and 5 more with the first way for all.)
//
//  * Rows alone: one pass, a row in the registers of a wave, of four or of sixteen.  (14336 x 4096 fp32 52.6
//    us, 5.6 TB/s.)
//  * Columns of up to 2048 rows: strips of columns with all their rows in a workgroup's registers, one launch;
//    with both sides, other workgroups of it take the rows, which they read by themselves.
//  * Columns of more, or rows of over 65536: a first kernel leaves maxima of rows and columns over parts of
//    x, at most 16 of a row and some 64 of a column; the second one's workgroups, 128 x 128 elements
//    each, take the largest of their rows' and columns' parts themselves.  It reads x again, from the
//    memory-side cache of 256 MB where x fits.
//
// Bound by memory, small ones by a launch and their trips to it.
#include "../../include/gemm_ops.h"
#include "ops_common.h"

#include <algorithm>

namespace dg {
namespace {

struct RowQuantArgs {
  const void *x;
  int64_t rows, cols, stride;
  uint8_t *codes, *codes_t;
  float *scales, *scales_t;
  int64_t pitch, pitch_t;
  uint32_t *row_parts, *col_parts;   // [part][rows], [part][cols]: bits of largest magnitudes
  int32_t parts_r, parts_c;
  int32_t wide, high;                // of a part: blocks of 128 columns, and rows
  int32_t col_tiles;
  int32_t groups;                    // of eight columns a strip
};

template <bool ONCE, class V>
__device__ __forceinline__ void put(V *p, V v) {   // ONCE: past the caches
  if constexpr (ONCE)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

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

// The scale of a row from the bits of its largest magnitude (NaN and infinity order above every number,
// so they carry through the integer maxima).
__device__ __forceinline__ float scale_of(uint32_t amax) {
  if (amax >= 0x7F800000u) return float_of(0x7FC00000u);
  return fmaxf(float_of(amax) / 127.0f, 0x1p-120f);
}

// Dividing by the scale of a row whose largest magnitude has the bits amax: r is negative where the rest of
// each value has to be looked at, and zero, as all codes are, for a NaN scale.
struct Divide {
  float s, r;
};
template <class T>
__device__ __forceinline__ Divide divide_by(uint32_t amax) {
  Divide d{scale_of(amax), 0.0f};
  if (d.s != d.s) return d;
  d.r = __builtin_amdgcn_rcpf(d.s);
  if constexpr (sizeof(T) == 2) {
    const float e = fmaf(-127.0f, d.s, float_of(amax));   // exact
    if (e == 0.0f || d.s == 0x1p-120f)
      d.r = -d.r;
    else
      d.r *= e > 0.0f ? 1.0f + 0x1p-18f : 1.0f - 0x1p-18f;
  } else {
    d.r = -d.r;
  }
  return d;
}

constexpr float kMagic = 0x1.8p23f;

__device__ __forceinline__ u32x2_t last_bytes(const uint32_t (&t)[8]) {
  u32x2_t c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(t[4 * h + 1], t[4 * h], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(t[4 * h + 3], t[4 * h + 2], 0x0C0C0400u);
    c[h] = lo | (hi << 16);
  }
  return c;
}
// Eight codes: element i is x(i) divided by d.
template <class T, class GetX>
__device__ __forceinline__ u32x2_t codes8(GetX x, const Divide &d) {
  uint32_t t[8];
  if (sizeof(T) == 2 && d.r >= 0.0f) {   // (a NaN in x, whose low bytes are zeros, stays one)
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = bits_of(fmaf(x(i), d.r, kMagic));
    return last_bytes(t);
  }
  const float half = 0.5f * d.s;
  bool off = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = fmaf(x(i), -d.r, kMagic);
    off |= fabsf(fmaf(kMagic - v, d.s, x(i))) >= half;
    t[i] = bits_of(v);
  }
  if (off) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = float_of(t[i]), rest = fmaf(kMagic - v, d.s, x(i));
      const bool wrong = fabsf(rest) > half || (fabsf(rest) == half && (t[i] & 1));
      if (wrong) t[i] = bits_of(v + (rest > 0.0f ? 1.0f : -1.0f));
    }
  }
  const uint32_t keep = d.s == d.s ? ~0u : 0u;
  const u32x2_t c = last_bytes(t);
  return u32x2_t{c[0] & keep, c[1] & keep};
}

template <class T>
__device__ __forceinline__ uint32_t largest(const Vec8<T> &v, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, bits_of(v.at(i)) & 0x7FFFFFFFu);
  return m;
}

// The bytes of the first n of eight codes; what lies past the matrix is stored as zeros.
__device__ __forceinline__ u32x2_t first_bytes(u32x2_t c, int64_t n) {
  if (n >= 8) return c;
  const uint64_t keep = n <= 0 ? 0 : ~0ull >> (64 - 8 * n);
  return u32x2_t{c[0] & (uint32_t)keep, c[1] & (uint32_t)(keep >> 32)};
}

// ---- rows alone -------------------------------------------------------------------------------

// ROWS rows of a workgroup with WAVES each, from `row0` on, V vectors of eight a lane.
template <class T, int ROWS, int WAVES, int V>
__device__ __forceinline__ void quantize_rows(const RowQuantArgs &a, int64_t row0) {
  constexpr int THREADS = WAVES * 64;
  __shared__ uint32_t slot[ROWS * WAVES];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, sub = ROWS > 1 ? wave / WAVES : 0;
  const int64_t row = row0 + sub;
  if (WAVES == 1 && row >= a.rows) return;
  const bool there = ROWS == 1 || row < a.rows;
  const int at = ((int)threadIdx.x - sub * THREADS) * 8;
  const T *const x = (const T *)a.x + row * a.stride;
  Vec8<T> v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t e = at + i * THREADS * 8;
    load8(v[i], x + e, there ? a.cols - e : 0);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = largest(v[i], m);
  m = row16_max(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  if constexpr (WAVES > 1) {
    if (lane == 0) slot[wave] = m;
    __syncthreads();
    if (!there) return;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = max(m, slot[sub * WAVES + w]);
  }
  const Divide d = divide_by<T>(m);
  if (at == 0) a.scales[row] = d.s;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t e = at + i * THREADS * 8;
    if (e >= a.pitch) break;
    *(u32x2_t *)(a.codes + row * a.pitch + e) = codes8<T>([&](int j) { return v[i].at(j); }, d);
  }
}

template <class T, int WAVES, int V>
__global__ void __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) rows_kernel(const RowQuantArgs a) {
  constexpr int ROWS = WAVES == 1 ? 4 : 1;
  quantize_rows<T, ROWS, WAVES, V>(a, (int64_t)blockIdx.x * ROWS);
}

// ---- columns of few rows --------------------------------------------------------------------------

// A workgroup takes 8 `groups` neighbouring columns with all their rows, a lane eight by eight of them.  ROWS: the
// workgroups behind take rows, four waves each, which they read by themselves.
template <class T, int THREADS, bool ROWS>
__global__ void __launch_bounds__(THREADS) strips_kernel(const RowQuantArgs a) {
  constexpr int WAVES = THREADS / 64;
  __shared__ uint32_t cmax[WAVES][128];
  __shared__ Divide dc[128];
  const int64_t strips = (a.cols + 8 * a.groups - 1) / (8 * a.groups);
  if (ROWS && blockIdx.x >= strips) {
    quantize_rows<T, WAVES / 4, 4, 8>(a, (blockIdx.x - strips) * (WAVES / 4));
    return;
  }
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int cg = tid & (a.groups - 1), rg = tid / a.groups;
  const int64_t c0 = ((int64_t)blockIdx.x * a.groups + cg) * 8, r0 = rg * 8;
  const int64_t nc = a.cols - c0, nr = a.rows - r0;
  Vec8<T> v[8];
#pragma unroll
  for (int p = 0; p < 8; ++p)
    load8(v[p], (const T *)a.x + (r0 + p) * a.stride + c0, p < nr ? nc : 0);
  uint32_t kmax[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    kmax[j] = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) kmax[j] = max(kmax[j], bits_of(v[p].at(j)) & 0x7FFFFFFFu);
  }
  for (int o = 32; o >= a.groups; o >>= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j) kmax[j] = max(kmax[j], (uint32_t)__shfl_xor((int)kmax[j], o, 64));
  if (lane < a.groups) {
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[wave][cg * 8 + j] = kmax[j];
  }
  __syncthreads();
  if (tid < 8 * a.groups) {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = max(m, cmax[w][tid]);
    dc[tid] = divide_by<T>(m);
    const int64_t c = (int64_t)blockIdx.x * a.groups * 8 + tid;
    if (c < a.cols) a.scales_t[c] = dc[tid].s;
  }
  __syncthreads();
  if (r0 >= a.pitch_t) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= nc) break;
    const u32x2_t c = codes8<T>([&](int i) { return v[i].at(j); }, dc[cg * 8 + j]);
    *(u32x2_t *)(a.codes_t + (c0 + j) * a.pitch_t + r0) = first_bytes(c, nr);
  }
}

// ---- maxima over parts, then tiles --------------------------------------------------------------

constexpr int kMostHigh = 4096;   // rows of a part: their maxima stay in LDS

template <class T, bool ROWS, bool COLS>
__global__ void __launch_bounds__(256) parts_kernel(const RowQuantArgs a) {
  __shared__ uint32_t rmax[ROWS ? kMostHigh : 1];
  __shared__ uint32_t cmax[4][128];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, cg = tid & 15, rg = tid >> 4;
  const int32_t pc = blockIdx.x % (uint32_t)a.parts_r, pr = blockIdx.x / (uint32_t)a.parts_r;
  const int64_t r0 = (int64_t)pr * a.high;
  const int high = (int)(a.rows - r0 < a.high ? a.rows - r0 : a.high);
  if constexpr (ROWS) {
    for (int i = tid; i < high; i += 256) rmax[i] = 0;
    __syncthreads();
  }
  const int64_t b1 = (int64_t)(pc + 1) * a.wide < a.col_tiles ? (int64_t)(pc + 1) * a.wide : a.col_tiles;
  for (int64_t b = (int64_t)pc * a.wide; b < b1; ++b) {
    const int64_t c0 = b * 128 + cg * 8, nc = a.cols - c0;
    uint32_t kmax[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) kmax[j] = 0;
    constexpr int AHEAD = 4;   // rows of a lane whose loads are in flight together
    for (int i0 = rg; i0 < high; i0 += 16 * AHEAD) {
      Vec8<T> v[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int i = i0 + 16 * u;
        load8(v[u], (const T *)a.x + (r0 + i) * a.stride + c0, i < high ? nc : 0);
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        if constexpr (COLS) {
#pragma unroll
          for (int j = 0; j < 8; ++j) kmax[j] = max(kmax[j], bits_of(v[u].at(j)) & 0x7FFFFFFFu);
        }
        if constexpr (ROWS) {
          const uint32_t m = row16_max(largest(v[u], 0));
          if (cg == 0 && i0 + 16 * u < high) atomicMax(&rmax[i0 + 16 * u], m);
        }
      }
    }
    if constexpr (COLS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        kmax[j] = max(kmax[j], (uint32_t)__shfl_xor((int)kmax[j], 16, 64));
        kmax[j] = max(kmax[j], (uint32_t)__shfl_xor((int)kmax[j], 32, 64));
      }
      __syncthreads();   // the block before has been read
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) cmax[wave][cg * 8 + j] = kmax[j];
      }
      __syncthreads();
      const int64_t c = b * 128 + tid;
      if (tid < 128 && c < a.cols)
        a.col_parts[pr * a.cols + c] =
            max(max(cmax[0][tid], cmax[1][tid]), max(cmax[2][tid], cmax[3][tid]));
    }
  }
  if constexpr (ROWS) {
    __syncthreads();
    for (int i = tid; i < high; i += 256) a.row_parts[pc * a.rows + r0 + i] = rmax[i];
  }
}

// The largest of the `parts` maxima of element i of `count`.
__device__ __forceinline__ uint32_t max_of_parts(const uint32_t *p, int parts, int64_t count,
                                                int64_t i) {
  uint32_t m = 0;
  for (int k = 0; k < parts; k += 8) {
    uint32_t u[8];   // loads in flight together
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = k + j < parts ? p[(k + j) * count + i] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, u[j]);
  }
  return m;
}

template <class T, bool ROWS, bool COLS, bool ONCE>
__global__ void __launch_bounds__(256) tiles_kernel(const RowQuantArgs a) {
  __shared__ Divide dr[128], dc[128];
  __shared__ __align__(16) uint8_t turned[COLS ? 128 * 128 : 16];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  // What the parts' kernel read last comes first and, where its parts divide among them, on the same XCD
  // (workgroup mod 8): part of it is still in that L2.
  const uint32_t back = gridDim.x - 1 - blockIdx.x;
  int64_t ct = blockIdx.x % (uint32_t)a.col_tiles, rt = back / (uint32_t)a.col_tiles;
  if (a.col_tiles % (8 * a.wide) == 0) {
    const uint32_t j = (uint32_t)ct / 8;
    ct = (j / a.wide * 8 + (uint32_t)ct % 8) * a.wide + j % a.wide;
  }
  const int64_t c0 = ct * 128 + cg * 8, r0 = rt * 128 + rg * 8;
  const int64_t nc = a.cols - c0, nr = a.rows - r0;
  Vec8<T> v[8];
#pragma unroll
  for (int p = 0; p < 8; ++p)
    load8(v[p], (const T *)a.x + (r0 + p) * a.stride + c0, p < nr ? nc : 0);
  if (tid < 128) {
    const int64_t r = rt * 128 + tid;
    if (ROWS && r < a.rows) {
      const Divide d = divide_by<T>(max_of_parts(a.row_parts, a.parts_r, a.rows, r));
      dr[tid] = d;
      if (ct == 0) a.scales[r] = d.s;
    }
  } else {
    const int64_t c = ct * 128 + tid - 128;
    if (COLS && c < a.cols) {
      const Divide d = divide_by<T>(max_of_parts(a.col_parts, a.parts_c, a.cols, c));
      dc[tid - 128] = d;
      if (rt == 0) a.scales_t[c] = d.s;
    }
  }
  __syncthreads();
  if constexpr (ROWS) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const u32x2_t c = first_bytes(
          codes8<T>([&](int i) { return v[p].at(i); }, p < nr ? dr[rg * 8 + p] : Divide{1.0f, 0.0f}), nc);
      if (p < nr && c0 < a.pitch) put<ONCE>((u32x2_t *)(a.codes + (r0 + p) * a.pitch + c0), c);
    }
  }
  if constexpr (COLS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = cg * 8 + j;
      const u32x2_t c = first_bytes(
          codes8<T>([&](int i) { return v[i].at(j); }, j < nc ? dc[col] : Divide{1.0f, 0.0f}), nr);
      *(u32x2_t *)&turned[col * 128 + (((rg >> 1) ^ (cg & 7)) << 4) + (rg & 1) * 8] = c;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = i * 32 + (tid >> 3), chunk = tid & 7;
      const u32x4_t w = *(const u32x4_t *)&turned[col * 128 + ((chunk ^ ((col >> 3) & 7)) << 4)];
      const int64_t row_t = ct * 128 + col, at = rt * 128 + chunk * 16;
      if (row_t < a.cols && at < a.pitch_t) put<ONCE>((u32x4_t *)(a.codes_t + row_t * a.pitch_t + at), w);
    }
  }
}

// ---- choice -----------------------------------------------------------------------------------

constexpr int64_t kMostInRow = 65536;   // columns that sixteen waves hold, eight vectors a lane

// Elements from which on the tiles' codes go past the caches, which x then has for itself.  (us so and not:
// 8192 x 4096 bf16, both sides 42, 45; 4096 x 4096 22.6, 25.2; 3001 x 3001 fp32 26.7, 28.0; 2048 x 4096 bf16
// alike.)
constexpr int64_t kPassing = 8 << 20;
template <class T>
void launch_rows(const RowQuantArgs &a, hipStream_t s) {
  const dim3 grid((uint32_t)a.rows), four((uint32_t)((a.rows + 3) / 4));
  const int64_t n = a.cols;
#define DG_ROWS(grid, waves, v) \
  hipLaunchKernelGGL((rows_kernel<T, waves, v>), grid, dim3(waves == 1 ? 256 : waves * 64), 0, s, a)
  if (n <= 512)
    DG_ROWS(four, 1, 1);
  else if (n <= 1024)
    DG_ROWS(four, 1, 2);
  else if (n <= 2048)
    DG_ROWS(grid, 4, 1);
  else if (n <= 4096)
    DG_ROWS(grid, 4, 2);
  else if (n <= 8192)
    DG_ROWS(grid, 4, 4);
  else if (n <= 16384)
    DG_ROWS(grid, 16, 2);
  else if (n <= 32768)
    DG_ROWS(grid, 16, 4);
  else
    DG_ROWS(grid, 16, 8);
#undef DG_ROWS
}

template <class T, bool ROWS, bool COLS>
void launch_parts(const RowQuantArgs &a, hipStream_t s) {
  const uint32_t parts = (uint32_t)a.parts_r * (uint32_t)a.parts_c;
  const uint32_t tiles = (uint32_t)((a.rows + 127) / 128) * (uint32_t)a.col_tiles;
  hipLaunchKernelGGL((parts_kernel<T, ROWS, COLS>), dim3(parts), dim3(256), 0, s, a);
  if (a.rows * a.cols >= kPassing)
    hipLaunchKernelGGL((tiles_kernel<T, ROWS, COLS, true>), dim3(tiles), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((tiles_kernel<T, ROWS, COLS, false>), dim3(tiles), dim3(256), 0, s, a);
}
// Columns in strips where a workgroup has room for all rows; 0: not in strips.  (us in strips and on tiles: 2 x
// 20564 bf16, columns, 5.8, 16.5; 300 x 9000 bf16, both sides, 9.6, 17.3; 1024 x 4096 10.3, 14.8; 512 x 16384 16.4,
// 21.6; 2048 x 4096 16.9, 16.5.  Four waves or sixteen: 600 x 600 5.2, 6.8, 300 x 40000 13.6, 15.0, 1000 x
// 8192 19, 14.)
struct Strip {
  int threads, groups;
};
Strip strip_of(int64_t rows, int64_t cols, bool rows_side, bool cols_side) {
  const int64_t high = (rows + 15) / 16 * 16;   // a lane has eight of them
  if (!cols_side || high > 2048 || cols > (rows_side ? kMostInRow : 1 << 22)) return {0, 0};
  const int threads = high <= 512 || (high <= 1024 && cols <= 2048) ? 256 : 1024;
  int groups = 16;
  while (threads / groups * 8 < high) groups /= 2;
  while (groups > 2 && cols < 8 * groups * 128) groups /= 2;   // 128 workgroups where there is room
  return {threads, groups};
}
constexpr int64_t kMostWithStrips = 16384;   // columns of a row that four waves hold, eight vectors a lane

template <class T, int THREADS, bool ROWS>
void launch_strips(const RowQuantArgs &a, hipStream_t s) {
  const int64_t strips = (a.cols + 8 * a.groups - 1) / (8 * a.groups);
  const int64_t rows = ROWS ? (a.rows + THREADS / 256 - 1) / (THREADS / 256) : 0;
  hipLaunchKernelGGL((strips_kernel<T, THREADS, ROWS>), dim3((uint32_t)(strips + rows)), dim3(THREADS), 0, s,
                     a);
}

template <class T>
void launch(RowQuantArgs a, hipStream_t s) {
  const Strip strip = strip_of(a.rows, a.cols, a.codes, a.codes_t);
  const bool together = a.codes && a.cols <= kMostWithStrips;
  a.groups = strip.groups;
  if (strip.threads && a.codes && !together) launch_rows<T>(a, s);
  if (strip.threads == 256)
    together ? launch_strips<T, 256, true>(a, s) : launch_strips<T, 256, false>(a, s);
  else if (strip.threads)
    together ? launch_strips<T, 1024, true>(a, s) : launch_strips<T, 1024, false>(a, s);
  else if (!a.codes_t && a.cols <= kMostInRow)
    launch_rows<T>(a, s);
  else if (!a.codes_t)
    launch_parts<T, true, false>(a, s);
  else if (a.codes)
    launch_parts<T, true, true>(a, s);
  else
    launch_parts<T, false, true>(a, s);
}

struct Parts {
  int32_t parts_r, parts_c, wide, high;   // parts_r: of a row, so along the columns
  size_t row_bytes, col_bytes;
};
Parts parts_of(int64_t rows, int64_t cols, bool rows_side, bool cols_side) {
  Parts p{};
  if ((!cols_side && cols <= kMostInRow) || strip_of(rows, cols, rows_side, cols_side).threads) return p;
  const int64_t ct = (cols + 127) / 128;
  p.wide = (int32_t)((ct + 15) / 16);
  p.parts_r = (int32_t)((ct + p.wide - 1) / p.wide);
  int64_t parts_c = std::min<int64_t>({64, 512 / p.parts_r, (rows + 31) / 32});
  parts_c = std::max(parts_c, (rows + kMostHigh - 1) / kMostHigh);
  p.high = (int32_t)((rows + parts_c - 1) / parts_c);
  p.parts_c = (int32_t)((rows + p.high - 1) / p.high);
  if (rows_side) p.row_bytes = (size_t)p.parts_r * (size_t)rows * 4;
  if (cols_side) p.col_bytes = (size_t)p.parts_c * (size_t)cols * 4;
  return p;
}

int check(int64_t rows, int64_t cols, bool rows_side, bool cols_side) {
  if (rows < 0 || cols < 0 || (!rows_side && !cols_side)) return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_OK;
  // 2^32 work-items, in tiles and in rows
  if ((rows + 127) / 128 > 0xFFFFFF / ((cols + 127) / 128)) return GEMM_ERR_UNSUPPORTED;
  if (!cols_side && rows > 0xFFFFFF / 4) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

struct Span {
  uintptr_t first, last;
};
Span span(const void *p, uintptr_t bytes) {
  return p ? Span{(uintptr_t)p, (uintptr_t)p + bytes} : Span{0, 0};
}

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace
}  // namespace dg

extern "C" int gemm_int8_quantize_workspace(int64_t rows, int64_t cols, int rows_side,
                                            int cols_side, size_t *bytes) {
  using namespace dg;
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  const int st = check(rows, cols, rows_side != 0, cols_side != 0);
  if (st != GEMM_OK) return st;
  *bytes = 0;
  if (rows == 0 || cols == 0) return GEMM_OK;
  const Parts p = parts_of(rows, cols, rows_side != 0, cols_side != 0);
  *bytes = p.row_bytes + p.col_bytes;
  return GEMM_OK;
}

extern "C" int gemm_int8_quantize(const void *x, int dtype, int64_t rows, int64_t cols,
                                  int64_t stride, void *codes, int64_t pitch, float *scales,
                                  void *codes_t, int64_t pitch_t, float *scales_t, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  using namespace dg;
  if (dtype != GEMM_BF16 && dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
  const int st = check(rows, cols, codes != nullptr, codes_t != nullptr);
  if (st != GEMM_OK) return st;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (!x || (codes && !scales) || (codes_t && !scales_t)) return GEMM_ERR_INVALID_ARG;
  if (stride < 0 || (rows > 1 && stride < cols && stride != 0)) return GEMM_ERR_INVALID_ARG;
  if (codes && (pitch < cols || pitch % 16 || pitch >= cols + 16)) return GEMM_ERR_INVALID_ARG;
  if (codes_t && (pitch_t < rows || pitch_t % 16 || pitch_t >= rows + 16))
    return GEMM_ERR_INVALID_ARG;
  const Parts p = parts_of(rows, cols, codes != nullptr, codes_t != nullptr);
  const size_t need = p.row_bytes + p.col_bytes;
  if (need && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
  if (!aligned(x, dtype == GEMM_BF16 ? 2 : 4) || !aligned(codes, 16) || !aligned(codes_t, 16) ||
      !aligned(scales, 4) || !aligned(scales_t, 4) || !aligned(workspace, 4))
    return GEMM_ERR_ALIGNMENT;
  // workgroups read x again after others have written: nothing of what is written may overlap anything else
  const uintptr_t es = dtype == GEMM_BF16 ? 2 : 4;
  const Span spans[] = {
      span(x, ((uintptr_t)(rows - 1) * (uintptr_t)stride + (uintptr_t)cols) * es),
      span(codes, (uintptr_t)rows * (uintptr_t)pitch),
      span(codes ? scales : nullptr, (uintptr_t)rows * 4),
      span(codes_t, (uintptr_t)cols * (uintptr_t)pitch_t),
      span(codes_t ? scales_t : nullptr, (uintptr_t)cols * 4),
      span(workspace, need),
  };
  for (int i = 0; i < 6; ++i)
    for (int j = i + 1; j < 6; ++j)
      if (spans[i].first < spans[j].last && spans[j].first < spans[i].last) return GEMM_ERR_INVALID_ARG;
  RowQuantArgs a{};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.stride = stride;
  a.codes = (uint8_t *)codes;
  a.codes_t = (uint8_t *)codes_t;
  a.scales = scales;
  a.scales_t = scales_t;
  a.pitch = pitch;
  a.pitch_t = pitch_t;
  a.row_parts = (uint32_t *)workspace;
  a.col_parts = (uint32_t *)((char *)workspace + p.row_bytes);
  a.parts_r = p.parts_r;
  a.parts_c = p.parts_c;
  a.wide = p.wide;
  a.high = p.high;
  a.col_tiles = (int32_t)((cols + 127) / 128);
  if (dtype == GEMM_BF16)
    launch<bf16_t>(a, (hipStream_t)stream);
  else
    launch<float>(a, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}
