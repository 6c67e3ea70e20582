// Layer norm (gemm_layer_norm) and its backward pass (gemm_layer_norm_backward).
//
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps),  y = (x - mean) rstd w + b
//   h = (x - mean) rstd,  g = dy w,  dx = rstd (g - mean(g) - h mean(g h)),
//   dw = sum over rows of dy h,  db = sum over rows of dy
//
// A row is held in the registers of the waves that work on it, so x (and dy) are read once: the
// squares are summed about the mean, not as a difference of two large sums.  Workgroups stay for
// many rows: w and b, and the sums of dw and db for a thread's columns, stay in registers too, and
// the next row's loads are in flight while the present one is summed.  A workgroup's dw and db go
// to the workspace as one row of partial sums; a second kernel adds those in a fixed order, so
// results do not change from run to run.  Few rows take one launch.  All sums are in fp32.
//
// Bound by memory: forward 2, backward 3 elements a column.
#include "../../include/gemm_ops.h"
#include "ops_common.h"

#include <type_traits>

namespace dg {
namespace {

struct NormArgs {
  const void *x, *w, *b, *dy;
  void *y;              // forward: y, backward: dx
  float *mean, *rstd;   // written forward, read backward
  float *partials;      // backward: one row of 2 x cols sums per workgroup
  int64_t rows, cols, stride, dstride;
  int64_t row_groups;   // norm_grad_few_kernel
  float eps;
};

// WAVES waves hold a row as NV vectors of eight a thread; one wave a row: four rows a workgroup.
template <int WAVES>
struct Geo {
  static constexpr int ROWS = WAVES == 1 ? 4 : 1;
  static constexpr int THREADS = WAVES * 64 * ROWS;
};

template <class T, class W, int WAVES, int NV>
__global__ void __launch_bounds__(Geo<WAVES>::THREADS) norm_kernel(const NormArgs a) {
  constexpr int ROWS = Geo<WAVES>::ROWS, SPAN = WAVES * 64;
  __shared__ float red[2][WAVES][1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = ROWS == 1 ? threadIdx.x : lane;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS == 1 ? 0 : wave);

  float w[NV][8], b[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t e = (int64_t)(v * SPAN + t) * 8;
    Vec8<W> q;
    load8(q, (const W *)a.w + e, a.cols - e);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[v][i] = q.at(i);
    load8(q, (const W *)a.b + e, a.b ? a.cols - e : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[v][i] = q.at(i);
  }
  const float n = (float)a.cols;
  Vec8<T> next[NV];
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t e = (int64_t)(v * SPAN + t) * 8;
      load8(next[v], (const T *)a.x + r * a.stride + e, a.cols - e);
    }
  };
  // three vectors of fp32 leave no room for the next row's
  constexpr bool AHEAD = NV < 3 || sizeof(T) == 2;
  if (AHEAD && row < a.rows) fetch(row);
  for (; row < a.rows; row += step) {
    if constexpr (!AHEAD) fetch(row);
    Vec8<T> x[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) x[v] = next[v];
    if (AHEAD && row + step < a.rows) fetch(row + step);
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += x[v].at(i);
    group_sum<WAVES, 1>(s, red[0], wave, lane);
    const float mean = s[0] / n;
    float q[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t left = a.cols - (int64_t)(v * SPAN + t) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = i < left ? x[v].at(i) - mean : 0.0f;
        q[0] = fmaf(d, d, q[0]);
      }
    }
    group_sum<WAVES, 1>(q, red[1], wave, lane);
    const float rstd = 1.0f / sqrtf(q[0] / n + a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t e = (int64_t)(v * SPAN + t) * 8;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf((x[v].at(i) - mean) * rstd, w[v][i], b[v][i]);
      store8((T *)a.y + row * a.cols + e, y, a.cols - e);
    }
    if (t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
  }
}

// Rows too long for the registers: three passes over each, which the caches mostly serve.
template <class T, class W>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
  __shared__ float red[2][16][1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const float n = (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *x = (const T *)a.x + row * a.stride;
    Vec8<T> v;
    float s[1] = {0.0f}, q[1] = {0.0f};
    for (int64_t e = threadIdx.x * 8; e < a.cols; e += 8192) {
      load8(v, x + e, a.cols - e);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v.at(i);
    }
    group_sum<16, 1>(s, red[0], wave, lane);
    const float mean = s[0] / n;
    for (int64_t e = threadIdx.x * 8; e < a.cols; e += 8192) {
      load8(v, x + e, a.cols - e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = i < a.cols - e ? v.at(i) - mean : 0.0f;
        q[0] = fmaf(d, d, q[0]);
      }
    }
    group_sum<16, 1>(q, red[1], wave, lane);
    const float rstd = 1.0f / sqrtf(q[0] / n + a.eps);
    for (int64_t e = threadIdx.x * 8; e < a.cols; e += 8192) {
      load8(v, x + e, a.cols - e);
      Vec8<W> w, b;
      load8(w, (const W *)a.w + e, a.cols - e);
      load8(b, (const W *)a.b + e, a.b ? a.cols - e : 0);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf((v.at(i) - mean) * rstd, w.at(i), b.at(i));
      store8((T *)a.y + row * a.cols + e, y, a.cols - e);
    }
    if (threadIdx.x == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
  }
}

template <class T, class W, int WAVES, int NV>
__global__ void __launch_bounds__(Geo<WAVES>::THREADS) norm_grad_kernel(const NormArgs a) {
  constexpr int ROWS = Geo<WAVES>::ROWS, SPAN = WAVES * 64;
  __shared__ float red[2][WAVES][2];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = ROWS == 1 ? threadIdx.x : lane;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS == 1 ? 0 : wave);

  float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t e = (int64_t)(v * SPAN + t) * 8;
    Vec8<W> q;
    load8(q, (const W *)a.w + e, a.cols - e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[v][i] = q.at(i);
      dw[v][i] = db[v][i] = 0.0f;
    }
  }
  const float inv_n = 1.0f / (float)a.cols;
  // four vectors of fp32 x and dy leave no room for the next row's
  constexpr bool AHEAD = NV < 4 || sizeof(T) == 2;
  Vec8<T> nx[NV], ng[NV];
  float nmean = 0.0f, nrstd = 0.0f;
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t e = (int64_t)(v * SPAN + t) * 8;
      load8(nx[v], (const T *)a.x + r * a.stride + e, a.cols - e);
      load8(ng[v], (const T *)a.dy + r * a.dstride + e, a.cols - e);
    }
    nmean = a.mean[r];
    nrstd = a.rstd[r];
  };
  if (AHEAD && row < a.rows) fetch(row);
  int turn = 0;
  for (; row < a.rows; row += step, turn ^= 1) {
    if constexpr (!AHEAD) fetch(row);
    Vec8<T> x[NV], g[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      x[v] = nx[v];
      g[v] = ng[v];
    }
    const float mean = nmean, rstd = nrstd;
    if (AHEAD && row + step < a.rows) fetch(row + step);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t left = a.cols - (int64_t)(v * SPAN + t) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = g[v].at(i), h = i < left ? (x[v].at(i) - mean) * rstd : 0.0f;
        const float gw = d * w[v][i];
        s[0] += gw;
        s[1] = fmaf(gw, h, s[1]);
        dw[v][i] = fmaf(d, h, dw[v][i]);
        db[v][i] += d;
      }
    }
    group_sum<WAVES, 2>(s, red[turn], wave, lane);
    const float mg = s[0] * inv_n, mgh = s[1] * inv_n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t e = (int64_t)(v * SPAN + t) * 8;
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = (x[v].at(i) - mean) * rstd;
        dx[i] = rstd * (fmaf(g[v].at(i), w[v][i], -mg) - h * mgh);
      }
      store8((T *)a.y + row * a.cols + e, dx, a.cols - e);
    }
  }

  if constexpr (ROWS > 1) {   // the four waves' sums become the workgroup's
    __shared__ float part[ROWS][2][NV * SPAN * 8];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        part[wave][0][(v * 8 + i) * SPAN + t] = dw[v][i];
        part[wave][1][(v * 8 + i) * SPAN + t] = db[v][i];
      }
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[v][i] = db[v][i] = 0.0f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          dw[v][i] += part[r][0][(v * 8 + i) * SPAN + t];
          db[v][i] += part[r][1][(v * 8 + i) * SPAN + t];
        }
      }
  }
  float *const out = a.partials + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t e = (int64_t)(v * SPAN + t) * 8;
    store8(out + e, dw[v], a.cols - e);
    store8(out + a.cols + e, db[v], a.cols - e);
  }
}

// Few rows, where launches and trips to memory count and not bytes: one launch, whose first a.row_groups
// workgroups take the rows' dx, and the others the dw and db of 16 columns each, from their own reading of
// x and dy (out of the caches for the most part).  128 x 1000 fp32 3.2 us (6.5 with partial sums and a
// launch to join them), 515 x 1111 7.0 (10.1), 515 x 4096 11.1 (12.7).  With 8 columns a workgroup, which
// reads half as much of a line: 3.1, 6.7, 15.6.
constexpr int kFewCols = 16;
template <class T, class W, int WAVES, int NV>
__global__ void __launch_bounds__(256) norm_grad_few_kernel(const NormArgs a, W *dw, W *db) {
  static_assert(Geo<WAVES>::THREADS == 256, "");
  constexpr int ROWS = Geo<WAVES>::ROWS, SPAN = WAVES * 64;
  if ((int64_t)blockIdx.x >= a.row_groups) {
    constexpr int COLS = kFewCols, LANES = 256 / COLS;   // LANES threads take every LANES-th row
    __shared__ float part[2][LANES][COLS + 1];
    const int c = threadIdx.x % COLS, r0 = threadIdx.x / COLS;
    const int64_t col = ((int64_t)blockIdx.x - a.row_groups) * COLS + c;
    float sw = 0.0f, sb = 0.0f;
    const T *const x = (const T *)a.x + (col < a.cols ? col : 0);
    const T *const dy = (const T *)a.dy + (col < a.cols ? col : 0);
    // FLIGHT rows, loaded together; a row past the last is read as row 0 and counts nothing
    auto take = [&](int64_t r, auto flight_c) {
      constexpr int FLIGHT = decltype(flight_c)::value;
      float xv[FLIGHT], gv[FLIGHT], mean[FLIGHT], rstd[FLIGHT];
#pragma unroll
      for (int u = 0; u < FLIGHT; ++u) {
        const int64_t at = r + LANES * u < a.rows ? r + LANES * u : 0;
        xv[u] = load1(x + at * a.stride);
        gv[u] = load1(dy + at * a.dstride);
        mean[u] = a.mean[at];
        rstd[u] = a.rstd[at];
      }
#pragma unroll
      for (int u = 0; u < FLIGHT; ++u)
        if (r + LANES * u < a.rows) {
          sw = fmaf(gv[u], (xv[u] - mean[u]) * rstd[u], sw);
          sb += gv[u];
        }
    };
    int64_t r = 0;
    for (; r + LANES * 4 < a.rows; r += LANES * 16) take(r + r0, std::integral_constant<int, 16>());
    for (; r < a.rows; r += LANES * 4) take(r + r0, std::integral_constant<int, 4>());
    part[0][r0][c] = sw;
    part[1][r0][c] = sb;
    __syncthreads();
    if (r0 < 2 && col < a.cols) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < LANES; ++i) s += part[r0][i][c];
      store1((r0 ? db : dw) + col, s);
    }
    return;
  }
  __shared__ float red[WAVES][2];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = ROWS == 1 ? threadIdx.x : lane;
  const int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS == 1 ? 0 : wave);
  if (row >= a.rows) return;   // a whole wave, and with one row a workgroup none
  Vec8<T> x[NV], g[NV];
  Vec8<W> w[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t e = (int64_t)(v * SPAN + t) * 8;
    load8(x[v], (const T *)a.x + row * a.stride + e, a.cols - e);
    load8(g[v], (const T *)a.dy + row * a.dstride + e, a.cols - e);
    load8(w[v], (const W *)a.w + e, a.cols - e);
  }
  const float mean = a.mean[row], rstd = a.rstd[row], inv_n = 1.0f / (float)a.cols;
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t left = a.cols - (int64_t)(v * SPAN + t) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float h = i < left ? (x[v].at(i) - mean) * rstd : 0.0f, gw = g[v].at(i) * w[v].at(i);
      s[0] += gw;
      s[1] = fmaf(gw, h, s[1]);
    }
  }
  group_sum<WAVES, 2>(s, red, wave, lane);
  const float mg = s[0] * inv_n, mgh = s[1] * inv_n;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t e = (int64_t)(v * SPAN + t) * 8;
    float dx[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float h = (x[v].at(i) - mean) * rstd;
      dx[i] = rstd * (fmaf(g[v].at(i), w[v].at(i), -mg) - h * mgh);
    }
    store8((T *)a.y + row * a.cols + e, dx, a.cols - e);
  }
}

// Long rows: two passes over each; a workgroup's sums of dw and db grow in its own row of the
// workspace (each element is read and written by one thread only).
template <class T, class W>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(const NormArgs a) {
  __shared__ float red[2][16][2];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const float inv_n = 1.0f / (float)a.cols;
  float *const out = a.partials + (int64_t)blockIdx.x * 2 * a.cols;
  bool first = true;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false, turn ^= 1) {
    const T *x = (const T *)a.x + row * a.stride, *dy = (const T *)a.dy + row * a.dstride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.0f, 0.0f};
    Vec8<T> v, g;
    Vec8<W> w;
    Vec8<float> pw, pb;
    for (int64_t e = threadIdx.x * 8; e < a.cols; e += 8192) {
      load8(v, x + e, a.cols - e);
      load8(g, dy + e, a.cols - e);
      load8(w, (const W *)a.w + e, a.cols - e);
      pw.zero();
      pb.zero();
      if (!first) {
        load8(pw, out + e, a.cols - e);
        load8(pb, out + a.cols + e, a.cols - e);
      }
      float dw[8], db[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = g.at(i), h = i < a.cols - e ? (v.at(i) - mean) * rstd : 0.0f;
        const float gw = d * w.at(i);
        s[0] += gw;
        s[1] = fmaf(gw, h, s[1]);
        dw[i] = fmaf(d, h, pw.at(i));
        db[i] = d + pb.at(i);
      }
      store8(out + e, dw, a.cols - e);
      store8(out + a.cols + e, db, a.cols - e);
    }
    group_sum<16, 2>(s, red[turn], wave, lane);
    const float mg = s[0] * inv_n, mgh = s[1] * inv_n;
    for (int64_t e = threadIdx.x * 8; e < a.cols; e += 8192) {
      load8(v, x + e, a.cols - e);
      load8(g, dy + e, a.cols - e);
      load8(w, (const W *)a.w + e, a.cols - e);
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = (v.at(i) - mean) * rstd;
        dx[i] = rstd * (fmaf(g.at(i), w.at(i), -mg) - h * mgh);
      }
      store8((T *)a.y + row * a.cols + e, dx, a.cols - e);
    }
  }
}

// Adds the rows of partial sums: a workgroup takes 32 columns (one 128-byte line a row), its 32
// groups of lanes every 32nd row, and joins them through LDS.
template <class W>
__global__ void __launch_bounds__(1024)
    norm_join_kernel(const float *partials, int64_t count, int64_t cols, W *dw, W *db) {
  __shared__ float part[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;   // of 2 x cols
  float s = 0.0f;
  if (col < 2 * cols)
    for (int64_t r = g; r < count; r += 32 * 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)   // loads in flight together
        v[u] = r + 32 * u < count ? partials[(r + 32 * u) * 2 * cols + col] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
  part[g][c] = s;
  __syncthreads();
  if (g == 0 && col < 2 * cols) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i][c];
    if (col < cols)
      store1(dw + col, s);
    else
      store1(db + col - cols, s);
  }
}

constexpr int kCUs = 256;
constexpr int64_t kMost = 1 << 24;   // columns: the join's work-items stay under 2^32
constexpr int64_t kLong = 1024 * 8 * 3, kGradLong = 512 * 8 * 4;   // the longest rows in registers

// Workgroups of a backward pass: one a CU.  515 x 1111 fp32 takes 17.6 us on 64, 11.8 on 128, 9.8 on
// 256, 10.5 on 512 (more partial sums to join); 16384 x 4096 bf16 273, 141, 79.6 and 80.9 us.
int grad_groups(int64_t rows, int64_t cols) {
  const int64_t per = cols <= 1024 ? 4 : 1;
  const int64_t need = (rows + per - 1) / per;
  return (int)(need < kCUs ? need : kCUs);
}

// One launch for dx, dw and db, up to two trips of 16 rows and one of 4 a thread: 1024 rows take 10.1 us
// at 1000 columns and 24.7 at 4096, and 9.0 and 15.2 the other way.  dx written over x or dy would
// change what the columns' workgroups read.
bool few_rows(const NormArgs &a) {
  return a.rows > 0 && a.rows <= 256 / kFewCols * 36 && a.cols <= 4096 && a.y != a.x && a.y != a.dy;
}

// How many waves hold a row, and as how many vectors of eight a thread: one wave up to 1024 columns
// (no barrier), then few enough vectors that the next row's loads find registers beside this one's.
#define DG_NORM_SHAPES(KERNEL, cols)          \
  do {                                        \
    if ((cols) <= 512) KERNEL(1, 1);          \
    else if ((cols) <= 1024) KERNEL(1, 2);    \
    else if ((cols) <= 2048) KERNEL(4, 1);    \
    else if ((cols) <= 4096) KERNEL(4, 2);    \
    else if ((cols) <= 8192) KERNEL(8, 2);    \
    else if ((cols) <= 16384) KERNEL(16, 2);  \
    else KERNEL(16, 3);                       \
  } while (0)
#define DG_NORM_GRAD_SHAPES(KERNEL, cols)     \
  do {                                        \
    if ((cols) <= 512) KERNEL(1, 1);          \
    else if ((cols) <= 1024) KERNEL(1, 2);    \
    else if ((cols) <= 2048) KERNEL(4, 1);    \
    else if ((cols) <= 4096) KERNEL(4, 2);    \
    else if ((cols) <= 8192) KERNEL(8, 2);    \
    else KERNEL(8, 4);                        \
  } while (0)

template <class T, class W>
void launch_norm(const NormArgs &a, hipStream_t s) {
  if (a.cols > kLong) {
    const int64_t grid = a.rows < 2 * kCUs ? a.rows : 2 * kCUs;
    hipLaunchKernelGGL((norm_long_kernel<T, W>), dim3((uint32_t)grid), dim3(1024), 0, s, a);
    return;
  }
#define DG_RUN(WV, NV)                                                                        \
  do {                                                                                        \
    const int64_t need = (a.rows + Geo<WV>::ROWS - 1) / Geo<WV>::ROWS;                        \
    const int64_t most = kCUs * (1024 / Geo<WV>::THREADS);                                    \
    hipLaunchKernelGGL((norm_kernel<T, W, WV, NV>), dim3((uint32_t)(need < most ? need : most)), \
                       dim3(Geo<WV>::THREADS), 0, s, a);                                      \
  } while (0)
  DG_NORM_SHAPES(DG_RUN, a.cols);
#undef DG_RUN
}

template <class T, class W>
void launch_norm_grad(const NormArgs &a, W *dw, W *db, hipStream_t s) {
  const int grid = grad_groups(a.rows, a.cols);
  if (few_rows(a)) {
    NormArgs f = a;
#define DG_FEW(WV, NV)                                                                           \
  do {                                                                                           \
    f.row_groups = (a.rows + Geo<WV>::ROWS - 1) / Geo<WV>::ROWS;                                 \
    hipLaunchKernelGGL((norm_grad_few_kernel<T, W, WV, NV>),                                     \
                       dim3((uint32_t)(f.row_groups + (a.cols + kFewCols - 1) / kFewCols)), \
                       dim3(256), 0, s, f, dw, db);                                                                  \
  } while (0)
    if (a.cols <= 512) DG_FEW(1, 1);
    else if (a.cols <= 1024) DG_FEW(1, 2);
    else if (a.cols <= 2048) DG_FEW(4, 1);
    else DG_FEW(4, 2);
#undef DG_FEW
    return;
  }
  if (grid) {
    if (a.cols > kGradLong) {
      hipLaunchKernelGGL((norm_grad_long_kernel<T, W>), dim3(grid), dim3(1024), 0, s, a);
    } else {
#define DG_RUN(WV, NV)                                                                      \
  hipLaunchKernelGGL((norm_grad_kernel<T, W, WV, NV>), dim3(grid), dim3(Geo<WV>::THREADS), 0, \
                     s, a)
      DG_NORM_GRAD_SHAPES(DG_RUN, a.cols);
#undef DG_RUN
    }
  }
  hipLaunchKernelGGL((norm_join_kernel<W>), dim3((uint32_t)((2 * a.cols + 31) / 32)), dim3(1024),
                     0, s, a.partials, (int64_t)grid, a.cols, dw, db);
}

size_t elem(int dtype) { return dtype == GEMM_BF16 ? 2 : 4; }
bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool types_ok(int dtype, int wtype) {
  return (dtype == GEMM_BF16 || dtype == GEMM_F32) && (wtype == GEMM_F32 || wtype == dtype);
}
bool stride_ok(int64_t rows, int64_t cols, int64_t stride) {
  return stride >= 0 && (rows <= 1 || stride == 0 || stride >= cols);
}
// Whether packed rows may be written to `to` while rows of `from` are read: apart from each of them, or each
// over its own.  (Over rows with another stride, a workgroup's row would fall on one that another workgroup
// has yet to read.)
bool apart_or_same(const void *to, const void *from, int64_t rows, int64_t cols, int64_t stride,
                   size_t es) {
  if (to == from && (rows <= 1 || stride == cols)) return true;
  const uintptr_t t0 = (uintptr_t)to, t1 = t0 + (uintptr_t)(rows * cols) * es, f0 = (uintptr_t)from;
  const uintptr_t row = (uintptr_t)cols * es, step = (uintptr_t)stride * es;
  if (rows <= 1 || stride == 0) return t1 <= f0 || f0 + row <= t0;
  const uintptr_t r = t0 < f0 + row ? 0 : (t0 - f0 - row) / step + 1;   // the first row that ends behind t0
  return r >= (uintptr_t)rows || f0 + r * step >= t1;
}

}  // namespace
}  // namespace dg

extern "C" int gemm_layer_norm(const void *x, int dtype, int64_t rows, int64_t cols,
                               int64_t stride, const void *w, const void *b, int wtype, float eps,
                               void *y, float *mean, float *rstd, void *stream) {
  using namespace dg;
  if (rows < 0 || cols <= 0 || !types_ok(dtype, wtype) || !stride_ok(rows, cols, stride))
    return GEMM_ERR_INVALID_ARG;
  if (cols > kMost) return GEMM_ERR_UNSUPPORTED;
  if (rows == 0) return GEMM_OK;
  if (!x || !w || !y || !mean || !rstd) return GEMM_ERR_INVALID_ARG;
  if (!aligned(x, elem(dtype)) || !aligned(y, elem(dtype)) || !aligned(w, elem(wtype)) ||
      !aligned(b, elem(wtype)) || !aligned(mean, 4) || !aligned(rstd, 4))
    return GEMM_ERR_ALIGNMENT;
  NormArgs a{};
  a.x = x;
  a.w = w;
  a.b = b;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = cols;
  a.stride = stride;
  a.eps = eps;
  hipStream_t s = (hipStream_t)stream;
  if (dtype == GEMM_F32)
    launch_norm<float, float>(a, s);
  else if (wtype == GEMM_F32)
    launch_norm<bf16_t, float>(a, s);
  else
    launch_norm<bf16_t, bf16_t>(a, s);
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

extern "C" int gemm_layer_norm_backward_workspace(int64_t rows, int64_t cols, size_t *bytes) {
  if (rows < 0 || cols <= 0 || !bytes) return GEMM_ERR_INVALID_ARG;
  if (cols > dg::kMost) return GEMM_ERR_UNSUPPORTED;
  *bytes = (size_t)dg::grad_groups(rows, cols) * 2 * (size_t)cols * sizeof(float);
  return GEMM_OK;
}

extern "C" int gemm_layer_norm_backward(const void *dy, int64_t dstride, const void *x,
                                        int64_t stride, int dtype, int64_t rows, int64_t cols,
                                        const void *w, int wtype, const float *mean,
                                        const float *rstd, void *dx, void *dw, void *db,
                                        void *workspace, size_t workspace_bytes, void *stream) {
  using namespace dg;
  if (rows < 0 || cols <= 0 || !types_ok(dtype, wtype) || !stride_ok(rows, cols, stride) ||
      !stride_ok(rows, cols, dstride) || !w || !dw || !db)
    return GEMM_ERR_INVALID_ARG;
  if (cols > kMost) return GEMM_ERR_UNSUPPORTED;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return GEMM_ERR_INVALID_ARG;
  if (!aligned(x, elem(dtype)) || !aligned(dy, elem(dtype)) || !aligned(dx, elem(dtype)) ||
      !aligned(w, elem(wtype)) || !aligned(dw, elem(wtype)) || !aligned(db, elem(wtype)) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
    return GEMM_ERR_ALIGNMENT;
  if (rows > 0 && (!apart_or_same(dx, x, rows, cols, stride, elem(dtype)) ||
                   !apart_or_same(dx, dy, rows, cols, dstride, elem(dtype))))
    return GEMM_ERR_INVALID_ARG;
  size_t need = 0;
  gemm_layer_norm_backward_workspace(rows, cols, &need);
  if (need && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
  NormArgs a{};
  a.x = x;
  a.w = w;
  a.dy = dy;
  a.y = dx;
  a.mean = (float *)mean;
  a.rstd = (float *)rstd;
  a.partials = (float *)workspace;
  a.rows = rows;
  a.cols = cols;
  a.stride = stride;
  a.dstride = dstride;
  hipStream_t s = (hipStream_t)stream;
  if (dtype == GEMM_F32)
    launch_norm_grad<float, float>(a, (float *)dw, (float *)db, s);
  else if (wtype == GEMM_F32)
    launch_norm_grad<bf16_t, float>(a, (float *)dw, (float *)db, s);
  else
    launch_norm_grad<bf16_t, bf16_t>(a, (bf16_t *)dw, (bf16_t *)db, s);
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}
