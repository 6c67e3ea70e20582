// Global norm of a list of gradients (gemm_grad_norm) and the list scaled to a largest norm
// (gemm_clip_grad_norm).
//
//   norm = sqrt(sum over all elements of g^2),  c = min(1, max_norm / (norm + 1e-6)),  g' = c g
//
// The list goes to the kernels as a table in their arguments (no copy to the device, nothing that
// a captured graph would have to keep alive), at most kTable tensors a launch, cut into chunks
// that workgroups take in turn.  Squares are summed in fp64, which vector units here do at the
// rate of fp32: no square of a finite fp32 gradient overflows, and the sum's own error is nothing.
// Each workgroup leaves one partial sum; every workgroup of the scaling pass adds all of them by
// itself, in one order, instead of waiting for a launch of its own that would.
//
// The scaling pass goes backwards: what the first pass read last is still in the memory-side cache of
// 256 MB, and where a list is long, the pass neither keeps there what it writes nor what it has read
// (260 M elements, 521 MB: 306 us otherwise, 267 so; 96 of them the norm, at 5.4 TB/s).
//
// Bound by memory: the list read twice and written once.
#include "../../include/gemm_ops.h"
#include "ops_common.h"

#include <stdlib.h>

#include <algorithm>

namespace dg {
namespace {

constexpr int kTable = 128;          // tensors a launch: the table stays under 4 KB of arguments
// Elements a workgroup takes at once: the least and the most.  A short list is cut small, so that it
// reaches many CUs; a long one in pieces that keep the search for their tensor rare.
constexpr int kChunkLeast = 2048, kChunkMost = 16384;
constexpr int64_t kLongest = (int64_t)1 << 37;   // of a tensor: a table's chunks fit 31 bits
constexpr int64_t kPassing = 96 << 20;             // bytes: with its scaled form, most of the cache
constexpr int kGroups = 1024;        // workgroups a launch, at most
constexpr int kThreads = 256;

struct Table {
  const void *in[kTable];
  int64_t n[kTable];
  uint32_t first[kTable + 1];   // first chunk of each tensor; first[count] = all of them
  uint32_t f32[kTable / 32];    // bit i: tensor i is fp32, else bf16
  int32_t count, chunk;
  int32_t passing;              // the list is too long for the caches to keep
};
struct OutTable {
  void *out[kTable];
};
static_assert(sizeof(Table) + sizeof(OutTable) + 32 <= 4096, "kernel arguments");

__device__ __forceinline__ int tensor_of(const Table &t, uint32_t chunk) {
  int lo = 0, hi = t.count - 1;   // the last tensor whose first chunk is not past it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Sum over the workgroup, in every thread.
__device__ __forceinline__ double group_total(double v, double *slot) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += slot[w];
  return s;
}

constexpr int kAhead = 4;   // vectors of a thread whose loads are in flight together

template <class T>
__device__ __forceinline__ double squares(const T *p, int64_t n) {
  double s[2] = {0.0, 0.0};
  int64_t e = threadIdx.x * 8;
  for (; e + (kAhead - 1) * kThreads * 8 + 8 <= n; e += kAhead * kThreads * 8) {
    Vec8<T> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u].load(p + e + u * kThreads * 8);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double d = (double)v[u].at(i);
        s[i & 1] = fma(d, d, s[i & 1]);
      }
  }
  for (; e < n; e += kThreads * 8) {
    Vec8<T> v;
    load8(v, p + e, n - e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = (double)v.at(i);
      s[i & 1] = fma(d, d, s[i & 1]);
    }
  }
  return s[0] + s[1];
}

__global__ void __launch_bounds__(kThreads) squares_kernel(const Table t, double *partials) {
  __shared__ double slot[kThreads / 64];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[i]) * t.chunk;
    const int64_t n = t.n[i] - at < t.chunk ? t.n[i] - at : t.chunk;
    s += (t.f32[i / 32] >> (i % 32)) & 1 ? squares((const float *)t.in[i] + at, n)
                                         : squares((const bf16_t *)t.in[i] + at, n);
  }
  s = group_total(s, slot);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

__device__ __forceinline__ float norm_of(const double *partials, int count, double *slot) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kThreads) s += partials[i];
  return (float)sqrt(group_total(s, slot));
}

__global__ void __launch_bounds__(kThreads)
    norm_only_kernel(const double *partials, int count, float *norm) {
  __shared__ double slot[kThreads / 64];
  const float v = norm_of(partials, count, slot);
  if (threadIdx.x == 0) *norm = v;
}

template <bool PASSING, class T>
__device__ __forceinline__ void scale_chunk(const T *p, T *q, int64_t n, float c) {
  int64_t e = threadIdx.x * 8;
  for (; e + (kAhead - 1) * kThreads * 8 + 8 <= n; e += kAhead * kThreads * 8) {
    Vec8<T> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if constexpr (PASSING)
        v[u].load_once(p + e + u * kThreads * 8);
      else
        v[u].load(p + e + u * kThreads * 8);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = v[u].at(i) * c;
      if constexpr (PASSING)
        store8_once(q + e + u * kThreads * 8, o);
      else
        store8_full(q + e + u * kThreads * 8, o);
    }
  }
  for (; e < n; e += kThreads * 8) {
    Vec8<T> v;
    load8(v, p + e, n - e);
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v.at(i) * c;
    store8(q + e, o, n - e);
  }
}

__global__ void __launch_bounds__(kThreads)
    scale_kernel(const Table t, const OutTable o, const double *partials, int count,
                 float max_norm, float *norm) {
  __shared__ double slot[kThreads / 64];
  const float v = norm_of(partials, count, slot);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  float c = max_norm / (v + 1e-6f);
  if (c > 1.0f) c = 1.0f;   // a NaN stays
  const uint32_t all = t.first[t.count];
  for (uint32_t j = blockIdx.x; j < all; j += gridDim.x) {
    const uint32_t k = all - 1 - j;
    const int i = tensor_of(t, k);
    const int64_t at = (int64_t)(k - t.first[i]) * t.chunk;
    const int64_t n = t.n[i] - at < t.chunk ? t.n[i] - at : t.chunk;
    if (c == 1.0f && o.out[i] == t.in[i]) continue;   // in place and not clipped: as it is
    auto scale = [&](auto type) {
      using T = decltype(type);
      const T *p = (const T *)t.in[i] + at;
      T *q = (T *)o.out[i] + at;
      if (t.passing)
        scale_chunk<true>(p, q, n, c);
      else
        scale_chunk<false>(p, q, n, c);
    };
    if ((t.f32[i / 32] >> (i % 32)) & 1)
      scale(float());
    else
      scale(bf16_t());
  }
}

// Fills a table from list entries [from, count) and returns the first entry that is not in it.
int64_t fill(Table &t, OutTable *o, const gemm_tensor *list, int64_t from, int64_t count,
             int chunk) {
  t.count = 0;
  t.chunk = chunk;
  t.first[0] = 0;
  for (auto &w : t.f32) w = 0;
  int64_t i = from;
  for (; i < count && t.count < kTable; ++i) {
    const int64_t chunks = (list[i].numel + chunk - 1) / chunk;
    if (chunks == 0) continue;
    const int k = t.count;
    t.in[k] = list[i].data;
    t.n[k] = list[i].numel;
    if (o) o->out[k] = list[i].out;
    if (list[i].dtype == GEMM_F32) t.f32[k / 32] |= 1u << (k % 32);
    t.first[k + 1] = t.first[k] + (uint32_t)chunks;
    t.count = k + 1;
  }
  return i;
}

int check(const gemm_tensor *list, int64_t count, bool out) {
  if (count < 0 || (count && !list)) return GEMM_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    if (list[i].numel < 0 || (list[i].dtype != GEMM_BF16 && list[i].dtype != GEMM_F32))
      return GEMM_ERR_INVALID_ARG;
    if (list[i].numel > kLongest) return GEMM_ERR_UNSUPPORTED;
    if (list[i].numel && (!list[i].data || (out && !list[i].out))) return GEMM_ERR_INVALID_ARG;
    const uintptr_t mask = list[i].dtype == GEMM_F32 ? 3 : 1;
    if (((uintptr_t)list[i].data | (out ? (uintptr_t)list[i].out : 0)) & mask)
      return GEMM_ERR_ALIGNMENT;
  }
  return GEMM_OK;
}

struct Span {
  uintptr_t begin, end;
  bool written;
};
// The bytes of entry i: its data and its output, or one span where they are the same.  How many.
int spans_of(const gemm_tensor &t, Span (&s)[2]) {
  if (t.numel == 0) return 0;
  const uintptr_t bytes = (uintptr_t)t.numel * (t.dtype == GEMM_F32 ? 4 : 2);
  s[0] = Span{(uintptr_t)t.out, (uintptr_t)t.out + bytes, true};
  s[1] = Span{(uintptr_t)t.data, (uintptr_t)t.data + bytes, false};
  return t.out == t.data ? 1 : 2;
}

// GEMM_OK where no output overlaps another output, or data that are not exactly its own: workgroups
// scale what they share in any order, so parts of it would be scaled twice.
int check_apart(const gemm_tensor *list, int64_t count) {
  // Most lists are cut from a few buffers, or allocated in order: a few runs of rising addresses that lie
  // apart as wholes (0.7 us for 153 tensors into others, 5 to sort them).
  constexpr int RUNS = 8;
  constexpr uintptr_t NEAR = 512;   // an allocator's rounding
  Span run[RUNS], s[2];
  int runs = 0;
  bool simple = true;
  for (int64_t i = 0; i < count && simple; ++i)
    for (int k = spans_of(list[i], s) - 1; k >= 0 && simple; --k) {
      int to = 0;   // a run that ends just before it
      while (to < runs && s[k].begin - run[to].end >= NEAR) ++to;
      if (to < runs)
        run[to].end = s[k].end;
      else if (runs < RUNS)
        run[runs++] = s[k];
      else
        simple = false;
    }
  const auto before = [](const Span &a, const Span &b) { return a.begin < b.begin; };
  std::sort(run, run + runs, before);
  for (int r = 1; r < runs; ++r) simple = simple && run[r - 1].end <= run[r].begin;
  if (simple) return GEMM_OK;

  Span *const all = (Span *)malloc((size_t)count * 2 * sizeof(Span));
  if (!all) return GEMM_ERR_UNSUPPORTED;
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i)
    for (int k = spans_of(list[i], s) - 1; k >= 0; --k) all[n++] = s[k];
  std::sort(all, all + n, before);
  uintptr_t read = 0, written = 0;   // where those so far end
  bool apart = true;
  for (int64_t i = 0; i < n; ++i) {
    apart = apart && all[i].begin >= written && !(all[i].written && all[i].begin < read);
    uintptr_t &end = all[i].written ? written : read;
    end = std::max(end, all[i].end);
  }
  free(all);
  return apart ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

// The size of chunk that gives a list at least kGroups of them, within its bounds.
int chunk_of(const gemm_tensor *list, int64_t count) {
  int64_t all = 0;
  for (int64_t i = 0; i < count; ++i) all += list[i].numel;
  int chunk = kChunkMost;
  while (chunk > kChunkLeast && all / chunk < kGroups) chunk /= 2;
  return chunk;
}

int64_t launches(int64_t count) { return (count + kTable - 1) / kTable; }

// Enqueues the sums of squares; *partial_count is how many the workspace then holds.
int sum_squares(const gemm_tensor *list, int64_t count, void *workspace, size_t bytes,
                hipStream_t s, int *partial_count) {
  const int chunk = chunk_of(list, count);
  int64_t from = 0;
  int n = 0;
  Table t;
  while (from < count) {
    from = fill(t, nullptr, list, from, count, chunk);
    if (t.count == 0) break;
    const uint32_t all = t.first[t.count];
    const int grid = all < (uint32_t)kGroups ? (int)all : kGroups;
    if ((size_t)(n + grid) * sizeof(double) > bytes) return GEMM_ERR_WORKSPACE;
    hipLaunchKernelGGL(squares_kernel, dim3(grid), dim3(kThreads), 0, s, t,
                       (double *)workspace + n);
    if (hipGetLastError() != hipSuccess) return GEMM_ERR_HIP;
    n += grid;
  }
  *partial_count = n;
  return GEMM_OK;
}

}  // namespace
}  // namespace dg

extern "C" int gemm_grad_norm_workspace(const gemm_tensor *list, int64_t count, size_t *bytes) {
  using namespace dg;
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  const int st = check(list, count, false);
  if (st != GEMM_OK) return st;
  // a launch leaves one sum a workgroup, of which it has kGroups at most
  const int chunk = chunk_of(list, count);
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) chunks += (list[i].numel + chunk - 1) / chunk;
  const int64_t most = launches(count) * kGroups;
  *bytes = (size_t)(chunks < most ? chunks : most) * sizeof(double);
  return GEMM_OK;
}

extern "C" int gemm_grad_norm(const gemm_tensor *list, int64_t count, float *norm,
                              void *workspace, size_t workspace_bytes, void *stream) {
  using namespace dg;
  const int st = check(list, count, false);
  if (st != GEMM_OK) return st;
  if (!norm) return GEMM_ERR_INVALID_ARG;
  size_t need = 0;
  gemm_grad_norm_workspace(list, count, &need);
  if (need && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
  if (((uintptr_t)workspace & 7) || ((uintptr_t)norm & 3)) return GEMM_ERR_ALIGNMENT;
  hipStream_t s = (hipStream_t)stream;
  int n = 0;
  const int run = sum_squares(list, count, workspace, workspace_bytes, s, &n);
  if (run != GEMM_OK) return run;
  hipLaunchKernelGGL(norm_only_kernel, dim3(1), dim3(kThreads), 0, s, (const double *)workspace, n,
                     norm);
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

extern "C" int gemm_clip_grad_norm(const gemm_tensor *list, int64_t count, float max_norm,
                                   float *norm, void *workspace, size_t workspace_bytes,
                                   void *stream) {
  using namespace dg;
  int st = check(list, count, true);
  if (st != GEMM_OK) return st;
  if (!norm || !(max_norm >= 0.0f)) return GEMM_ERR_INVALID_ARG;
  st = check_apart(list, count);
  if (st != GEMM_OK) return st;
  size_t need = 0;
  gemm_grad_norm_workspace(list, count, &need);
  if (need && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
  if (((uintptr_t)workspace & 7) || ((uintptr_t)norm & 3)) return GEMM_ERR_ALIGNMENT;
  if (need == 0) return gemm_grad_norm(list, count, norm, workspace, workspace_bytes, stream);
  hipStream_t s = (hipStream_t)stream;
  int n = 0;
  const int run = sum_squares(list, count, workspace, workspace_bytes, s, &n);
  if (run != GEMM_OK) return run;
  // the tables of the list's end first
  const int chunk = chunk_of(list, count);
  int64_t bytes = 0;
  for (int64_t i = 0; i < count; ++i) bytes += list[i].numel * (list[i].dtype == GEMM_F32 ? 4 : 2);
  Table t;
  t.passing = bytes > kPassing;
  OutTable o;
  for (int64_t k = launches(count) - 1; k >= 0; --k) {
    const int64_t last = (k + 1) * kTable;
    fill(t, &o, list, k * kTable, last < count ? last : count, chunk);
    if (t.count == 0) continue;
    const uint32_t all = t.first[t.count];
    const int grid = all < (uint32_t)(2 * kGroups) ? (int)all : 2 * kGroups;
    hipLaunchKernelGGL(scale_kernel, dim3(grid), dim3(kThreads), 0, s, t, o,
                       (const double *)workspace, n, max_norm, norm);
    if (hipGetLastError() != hipSuccess) return GEMM_ERR_HIP;
    norm = nullptr;   // written once
  }
  return GEMM_OK;
}
