// An AdamW step over a list of parameters (gemm_adamw_step):
//
//   c = min(1, max_norm / (norm + 1e-6)) or 1,  g' = c g
//   m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2
//   p' = p - lr (wd p + (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps))
//
// in fp32, each parameter rounded once.  States are fp32, or e4m3: then m and the root of v are held as
// codes with an fp32 scale s = max(amax / 448, 2^-126) per 128 neighbours, x ~ s q.  (The root spans half of
// v's powers of two, and is what divides.  One that is not zero keeps the smallest code at least: a first
// moment over a root that was rounded to zero would be as large as 1 / eps.)  Codes are those of
// x * (1 / s), so a quotient within 2^-22 of a border may go to either neighbour.  A change of less than half a
// code is lost: roots follow gradients that fall for b2 up to 0.95.
//
// The list goes to the kernels as a table in their arguments, as in ops_clip.hip, cut into chunks that
// workgroups take in turn.  A lane takes eight neighbours, so a scale's 128 are a DPP row of 16 lanes.
//
// Bound by memory: parameters and states read and written once, gradients read once.  Many short workgroups
// come nearest to it (260 M bf16 parameters with e4m3 states, 2.6 GB, in chunks of 2048, 4096, 8192, 16384:
// 511, 466, 469, 498 us, 5.65 TB/s at best; 134 M fp32 ones with fp32 states and copies, 3.8 GB, of 1024, 2048,
// 4096, 16384: 640, 676, 733, 768 us, 5.9 TB/s; 2048 workgroups that stay: 556, 831), and loads and stores
// past the caches (583 and 860 without).
#include "../../include/gemm_ops.h"
#include "ops_common.h"
#include "ops_spans.h"

#include <math.h>

#include <type_traits>

namespace dg {
namespace {

constexpr int kTable = 120, kTableCopies = 96;   // tensors a launch: a table stays under 4 KB of arguments
constexpr int kBlock = 128;          // neighbours of one scale; each tensor's state starts at a multiple
constexpr int kThreads = 256;
constexpr int kGroups = 1 << 22;     // workgroups a launch, at most: chunks past them are second ones
constexpr int64_t kLongest = (int64_t)1 << 37;   // of all tensors: chunks and blocks fit 32 bits
constexpr int64_t kPassing = 96 << 20;   // bytes of a step that the caches could keep for the next pass

template <int N>
struct Copies {
  void *copy[N];
};
struct NoCopies {};
template <bool COPIES>
struct Table : std::conditional_t<COPIES, Copies<kTableCopies>, NoCopies> {
  static constexpr int N = COPIES ? kTableCopies : kTable;
  void *param[N];
  const void *grad[N];
  int64_t n[N];
  uint32_t block[N];            // the first block of 128 of each tensor's state
  uint32_t first[N + 1];        // first chunk of each tensor; first[count] = all of them
  uint32_t f32[4];              // bit i: tensor i's parameters are fp32, else bf16
  uint32_t grad_f32[4];
  int32_t count, chunk;
};
struct Step {
  void *m, *v;
  float *ms, *vs;
  const float *norm, *lr_at;
  const int64_t *step_at;
  double beta1, beta2;          // for what step_at and lr_at say
  float b1, b1_rest, b2, b2_rest, eps, decay, max_norm;
  float lr, rate, root;         // rate = lr / (1 - b1^t), root = 1 / sqrt(1 - b2^t)
  float up;                     // a power of two for both sides of the quotient (eps has it already)
};
static_assert(sizeof(Table<false>) + sizeof(Step) + 16 <= 4096, "kernel arguments");
static_assert(sizeof(Table<true>) + sizeof(Step) + 16 <= 4096, "kernel arguments");
static_assert(kTable <= 128, "bits of the types, two tensors a lane");

// The last tensor whose first chunk is not past this one.  Arguments may lie in the host's memory: all first
// chunks in one trip there, not the seven of a search that halves them.
template <class T>
__device__ __forceinline__ int tensor_of(const T &t, uint32_t chunk) {
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 64 * k;
    const bool at = i < t.count && t.first[i < T::N ? i : 0] <= chunk;
    n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(at));
  }
  return __builtin_amdgcn_readfirstlane(n - 1);
}

__device__ __forceinline__ double power(double b, int64_t t) {
  double r = 1.0;
  for (uint64_t n = t > 0 ? (uint64_t)t : 0; n; n >>= 1) {
    if (n & 1) r *= b;
    b *= b;
  }
  return r;
}

// Largest over the 16 lanes of a DPP row, in each of them; a NaN is the largest.
__device__ __forceinline__ float row16_amax(float x) {
  uint32_t v = bits_of(x) & 0x7FFFFFFFu;
#define DG_ROR(n) \
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xF, 0xF, false))
  DG_ROR(8);
  DG_ROR(4);
  DG_ROR(2);
  DG_ROR(1);
#undef DG_ROR
  return float_of(v);
}

// The instruction flushes small operands and results.
__device__ __forceinline__ float root_of(float v) {
  const bool small = v < 0x1p-96f;
  const float r = __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v);
  return small ? r * 0x1p-32f : r;
}

__device__ __forceinline__ void decode8(float (&x)[8], u32x2_t c, float s) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], true);
    x[4 * h] = a[0] * s;
    x[4 * h + 1] = a[1] * s;
    x[4 * h + 2] = b[0] * s;
    x[4 * h + 3] = b[1] * s;
  }
}

// Codes of eight values of a block, whose scale goes to *s.
template <bool ROOT>
__device__ __forceinline__ u32x2_t encode8(const float (&x)[8], float *s) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, bits_of(x[i]) & 0x7FFFFFFFu);
  const float amax = row16_amax(float_of(top));
  // the quotient rounded to nearest: one step of correction makes amax * (1 / 448) exact
  const float y = 1.0f / 448.0f, near = amax * y;
  float scale = fmaxf(fmaf(fmaf(-448.0f, near, amax), y, near), 0x1p-126f);
  if (!(amax < __builtin_inff())) scale = float_of(0x7FC00000u);
  *s = scale;
  const float r = scale == scale ? __builtin_amdgcn_rcpf(scale) : scale;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = x[i] * r;
    if (ROOT) q[i] = x[i] > 0.0f ? __builtin_elementwise_maximum(q[i], 0x1p-9f) : q[i];
  }
  u32x2_t c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
    c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], w, true);
  }
  return c;
}

struct Now {   // what is the same for every element
  float c, rate, root, decay;   // decay: lr wd
};

__device__ __forceinline__ void update(const Step &a, const Now &now, float g, float &p, float &m,
                                       float &v, float &r) {
  g *= now.c;
  m = fmaf(a.b1, m, a.b1_rest * g);
  v = fmaf(a.b2, v, a.b2_rest * g * g);
  r = root_of(v);
  // (1 - lr wd would lose the places of lr wd: p less its share instead)
  const float way = now.rate * m * __builtin_amdgcn_rcpf(fmaf(r, now.root, a.eps));
  p = fmaf(-now.decay, p, p) - way;
}

// W neighbours of a tensor as fp32, of which n are there; ONCE: past the caches, for lists too long for them.
template <int W, bool ONCE, class T>
__device__ __forceinline__ void take(float (&x)[W], const T *p, int64_t n) {
  if (n >= W) {
    if constexpr (W == 8) {
      Vec8<T> v;
      if constexpr (ONCE)
        v.load_once(p);
      else
        v.load(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = v.at(i);
    } else if constexpr (sizeof(T) == 4) {
      const u32x4_t v = ONCE ? __builtin_nontemporal_load((const u32x4_any *)p) : *(const u32x4_any *)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = float_of(v[i]);
    } else {
      const u32x2_t v = ONCE ? __builtin_nontemporal_load((const u32x2_any *)p) : *(const u32x2_any *)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = float_of(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = i < n ? load1(p + i) : 0.0f;
  }
}
template <int W, bool ONCE, class T>
__device__ __forceinline__ void give(T *p, const float (&x)[W], int64_t n) {
  if (n >= W) {
    if constexpr (W == 8) {
      if constexpr (ONCE)
        store8_once(p, x);
      else
        store8_full(p, x);
    } else if constexpr (sizeof(T) == 4) {
      const u32x4_t v = {bits_of(x[0]), bits_of(x[1]), bits_of(x[2]), bits_of(x[3])};
      if constexpr (ONCE)
        __builtin_nontemporal_store(v, (u32x4_any *)p);
      else
        *(u32x4_any *)p = v;
    } else {
      const u32x2_t v = {bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
      if constexpr (ONCE)
        __builtin_nontemporal_store(v, (u32x2_any *)p);
      else
        *(u32x2_any *)p = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < n) store1(p + i, x[i]);
  }
}
template <bool ONCE>
__device__ __forceinline__ u32x2_t take_codes(const void *p, int64_t at) {
  const u32x2_t *q = (const u32x2_t *)((const uint8_t *)p + at);
  return ONCE ? __builtin_nontemporal_load(q) : *q;
}
template <bool ONCE>
__device__ __forceinline__ void give_codes(void *p, int64_t at, u32x2_t c) {
  u32x2_t *q = (u32x2_t *)((uint8_t *)p + at);
  if (ONCE)
    __builtin_nontemporal_store(c, q);
  else
    *q = c;
}

// Neighbours of a lane: eight of a block's 128 with e4m3 states; four with fp32 states, whose 16 bytes then
// lie next to the next lane's.
template <bool E4M3>
constexpr int kWidth = E4M3 ? 8 : 4;

// One vector of a tensor, of which `n` elements are left.
template <class P, class G, bool E4M3, bool ONCE>
__device__ __forceinline__ void vector_step(const Step &a, const Now &now, P *p, const G *g,
                                            bf16_t *copy, int64_t state, int64_t n) {
  constexpr int W = kWidth<E4M3>;
  float m[W], v[W], x[W], d[W], r[W];
  take<W, ONCE>(x, p, n);
  take<W, ONCE>(d, g, n);
  if constexpr (E4M3) {
    u32x2_t mc = {0, 0}, vc = {0, 0};
    float ms = 0.0f, vs = 0.0f;
    if (n > 0) {
      mc = take_codes<ONCE>(a.m, state);
      vc = take_codes<ONCE>(a.v, state);
      ms = a.ms[state / kBlock];
      vs = a.vs[state / kBlock];
    }
    decode8(m, mc, ms);
    decode8(v, vc, vs);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= v[i];
  } else {
    take<W, ONCE>(m, (const float *)a.m + state, n);
    take<W, ONCE>(v, (const float *)a.v + state, n);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) update(a, now, d[i], x[i], m[i], v[i], r[i]);
  give<W, ONCE>(p, x, n);
  if (copy) give<W, ONCE>(copy, x, n);
  if constexpr (E4M3) {
    // what lies behind the tensor's end is no part of its last block
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i >= n) m[i] = r[i] = 0.0f;
    float ms, vs;
    const u32x2_t mc = encode8<false>(m, &ms), vc = encode8<true>(r, &vs);
    if (n > 0) {
      give_codes<ONCE>(a.m, state, mc);
      give_codes<ONCE>(a.v, state, vc);
      if (state % kBlock == 0) {
        a.ms[state / kBlock] = ms;
        a.vs[state / kBlock] = vs;
      }
    }
  } else {
    give<W, ONCE>((float *)a.m + state, m, n);
    give<W, ONCE>((float *)a.v + state, v, n);
  }
}

template <bool E4M3, bool COPIES, bool ONCE>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const Table<COPIES> t, const Step a) {
  Now now{1.0f, a.rate, a.root, a.lr * a.decay};
  if (a.step_at || a.lr_at) {
    float lr = a.lr;
    if (a.lr_at) {
      lr = *a.lr_at;
      now.decay = lr * a.decay;
    }
    if (a.step_at) {
      const int64_t step = *a.step_at;
      now.rate = (float)((double)lr / (1.0 - power(a.beta1, step)));
      now.root = (float)(1.0 / sqrt(1.0 - power(a.beta2, step)));
    } else {
      now.rate = lr * a.rate;   // of a rate of one
    }
  }
  now.rate *= a.up;
  now.root *= a.up;
  if (a.norm) {
    now.c = a.max_norm / (*a.norm + 1e-6f);
    if (now.c > 1.0f) now.c = 1.0f;   // a NaN stays
  }
  for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[i]) * t.chunk;
    const int64_t n = t.n[i] - at < t.chunk ? t.n[i] - at : t.chunk;
    const int64_t state = (int64_t)t.block[i] * kBlock + at;
    bf16_t *copy = nullptr;
    if constexpr (COPIES)
      if (t.copy[i]) copy = (bf16_t *)t.copy[i] + at;
    auto run = [&](auto param, auto grad) {
      using P = decltype(param);
      using G = decltype(grad);
      P *const p = (P *)t.param[i] + at;
      const G *const g = (const G *)t.grad[i] + at;
      constexpr int W = kWidth<E4M3>;
      for (int64_t e = threadIdx.x * W; e - threadIdx.x * W < n; e += kThreads * W)
        vector_step<P, G, E4M3, ONCE>(a, now, p + e, g + e, copy ? copy + e : nullptr, state + e,
                                      n - e);
    };
    const bool pf = (t.f32[i / 32] >> (i % 32)) & 1, gf = (t.grad_f32[i / 32] >> (i % 32)) & 1;
    if (pf && gf)
      run(float(), float());
    else if (pf)
      run(float(), bf16_t());
    else if (gf)
      run(bf16_t(), float());
    else
      run(bf16_t(), bf16_t());
  }
}

bool number(double v) { return v - v == 0.0; }

int check(const gemm_adamw_tensor *list, int64_t count, const gemm_adamw_desc *d) {
  if (!d || count < 0 || (count && !list)) return GEMM_ERR_INVALID_ARG;
  if (d->dtype_state != GEMM_F32 && d->dtype_state != GEMM_FP8_E4M3) return GEMM_ERR_INVALID_ARG;
  if (!(d->beta1 >= 0.0 && d->beta1 < 1.0) || !(d->beta2 >= 0.0 && d->beta2 < 1.0) ||
      !(d->eps >= 0.0) || !number(d->eps) || !number(d->weight_decay) ||
      (!d->lr_at && !number(d->lr)) || (!d->step_at && d->step < 1) ||
      (d->norm && !(d->max_norm >= 0.0)))
    return GEMM_ERR_INVALID_ARG;
  int64_t all = 0;
  for (int64_t i = 0; i < count; ++i) {
    const gemm_adamw_tensor &t = list[i];
    if (t.numel < 0 || (t.dtype != GEMM_BF16 && t.dtype != GEMM_F32) ||
        (t.dtype_grad != GEMM_BF16 && t.dtype_grad != GEMM_F32))
      return GEMM_ERR_INVALID_ARG;
    if (t.numel > kLongest || (all += t.numel + kBlock) > kLongest) return GEMM_ERR_UNSUPPORTED;
    if (t.numel == 0) continue;
    if (!t.param || !t.grad || !d->m || !d->v) return GEMM_ERR_INVALID_ARG;
    if (d->dtype_state == GEMM_FP8_E4M3 && (!d->m_scales || !d->v_scales))
      return GEMM_ERR_INVALID_ARG;
    if (((uintptr_t)t.param & (t.dtype == GEMM_F32 ? 3 : 1)) ||
        ((uintptr_t)t.grad & (t.dtype_grad == GEMM_F32 ? 3 : 1)) || ((uintptr_t)t.copy & 1))
      return GEMM_ERR_ALIGNMENT;
  }
  const uintptr_t state = d->dtype_state == GEMM_F32 ? 3 : 7;
  if ((((uintptr_t)d->m | (uintptr_t)d->v) & state) ||
      (((uintptr_t)d->m_scales | (uintptr_t)d->v_scales | (uintptr_t)d->norm |
        (uintptr_t)d->lr_at) & 3) || ((uintptr_t)d->step_at & 7))
    return GEMM_ERR_ALIGNMENT;
  return GEMM_OK;
}

// GEMM_OK where nothing that is written overlaps anything else: a parameter that is in the list twice would
// be stepped by two workgroups at once.
int check_apart(const gemm_adamw_tensor *list, int64_t count, const gemm_adamw_desc *d) {
  const bool e4m3 = d->dtype_state == GEMM_FP8_E4M3;
  uintptr_t blocks = 0;
  for (int64_t i = 0; i < count; ++i) blocks += (uintptr_t)((list[i].numel + kBlock - 1) / kBlock);
  if (blocks == 0) return GEMM_OK;
  return spans_apart<3>(count + 3, [=](int64_t i, Span (&s)[3]) {
    int n = 0;
    const auto add = [&](const void *p, uintptr_t bytes, bool written) {
      if (p && bytes) s[n++] = Span{(uintptr_t)p, (uintptr_t)p + bytes, written};
    };
    if (i < count) {
      const gemm_adamw_tensor &t = list[i];
      add(t.numel ? t.param : nullptr, (uintptr_t)t.numel * (t.dtype == GEMM_F32 ? 4 : 2), true);
      add(t.numel ? t.grad : nullptr, (uintptr_t)t.numel * (t.dtype_grad == GEMM_F32 ? 4 : 2), false);
      add(t.numel ? t.copy : nullptr, (uintptr_t)t.numel * 2, true);
    } else if (i == count) {
      add(d->m, blocks * (e4m3 ? kBlock : 4 * kBlock), true);
      add(d->v, blocks * (e4m3 ? kBlock : 4 * kBlock), true);
    } else if (i == count + 1) {
      add(e4m3 ? d->m_scales : nullptr, blocks * 4, true);
      add(e4m3 ? d->v_scales : nullptr, blocks * 4, true);
    } else {
      add(d->norm, 4, false);
      add(d->lr_at, 4, false);
      add(d->step_at, 8, false);
    }
    return n;
  });
}

// Enqueues a launch for each table that the list fills; `all` elements are in it.
template <bool E4M3, bool COPIES, bool ONCE>
int step_list(const gemm_adamw_tensor *list, int64_t count, const Step &a, int64_t all,
              hipStream_t s) {
  Table<COPIES> t;
  // a vector a thread; two with e4m3 states where that leaves every CU some workgroups
  t.chunk = kThreads * kWidth<E4M3>;
  if (E4M3 && all >= (int64_t)4096 * t.chunk) t.chunk *= 2;
  int64_t i = 0, block = 0;
  while (i < count) {
    t.count = 0;
    t.first[0] = 0;
    for (int w = 0; w < 4; ++w) t.f32[w] = t.grad_f32[w] = 0;
    for (; i < count && t.count < t.N; ++i) {
      const gemm_adamw_tensor &x = list[i];
      if (x.numel == 0) continue;
      const int k = t.count++;
      t.param[k] = x.param;
      t.grad[k] = x.grad;
      if constexpr (COPIES) t.copy[k] = x.copy;
      t.n[k] = x.numel;
      t.block[k] = (uint32_t)block;
      if (x.dtype == GEMM_F32) t.f32[k / 32] |= 1u << (k % 32);
      if (x.dtype_grad == GEMM_F32) t.grad_f32[k / 32] |= 1u << (k % 32);
      t.first[k + 1] = t.first[k] + (uint32_t)((x.numel + t.chunk - 1) / t.chunk);
      block += (x.numel + kBlock - 1) / kBlock;
    }
    if (t.count == 0) break;
    const uint32_t chunks = t.first[t.count];
    const dim3 grid(chunks < (uint32_t)kGroups ? chunks : kGroups);
    hipLaunchKernelGGL((adamw_kernel<E4M3, COPIES, ONCE>), grid, dim3(kThreads), 0, s, t, a);
    if (hipGetLastError() != hipSuccess) return GEMM_ERR_HIP;
  }
  return GEMM_OK;
}

}  // namespace
}  // namespace dg

extern "C" int gemm_adamw_step(const gemm_adamw_tensor *list, int64_t count,
                               const gemm_adamw_desc *d, void *stream) {
  using namespace dg;
  int st = check(list, count, d);
  if (st != GEMM_OK) return st;
  st = check_apart(list, count, d);
  if (st != GEMM_OK) return st;
  Step a{};
  a.m = d->m;
  a.v = d->v;
  a.ms = d->m_scales;
  a.vs = d->v_scales;
  a.norm = d->norm;
  a.lr_at = d->lr_at;
  a.step_at = d->step_at;
  a.beta1 = d->beta1;
  a.beta2 = d->beta2;
  a.b1 = (float)d->beta1;
  a.b1_rest = (float)(1.0 - d->beta1);
  a.b2 = (float)d->beta2;
  a.b2_rest = (float)(1.0 - d->beta2);
  // The reciprocal's instruction takes a number under 2^-126 for zero, and a moment of zero over that would be
  // NaN: where eps may be one, both sides of the quotient are 2^24 times as large, eps 2^-149 at least.
  const bool tiny = d->eps > 0.0 && d->eps < 0x1p-100;
  a.up = tiny ? 0x1p24f : 1.0f;
  a.eps = tiny ? fmaxf((float)(d->eps * 0x1p24), 0x1p-125f) : (float)d->eps;
  a.decay = (float)d->weight_decay;
  a.max_norm = (float)d->max_norm;
  a.lr = (float)d->lr;
  if (!d->step_at) {
    a.rate = (float)((d->lr_at ? 1.0 : d->lr) / (1.0 - pow(d->beta1, (double)d->step)));
    a.root = (float)(1.0 / sqrt(1.0 - pow(d->beta2, (double)d->step)));
  }
  bool copies = false;
  int64_t all = 0, bytes = 0;
  for (int64_t i = 0; i < count; ++i) {
    const gemm_adamw_tensor &x = list[i];
    copies = copies || (x.numel && x.copy);
    all += x.numel;
    bytes += x.numel * ((x.dtype == GEMM_F32 ? 8 : 4) + (x.dtype_grad == GEMM_F32 ? 4 : 2) +
                        (d->dtype_state == GEMM_F32 ? 16 : 4) + (x.copy ? 2 : 0));
  }
  const bool once = bytes > kPassing, e4m3 = d->dtype_state == GEMM_FP8_E4M3;
  hipStream_t s = (hipStream_t)stream;
  const auto go = [&](auto e4m3_c, auto copies_c, auto once_c) {
    return step_list<decltype(e4m3_c)::value, decltype(copies_c)::value, decltype(once_c)::value>(
        list, count, a, all, s);
  };
  const auto with_once = [&](auto e4m3_c, auto copies_c) {
    return once ? go(e4m3_c, copies_c, std::true_type()) : go(e4m3_c, copies_c, std::false_type());
  };
  const auto with_copies = [&](auto e4m3_c) {
    return copies ? with_once(e4m3_c, std::true_type()) : with_once(e4m3_c, std::false_type());
  };
  return e4m3 ? with_copies(std::true_type()) : with_copies(std::false_type());
}
