// Large tiles of the int8 product: 256 rows by 256 columns, four waves, each alone on its SIMD with
// half of the tile's rows and columns, so the instruction stream is laid out by hand, one k-block of 128 a
// step, as in the block-scaled product's wide kernel: in each slot behind a block's two MFMAs goes a share of
// what the next steps need.  A fragment is read again right behind its last MFMA, and the loads of the step
// after the next go out once the waves have met (the next step's have landed, this step's fragments are all
// read).  The first two and the last two rows of blocks are taken column by column, so that the reads of
// B's fragments have 2 FN slots, and as many before their next MFMA.
//
// Workgroups stay for tile after tile: the loads of the next one are under way when a tile ends, and a
// tile that was left in the registers is scaled and written out beside the next one's first step.
//
// Bound by the matrix units and the power that they may draw: 8192 x 8192 x 8192 takes 386 us, 2.85 POP/s, the units
// busy 0.75 of the time at 1.9 GHz (354 us on zeros); 4096 x 14336 x 4096 to bf16 184 to 188, of which an eighth is the
// half-empty fourth round, 208 with stores through the caches.  Loads in all of a step's slots behind the
// handshake rather than in its first few: 420 to 390 us.
#include "ops_int8.h"

namespace dg {
namespace {

constexpr int kWorkers = 256;   // one a CU
constexpr int kNonTemporal = 2;

// Corner of the tile of worker b in a round; false if it has none.  The workers of an XCD (b mod 8)
// take neighbouring tiles: strips of eight rows of tiles, walked down first.
__device__ __forceinline__ bool tile_at(const Int8Args &a, int32_t b, int32_t round, int bm, int bn,
                                        int64_t &m0, int64_t &n0) {
  const int32_t left = a.mt * a.nt - round * kWorkers;
  const int32_t now = left < kWorkers ? left : kWorkers;
  const int32_t per = now >> 3, more = now & 7, x = b & 7, i = b >> 3;
  if (now <= 0 || i >= per + (x < more)) return false;
  const int32_t t = round * kWorkers + x * per + (x < more ? x : more) + i;
  const int32_t strip = t / (8 * a.nt), in = t % (8 * a.nt);
  const int32_t high = a.mt - strip * 8 < 8 ? a.mt - strip * 8 : 8;
  m0 = (int64_t)(strip * 8 + in % high) * bm;
  n0 = (int64_t)(in / high) * bn;
  return true;
}

// The output of a wave's FM x FN blocks of 16 x 16, written out one block at a time: block (f, g) goes as it
// is into one of two halves of a row of blocks in the wave's LDS (4 KB each, 16-byte chunks swizzled).
// Beside the other half's blocks it comes back as rows, four columns a lane -- so that a lane needs the scales
// and the bias of eight columns only -- and is scaled, finished and stored.
template <int FM, int FN, class OUT>
struct OutRows {
  static constexpr uint32_t ES = sizeof(OUT);
  static constexpr int HALF = FN / 2;   // blocks of a half
  static_assert(HALF == 4, "a half is 64 columns, 16 lanes of four");
  typedef i32x4 __attribute__((address_space(3))) *p128;
  __amdgpu_buffer_rsrc_t cr;
  uint32_t st_off[2], pitch;
  uint32_t wa, ra;   // LDS addresses of the lane's write of block column 0 and read 0
  i32x4 v;
  f32x4 sb[2], bias[2];   // of the lane's four columns in each half
  f32x4 sa[FM];           // of its four rows in each row of blocks

  __device__ __forceinline__ void init(const Int8Args &a, lds_t *slice, int lane) {
    clear(a);   // nothing is carried: the stores go to an empty range
    const uint32_t base = (uint32_t)(size_t)slice;
    const int row = lane & 15, q = lane >> 4;   // writes: row `row`, chunk (4 g + q) ^ row of a half
    wa = base + row * 256 + ((q ^ row) * 16);
    ra = base + q * 1024 + ((row ^ (4 * q)) * 16);   // reads: row 4 q (+ j), chunk `row` ^ 4 q (^ j)
#pragma unroll
    for (int h = 0; h < 2; ++h) sb[h] = bias[h] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = f32x4{0, 0, 0, 0};
  }
  // The scales and the bias of a tile: what lies past M or N reads as zeros.
  __device__ __forceinline__ void load(const Int8Args &a, int64_t m0, int64_t n0, int lane) {
    const bool inside = m0 < a.M && n0 < a.N;
    const int64_t m = inside ? m0 : 0, n = inside ? n0 : 0;
    const auto rows = uniform_rsrc(a.sa + m, inside ? (a.M - m) * 4 : 0);
    const auto cols = uniform_rsrc(a.sb + n, inside ? (a.N - n) * 4 : 0);
    const auto br = uniform_rsrc(a.bias + n, a.bias && inside ? (a.N - n) * 4 : 0);
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sa[f][e] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            rows, (lane >> 4) * 16 + f * 64 + e * 4, 0, 0));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = (lane & 15) * 16 + h * (HALF * 64) + e * 4;
        sb[h][e] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(cols, at, 0, 0));
        bias[h][e] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(br, at, 0, 0));
      }
  }
  // Whether a scale of A is so large that B's has to come first.
  __device__ __forceinline__ bool large() const {
    bool any = false;
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) any |= fabsf(sa[f][e]) > kLargeScale;
    return __builtin_amdgcn_readfirstlane((int)(__builtin_amdgcn_ballot_w64(any) != 0)) != 0;
  }
  // the tile that is carried: rows past M lie outside the buffer's range, lanes whose columns lie past
  // N (a multiple of four) store outside it
  __device__ __forceinline__ void set(const Int8Args &a, int64_t m0, int64_t n0, int lane) {
    const bool inside = m0 < a.M && n0 < a.N;
    const int64_t origin = inside ? m0 * a.N + n0 : 0;
    cr = uniform_rsrc(a.C + origin * ES, (a.M * a.N - origin) * ES);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = (lane & 15) * 4;
      const bool ok = inside && n0 + h * (HALF * 16) + at < a.N;
      st_off[h] =
          ok ? (uint32_t)(lane >> 4) * 4 * pitch_of(a) + (h * (HALF * 16) + at) * ES : kOOB;
    }
  }
  static __device__ __forceinline__ uint32_t pitch_of(const Int8Args &a) { return (uint32_t)a.N * ES; }
  __device__ __forceinline__ void clear(const Int8Args &a) {
    cr = uniform_rsrc(a.C, 0);
    st_off[0] = st_off[1] = 0;
  }
  __device__ __forceinline__ void begin(const Int8Args &a) {
    pitch = pitch_of(a);
    // keeps the compiler from forming the addresses of all writes ahead of time
    asm volatile("" : "+v"(wa), "+v"(ra));
    asm volatile("" : "+s"(pitch));
  }
  template <int H, int J>
  __device__ __forceinline__ i32x4 read() {
    return *(p128)(size_t)((ra ^ (J * 16)) + H * 4096 + J * 256);
  }
  template <int F, int H, int J>
  __device__ __forceinline__ void store(const i32x4 &t) {
    f32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf((float)t[e] * sa[F][J], sb[H][e], bias[H][e]);
    // rows are whole: past M the lane's offset, of its row in it, leaves the range
    const uint32_t off = st_off[H] + (uint32_t)(F * 16 + J) * pitch;
    if constexpr (ES == 2)
      __builtin_amdgcn_raw_buffer_store_b64(
          u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])}, cr, off, 0, kNonTemporal);
    else
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), cr, off, 0, kNonTemporal);
  }
  // a block's sums to half H, where it is block E
  template <int H, int E>
  __device__ __forceinline__ void put(const i32x4 &block) {
    *(p128)(size_t)((wa ^ (E * 64)) + H * 4096) = block;
  }
  template <int F, int G>
  __device__ __forceinline__ void slot(const i32x4 &block) {
    // of the half that was written before this one, read j in slot j and its store in the next
    constexpr int H = G / HALF, j = G % HALF, OF = H ? F : F - 1;
    if constexpr (j > 0 && OF >= 0) store<OF, 1 - H, j - 1>(v);
    if constexpr (j == 0 && F >= 1) store<F - 1, H, 3>(v);
    if constexpr (OF >= 0) v = read<1 - H, j>();
    put<H, j>(block);
  }
  __device__ __forceinline__ void finish() {
    store<FM - 1, 0, 3>(v);
    const i32x4 x0 = read<1, 0>(), x1 = read<1, 1>(), x2 = read<1, 2>(), x3 = read<1, 3>();
    store<FM - 1, 1, 0>(x0);
    store<FM - 1, 1, 1>(x1);
    store<FM - 1, 1, 2>(x2);
    store<FM - 1, 1, 3>(x3);
    __builtin_amdgcn_sched_barrier(0);
  }
  template <class ACC>
  __device__ __forceinline__ void flush(const Int8Args &a, const ACC &acc) {
    begin(a);
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (
          [&] {
            slot<I / FN, I % FN>(acc[I / FN][I % FN]);
            __builtin_amdgcn_sched_barrier(0);
          }(),
          ...);
    }(std::make_integer_sequence<int, FM * FN>());
    finish();
  }
};

template <class OUT>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
wide_int8_kernel(const Int8Args a) {
  constexpr int BM = 256, BN = 256, NW = 4, WM = BM / 2, WN = BN / 2;
  constexpr int FM = WM / 16, FN = WN / 16;
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW, L = LA + LB;
  constexpr int STAGE = (BM + BN) * 128;
  __shared__ __align__(1024) char smem_[2 * STAGE + NW * kWideSlice];
  static_assert(sizeof(smem_) <= 160 * 1024, "LDS");
  lds_t *const smem = (lds_t *)smem_;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  typedef f32x4 __attribute__((address_space(3))) *f4p;
  lds_t *const slice = smem + 2 * STAGE + wave * kWideSlice;
  const int wm = wave / 2, wn = wave % 2, r16 = lane & 15, g4 = lane >> 4;

  // ---- producer: the k-block to load next, and where its tile lies
  int32_t pround = 0, pk = 0;
  __amdgpu_buffer_rsrc_t ra = uniform_rsrc(a.A, 0), rb = ra;
  const uint32_t row0 = wave * 8 + lane / 8;
  const uint32_t chunk = ((lane % 8) ^ ((row0 >> 1) & 7)) * 16;
  const uint32_t stepa = NW * 8 * (uint32_t)a.lda, stepb = NW * 8 * (uint32_t)a.ldb;
  const uint32_t oa = row0 * (uint32_t)a.lda + chunk, ob = row0 * (uint32_t)a.ldb + chunk;
  auto producer_tile = [&] {
    int64_t m0, n0;
    if (tile_at(a, blockIdx.x, pround, BM, BN, m0, n0)) {
      const int32_t rows_a = (int32_t)(a.M - m0 < BM ? a.M - m0 : BM);
      const int32_t rows_b = (int32_t)(a.N - n0 < BN ? a.N - n0 : BN);
      ra = uniform_rsrc(a.A + m0 * a.lda, rows_a * a.lda);
      rb = uniform_rsrc(a.B + n0 * a.ldb, rows_b * a.ldb);
    } else {   // empty ranges read as zeros
      ra = uniform_rsrc(a.A, 0);
      rb = ra;   // (in the order of the other branch, or both are kept in memory)
    }
  };
  uint32_t la, lb;
  lds_t *to;
  auto begin = [&](int stage) {
    const uint32_t k = (uint32_t)pk * 128;
    const bool past = k + chunk >= (uint32_t)a.kbytes;
    la = past ? kOOB : oa + k;
    lb = past ? kOOB : ob + k;
    to = smem + stage * STAGE + wave * 1024;
  };
  // load J of the k-block: eight rows of A or of B.  A row past the tile's edge lies past its
  // buffer's range and reads as zeros.
  auto load = [&](auto j_c) {
    constexpr int J = decltype(j_c)::value;
    if constexpr (J < LA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to + J * NW * 1024, 16, la + J * stepa, 0, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, to + BM * 128 + (J - LA) * NW * 1024, 16,
                                               lb + (J - LA) * stepb, 0, 0, 0);
  };
  auto end = [&] {
    if (++pk == a.kb) {
      pk = 0;
      ++pround;
      producer_tile();
    }
  };
  auto load_all = [&] {
    [&]<int... J>(std::integer_sequence<int, J...>) {
      (load(std::integral_constant<int, J>()), ...);
    }(std::make_integer_sequence<int, L>());
  };

  // ---- consumer
  const uint32_t x = (r16 >> 1) & 7;
  const uint32_t arow = (wm * WM + r16) * 128, brow = BM * 128 + (wn * WN + r16) * 128;
  typedef const i32x4 __attribute__((address_space(3))) *frag;
  i32x4 fa[2][FM], fb[2][FN], acc[FM][FN];
  const uint32_t ck[2] = {(g4 ^ x) * 16, ((g4 + 4) ^ x) * 16};
  // fragment E of a half: B's first
  auto read = [&](const lds_t *st, auto half_c, auto e_c) {
    constexpr int H = decltype(half_c)::value, E = decltype(e_c)::value;
    if constexpr (E < FN)
      fb[H][E] = *(frag)(st + brow + ck[H] + E * 2048);
    else
      fa[H][E - FN] = *(frag)(st + arow + ck[H] + (E - FN) * 2048);
  };

  int c = 0;
  auto handshake = [&](int step) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    begin((step + 1) & 1);
  };
  producer_tile();
  begin(0);
  load_all();
  end();
  begin(1);
  load_all();
  end();
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(L) : "memory");
  [&]<int... E>(std::integer_sequence<int, E...>) {
    (read(smem, std::integral_constant<int, 0>(), std::integral_constant<int, E>()), ...);
  }(std::make_integer_sequence<int, FM + FN>());

  OutRows<FM, FN, OUT> out;
  out.init(a, slice, lane);

  // One step.  FIRST of a tile: a block's last sums are taken from its accumulators before they start again.
  auto kstep = [&](auto first_c) {
    constexpr bool FIRST = decltype(first_c)::value;
    const lds_t *const now = smem + (c & 1) * STAGE, *const next = smem + ((c + 1) & 1) * STAGE;
    if constexpr (FIRST) out.begin(a);
    // what was moved or made ready between steps is two wait states old before an MFMA reads it
    asm volatile("s_nop 1" ::: "memory");
    int8_step<FM, FN, L>(
        [&](auto half_c, auto f_c, auto g_c) {
          constexpr int H = decltype(half_c)::value, f = decltype(f_c)::value, g = decltype(g_c)::value;
          if constexpr (FIRST && H == 0) {
            out.template slot<f, g>(acc[f][g]);
            mfma_int8_zero(acc[f][g], fb[H][g], fa[H][f]);
          } else {
            mfma_int8_inplace(acc[f][g], fb[H][g], fa[H][f]);
          }
        },
        [&](auto half_c, auto e_c) { read(decltype(half_c)::value ? now : next, half_c, e_c); },
        [&] { handshake(c + 1); }, load);
    end();
    ++c;
  };

  using ON = std::true_type;
  using OFF = std::false_type;
  int64_t m0, n0;
  bool any = tile_at(a, blockIdx.x, 0, BM, BN, m0, n0);
  // the first tile's first step writes these (unset) values out to nowhere
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < FN; ++g) acc[f][g] = __builtin_nondeterministic_value(acc[f][g]);
  for (int32_t round = 1; any; ++round) {
    kstep(ON());
    out.finish();
    const int64_t tm = m0 + wm * WM, tn = n0 + wn * WN;
    out.load(a, tm, tn, lane);   // used when the tile ends
    for (int32_t k = 1; k < a.kb; ++k) kstep(OFF());
    mfma_wait_states();
    any = tile_at(a, blockIdx.x, round, BM, BN, m0, n0);
    if (a.plain_rows && !out.large()) {
      out.set(a, tm, tn, lane);
      if (!any) out.flush(a, acc);
      continue;
    }
    // A source, columns that are no multiple of four, or a scale of A that B's has to come before: the sums go
    // through the wave's LDS, half a row of blocks at a time, the source of the next three on its way.  (8192 x
    // 8192 x 1024, fp32 C and source: 155 us, 208 with each half's source loaded in its turn.)
    out.clear(a);
    with_source(a, [&](auto src_c) {
      constexpr int SRC = decltype(src_c)::value, HALF = out.HALF;
      constexpr int DEEP = 3;   // halves of rows of blocks whose source is on its way
      u32x4 src[DEEP][4];
      const int64_t lm = tm + lane / 16 * 4, ln = tn + lane % 16 * 4;
      const auto fetch = [&](auto i_c) {
        constexpr int f = decltype(i_c)::value / 2, h = decltype(i_c)::value % 2;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          src[decltype(i_c)::value % DEEP][u] = source_at<SRC>(a, lm + f * 16 + u, ln + h * (HALF * 16));
      };
      if constexpr (SRC != SRC_NONE)
        [&]<int... I>(std::integer_sequence<int, I...>) {
          (fetch(std::integral_constant<int, I>()), ...);
        }(std::make_integer_sequence<int, DEEP>());
      [&]<int... I>(std::integer_sequence<int, I...>) {
        (
            [&] {
              constexpr int f = I / 2, h = I % 2, deep = I % DEEP;
              [&]<int... E>(std::integer_sequence<int, E...>) {
                (out.template put<h, E>(acc[f][h * HALF + E]), ...);
              }(std::make_integer_sequence<int, HALF>());
              [&]<int... U>(std::integer_sequence<int, U...>) {
                (
                    [&] {
                      const int64_t m = lm + f * 16 + U, n = ln + h * (HALF * 16);
                      const i32x4 sum = out.template read<h, U>();
                      f32x4 v;
#pragma unroll
                      for (int e = 0; e < 4; ++e)
                        v[e] = scaled((float)sum[e], out.sa[f][U], out.sb[h][e], out.bias[h][e]);
                      if constexpr (SRC != SRC_NONE) v += source_four<SRC>(a, n, src[deep][U]);
                      if (m < a.M && n < a.N) put_four_once(a, m, n, v);
                    }(),
                    ...);
              }(std::make_integer_sequence<int, 4>());
              if constexpr (SRC != SRC_NONE && I + DEEP < 2 * FM)
                fetch(std::integral_constant<int, I + DEEP>());
              __builtin_amdgcn_sched_barrier(0);
            }(),
            ...);
      }(std::make_integer_sequence<int, 2 * FM>());
    });
  }
  wait_vmcnt<0>();   // no load is on its way into LDS that the workgroup no longer has
}

}  // namespace

hipError_t launch_int8_wide(const Int8Args &a, hipStream_t s) {
  const int64_t tiles = (int64_t)a.mt * a.nt;
  const dim3 grid((uint32_t)(tiles < kWorkers ? tiles : kWorkers));
  if (a.out_bf16)
    hipLaunchKernelGGL((wide_int8_kernel<uint16_t>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((wide_int8_kernel<float>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace dg
