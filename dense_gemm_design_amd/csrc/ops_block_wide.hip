// Large tiles of the block-scaled product with a bf16 C: four waves, each alone on its SIMD with 128
// columns and half of the tile's rows, so the instruction stream is laid out by hand, one k-block a
// step.  In each slot between two MFMAs goes a share of what the next steps need: a fragment is read
// again right after its last MFMA, and the loads of the step after the next go out once the waves have
// met (the next step's have landed, this step's fragments are all read).  The first two and the last
// two rows of blocks are taken column by column, so that the reads of B's fragments have 16 slots,
// about what LDS takes for them, and 14 more before their next MFMA.
//  * Powers of two, 256 x 256: the 256 accumulators of a lane stay in accumulation registers, and
//    the MFMA adds to them.  8192^3 in 401 us on inputs that change from call to call, 2.74 PFLOP/s (the
//    product with one scale a tensor takes as long); the matrix units are busy 0.70 of the time, at the
//    2.01 GHz that the card then holds.
//  * fp32 scales of 128 x 128 blocks of B, 192 x 256: vector instructions reach only the other 256
//    registers, so there the 192 accumulators have to be, and the fragments go to the accumulation
//    registers.  A wave's columns are one block of B, whose power of two the MFMA applies; what is left of
//    that scale, times A's, is one a row.  An MFMA's four results are added two slots later, when they
//    have left the matrix unit.  4096 x 14336 x 4096 with a bias in 247 us between other launches, 1.95
//    PFLOP/s, and 265 one after the other (4 % less with the scales' product formed first, which left the
//    range of fp32 where C does not).  The matrix units are busy 0.44 of the time, a wave issues for 0.58,
//    waits to issue for 0.16 and for memory, LDS or the barrier for 0.17: none of them fills it, and the time
//    is near the sum of the MFMAs' and the additions', as if they overlapped little.  Why is not known.
// Workgroups stay for tile after tile: the loads of the next one are under way when a tile ends, and
// what a tile leaves in the registers is written out beside the next one's first step (written at
// once by all CUs, the 33 MB of a round took 8 us in which nothing was multiplied).
#include "ops_block.h"

namespace dg {
namespace {

constexpr int kWorkers = 256;   // one a CU

__device__ __forceinline__ void mfma_scaled_inplace(f32x4 &c, const i32x8 &b, const i32x8 &a,
                                                    int eb, int ea) {
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
               : "+a"(c)
               : "v"(b), "v"(a), "v"(eb), "v"(ea));
}
__device__ __forceinline__ void mfma_scaled_zero(f32x4 &c, const i32x8 &b, const i32x8 &a, int eb,
                                                 int ea) {
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel_hi:[0,0,0]"
               : "=a"(c)
               : "v"(b), "v"(a), "v"(eb), "v"(ea));
}

// Corner of the tile of worker b in a round; false if it has none.  The workers of an XCD (b mod 8)
// take neighbouring tiles: strips of eight rows of tiles, walked down first.
__device__ __forceinline__ bool tile_at(const BlockArgs &a, int32_t b, int32_t round, int bm, int bn,
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

// c += z p and c = z p for the four results p of an MFMA.  Written out, they stay where they are put;
// the compiler does not see that they read p, which is two MFMAs old at the earliest (8 passes each,
// where 11 wait states are asked for), or behind mfma_wait_states().
__device__ __forceinline__ void add_scaled(f32x4 &c, const f32x4 &p, int z) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    asm volatile("v_fmac_f32 %0, %1, %2" : "+v"(c[e]) : "v"(p[e]), "v"(z));
}
__device__ __forceinline__ void set_scaled(f32x4 &c, const f32x4 &p, int z) {
#pragma unroll
  for (int e = 0; e < 4; ++e) asm volatile("v_mul_f32 %0, %1, %2" : "=v"(c[e]) : "v"(p[e]), "v"(z));
}

// The output of a wave's FM x 8 blocks of 16 x 16, written out one block at a time: block (f, g) goes
// as bf16 into one of two rows of blocks in the wave's LDS (4 KB each, 16-byte chunks swizzled), and
// beside row f's blocks row f - 1 comes back as whole rows of 256 bytes and is stored.
template <int FM, bool AGPR>
struct OutRows {
  typedef u32x2 __attribute__((address_space(3))) *p64;
  typedef u32x4 __attribute__((address_space(3))) *p128;
  __amdgpu_buffer_rsrc_t cr;
  uint32_t st_off, pitch;
  uint32_t wa, ra;   // LDS addresses of the lane's write of block column 0 and read 0
  u32x4 v[2];
  f32x4 bias[8];     // of the lane's four columns in each block column

  __device__ __forceinline__ void init(const BlockArgs &a, lds_t *slice, int lane) {
    clear(a);
    const uint32_t base = (uint32_t)(size_t)slice;
    const int row = lane & 15, q = lane >> 4;   // writes: chunk (2 g + q / 2) ^ row, half q mod 2
    wa = base + row * 256 + ((q >> 1) ^ (row & 1)) * 16 + (row >> 1) * 32 + (q & 1) * 8;
    ra = base + q * 256 + ((row ^ q) * 16);     // reads: row q (+ 4 j), chunk row ^ q (^ 4 j)
  }
  // the tile that is carried: rows past M lie outside the buffer's range, lanes whose columns lie past
  // N store outside it
  __device__ __forceinline__ void set(const BlockArgs &a, int64_t m0, int64_t n0, int lane) {
    const bool inside = m0 < a.M && n0 < a.N;
    const int64_t origin = inside ? m0 * a.N + n0 : 0;
    cr = make_rsrc(a.C + origin * 2, (a.M * a.N - origin) * 2);
    const bool ok = inside && n0 + (lane & 15) * 8 < a.N;
    st_off = ok ? (uint32_t)(lane >> 4) * ((uint32_t)a.N * 2) + (lane & 15) * 16 : kOOB;
    const auto br = make_rsrc((const char *)(a.bias + (inside ? n0 : 0)),
                              a.bias && inside ? (a.N - n0) * 4 : 0);
#pragma unroll
    for (int g = 0; g < 8; ++g)
      bias[g] = __builtin_bit_cast(
          f32x4, __builtin_amdgcn_raw_buffer_load_b128(br, (lane >> 4) * 16 + g * 64, 0, 0));
  }
  // nothing is carried: the stores go to an empty range
  __device__ __forceinline__ void clear(const BlockArgs &a) {
    cr = make_rsrc(a.C, 0);
    st_off = 0;
#pragma unroll
    for (int g = 0; g < 8; ++g) bias[g] = f32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void begin(const BlockArgs &a) {
    pitch = (uint32_t)a.N * 2;
    // keeps the compiler from forming the addresses of all writes ahead of time
    asm volatile("" : "+v"(wa), "+v"(ra));
    asm volatile("" : "+s"(pitch));
  }
  template <int F, int J>
  __device__ __forceinline__ u32x4 read() {
    return *(p128)(size_t)((ra ^ (J * 64)) + ((F % 2) * 4 + J) * 1024);
  }
  template <int F, int J>
  __device__ __forceinline__ void store(const u32x4 &x) {
    // rows are whole: past M the lane's offset, of its row in it, leaves the range
    __builtin_amdgcn_raw_buffer_store_b128(x, cr, st_off + (uint32_t)(F * 16 + J * 4) * pitch, 0, 0);
  }
  template <int F, int G>
  __device__ __forceinline__ void slot(const f32x4 &block) {
    if constexpr (F >= 1 && G % 2 == 0) {
      if constexpr (G >= 2)
        store<F - 1, G / 2 - 1>(v[(G / 2 - 1) % 2]);
      else if constexpr (F >= 2)
        store<F - 2, 3>(v[1]);
      v[(G / 2) % 2] = read<F - 1, G / 2>();
    }
    const f32x4 x = quad_of<AGPR>(block, 0) + bias[G];
    *(p64)(size_t)((wa ^ (G * 32)) + (F % 2) * 4096) =
        u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
  }
  __device__ __forceinline__ void finish() {
    constexpr int F = FM - 1;
    store<F - 1, 3>(v[1]);
    const u32x4 x0 = read<F, 0>(), x1 = read<F, 1>(), x2 = read<F, 2>(), x3 = read<F, 3>();
    store<F, 0>(x0);
    store<F, 1>(x1);
    store<F, 2>(x2);
    store<F, 3>(x3);
    __builtin_amdgcn_sched_barrier(0);
  }
  template <class ACC>
  __device__ __forceinline__ void flush(const BlockArgs &a, const ACC &acc) {
    begin(a);
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (
          [&] {
            slot<I / 8, I % 8>(acc[I / 8][I % 8]);
            __builtin_amdgcn_sched_barrier(0);
          }(),
          ...);
    }(std::make_integer_sequence<int, FM * 8>());
    finish();
  }
};

// The block of each of a step's slots: row by row, or PAIRED, with the first and the last two rows
// taken column by column; and the last slot of a row, or of a column, of blocks.
template <int FM, bool PAIRED>
struct Order {
  static constexpr int NM = FM * 8;
  static constexpr int row(int i) {
    if (PAIRED && i < 16) return i % 2;
    if (PAIRED && i >= NM - 16) return FM - 2 + i % 2;
    return i / 8;
  }
  static constexpr int col(int i) {
    return PAIRED && (i < 16 || i >= NM - 16) ? i % 16 / 2 : i % 8;
  }
  static constexpr int last_of_row(int f) {
    int last = 0;
    for (int i = 0; i < NM; ++i) last = row(i) == f ? i : last;
    return last;
  }
  static constexpr int last_of_col(int g) {
    int last = 0;
    for (int i = 0; i < NM; ++i) last = col(i) == g ? i : last;
    return last;
  }
};

template <bool POW2, bool ROWB>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
wide_block_kernel(const BlockArgs a) {
  constexpr int BM = wide_rows(POW2), BN = 256, NW = 4, WM = BM / 2, WN = 128;
  constexpr int FM = WM / 16, FN = WN / 16, NM = FM * FN;
  static_assert(POW2 || !ROWB, "fp32 scales are one a row of the wave's sub-tile");
  static_assert(NM % 4 == 0, "the ring of results turns a whole number of times a step");
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
  struct Scales {   // of the wave's rows and columns in one k-block, and how many bytes of them there are
    const float *a, *b;
    int32_t rows, cols;
  };
  int32_t pround = 0, pk = 0;
  __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, 0), rb = ra;
  Scales ps{a.sa, a.sb, 0, 0};
  const uint32_t row0 = wave * 8 + lane / 8;
  const uint32_t chunk = ((lane % 8) ^ ((row0 >> 1) & 7)) * 16;
  const uint32_t stepa = NW * 8 * (uint32_t)a.lda, stepb = NW * 8 * (uint32_t)a.ldb;
  const uint32_t oa = row0 * (uint32_t)a.lda + chunk, ob = row0 * (uint32_t)a.ldb + chunk;
  auto producer_tile = [&] {
    int64_t m0, n0;
    if (tile_at(a, blockIdx.x, pround, BM, BN, m0, n0)) {
      const int32_t rows_a = (int32_t)(a.M - m0 < BM ? a.M - m0 : BM);
      const int32_t rows_b = (int32_t)(a.N - n0 < BN ? a.N - n0 : BN);
      ra = make_rsrc(a.A + m0 * a.lda, rows_a * a.lda);
      rb = make_rsrc(a.B + n0 * a.ldb, rows_b * a.ldb);
      // a sub-tile wholly past the edge reads no scales, from the start of the tile's
      const int32_t rm = rows_a - wm * WM, rn = rows_b - wn * WN;
      ps.rows = __builtin_amdgcn_readfirstlane(rm > 0 ? rm * 4 : 0);
      ps.cols = __builtin_amdgcn_readfirstlane(rn > 0 ? (ROWB ? rn : 1) * 4 : 0);
      ps.a = a.sa + m0 + (rm > 0 ? wm * WM : 0);
      ps.b = a.sb + (ROWB ? n0 + (rn > 0 ? wn * WN : 0) : n0 / 128 + (rn > 0 ? wn : 0));
    } else {   // empty ranges read as zeros
      ra = rb = make_rsrc(a.A, 0);
      ps = Scales{a.sa, a.sb, 0, 0};
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
    ps.a += a.lsa;
    ps.b += a.lsb;
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
  const uint32_t c0 = (g4 ^ x) * 16, c1 = ((g4 + 4) ^ x) * 16;
  const uint32_t arow = (wm * WM + r16) * 128, brow = BM * 128 + (wn * WN + r16) * 128;
  i32x8 fa[FM], fb[FN];
  f32x4 acc[FM][FN], p[4];
  // The next step's scales as they are in memory, one of 64 rows (columns) a lane, and this step's in
  // use: exponents (POW2), or A's times what is left of B's, spread to the lanes of each block's rows,
  // and the power of two of B's.
  constexpr int XB = ROWB ? 2 : 1;
  int raw_a[2], raw_b[XB], sa[8], sb[ROWB ? 8 : 1];
  TileScale tile(0);
  auto read_a = [&](const lds_t *st, int f) {
    fa[f] = lds_frag<DT_FP8>(st + arow + c0 + f * 2048, st + arow + c1 + f * 2048);
  };
  auto read_b = [&](const lds_t *st, int g) {
    fb[g] = lds_frag<DT_FP8>(st + brow + c0 + g * 2048, st + brow + c1 + g * 2048);
  };
  __amdgpu_buffer_rsrc_t rsa, rsb;
  auto scales_at = [&](const Scales &s) {
    rsa = __builtin_amdgcn_make_buffer_rsrc((void *)s.a, (short)0, s.rows, 0x00020000);
    rsb = __builtin_amdgcn_make_buffer_rsrc((void *)s.b, (short)0, s.cols, 0x00020000);
  };
  auto read_scale = [&](int j) {
    if (j < XB)
      raw_b[j] = __builtin_amdgcn_raw_buffer_load_b32(rsb, ROWB ? lane * 4 + j * 256 : 0, 0, 0);
    else
      raw_a[j - XB] = __builtin_amdgcn_raw_buffer_load_b32(rsa, lane * 4 + (j - XB) * 256, 0, 0);
  };
  // lanes 16 f .. 16 f + 15 of x to every 16 lanes of to[f]
  auto spread = [](int x, int *to) {
    const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    to[0] = a[0];
    to[1] = a[1];
    to[2] = b[0];
    to[3] = b[1];
  };
  auto use_a = [&](int x) {   // of rows 64 x .. 64 x + 63
    if constexpr (POW2)
      spread((int)((uint32_t)raw_a[x] >> 23), sa + 4 * x);
    else
      spread(__float_as_int(tile.times(__int_as_float(raw_a[x]))), sa + 4 * x);
  };
  auto use_b = [&](int x) {
    if constexpr (ROWB)
      spread((int)((uint32_t)raw_b[x] >> 23), sb + 4 * x);
    else if constexpr (POW2)
      sb[0] = (int)((uint32_t)raw_b[0] >> 23);
    else
      sb[0] = (int)tile.bytes;
  };

  int c = 0;
  // LATER: loads that were issued after the operands' and need not have arrived
  auto handshake = [&](int step, auto later_c) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(later_c)::value)
                 : "memory");
    begin((step + 1) & 1);
  };
  producer_tile();
  begin(0);
  load_all();
  Scales cs = ps;   // of the step whose fragments are read next
  end();
  handshake(0, std::integral_constant<int, 0>());
  load_all();
  scales_at(cs);
#pragma unroll
  for (int j = 0; j < XB + 2; ++j) read_scale(j);
#pragma unroll
  for (int g = 0; g < FN; ++g) read_b(smem, g);
#pragma unroll
  for (int f = 0; f < FM; ++f) read_a(smem, f);
  cs = ps;
  end();
  if constexpr (!POW2) tile = TileScale(raw_b[0]);
  use_a(0);
  use_b(0);

  OutRows<FM, POW2> out;
  out.init(a, slice, lane);

  // adds the results of slot J of a step (the FIRST of a tile, or not) in order O
  auto add = [&](auto order, auto j_c, auto first_c) {
    using O = decltype(order);
    constexpr int J = decltype(j_c)::value, f = O::row(J), g = O::col(J);
    if constexpr (decltype(first_c)::value) {
      out.template slot<f, g>(acc[f][g]);
      set_scaled(acc[f][g], p[J % 4], sa[f]);
    } else {
      add_scaled(acc[f][g], p[J % 4], sa[f]);
    }
  };
  // One step.  FIRST of a tile: row by row, as the output wants it.  PENDING: the last two slots'
  // results of the step before are still to be added.  After the MFMA of a slot:
  //  * the scales that step c + 1 needs are loaded (raw, one load for 64 rows: a load for each of the
  //    16 rows of a block kept the path to the caches busier than the operands, 8192^3 410 us) from slot
  //    4 on.  They come into use when they have arrived and this step is done with the ones before: the
  //    first four rows' (columns') of blocks in its last slots, the others' in slots 2 and 3 of their
  //    own step;
  //  * the handshake, after slot HS; then reads of step c + 1 and loads of step c + 2.  (After slot 7,
  //    11, 15, 19, 23, 31: 8192^3 with powers of two 402, 392, 383, 380, 379, 385 us -- the loads have
  //    longer to land, the reads less time.)
  using Paired = Order<FM, true>;
  using Rows = Order<FM, false>;
  static_assert(4 + XB + 2 <= 19, "the scales' loads come before the handshake");
  constexpr int HS = 19, LW = HS + 1 + (NM - HS) * 3 / 4;
  auto kstep = [&](auto first_c, auto pending_c) {
    constexpr bool FIRST = decltype(first_c)::value, PENDING = decltype(pending_c)::value;
    using O = std::conditional_t<FIRST, Rows, Paired>;
    const lds_t *const next = smem + ((c + 1) & 1) * STAGE;
    if constexpr (FIRST) out.begin(a);
    // what was moved or made ready between steps is two wait states old before an MFMA reads it
    asm volatile("s_nop 1" ::: "memory");
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (
          [&] {
            constexpr int i = I, f = O::row(i), g = O::col(i);
            if constexpr (!POW2) {
              p[i % 4] = mfma_block_b(fb[g], fa[f], sb[0]);
              // results that are added in the next step: their MFMAs must not be moved there
              if constexpr (i >= NM - 2) asm volatile("" : "+v"(p[i % 4]));
              __builtin_amdgcn_sched_barrier(0);   // before what follows, which counts on it
              if constexpr (i >= 2)
                add(O(), std::integral_constant<int, i - 2>(), first_c);
              else if constexpr (PENDING)
                add(Paired(), std::integral_constant<int, NM - 2 + i>(), std::false_type());
            } else if constexpr (FIRST) {
              out.template slot<f, g>(acc[f][g]);
              mfma_scaled_zero(acc[f][g], fb[g], fa[f], sb[ROWB ? g : 0], sa[f]);
            } else {
              mfma_scaled_inplace(acc[f][g], fb[g], fa[f], sb[ROWB ? g : 0], sa[f]);
            }
            if constexpr (ROWB && i == 2) use_b(1);
            if constexpr (i == 3) {
              use_a(1);
              scales_at(cs);
            }
            if constexpr (i >= 4 && i - 4 < XB + 2) read_scale(i - 4);
            if constexpr (!POW2 && i == NM - 4) tile = TileScale(raw_b[0]);
            if constexpr (i == NM - 4) use_a(0);
            if constexpr (ROWB && i == NM - 3) use_b(0);
            if constexpr (i == HS) handshake(c + 1, std::integral_constant<int, XB + 2>());
            if constexpr (i >= HS) {
              // (rows that were done before it at the handshake)
              [&]<int... F>(std::integer_sequence<int, F...>) {
                (((O::last_of_row(F) > HS ? O::last_of_row(F) : HS) == i ? read_a(next, F) : void()),
                 ...);
              }(std::make_integer_sequence<int, FM>());
              if constexpr (O::last_of_col(g) == i) read_b(next, g);
              constexpr int plo = ops_before(i, L, HS, LW), phi = ops_before(i + 1, L, HS, LW);
              [&]<int... J>(std::integer_sequence<int, J...>) {
                (load(std::integral_constant<int, plo + J>()), ...);
              }(std::make_integer_sequence<int, phi - plo>());
            }
            __builtin_amdgcn_sched_barrier(0);
          }(),
          ...);
    }(std::make_integer_sequence<int, NM>());
    if constexpr (!ROWB) use_b(0);
    cs = ps;
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
    kstep(ON(), OFF());
    if constexpr (!POW2) {   // the last two slots' results, and the blocks they replace
      mfma_wait_states();
      add(Rows(), std::integral_constant<int, NM - 2>(), ON());
      add(Rows(), std::integral_constant<int, NM - 1>(), ON());
    }
    out.finish();
    if (a.kb > 1) kstep(OFF(), OFF());
    for (int32_t k = 2; k < a.kb; ++k) kstep(OFF(), ON());
    mfma_wait_states();
    if constexpr (!POW2) {
      if (a.kb > 1) {
        add(Paired(), std::integral_constant<int, NM - 2>(), OFF());
        add(Paired(), std::integral_constant<int, NM - 1>(), OFF());
      }
    }
    const int64_t tm = m0 + wm * WM, tn = n0 + wn * WN;
    any = tile_at(a, blockIdx.x, round, BM, BN, m0, n0);
    if (a.plain_rows) {
      out.set(a, tm, tn, lane);
      if (!any) out.flush(a, acc);
      continue;
    }
    // With a source, or rows that are not 16-byte aligned: through the wave's LDS as fp32,
    // half a row of blocks at a time, the source's next half on its way.
    out.clear(a);
    with_source(a, [&](auto src_c) {
      constexpr int SRC = decltype(src_c)::value;
      constexpr int QUADS = WN / 8, U = 16 * QUADS / 64;   // of half a row: a row's, and a lane's
      f32x4 bias[2];
      u32x4 src[2][U];
      const int64_t lm = tm + lane / QUADS, ln = tn + lane % QUADS * 4;
      auto fetch = [&](auto i_c) {
        constexpr int f = decltype(i_c)::value / 2, h = decltype(i_c)::value % 2;
#pragma unroll
        for (int u = 0; u < U; ++u)
          src[h][u] = source_at<SRC>(a, lm + f * 16 + u * (16 / U), ln + h * (WN / 2));
      };
#pragma unroll
      for (int h = 0; h < 2; ++h) bias[h] = bias_four(a, ln + h * (WN / 2));
      if constexpr (SRC != SRC_NONE) fetch(std::integral_constant<int, 0>());
      [&]<int... I>(std::integer_sequence<int, I...>) {
        (
            [&] {
              constexpr int f = I / 2, h = I % 2, PITCH = (WN / 2 + 4) * 4;
              [&]<int... E>(std::integer_sequence<int, E...>) {
                ((*(f4p)(slice + r16 * PITCH + E * 64 + g4 * 16) =
                      quad_of<POW2>(acc[f][h * (FN / 2) + E], 0)),
                 ...);
              }(std::make_integer_sequence<int, FN / 2>());
              if constexpr (I + 1 < 2 * FM && SRC != SRC_NONE)
                fetch(std::integral_constant<int, I + 1 < 2 * FM ? I + 1 : I>());
#pragma unroll
              for (int u = 0; u < U; ++u) {
                const int64_t m = lm + f * 16 + u * (16 / U), n = ln + h * (WN / 2);
                f32x4 v = *(f4p)(slice + (lane / QUADS + u * (16 / U)) * PITCH + lane % QUADS * 16);
                if (a.bias) v += bias[h];
                if constexpr (SRC != SRC_NONE) v += source_four<SRC>(a, n, src[h][u]);
                if (m < a.M && n < a.N) put_four(a, m, n, v);
              }
              __builtin_amdgcn_sched_barrier(0);
            }(),
            ...);
      }(std::make_integer_sequence<int, 2 * FM>());
    });
  }
  wait_vmcnt<0>();   // no load is on its way into LDS that the workgroup no longer has
}

}  // namespace

hipError_t launch_block_wide(const BlockArgs &a, bool rowb, bool pow2, hipStream_t s) {
  const int64_t tiles = (int64_t)a.mt * a.nt;
  const dim3 grid((uint32_t)(tiles < kWorkers ? tiles : kWorkers));
  if (!pow2)
    hipLaunchKernelGGL((wide_block_kernel<false, false>), grid, dim3(256), 0, s, a);
  else if (rowb)
    hipLaunchKernelGGL((wide_block_kernel<true, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((wide_block_kernel<true, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace dg
