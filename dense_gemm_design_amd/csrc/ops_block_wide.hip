// Large tiles of the block-scaled product with a bf16 C: four waves of 128 x (BN / 2), each alone on
// its SIMD, so the instruction stream is laid out by hand.  The MFMAs of a k-block go row by row;
// after row 0 the waves meet (the next block's loads have landed, this block's fragments are all
// read), and from there on each slot between two MFMAs takes a share of the next block's fragment
// reads and of the loads after that.  A has one buffer of fragments (row f is read again right after
// its last MFMA), B two.
//  * Powers of two, BN = 256: the 256 accumulators stay in accumulation registers.
//  * fp32 scales, BN = 192: vector instructions reach only the other 256 registers, so there the
//    accumulators of 128 x 96 have to be, and the fragments go to the accumulation registers.  An
//    MFMA's results are added two slots later, when they have left the matrix unit.
// Workgroups stay for tile after tile: the loads of the next one are under way when a tile ends.
#include "launch.h"
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

template <bool ROWB>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
wide_block_kernel(const BlockArgs a) {
  using CFG = CfgFp8_256w;
  constexpr int BM = 256, BN = 256, NW = 4, WM = 128, WN = 128, FM = 8, FN = 8, NM = FM * FN;
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
  struct Scales {   // of the wave's rows and columns in one k-block, and how many there are
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
      ps.rows = rm > 0 ? rm : 0;
      ps.cols = rn > 0 ? (ROWB ? rn : 1) : 0;
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
  constexpr int SB = ROWB ? FN : 1;   // scales of B a wave and k-block
  i32x8 fa[FM], fb[2][FN];
  f32x4 acc[FM][FN];
  int ea[FM], eb[2][SB];   // bits of the scales as read, then their exponents
  __amdgpu_buffer_rsrc_t rsa, rsb;
  auto scales_at = [&](const Scales &s) {
    rsa = make_rsrc((const char *)s.a, (int64_t)__builtin_amdgcn_readfirstlane(s.rows) * 4);
    rsb = make_rsrc((const char *)s.b, (int64_t)__builtin_amdgcn_readfirstlane(s.cols) * 4);
  };
  auto read_a = [&](const lds_t *st, int f) {
    fa[f] = lds_frag<DT_FP8>(st + arow + c0 + f * 2048, st + arow + c1 + f * 2048);
    ea[f] = __builtin_amdgcn_raw_buffer_load_b32(rsa, r16 * 4 + f * 64, 0, 0);
  };
  auto read_b = [&](const lds_t *st, int q, int g) {
    fb[q][g] = lds_frag<DT_FP8>(st + brow + c0 + g * 2048, st + brow + c1 + g * 2048);
    if (g < SB) eb[q][g] = __builtin_amdgcn_raw_buffer_load_b32(rsb, ROWB ? r16 * 4 + g * 64 : 0, 0, 0);
  };
  auto shift = [](int &s) { s = (int)((uint32_t)s >> 23); };

  int c = 0;
  auto handshake = [&](int step) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    begin((step + 1) & 1);
  };
  producer_tile();
  begin(0);
  load_all();
  Scales cs = ps;   // of the k-block whose fragments are read next
  end();
  handshake(0);
  load_all();
  scales_at(cs);
#pragma unroll
  for (int g = 0; g < FN; ++g) read_b(smem, 0, g);
#pragma unroll
  for (int f = 0; f < FM; ++f) read_a(smem, f);
  cs = ps;
  end();
  shift(ea[0]);
#pragma unroll
  for (int g = 0; g < SB; ++g) shift(eb[0][g]);

  // the finished tile's output, written out during the next one's first k-block
  KernelArgs ka{};
  ka.C = a.C;
  ka.M = a.M;
  ka.N = ka.ldc = a.N;
  DeferredOut<CFG> dout;
  dout.init(ka, slice, lane);

  // k-block c on buffer P of B: MFMA (f, g); then at its slot the handshake, the reads of the next
  // block (A's row f after its last MFMA, B's spread over the slots), the shifts that make exponents
  // of scales (a row's before it begins, a column's in the last slots: well after the read and two
  // slots before their first MFMA), and the loads of the block after that, over half of the slots.
  constexpr int HS = FN, RB = NM - 2 * FN, LW = HS + (NM - HS) / 2;
  auto kstep = [&](auto p_c, auto first_c) {
    constexpr int P = decltype(p_c)::value, Q = P ^ 1;
    constexpr bool FIRST = decltype(first_c)::value;
    const lds_t *const next = smem + ((c + 1) & 1) * STAGE;
    scales_at(cs);
    if constexpr (FIRST) dout.begin();
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (
          [&] {
            constexpr int i = I, f = i / FN, g = i % FN;
            if constexpr (FIRST) {
              dout.template slot<f, g>(acc[f][g], 1.0f);
              mfma_scaled_zero(acc[f][g], fb[P][g], fa[f], eb[P][ROWB ? g : 0], ea[f]);
            } else {
              mfma_scaled_inplace(acc[f][g], fb[P][g], fa[f], eb[P][ROWB ? g : 0], ea[f]);
            }
            if constexpr (g == FN - 4) shift(ea[(f + 1) % FM]);
            if constexpr (i + 1 == HS) handshake(c + 1);
            if constexpr (i + 1 >= HS) {
              if constexpr (g == FN - 1) read_a(next, f);
              constexpr int blo = ops_before(i, FN, HS, RB), bhi = ops_before(i + 1, FN, HS, RB);
              [&]<int... E>(std::integer_sequence<int, E...>) {
                (read_b(next, Q, blo + E), ...);
              }(std::make_integer_sequence<int, bhi - blo>());
              if constexpr (f == FM - 1 && g < FN - 2) {
                if constexpr (g < SB) shift(eb[Q][g]);
                if constexpr (g < 2 && FN - 2 + g < SB) shift(eb[Q][FN - 2 + g]);
              }
              constexpr int plo = ops_before(i, L, HS, LW), phi = ops_before(i + 1, L, HS, LW);
              [&]<int... J>(std::integer_sequence<int, J...>) {
                (load(std::integral_constant<int, plo + J>()), ...);
              }(std::make_integer_sequence<int, phi - plo>());
            }
            __builtin_amdgcn_sched_barrier(0);
          }(),
          ...);
    }(std::make_integer_sequence<int, NM>());
    cs = ps;
    end();
    ++c;
  };

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  int64_t m0, n0;
  bool any = tile_at(a, blockIdx.x, 0, BM, BN, m0, n0);
  // the first tile's first k-block writes these (unset) values out to nowhere
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < FN; ++g) acc[f][g] = __builtin_nondeterministic_value(acc[f][g]);
  for (int32_t round = 1; any; ++round) {
    dout.ldc_b = (uint32_t)a.N * 2;
    // a tile starts on buffer 0; after an odd count of k-blocks what is in buffer 1 moves over
    kstep(I0(), std::true_type());
    dout.finish();
    int32_t k = 1;
    for (; k + 2 <= a.kb; k += 2) {
      kstep(I1(), std::false_type());
      kstep(I0(), std::false_type());
    }
    if (k < a.kb) {
      kstep(I1(), std::false_type());
    } else {
#pragma unroll
      for (int g = 0; g < FN; ++g) fb[0][g] = fb[1][g];
#pragma unroll
      for (int g = 0; g < SB; ++g) eb[0][g] = eb[1][g];
    }
    const int64_t tm = m0, tn = n0;
    any = tile_at(a, blockIdx.x, round, BM, BN, m0, n0);
    if (a.plain_rows) {
      WorkItem w{};
      w.m = (int32_t)(tm / BM);
      w.n = (int32_t)(tn / BN);
      dout.set(ka, w, wm, wn, lane);
      if (!any) {
        mfma_wait_states();
        dout.flush(acc, 1.0f);
      }
      continue;
    }
    // With a bias, a source or rows that are not 16-byte aligned: through the wave's LDS as fp32,
    // half a row of blocks at a time, and an epilogue that is not unrolled over the accumulators.
    dout.clear(ka);
    mfma_wait_states();
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (
          [&] {
            constexpr int f = I / 2, h = I % 2, PITCH = (WN / 2 + 4) * 4;
            [&]<int... E>(std::integer_sequence<int, E...>) {
              ((*(f4p)(slice + r16 * PITCH + E * 64 + g4 * 16) =
                    quad_of<true>(acc[f][h * (FN / 2) + E], 0)),
               ...);
            }(std::make_integer_sequence<int, FN / 2>());
            constexpr int QUADS = WN / 8;   // of half a row
#pragma unroll 1
            for (int q = lane; q < 16 * QUADS; q += 64) {
              const int64_t m = tm + wm * WM + f * 16 + q / QUADS;
              const int64_t n = tn + wn * WN + h * (WN / 2) + q % QUADS * 4;
              if (m < a.M && n < a.N)
                store_four(a, m, n, *(f4p)(slice + q / QUADS * PITCH + q % QUADS * 16));
            }
          }(),
          ...);
    }(std::make_integer_sequence<int, 2 * FM>());
  }
  wait_vmcnt<0>();   // no load is on its way into LDS that the workgroup no longer has
}

}  // namespace

hipError_t launch_block_wide(const BlockArgs &a, bool rowb, hipStream_t s) {
  const int64_t tiles = (int64_t)a.mt * a.nt;
  const dim3 grid((uint32_t)(tiles < kWorkers ? tiles : kWorkers));
  if (rowb)
    hipLaunchKernelGGL(wide_block_kernel<true>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(wide_block_kernel<false>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace dg
