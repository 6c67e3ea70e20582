// Which kernels a product of int8 operands takes (host code): an estimate of the time that each would take.
#pragma once
#include <stdint.h>

#include <initializer_list>

#include "../../include/gemm_ops.h"

namespace dg {

constexpr int kCUs = 256;

// Sums stay in int32 up to this many blocks of 128 along K (128^2 K < 2^31); past it K is cut.
constexpr int32_t kMostBlocks = 1023;

// Kernels for tiles, and what a launch of one takes by measurement (us): each of a workgroup's items `fix`
// and, for each k-block, `alone` where few CUs are at work to `full` where all are, which then share the way
// to the caches and the power.  (At 4096 x 4096, rows against us by each kernel, smallest tile to largest:
// 64: 10.2, 14.1, 17.1; 256: 11.5, 14.4, 18.0; 512: 20, 15.7, 18.3; 1024: 36, 27, 22.0, 24.8, 30.4, 28.6, 47;
// 2048: 71, 55, 40, 46, 36, 34.8, 47.  `shifted`: 1000 x 4104 x 8192 and x 8201: 64, 71 on 64 x 128; 58, 64; 42,
// 45; 42, 45; 51, 57; 48, 60; 48, 60.)
struct TileKind {
  int32_t bm, bn;
  double fix, alone, full;
  double shifted;   // times a k-block's, where rows do not start at multiples of 128 bytes
};
constexpr TileKind kTiles[] = {
    {64, 64, 1.2, 0.185, 0.245, 1.25},
    {64, 128, 2.0, 0.32, 0.36, 1.1},
    {128, 128, 3.2, 0.385, 0.51, 1.08},
    {128, 192, 3.8, 0.52, 0.64, 1.1},
    {192, 128, 3.8, 0.52, 0.64, 1.1},
    {192, 192, 4.5, 0.70, 0.93, 1.13},
    {128, 256, 4.6, 0.64, 0.88, 1.27},
    {256, 128, 4.6, 0.64, 0.88, 1.27},
};
constexpr int kKinds = sizeof(kTiles) / sizeof(kTiles[0]);
constexpr int kWide = 256;                       // of the wide kernel's tiles
constexpr double kWideAlone = 0.95, kWideFull = 1.37, kWideShifted = 1.25;
inline bool is_shifted(const gemm_int8_desc &d) { return (d.lda | d.ldb) % 128 != 0; }
// Its rounds write beside the next one's first step; rows that are no multiple of four columns are written
// before it.  (Four rounds, 8192 x 8192 x 2048: bf16 115 us, fp32 145, and 174 on tiles of 192 x 192.)
inline double wide_fix(const gemm_int8_desc &d) {
  return d.N % 4 != 0 ? 13.0 : d.dtype_c == GEMM_BF16 ? 3.7 : 9.0;
}
constexpr double kWideOnce = 6.0;   // us before the first round and behind the last
constexpr double kLaunch = 2.2, kBytes = 5.0e6;  // us of a launch; bytes a us from memory

struct Int8Plan {
  int tiles;               // of kTiles; -1: few rows; -2: none, all columns are the wide kernel's
  int32_t wide;            // columns of the wide kernel's tiles in front
  int32_t splits, mt, nt, whole;   // whole: the tiles whose K is not cut
};

inline double rounds_of(double items, double blocks, double fix, double alone, double full) {
  const double rounds = (double)((int64_t)items / kCUs), rest = items - rounds * kCUs;
  double us = rounds * (fix + blocks * full);
  if (rest > 0) us += fix + blocks * (alone + (full - alone) * rest / kCUs);
  return us;
}

// The best of kTiles for N columns, and its time.
inline double best_tiles(const gemm_int8_desc &d, int64_t N, int64_t kb, int64_t least, Int8Plan &best) {
  double us = 1e30;
  for (int k = 0; k < kKinds; ++k) {
    TileKind t = kTiles[k];
    if (is_shifted(d)) {
      t.alone *= t.shifted;
      t.full *= t.shifted;
    }
    const int64_t mt = (d.M + t.bm - 1) / t.bm, nt = (N + t.bn - 1) / t.bn, all = mt * nt;
    const auto offer = [&](double time, int64_t splits, int64_t whole) {
      if (time >= us) return;
      us = time;
      best.tiles = k;
      best.splits = (int32_t)splits;
      best.mt = (int32_t)mt;
      best.nt = (int32_t)nt;
      best.whole = (int32_t)whole;
    };
    if (least == 1) offer(kLaunch + rounds_of((double)all, (double)kb, t.fix, t.alone, t.full), 1, all);
    // K cut for the tiles that do not fill a round: a launch, and 8 bytes an element and piece
    const int64_t whole = least == 1 ? all / kCUs * kCUs : 0, rest = all - whole;
    if (rest == 0 || (least == 1 && rest > kCUs / 2)) continue;
    for (int64_t s : {least, 2l, 3l, 4l, 6l, 8l, 12l, 16l, 24l, 32l, 48l, 64l}) {
      if (s == 1 || s < least || (s > least && (s * 4 > kb || rest * s > 2 * kCUs))) continue;
      const double items = (double)(rest * s), blocks = (double)((kb + s - 1) / s);
      offer(kLaunch + rounds_of((double)whole, (double)kb, t.fix, t.alone, t.full) +
                rounds_of(items, blocks, t.fix, t.alone, t.full) + 3.6 +
                items * (double)(t.bm * t.bn) * 2.8e-6,
            s, whole);
    }
  }
  return us;
}

inline Int8Plan plan_of(const gemm_int8_desc &d) {
  const int64_t kb = (d.K + 127) / 128;
  const int64_t least = kb > kMostBlocks ? (kb + kMostBlocks - 1) / kMostBlocks : 1;   // of pieces
  Int8Plan best{};
  double us = best_tiles(d, d.N, kb, least, best);
  const double memory = (double)(d.M + d.N) * (double)d.K / kBytes;
  if (us < kLaunch + memory) us = kLaunch + memory;
  if (d.M <= 32) {
    // Few rows: 16 columns a workgroup, that reads them and all rows of A at 34 bytes a ns, all together
    // at 7600; K in pieces where there are few columns and much of it.  (us so, and on tiles: 1 x 4096 x 4096
    // 5.9, 9.4; 16 x 4096 x 4096 6.9, 9.6; 1 x 14336 x 4096 13.0, 11.8; 16 x 16384 x 16384 76, 62.)
    const int64_t nt = (d.N + 15) / 16;
    const double group = (double)(16 + d.M) * (double)d.K;
    for (int64_t s = least; s <= 64; s = s * 2) {
      if (s > least && (nt * s > kCUs || s * 8 > kb)) break;
      double t = group / 34e3 / (double)s;
      const double way = (double)nt * group / 7.6e6;
      t = t < way ? way : t;
      t = 2.4 + (t < memory ? memory : t);
      if (s > 1) t += 2.4 + (double)(s * d.M * d.N) * 2.8e-6;
      if (t < us) {
        us = t;
        best = {-1, 0, (int32_t)s, 1, (int32_t)nt, 0};
      }
    }
    return best;
  }
  if (d.N < 4 || kb == 0 || least > 1) return best;
  // Tiles of 256 x 256: all columns or, where that leaves a last round less than half full, as many of them as
  // fill rounds of all CUs, and the others' tiles in a launch behind them.  (4096 x 14336 x 4096, 3.5 rounds:
  // all 184 us, three rounds and 256 tiles of 128 x 256 192; 4096 x 6144 x 4096, 1.5: 90, 91; 6144 x 6144 x
  // 2048, 2.25: 83, 79; 4096 x 4352 x 4096, 1.06: 89, 66.)
  const int64_t mt = (d.M + kWide - 1) / kWide, nt = (d.N + kWide - 1) / kWide;
  const double fix = wide_fix(d), times = is_shifted(d) ? kWideShifted : 1.0;
  const double alone = kWideAlone * times, full = kWideFull * times;
  const double all =
      kLaunch + kWideOnce + rounds_of((double)(mt * nt), (double)kb, fix, alone, full);
  if (all < us) {
    us = all;
    best = {-2, (int32_t)nt, 1, 0, 0, 0};
  }
  const int64_t front = mt * nt / kCUs * kCUs / mt;   // columns of tiles
  if (front > 0 && front < nt && mt * nt % kCUs < kCUs / 2) {
    Int8Plan rest{};
    const double t =
        kWideOnce + rounds_of((double)(mt * front), (double)kb, fix, alone, full) +
        best_tiles(d, d.N - front * kWide, kb, 1, rest);
    if (t < us) {
      best = rest;
      best.wide = (int32_t)front;
    }
  }
  return best;
}

}  // namespace dg
