// Which form multiplies E4M3 codes with block scales: of few tokens (block_few.hip), or which tile (block_gemm.hip) in
// how many parts of K.  Host code by itself, for the launches, the workspace's size and the tests of both.
#pragma once

#include <algorithm>
#include <cstdint>
#include <iterator>

#include "layer.h"

namespace w8a8 {
namespace block_choice {

constexpr int kCus = 256;

// Up to 16 tokens the form of few tokens reads the weight about as fast as memory gives it.  For more, whose codes every
// workgroup reads again, up to weights of 48 Mi: 64 tokens of 5,120 x 7,168 11.4 us (12.7 with tiles), but 17,408 x 5,120
// 34.4 (22.8 with tiles).
inline bool few_fits(int64_t M, int64_t N, int64_t K) { return M <= 16 || (M <= 64 && N * K <= (48 << 20)); }

// Its workgroups quantize x themselves, a launch less, where a wave has four steps at most and the weight few blocks in
// all.  1 and 16 tokens, in us, made so and by a launch of their own: 1,024 x 1,024 3.4 and 3.8, 5.8 and 6.7; 2,048 x
// 4,096 4.9 and 6.7, 6.5 and 7.4; with four steps 4,096 x 1,024 6.7 and 8.3, 6.3 and 6.9, but 6.8 and 8.5, 8.8 and 8.9
// for calls from Python one behind the other, which a second launch holds up; with eight 8,192 x 1,024 11.0 and 13.1,
// 9.2 and 10.9, and with 128 131,072 x 64 138 and 147, 62 and 77.  (5,120 x 5,120, one token: 8.8 against 6.6 and the
// quantizer.)
constexpr int kFusedWaves = 8;
inline bool fused_fits(int64_t M, int64_t N, int64_t K) {
  return M <= 16 && K / kScaleBlock <= 4 * kFusedWaves && (N + 15) / 16 * (K / kScaleBlock) <= 4096;
}

// Tile and parts of K.  Tiles are ranked by what a launch takes, in us, of its own work (what they have in common, the
// weight's bytes, which bound few tokens, is left out: 64 x 5,120 x 34,816 counts 24 and takes 38): `begin`, `again`
// for each further round (workgroups over what the CUs hold), and for each stage of a round from `one`, where there is
// a workgroup for each CU or fewer, to `full`, where they hold all they can or take turns; parts cost a launch and the
// sums' way through memory.  Fitted to 141 shapes of 24 to 5,729 tokens, weights of 512 x 1,024 to 34,816 x 17,408: of
// the forms measured for each (every tile in one part, for 57 of the shapes in up to 16) the one that is chosen is the
// fastest or, on the mean, 0.5% behind it, 9% at most. 1,502 x 4,096 x 4,096 25.9 us with 192 x 128, 28.1 with 128 x
// 256, 42.2 with 256 x 256; 2,270 x 5,120 x 5,120 52 with 192 x 256, 56 with 256 x 256; 1,024 x 4,096 x 4,096 20.0 with
// 128 x 128, 21.4 with 64 x 256; 330 x 4,096 x 4,096 13.1 with 64 x 128, 15.0 with 64 x 64; 100 x 5,120 x 17,408 26.8
// with 128 x 128, 31.7 with 64 x 256; 64 x 5,120 x 34,816 38.1 with 64 x 256, 43.2 with 64 x 64.
struct Tile {
  int bm, bn, per_cu;
  double begin, again, one, full;
};
constexpr Tile kTiles[] = {{256, 256, 1, 7.6, 4.7, 1.219, 1.336}, {192, 256, 1, 6.5, 5.4, 1.052, 1.129}, {128, 256, 1, 5.0, 4.7, 0.646, 0.798},
                           {64, 256, 1, 3.8, 2.9, 0.501, 0.566},  {192, 128, 1, 4.9, 3.5, 0.545, 0.614}, {128, 128, 1, 4.3, 2.5, 0.429, 0.486},
                           {64, 128, 2, 4.0, 1.7, 0.267, 0.594},  {64, 64, 3, 3.5, 1.3, 0.257, 0.571}};
inline double time_of(const Tile& c, int64_t groups, int stages) {
  const int64_t room = (int64_t)kCus * c.per_cu, rounds = groups <= room ? 1 : (groups + room - 1) / room;
  const int64_t held = std::min<int64_t>((groups + kCus - 1) / kCus, c.per_cu);
  const double busy = c.per_cu == 1 ? groups > kCus : (double)(held - 1) / (c.per_cu - 1);
  return c.begin + c.again * (rounds - 1) + (double)rounds * stages * (c.one + (c.full - c.one) * busy);
}
struct Choice {
  int tile, splits;
};
inline Choice choose(int64_t M, int64_t N, int64_t K) {
  const int blocks = (int)(K / kScaleBlock);
  Choice best{0, 1};
  double least = 1e30;
  for (int t = 0; t < (int)std::size(kTiles); ++t) {
    const Tile& c = kTiles[t];
    const int64_t tiles = (M + c.bm - 1) / c.bm * ((N + c.bn - 1) / c.bn);
    // (walking needs a few blocks of columns, and rows of outputs within 2^31 bytes of a tile's first)
    if (t == 0 && (blocks < 4 || N > (1 << 21))) continue;
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (t == 0 || blocks < 4 * splits || tiles * splits > 2 * kCus * c.per_cu)) break;
      const int stages = (blocks + splits - 1) / splits;
      if (splits > 1 && (splits - 1) * stages >= blocks) continue;   // (a part without a block)
      const double time = time_of(c, tiles * splits, stages) + (splits > 1 ? 2.8 + splits * 1.5e-6 * M * N : 0.0);
      if (time < least) least = time, best = {t, splits};
    }
  }
  return best;
}

}  // namespace block_choice
}  // namespace w8a8
