// Which kernel a product of sv_linear takes, by its sizes alone (plain C++, so
// that the choice can be looked at without a GPU).
#pragma once

#include <algorithm>
#include <cstdint>

namespace sv {

// The tiles to choose from: rows, columns, steps of k a round, workgroups a
// compute unit holds, and the time of a round in nanoseconds, alone on its
// compute unit (lat) and among others (thr), fitted to bfloat16 products of 32
// to 1024 rows; e4m3 operands take them in the same order (pick_tile).
struct TileCost {
  int tm, tn, wk, per_cu;
  float lat, thr;
};
constexpr TileCost kTiles[] = {
    {32, 32, 4, 2, 530.0f, 450.0f},  {32, 64, 4, 1, 770.0f, 770.0f},    {64, 64, 2, 2, 550.0f, 490.0f},
    {64, 128, 2, 1, 720.0f, 900.0f}, {128, 128, 1, 2, 600.0f, 590.0f},  {128, 256, 1, 1, 850.0f, 1050.0f},
    {192, 256, 1, 1, 1150.0f, 1360.0f}, {224, 256, 1, 1, 1300.0f, 1570.0f},
};

// The tile with the least estimated time: that of the compute unit with the
// most tiles, per_cu of them at a time, their rounds and 2.5 us around each
// such turn.  Tiles of 32 rows are for products whose tiles all run at once:
// in turns they reach less of the memory's bandwidth (32 x 24576 x 4096: 45 us,
// 38 with 64 x 128).  Measured against each of them on 29 shapes, the choice is
// behind the fastest by 0.9% in the mean for bfloat16 operands, 1.3 for e4m3 to
// float32 and 0.7 for e4m3 to bfloat16, and by 15, 14 and 8% at most; 64 x 64
// everywhere, for one, takes twice as long at 448 x 128256 x 2048 (471 against
// 225 us), and 224 x 256 five times as long at 128 x 4096 x 4096 (78 against 16
// us).
inline int pick_tile(int64_t M, int64_t N, int64_t steps) {
  int best = -1;
  double least = 0.0;
  for (int i = 0; i < (int)(sizeof kTiles / sizeof *kTiles); ++i) {
    const TileCost& c = kTiles[i];
    const int64_t tiles = ((M + c.tm - 1) / c.tm) * ((N + c.tn - 1) / c.tn);
    if (c.tm == 32 && tiles > 256 * c.per_cu) continue;
    const double rounds = (double)((steps + c.wk - 1) / c.wk);
    const int64_t most = (tiles + 255) / 256, turns = most / c.per_cu, left = most % c.per_cu;
    double ns = turns * (rounds * std::max(c.lat, c.per_cu * c.thr) + 2500.0);
    if (left) ns += rounds * std::max(c.lat, left * c.thr) + 2500.0;
    if (best < 0 || ns < least) {
      least = ns;
      best = i;
    }
  }
  return best;
}

// The kernel of a product: an index of kTiles, or one of these for up to 16 rows.
enum Few : int { ROWS_16 = -1, ROWS_32 = -2 };  // 16 and 32 columns a workgroup

inline int pick_kernel(int64_t M, int64_t N, int64_t kbytes) {
  const int64_t steps = (kbytes + 127) / 128;
  if (M > 16) return pick_tile(M, N, steps);
  // Up to 8192 columns: 16 a workgroup, whose eight waves share k, so that
  // there are enough of them (16 x 1000 x 16384 bfloat16: 15.5 us, 24 with 32
  // columns and four waves; 16 x 4096 x 4096: 9.1 against 11.4).  Then 32
  // columns where rows are short, since each wave has only a few steps of one (k
  // of 4096 bytes, 16 x 128256 e4m3: 94 against 111 us; of 2048, 16 x 24576: 10.7
  // against 12.3), and 16 where they are longer (8192 bytes, 1 x 128256: 164
  // against 183 us).  Many columns with more than 8 long rows share the rows of
  // x in the tiles of larger products (16 x 128256 x 4096 bfloat16: 182 against
  // 202 us; 8 rows 181 against 177, 1 row 177 against 164).  Between 24576 and
  // 128256 columns the two are close: 16 rows of 4096 take 47 against 51 us at
  // 32000 columns, 78 against 77 at 49152, 101 against 103 at 65536, and 9 rows,
  // the other end, 47, 78 and 100 against 47, 71 and 93.
  if (N <= 8192) return ROWS_16;
  if (kbytes <= 4096) return ROWS_32;
  return M <= 8 || N <= 24576 ? ROWS_16 : pick_tile(M, N, steps);
}

}  // namespace sv
