// mx_plan.h -- which tile a dense fused product and a dense gradient take, by an estimate of
// the time from the sizes alone (host only; internal to libnf4).
#pragma once

#include <stdint.h>

namespace nf4 {
namespace mx {

// Workgroups that a CU of the fullest XCD gets of `tiles` x `cols` ones: make_grid deals
// groups of eight row tiles times a column block out to eight XCDs of 32 CUs.
inline int64_t workgroups_a_cu(int64_t tiles, int64_t cols) {
  const int64_t group = tiles < 8 ? tiles : 8, whole = tiles < 8 ? 1 : tiles >> 3, rest = tiles < 8 ? 0 : tiles & 7;
  return (((whole * cols + 7) >> 3) * group + ((cols + 7) >> 3) * rest + 31) >> 5;
}

// The tile of a dense product with an epilogue, of more than 16 rows, by an estimate of the
// time: a CU takes up to `places` workgroups at once, which take `full` us for 64 k of a
// K-group, and one alone `one`; kFill is what start and epilogue cost, in such stages.  Fitted to 1200
// measurements of mx_linear, 117 sizes of 17 to 4096 rows with all tiles.  The estimate's choice is
// 1.5 % off the fastest on average (24 % at most); the rules by counts of tiles that the plain
// products keep (so that their bits stay) 7 % (54 %).  The loss takes it, too: over 28 sizes of
// 24 to 2047 rows of heads of 32000 x 4096, 50257 x 1600 and 128256 x 4096 it is 1.2 % off (12 %
// at most, 1000 x 50257 x 1600: 96 x 128 174 us, 128 x 256 155).
// Us on four cards, weights from memory, M x N x K with a bias, taken, and others:
//   96 x 128    700 x 11008 x 4096   65-68   128 x 256: 95-99 (258 tiles on 256 CUs)
//   96 x 128    333 x 13824 x 5120   57-62   64 x 128: 64-65
//   32 x 64     411 x 1703 x 3744       17   64 x 128: 25
//   32 x 64     31 x 17241 x 5216    30-31   32 x 128: 35; two K-groups: 36
constexpr int kDenseTiles = 11;
inline int dense_tile(int64_t M, int64_t N, int64_t K) {
  struct Tile {
    int rows, col_shift, groups, places;  // columns as log2, 0: 192; groups: K-groups of a workgroup
    float one, full;
  };
  static constexpr Tile kTiles[kDenseTiles] = {
      {128, 8, 1, 2, 0.775f, 1.266f}, {128, 0, 1, 2, 0.67f, 0.953f},  {128, 7, 1, 2, 0.507f, 0.683f},
      {96, 7, 1, 3, 0.489f, 0.702f},  {64, 7, 1, 2, 0.255f, 0.414f},  {32, 7, 1, 3, 0.23f, 0.415f},
      {32, 6, 1, 2, 0.143f, 0.229f},  {32, 6, 2, 1, 0.227f, 0.227f},  {16, 6, 1, 3, 0.126f, 0.23f},
      {16, 6, 2, 1, 0.177f, 0.177f},  {16, 5, 4, 1, 0.196f, 0.196f}};
  constexpr float kFill = 11.6f;
  int best = 0;
  float least = 0.f;
  for (int i = 0; i < kDenseTiles; ++i) {
    const Tile &t = kTiles[i];
    const int64_t cols = t.col_shift ? (N + (1 << t.col_shift) - 1) >> t.col_shift : (N + 191) / 192;
    const int64_t a_cu = workgroups_a_cu((M + t.rows - 1) / t.rows, cols);
    const int64_t turns = a_cu / t.places;
    const int left = (int)(a_cu - turns * t.places);
    float cost = (float)turns * t.full;
    if (left > 0) cost += t.one + (left > 1 ? (t.full - t.one) * (float)(left - 1) / (float)(t.places - 1) : 0.f);
    cost *= (float)K / (float)(64 * t.groups) + kFill;
    if (i > 0 && cost >= least) continue;
    best = i;
    least = cost;
  }
  return best;
}

// A dense gradient has few tiles where rows are few, so the n may be shared out over the
// workgroups of a tile: parts of the sum in fp32, added in order by whoever takes them.
struct DensePlan {
  int mf, wv, kg, splits;
};
// Tile and splits by an estimate of the time.  A CU takes two workgroups of 256 threads or one
// of 512 at once; a workgroup takes a time for every stage of 64 n of its K-groups, and two together
// less than twice that.  `one`, `two`, kFill (stages' worth of start and end) and the cost of
// the parts (us, and us a MB) are fitted to 1090 measurements, 43 sizes of 1 to 4096 rows
// each with all tiles and up to 32 splits, and the plan so found is the fastest measured or
// within 1 % at all but four of the small ones (4-6 %).  Measured, us with the sum of the
// parts, weights from memory, on four cards, M x N x K, taken (splits), and others:
//    16 x 28672 x 4096    16 x 256, two K-groups (16)     22   32 x 256 (16): 22.4
//    77 x 13824 x 5120    32 x 256, two K-groups (4)   30-31   (8): 31; 64 x 512, two (12): 34
//   200 x 19360 x 4992    64 x 512, two K-groups (6)   64-67   32 x 256, two (2): 100, (1): 125
//   512 x 4096 x 4096     32 x 256, two K-groups (1)   29-31   64 x 512, two (4): 42
//  1000 x 13824 x 5120    64 x 512 (3)               148-164   two K-groups (1): 166-171
//  2048 x 4096 x 4096     64 x 512, two K-groups (1)   62-72   64 x 512 (2): 90-93
//  2048 x 28672 x 4096    64 x 512, two K-groups (1) 381-392   64 x 512 (2): 400-407
inline DensePlan plan_dense(int64_t M, int64_t N, int64_t K) {
  struct Tile {
    DensePlan plan;
    int row_shift, col_shift;  // log2 of the tile
    float one, two;            // us a stage of one workgroup on a CU, of two
  };
  static constexpr Tile kTiles[] = {{{1, 2, 2, 1}, 4, 8, 0.65f, 1.12f},
                                    {{2, 2, 2, 1}, 5, 8, 0.72f, 1.13f},
                                    {{4, 4, 1, 1}, 6, 9, 0.88f, 1.43f},
                                    {{4, 4, 2, 1}, 6, 9, 1.5f, 3.f}};
  static constexpr int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32};
  constexpr float kFill = 2.35f, kParts = 4.5f, kPartsMb = 0.43f;
  constexpr int64_t kPartsBytes = int64_t(256) << 20;
  const int stages = (int)((N + 63) >> 6);
  DensePlan best{};
  float least = 0.f;
  for (const Tile &t : kTiles) {
    if (t.plan.mf == 1 ? M > 64 : t.plan.mf == 4 && M <= 16) continue;
    const int64_t rows = (M + (1 << t.row_shift) - 1) >> t.row_shift;
    const int64_t cols = (K + (1 << t.col_shift) - 1) >> t.col_shift;
    for (const int splits : kSplits) {
      const int shares = t.plan.kg * splits;
      // at least four stages for each share
      if (splits > 1 && (stages < 4 * shares || splits * M * K * 4 > kPartsBytes)) break;
      const int64_t blocks = cols * splits;
      const int64_t a_cu = workgroups_a_cu(rows, blocks);
      float cost = ((float)(a_cu >> 1) * t.two + (float)(a_cu & 1) * t.one) *
                   ((float)((stages + shares - 1) / shares) + kFill);
      if (splits > 1) cost += kParts + kPartsMb * 4e-6f * (float)(splits * M * K);
      if (best.mf != 0 && cost >= least) continue;
      best = t.plan;
      best.splits = splits;
      least = cost;
    }
  }
  return best;
}

}  // namespace mx
}  // namespace nf4
