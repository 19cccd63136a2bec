// Host-side choices of the 8-bit and mixture-of-experts operators, free of HIP so that they can be compiled and checked alone.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace fp4 {

// A grid of `groups` workgroups of `threads` threads. One dimension of a launch holds less than 2^32 work-items, so more than
// that continue in y; the kernel's workgroup is blockIdx.y * gridDim.x + blockIdx.x, and those from `groups` on leave.
// x is a multiple of 8 wherever y > 1: workgroups go to the 8 XCDs in turn by this number.
struct Grid {
  unsigned x, y;
};
inline Grid grid_of(int64_t groups, int threads) {
  const int64_t most = (int64_t)(0xFFFFFFFFu / (unsigned)threads) / 8 * 8;
  if (groups <= most) return {(unsigned)groups, 1};
  return {(unsigned)most, (unsigned)((groups + most - 1) / most)};
}

// ---- 8-bit GEMM --------------------------------------------------------------------------------------------------------

// The tile shapes: rows of X, rows of W, workgroups that run at once on a CU, and the time of one scale block of K in us
// (one round of workgroups at K = 4096, the launch taken off; at a short K the start and end of a tile, which grow with it, count
// for more than this says, and nothing was fitted there). The least rounds times a round's time is taken; up
// to 8 rows of X, which cost little beside W, go to 16 x 16. The first three split K over the waves of a workgroup
// (gemm_fp8_split.hip); several of their workgroups run on a CU, sharing what it reads.
//   rows x N (K 4096)   16 x 16   16 x 32   32 x 32   64 x 64   128 x 64   128 x 128   the same, two a CU   256 x 256   (us)
//   1 x 14336              10.7      10.6      10.9      12.1
//   16 x 4096               5.2       5.3       5.9
//   37 x 4100               8.0       7.2       8.7      12.1
//   64 x 4096               8.6       7.4       6.5      11.6       15.2        20.6                 24.7        37
//   128 x 4096             14.1      11.4       9.5      11.8
//   64 x 14336                       24.7      16.3      12.8       16.3        21.5                 25.6        37
//   100 x 14336                                          21.8       16.5        23.7                 28.4        39
//   200 x 14336                                          40.2       31.0        24.5                 28.9        39
//   300 x 14336                                          51.3       43.4        42.3                 32.1        41
//   1024 x 14336                                          137        108        93.4                 71.4        53
//   K 8192: 1 x 28672      40.5      43.3      41.3
//   8 x 28672              41.9      45.1      43.4
//   16 x 28672             48.3      44.9      43.7
struct Shape {
  int bm, bn, per_cu;
  float cost;
};
constexpr Shape kShapes[] = {{16, 16, 1, 0.047f}, {16, 32, 1, 0.061f}, {32, 32, 1, 0.095f}, {64, 64, 1, 0.26f},
                             {128, 64, 1, 0.41f}, {128, 128, 1, 0.65f}, {128, 128, 2, 1.16f}, {256, 256, 1, 1.27f}};

inline int best_shape(int64_t M, int64_t N, int64_t K, int cus) {
  int best = 0;
  double least = 0;
  if (M <= 8) return 0;
  for (int i = 0; i < (int)(sizeof kShapes / sizeof kShapes[0]); ++i) {
    const Shape& s = kShapes[i];
    if (s.bm == 256 && K < 512) break;  // its two wave groups start with four blocks of K
    const int64_t tiles = ((M + s.bm - 1) / s.bm) * ((N + s.bn - 1) / s.bn), slots = (int64_t)s.per_cu * cus;
    const double t = (double)((tiles + slots - 1) / slots) * s.cost;
    if (i == 0 || t < least) {
      best = i;
      least = t;
    }
  }
  return best;
}

// ---- experts -----------------------------------------------------------------------------------------------------------

// Two launches that read a pair's matrices for that pair (6 us, and 3.4 TB/s or 4.7 ns a workgroup, whichever is
// longer), or five that read those of the used experts once (22 us and 4.4 TB/s), as fitted to 2 .. 250 pairs of
// matrices from 512 x 384 to 7168 x 1408, whichever is sooner; the used experts are guessed as those of evenly
// spread ids. (Two launches and five: 8 of 128 experts of 2048 x 768, 4 tokens 25 and 41 us, 16 tokens 98 and 64; 2 of
// 128 of 4992 x 128, 51 tokens 88 and 49; 5 of 64 of 512 x 384, 49 tokens 43 and 31.)
inline bool few_pairs(int T, int k, int64_t E, int64_t D, int64_t I) {
  const double pairs = (double)T * k, bytes = 1.59 * (double)D * (double)I;  // bytes: of an expert
  const double spread = (double)E * (1.0 - std::pow(1.0 - std::min(1.0, (double)k / (double)E), (double)T));
  const double groups = pairs * (double)I / 16 + (double)T * (double)D / 16;
  const double few = 6.0 + std::max(pairs * bytes / 3.4e6, groups * 4.7e-3);
  return few < 22.0 + std::min(pairs, spread) * bytes / 4.4e6;
}

// Eight waves a workgroup where K has to be split to fill the chip, and where there are workgroups enough for four on
// every CU two, or one for a short K, of which two waves would have little or nothing each: more workgroups on a CU then
// hide each other's starts. Two waves and one, us a call: 64 tokens, 6 of 64 of 4096 x 1408 (down alone) 145 and 143;
// 8 of 128 of 2048 x 768 (down) 90 and 86; 4 of 256 of 768 x 512 (both) 42 and 37; 51 tokens, 2 of 128 of 4992 x 128
// (down) 50 and 43; but up alone, K = 4096, 82 and 85. Four and eight waves at the first: 168 and 230.
// Where the two meet (6 of 64 experts, one / two waves in the product of that K, us a call): K of the first 1536 56.4 / 58.4, 2048
// 66.0 / 68.8, 2560 86.0 / 82.4, 4096 124 / 111 for 64 tokens, and 41.9 / 44.3, 49.2 / 51.4, 55.2 / 57.8, 91.9 / 82.8 for 16;
// of the second, 64 tokens, 1536 91.7 / 93.4, 2048 112 / 112, 2560 138 / 130. So from 1536 to about 2048 one wave would be up to 4%
// sooner than the two that are taken.
constexpr int kShortK = 1536;
inline int expert_waves(int64_t K, int64_t workgroups) { return workgroups < 1024 ? 8 : K <= kShortK ? 1 : 2; }

}  // namespace fp4
