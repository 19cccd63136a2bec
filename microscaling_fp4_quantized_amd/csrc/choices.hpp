// Host-side choices of the 8-bit, mixture-of-experts and attention operators, free of HIP so that they can be compiled and checked alone.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/fp4.h"

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

// ---- attention ---------------------------------------------------------------------------------------------------------

// A call of the attention operators, as far as it decides which kernels it takes.
struct AttentionCall {
  int dim;
  bool e4m3;
  int64_t T, batch;  // rows (decode: batch)
  int q_heads, heads;
  int64_t room;  // tokens of a sequence that the table has room for
  int window, sinks;
  bool side_by_side;  // a token's heads follow each other in memory
};

constexpr int kDecodeTile = 32;     // tokens
constexpr int kPromptTokens = 64;   // of a tile
constexpr int kPromptMinTiles = 4;  // of a part, where a row's tokens are split over workgroups

// Key-value heads of a decode workgroup, side by side in memory; its other waves share a head's tiles. Four heads have two waves each:
// half the pieces to join (64 sequences of 1721 tokens, 8 bits: 57 -> 51 us).
constexpr int decode_waves(int beside) { return beside == 4 ? 8 : 4; }

struct DecodeWay {
  int beside;    // 1, 2 or 4
  bool whole;    // a workgroup has a sequence, without a second launch
  int64_t most;  // pieces at most
  int wide;      // query heads of a workgroup of the join; 0: no join
};

inline DecodeWay decode_way(const AttentionCall& c, int cus) {
  DecodeWay way{1, false, 1, 0};
  // heads that lie side by side, in rows of 256 bytes at most: up to 512 bytes of them to a workgroup
  const int bytes = c.dim * (c.e4m3 ? 1 : 2);
  if (c.side_by_side && bytes <= 256) way.beside = bytes <= 128 && c.heads % 4 == 0 ? 4 : c.heads % 2 == 0 ? 2 : 1;
  const int waves = decode_waves(way.beside), ways = waves / way.beside;
  const int blocks = (c.q_heads / c.heads + 15) / 16, together = c.heads / way.beside;
  // what the longest sequence that the table has room for can be cut into
  int64_t tokens = c.room;
  if (c.window && (int64_t)c.window + c.sinks + 2 * kDecodeTile < tokens) tokens = (int64_t)c.window + c.sinks + 2 * kDecodeTile;
  const int64_t longest = (tokens + kDecodeTile - 1) / kDecodeTile + (c.window ? 1 : 0);
  // Short sequences are not cut: a workgroup has one, and there is nothing to join. Up to 5 tiles a wave, and up to 10 where the workgroups
  // fill the CUs, four times over if lengths can differ. Us cut and whole, 32 over 8 heads of 128: 16 sequences of up to 101 tokens 11.6 / 5.0,
  // 64 of 251 16.2 / 11.5, 128 of 10 to 1001 35.8 / 30.6, 256 of them 67.8 / 65.7, 37 with a window of 1024 in 8 bits 23.3 / 21.2; but 1 of 1001
  // 9.4 / 17.6, 64 of 10 to 1001 22.1 / 23.1, 64 of 10 to 2001 27.8 / 40.0.
  const int64_t workgroups = c.batch * together * blocks * (waves / 4);
  way.whole = longest <= 5 * ways || (longest <= 10 * ways && workgroups >= (int64_t)cus * (tokens < c.room ? 1 : 4));
  const int64_t needed = (longest * c.batch + ways - 1) / ways;
  // more units can round up to more pieces than fewer do, and the workspace is for the fewest
  const int64_t pieces = std::min<int64_t>(FP4_ATTENTION_PIECES(c.batch, together * blocks * (waves / 4)),
                                           FP4_ATTENTION_PIECES(c.batch, FP4_ATTENTION_UNITS_(c.q_heads, c.heads)));
  way.most = std::min(needed, pieces);
  // few rows: all lanes to the pieces of one (both ways, us: 1 x 131000 tokens 90 / 93, 64 sequences 64.5 / 61.4)
  if (!way.whole && way.most > 1) way.wide = c.batch * c.q_heads >= 1024 ? 1024 / c.dim : 1;
  return way;
}

// Parts of so many tiles that are worth a workgroup each. Few rows are joined quickly: up to 32 parts of half the size for them. Us with and
// without: 16 tokens behind 1000 13.8 / 16.1, 8 of 16 heads of 256 behind 600 18.3 / 23.0; but 300 tokens, all for one of their own, 18.0 / 17.1,
// 64 of 16 heads behind 8000 in 64 parts and not 32 24.8 / 19.5.
constexpr int64_t worth(int64_t tiles, int64_t T, int q_heads, int dim) {
  const int64_t parts = (tiles + kPromptMinTiles - 1) / kPromptMinTiles, fine = (tiles + 1) / 2;
  return T * q_heads * dim > (1 << 18) || parts >= 32 ? parts : fine < 32 ? fine : 32;
}

// Whether eight waves share what is brought into LDS, where there are rows for them: 310 us at 8192 tokens and heads of 64, with workgroups
// of four waves 338; 582 and 623 with heads of 128 in 8 bits. Heads of 64 in 8 bits need more than the 128 registers that four waves of a
// SIMD have, and do better with three of 168 in workgroups of four waves (a window of 1024: 499 us, 607 with eight waves and 37 registers
// spilled); heads of 256 fill the registers of a SIMD with one wave. No variant may keep anything in scratch memory: the loop would wait for
// it, and with it for the next tile's loads. Where tokens are split, heads of 64 are sooner with four waves (512 rows of 64 heads in two
// parts 187 us, with eight 215).
constexpr bool prompt_eight(int dim, bool e4m3, bool split) { return dim == 128 || (dim == 64 && !e4m3 && !split); }

struct PromptWay {
  int waves;   // 4 or 8, of 32 rows each
  int splits;  // parts of a row's tokens at most
  int wide;    // query heads of a workgroup of the join; 0: no join
};

inline PromptWay prompt_way(const AttentionCall& c, int cus) {
  PromptWay way{4, 1, 0};
  // few rows: their tokens split over workgroups, as far as the longest sequence that the table has room for goes. Us with and without: two
  // pieces of 512 tokens behind 9000 and 16001 251 / 371, one token behind 60000 77 / 1381. No further than 256 tiles of 128 rows, so 1025 and
  // 1100 rows of those pieces take 415 and 417 (8 bits 491 and 495), 1000 to 1024 251 (283): two parts of more would help sequences of different
  // lengths (1025 rows 277, 1280 296 / 421) and cost others (2000 tokens behind nothing 76 / 61, behind 7000 301 / 286 and with heads of 256
  // 757 / 645).
  int64_t tokens = c.room;
  if (c.window && (int64_t)c.window + c.sinks + 32 * 8 < tokens) tokens = (int64_t)c.window + c.sinks + 32 * 8;
  const int64_t tiles = (tokens + kPromptTokens - 1) / kPromptTokens;
  const int64_t most = tiles > kPromptMinTiles ? worth(tiles, c.T, c.q_heads, c.dim) : 1;
  way.splits = (int)std::min<int64_t>(FP4_ATTENTION_SPLITS(c.T, c.batch, c.q_heads, c.heads), most);
  const int64_t tiles8 = (c.T * (c.q_heads / c.heads) + 255) / 256;  // of 256 rows
  if (way.splits > 1) {
    // 256 rows share what is brought into LDS: an eighth sooner where their workgroups are one round, every CU but a 32nd of them having one,
    // and none two, and where no part is so short that its start shows. Us with 128 and 256 rows (splits), two sequences behind 9000 and 16001, 32
    // over 8 heads of 128: 1000 to 1024 rows (2) 281 / 250, 500 (4) 148 / 134, 256 (8) 85 / 78; 128 (16) 57 / 84, 200 (9) 104 / 108; 641 (3: 264
    // workgroups) 199 / 200, in 8 bits 215 / 224; one behind 8000, 16 heads: 2000 (2) 185 / 168, 900 (4) 100 / 93, 500 (8) 62 / 60; 1200 (3: 240)
    // 117 / 172, 768 (5: 240) 83 / 120, 600 (6: 288) 99 / 104, 256 (16) 44 / 67.
    const int64_t groups = std::max(tiles8, c.batch) * c.heads * way.splits;
    if (prompt_eight(c.dim, c.e4m3, true) && way.splits <= 8 && groups <= cus && groups >= cus - cus / 32) way.waves = 8;
  } else {
    // Once they fill the CUs: 8192 tokens 540 with 256 rows, 588 with 128; below the line 4 sequences of 200 to 900 tokens 50.9 / 49.8.
    // (A grid has fewer than 2^32 work-items.)
    if (prompt_eight(c.dim, c.e4m3, false) && c.T * c.q_heads >= (int64_t)256 * cus && (tiles8 + c.batch) * c.heads < (1 << 23)) way.waves = 8;
  }
  if (way.splits > 1) {
    // heads of a workgroup of the join: fewer where they have many parts (one token behind 60000, 64 parts: 87 us with all, 76 so)
    way.wide = 1024 / c.dim;
    while (way.wide > 1 && way.splits * way.wide > 4 * (1024 / c.dim)) way.wide /= 2;
  }
  return way;
}

}  // namespace fp4
