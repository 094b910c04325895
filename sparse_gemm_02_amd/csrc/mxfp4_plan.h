// Host side: which kernel a 2:4 product on 4-bit codes takes (spmm_mxfp4.hip), by its sizes and the
// device's compute units.  `stages` is K in steps of 128, M the outputs.
#pragma once
#include <stdint.h>

#include <algorithm>

#include "tile_rounds.h"

namespace slope {

constexpr int kLdsBytes = 160 * 1024;                // of a compute unit
constexpr int kMostParts = 8;
constexpr int kMidRows = 128, kMidTokens = 64;       // of the smallest tiles

inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// LDS of the largest form for so many tokens: eight waves' X rows, and all of the scales.
inline int64_t decode_lds(int tokens, int64_t stages) { return 1024 * tokens + up(stages, 4) * 16 * tokens; }

// Up to 64 tokens.  64 rows a block draw X half as often as 32, and 32 spread better over
// the compute units; parts of K spread them too, and cost a second launch and their sums.
// A unit takes in 48 bytes a nanosecond of rows of weight (0.41 bytes a value) and tokens (0.53),
// and all of them 6400 of weight: what is estimated to take the least.  Parts have to win a tenth,
// over blocks of 32 rows a little more, which do better than estimated.  us, 64 rows / 32 rows / 64 rows in parts, the weight from HBM:
//   9216 -> 27648    1 token 18.7 / 20.4          16: 19.1 / 21.7          64: 27.9 / 42.2
//   5120 -> 20480            12.1 / 10.4              11.7 / 11.3              17.5 / 22.0
//   9216 -> 9216              9.8 / 10.1              10.8 / 11.6              16.0 / 21.4 / 18.3 (3)
//   20480 -> 5120            14.5 / 10.3 / 12.1 (3)   17.5 / 12.6 / 12.8 (3)   28.3 / 22.3 / 17.7 (3)
//   20480 -> 2560            13.7 /  9.3 /  9.4 (4)   16.4 / 11.6 / 10.0 (4)   26.1 / 20.8 / 13.9 (4)
//   16384 -> 6144            12.8 /  9.8 / 12.1 (2)   14.9 / 11.2 / 12.7 (4)   22.6 / 18.0 / 17.9 (2)
//   36864 -> 9216            25.5 / 28.0 / 26.3 (3)   30.2 / 37.9 / 27.2 (3)   47.2 / 67.4 / 40.9 (3)
// Waves and pairs in flight as measured best: two blocks a unit want four waves (5120 -> 20480 at
// 16 tokens 11.9 us, with eight 13.4), one wants eight (9216 -> 9216 at 16 10.8, with four 12.9).
// (More pairs of weight in flight, 128 rows a block and the scales' loads behind the first pairs'
// won nothing.)
//
// Of so long a K that 64 tokens' scales do not fit LDS (from 49153 on) a block has fewer tokens,
// or a part of K.
struct FewPlan {
  int tokens;                                        // of a block: 8, 16, 32 or 64; 0: they fit no block
  bool wide, one;                                    // 64 rows a block; a block a compute unit at most
  int parts;
};
inline int group_of(int64_t T) { return T <= 8 ? 8 : T <= 16 ? 16 : T <= 32 ? 32 : 64; }
inline FewPlan few_plan(int64_t T, int64_t M, int64_t stages, int64_t most_parts, int64_t cus) {
  const int64_t groups = up(stages, 4);
  const double k = 128.0 * (double)stages, sums = 4.0 * (double)T * (double)M, stream = k * (double)M * 0.41 / 6.4e6;
  auto intake = [&](int64_t rows, int64_t tokens, int64_t parts) {
    const double a_unit = (double)up(up(M, rows) * up(T, tokens) * parts, cus) / (double)parts;
    return k * a_unit * ((double)rows * 0.41 + 0.53 * (double)std::min(T, tokens)) / 48e3;
  };
  int tokens = group_of(T);
  while (tokens && decode_lds(tokens, stages) > kLdsBytes) tokens = tokens > 8 ? tokens / 2 : 0;
  FewPlan plan{tokens, false, false, 1};
  double least = 1e30;
  if (tokens) {
    const double wide = intake(64, tokens, 1), narrow = intake(32, tokens, 1);
    plan.wide = wide <= narrow;
    plan.one = up(M, plan.wide ? 64 : 32) * up(T, tokens) <= cus;
    least = std::max(plan.wide ? wide : 0.94 * narrow, stream);
  }
  tokens = group_of(T);
  for (int parts = 2; parts <= most_parts; ++parts) {
    const double us = std::max(intake(64, tokens, parts), stream) + 3.0 + 2.0 * parts * sums / 5e6;   // and the sums' way to memory and back
    if (us < 0.9 * least && decode_lds(tokens, up(groups, parts) * 4) <= kLdsBytes) {
      least = us;
      plan = FewPlan{tokens, true, up(M, 64) * parts <= cus, parts};
    }
  }
  return plan;
}
// Parts of one call: whole groups of four stages, and the scratch holds their sums.
inline int64_t most_parts(int64_t T, int64_t M, int64_t stages, int64_t scratch_bytes) {
  return std::max<int64_t>(1, std::min({(int64_t)kMostParts, up(stages, 4), scratch_bytes / (4 * T * M)}));
}

// Above 64 tokens, four kernels by their estimated time in units of a
// stage (us for 128 k), fitted to sweeps of 65 .. 8192 tokens over the shapes below:
//   large   0.0103 a unit of full_width_rows' cost (100 a round of full tiles, 65 of half tiles)
//   wide    256 x 128 tiles of four waves: 0.60 a round
//   mid     128 x 64 tiles: 0.13 + 0.205 a tile of each compute unit, 0.38 at least
//   direct  the few-token kernel over groups of 64 tokens: 0.10 + 0.14 a block of 64 rows of each
//           unit; 32 rows up to 128 such blocks (4096 -> 1024 at 512 tokens 6.6 us, with 64 8.5)
// Measured, us (large / wide / mid / direct, the weight from HBM), the rule's choice starred:
//   9216 -> 9216    128 tokens  47.8 /  45.3 /  29.2 /  20.1*
//                   256         47.3 /  45.5 /  33.0*/  32.3
//                   512         47.8 /  45.9 /  43.5*/  49.1
//                  1000         61.4*/  82.2 /  77.9 /  81.3
//                  8192        350 * / 392   / 535
//   20480 -> 5120    65         89.4 /  81.1 /  59.3 /  26.4*
//                   256         98.6 /  91.1 /  59.6 /  36.7*
//                   512         96.3 /  90.4 /  68.7*/  61.7     (estimated 61.8 and 72)
//                  1000         95.0 /  86.5*/  93.7 /  97.6
//                  2048        130.6*/ 170.6 / 170.2 / 180.9
//   9216 -> 27648    65         44.0 /  40.6 /  38.6*/  40.7
//                   256         51.5 /  49.1*/  76.3 /  76.8
//                   512         72.2*/  93.2 / 121.5 / 139.8
//   5120 -> 5120    256         29.1 /  28.8 /  18.0 /  13.9*
//                  1000         28.6 /  26.8*/  27.6 /  31.7
//   4096 -> 1024   1000         22.6 /  21.4 /  15.3 /   9.1*
//                  2048         23.3 /  21.7 /  16.0 /  13.8*
//   768 -> 2304    1000          9.3 /   9.6 /   7.1*/  10.0
enum class Many { Direct32, Direct64, Mid, Wide, Large };   // (direct, with so many rows a block)
struct ManyPlan {
  Many kernel;
  int64_t rows_full;                                 // of Large
};
inline ManyPlan many_plan(int64_t T, int64_t M, int64_t stages, int64_t cus) {
  const bool fits = decode_lds(64, stages) <= kLdsBytes && up(T, 64) <= 65535;   // (and a grid's second dimension)
  const int64_t rows = up(M, 256), cols = up(T, 256), halves = up(T, 128);
  const int64_t rows_full = full_width_rows(rows, cols, halves, cus);
  const double large = 0.0103 * (100 * (double)up(rows_full * cols, cus) +
                                 65 * (double)up((rows - rows_full) * halves, cus));
  const double wide = 0.60 * (double)up(rows * halves, cus);
  const double mid = std::max(0.38, 0.13 + 0.205 * (double)(up(M, kMidRows) * up(T, kMidTokens)) / (double)cus);
  const int64_t blocks = up(M, 64) * up(T, 64);
  const double direct = 0.10 + 0.14 * (double)blocks / (double)cus;
  if (fits && direct <= mid && direct <= wide && direct <= large)
    return {blocks <= 128 ? Many::Direct32 : Many::Direct64, 0};
  if (mid <= wide && mid <= large) return {Many::Mid, 0};
  return wide <= large ? ManyPlan{Many::Wide, 0} : ManyPlan{Many::Large, rows_full};
}

}  // namespace slope
