// act_tile.cuh -- the activation GEMM's choice of tile for ragged and
// middling shapes.  Host arithmetic only: plain C++, no CUDA headers.
#pragma once

#include <cstdint>

namespace hq {

// Tile of the activation GEMM for more than 128 rows where the CTA-pair rule
// (dispatch_gemm) does not hold (ragged N, N < 2048, middling M): the one of
// the least estimated time,
//   t_k nkb + (rounds - 1) max(t_k nkb, t_e) + t_e
// with t_k the time of a 128-byte K block and t_e of a tile's epilogue
// (silu, bias, residual), us, measured on one round of tiles; the 256 x 512
// tile has no second accumulator and pays both every round.  All tiles give
// the same bits.  Measured with that epilogue and the operands in L2, us, the
// choice in brackets:
//                         128x64  128x128  128x256  256x256  256x512
//    133 x  2096 x  1840   [9.3]     11.9     17.2     16.4     25.6
//   2047 x  1024 x  4096    20.3   [14.8]     19.8     21.3     34.1
//   2047 x  9216 x  2048    74.8     50.9   [42.1]     46.2     53.6
//   1460 x 24400 x  1776   174.0    119.2   [98.9]     94.5    110.1
//   1388 x  1880 x  4560    43.0     38.6     31.9   [29.7]     46.0
//    692 x  9208 x 28352   382.2    257.0    202.5    196.2  [153.3]
// The estimate is off by up to a quarter (where the result's stores bound
// every round it is that much too low), so candidates within some 5 % of one
// another may come in the wrong order, as in the fourth line; without bias
// and residual, at short K, the choice cost up to 18 % there (83 against 71).
enum ActTile { kT64, kT128, kT256, kPair256, kPair512 };
inline ActTile pick_act_tile(int64_t M, int64_t N, int64_t nkb, int64_t sms) {
  struct Cost {
    int rows, cols, units;  // units: SMs per tile
    double k, e;
  };
  const Cost costs[] = {{128, 64, 1, 0.27, 2.9},
                        {128, 128, 1, 0.385, 4.4},
                        {128, 256, 1, 0.44, 8.5},
                        {256, 256, 2, 0.42, 8.8},
                        {256, 512, 2, 0.75, 18.0}};
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < 5; ++i) {
    const Cost& c = costs[i];
    if (c.units > sms) continue;  // a share of one SM runs no pair of CTAs
    const int64_t at_once = sms / c.units;
    const int64_t tiles = ((M + c.rows - 1) / c.rows) * ((N + c.cols - 1) / c.cols);
    const double rounds = static_cast<double>((tiles + at_once - 1) / at_once);
    const double k = c.k * static_cast<double>(nkb);
    const double t = i == kPair512 ? rounds * (k + c.e) : k + (rounds - 1.0) * (k > c.e ? k : c.e) + c.e;
    if (i == 0 || t < least) { least = t; best = i; }
  }
  return static_cast<ActTile>(best);
}

}  // namespace hq
