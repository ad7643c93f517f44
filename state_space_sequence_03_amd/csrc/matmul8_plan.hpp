// matmul8_plan.hpp -- which form of the 8-bit product takes which sizes (matmul8.hip).  Host code without HIP,
// so that the tests can ask it too.
#pragma once
#include <cmath>
#include <cstdint>
#include <initializer_list>

namespace ssd {

enum Matmul8Form { kFew, kTile64, kTile128, kTile256 };
struct Matmul8Plan {
  Matmul8Form form;
  int parts, each;   // of the depth
};

// How a product is computed.  Up to 16 rows, each wave takes its own blocks straight from memory (1 x 10576 x
// 2560 7.1 us, in tiles of 64 x 64 9; more of them on their way at once change nothing), and up to 32 where one
// workgroup for each CU does and the depth is not large (32 x 2560 x 5120 9.7, in tiles 10.2; 20 x 4096 x 5120 8.5,
// 11.6; but 32 x 4096 x 8192 13.7, 13.0; 32 x 10576 x 2560 13.2, 9.6).  Beyond that the form and the parts of the
// depth whose time, by what was measured, is the least.  A step of 128 in the depth takes a CU (us) for as many
// tiles (times parts) as it has, at most those that fit it at once, and again for those behind them:
//                 bf16 results                 fp32 results
//   64 x 64       0.33, 0.42, 0.60, 0.80       0.49, 0.70, 0.98, 1.25  (64 x 16 a wave, not 32 x 32: 0.65, 1.07)
//   128 x 128     0.70, 1.10                   1.33, 1.95
//   256 x 256     1.9 (1.7 on up to 180 CUs)   (their operands take twice the registers)
// a launch 3, and a split depth 3 more, 0.15 for each part, and the parts' way through memory at 4.5 TB/s.
// Measured against it:
//   512 x 2560 x 5120 in tiles of 64 19.6 (19.8), of 128 29 (31); 256 x 10576 x 2560 16.9 (15), 17.3 (17);
//   2048 x 2560 x 5120 47 (48), 43 (47); 2048 x 10576 x 2560 in tiles of 128 73 (69), of 256 79 (79);
//   4096 x 10576 x 2560 146 (127), 117 (117); 128 x 2560 x 5120 whole 15.6 (16), in three parts 12.4 (13);
//   fp32 1111 x 770 x 2176 whole 11.7 (11), in two 16 (16); fp32 1500 x 1500 x 16384 in tiles of 128 whole 163
//   (173), in three parts 92 (104).
inline Matmul8Plan matmul8_plan(int64_t M, int64_t N, int64_t K, int out_bf16) {
  const int64_t blocks = K / 128;
  Matmul8Plan best{kFew, 1, (int)blocks};
  if (M <= 16 || (M <= 32 && N <= 4096 && K <= 5120)) return best;
  const auto tiles = [&](int64_t t) { return (double)((M + t - 1) / t) * (double)((N + t - 1) / t); };
  const double cells = (double)M * (double)N;
  double least = 0.0;
  const auto consider = [&](Matmul8Form form, double count, std::initializer_list<double> steps) {
    for (int parts = 1; parts <= 16; ++parts) {
      const int64_t each = (blocks + parts - 1) / parts;
      if (parts > 1 && (form == kTile256 || each < 4 || parts * cells * sizeof(float) > (1 << 28))) break;
      const double c = std::ceil(count * parts / 256.0), rounds = std::floor(c / (double)steps.size());
      const int rest = (int)(c - rounds * (double)steps.size());
      const double step = rounds * steps.end()[-1] + (rest ? steps.begin()[rest - 1] : 0.0);
      double t = 3.0 + step * (double)each;
      if (parts > 1) t += 3.0 + 0.15 * parts + cells * (8.0 * parts + (out_bf16 ? 2.0 : 4.0)) / 4.5e6;
      if (least == 0.0 || t < least) {
        least = t;
        best.form = form;
        best.each = (int)each;
        best.parts = (int)((blocks + each - 1) / each);
      }
    }
  };
  if (out_bf16) {
    consider(kTile64, tiles(64), {0.33, 0.42, 0.60, 0.80});
    consider(kTile128, tiles(128), {0.70, 1.10});
    consider(kTile256, tiles(256), {tiles(256) <= 180 ? 1.7 : 1.9});
  } else {
    consider(kTile64, tiles(64), {0.49, 0.70, 0.98, 1.25});
    consider(kTile128, tiles(128), {1.33, 1.95});
  }
  return best;
}

}  // namespace ssd
