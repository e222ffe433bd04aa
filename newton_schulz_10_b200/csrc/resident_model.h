// Which stacks the on-chip update (resident.cu) takes, and on how many CTAs a
// matrix: host arithmetic only.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace muon {
namespace res {

constexpr int MAX_N = 128;      // rows of the wide view
constexpr int MAX_M = 2048;     // columns of the wide view
constexpr int MAX_G = 8;        // 64-column groups per CTA (their accumulators fill TMEM)
constexpr int MAX_C = 16;       // CTAs per cluster (above 8 only where a smaller one cannot hold the matrix)
constexpr int MISC = 1024;
constexpr int SMEM_MAX = 232448;  // opt-in shared memory of one sm_100 CTA

// A 64-column group of a plane: np rows of 128 bytes.
constexpr int group_bytes(int np) { return np * 128; }
// X (g groups) and A (np rows and columns), two planes each, and with a
// cluster the np x np fp32 sums; the M side of a product reads 128 rows from
// a group's start, so as much must lie behind the last one. At least 120 KB,
// so that an SM holds one CTA (two would wait for each other's TMEM columns).
constexpr int smem_bytes(int g, int np, int C) {
  const int b = 1024 + 2 * (g + (np + 63) / 64) * group_bytes(np) + (C > 1 ? np * np * 4 : 0) + MISC + group_bytes(128 - np);
  return b > 120 * 1024 ? b : 120 * 1024;
}
static_assert(smem_bytes(4, MAX_N, 1) <= SMEM_MAX && smem_bytes(2, MAX_N, MAX_C) <= SMEM_MAX, "every shape fits");

// The cluster size, by a model of the step in cycles (measured with the clock
// register at np = 64 and 128, g = 1 to 4, C = 1 to 8): an instruction of the
// products takes at least 75 cycles, an epilogue 700 a group of X and 75 per
// four rows and columns of B', the exchange 1700 + 0.55 np^2 whatever C is,
// loads and stores 0.4 an element. Larger clusters halve the work on X and
// pay the exchange: 12 x 64 x 768 takes 45 us on 8 CTAs a matrix and 51 on 4,
// 1 x 128 x 128 takes 68 on 2 and 47 on 1, 16 x 128 x 512 (two waves of
// clusters of 8) 147 on 8 and 76 on 4.
//
// A stack of many matrices that need large clusters is left to the chain of
// launches, whose time is about 20 us a step for its latencies and its padded
// products at 0.8 PFLOP/s: 48 x 128 x 2048 takes 620 us here and 429 there,
// 48 x 64 x 2048 156 here and 342 there.
//
// capacity(C): clusters of C CTAs that run at once; 0 where none can (a part
// of a device may have no 16 SMs that can form one), which leaves the stack to
// a smaller cluster or to the chain.
template <typename F>
bool choose_cluster(int64_t rows, int64_t cols, int64_t count, int T, int planes, F capacity, int* C_out) {
  if (C_out) *C_out = 0;
  const int64_t n = std::min(rows, cols), m = std::max(rows, cols);
  if (n > MAX_N || m > MAX_M) return false;
  const int groups = (int)((m + 63) / 64), np = (int)((n + 15) / 16 * 16);
  double best = 0.0;
  int best_C = 0;
  for (int C = 1; C <= MAX_C; C *= 2) {
    const int g = (groups + C - 1) / C;
    if (g > MAX_G || smem_bytes(g, np, C) > SMEM_MAX) continue;
    if (C > 8 && best_C) break;  // only where a smaller cluster cannot hold the matrix
    const int64_t at_once = capacity(C);
    if (at_once < 1) continue;
    const double step = 2000.0 + 900.0 * g + 14.0 * np + std::max(14.0 * np * ((g + 3) / 4), 6.6 * np * g) + 700.0 * g + 19.0 * np +
                        (C > 1 ? 1700.0 + 0.55 * np * np : 1000.0);
    const double waves = (double)((count + at_once - 1) / at_once);
    const double t = waves * (12000.0 + 0.4 * n * 64 * g + T * step);
    if (!best_C || t < best) {
      best = t;
      best_C = C;
    }
  }
  const double N = 256.0, tile = (double)(m + 127) / 128 * 128;
  const double chain = 20.0 * T + 2.0 * count * T * (N * N * tile + N * N * np + N * tile * np) * (planes == 2 ? 3.0 : 1.0) / 0.8e9;
  if (C_out) *C_out = best_C;
  return best_C > 0 && 1.25 * best / 1850.0 <= chain;  // the model is 10 to 20% low
}

}  // namespace res
}  // namespace muon
