// int8_gemm.hip -- which kernel a product of 8-bit integer lines takes.
#include "nvfp4_launch.h"

#include <algorithm>

namespace nvfp4 {

// Sums of K products of two 8-bit integers (2^14 at most) in 32 bits; 32-bit
// offsets within a tile; the launch grids.
bool int8_gemm_supported(int64_t M, int64_t N, int64_t K, bool gated) {
  return K < ((int64_t)1 << 17) && N <= ((int64_t)1 << 26) && M <= ((int64_t)1 << 31) &&
         gemm_tiles(M, N, gated) <= ((int64_t)1 << 23);
}

// Which kernel runs: the few-lines one (0) or tiles of 64 WM lines of A (WM = 1, 2, 4; by
// 128, 128 and 256 lines of B). Up to 32 lines B's bytes count alone: few-lines. For more, a
// model of the four kernels' times in us, s stages of 128 k: a latency that a stage
// costs however few the workgroups, and what n workgroups cost together (L2's and the
// matrix pipe's share of a stage, the rest of a tile). Measured and modelled:
//                       few-lines      64 x 128       128 x 128      256 x 256
//   128 x 4096 x 4096   9.8  12.9      14.9  15.2     18.9  17.7     48.2  50.2
//   512 x 4096 x 4096   33.7 40.2      16.3  16.5     19.9  17.7     48.2  51.4
//   1024 x 4096 x 4096  64.6 76.8      27.0  28.6     25.3  26.0     50.3  53.9
//   4096 x 4096 x 4096  247              92.7  101    76.3  84.3     68.9  68.8
//   512 x 8192 x 8192   140  136       46.8  48.9     41.0  42.3     84.1  91.8
//   8192 x 1000 x 1000  92.4 62.5      26.1  21.9     21.2  20.8     32.8  29.4
//   300 x 3000 x 300    10.5 8.0       7.0   6.6      9.4   8.1      22.7  19.7
// Of 38 sizes from 1 x 64 x 64 to 4097 x 2880 x 2881 none took over 1.2 times the quickest
// kernel's time, most within 1.05.
static int tile_of(const GemmArgs& a) {
  if (a.M <= 32) return 0;
  const int64_t NB = a.act == 4 ? 2 * a.N : a.N;
  auto tiles = [&](int64_t m, int64_t n) { return (double)((a.M + m - 1) / m) * (double)((NB + n - 1) / n); };
  const double s = (double)((a.K + 127) / 128);
  const double few = tiles(64, 32), small = tiles(64, 128), mid = tiles(128, 128), large = tiles(256, 256);
  const double rounds = large <= 256 ? 1.0 : large / 256, share = large < 256 ? large / 256 : 1.0;
  const double limit = 1 << 22;  // (a launch holds fewer than 2^32 threads)
  const double t[4] = {few > limit ? 1e30 : 3.5 + std::max(0.135 * s, few * (0.0009 * s + 0.007)),
                       small > limit ? 1e30 : 4.5 + std::max(0.335 * s, small * (0.00125 * s + 0.007)),
                       mid > limit ? 1e30 : 6.5 + std::max(0.35 * s, mid * (0.002 * s + 0.012)),
                       6.0 + rounds * (10.0 + (1.03 + 0.62 * share) * s)};
  const int best = (int)(std::min_element(t, t + 4) - t);
  return best == 0 ? 0 : 1 << (best - 1);
}

int launch_int8_gemm(const GemmArgs& a, hipStream_t s) {
  const int wm = tile_of(a);
  if (wm == 0) launch_int8_rows_gemm(a, s);
  else launch_int8_tile(a, wm, s);
  return hipGetLastError() == hipSuccess ? 0 : -3;
}

}  // namespace nvfp4
