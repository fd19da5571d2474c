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
// 128, 128 and 256 lines of B). Up to 32 lines always few-lines (32 x 4096 x 4096 7.6 us, the
// quickest tile 16; 32 x 28672 x 8192 65 and 56). For more, a model of the four kernels'
// times in us, s stages of 128 k: a latency that a stage costs however few the workgroups,
// and what n workgroups cost together (L2's and the matrix pipe's share of a stage, the rest
// of a tile). B's bytes from HBM are not in it: where they bound, its times are too
// short, and only their order is of use. Measured and modelled:
//                       few-lines      64 x 128       128 x 128      256 x 256
//   128 x 4096 x 4096   10.3  12.7     15.0  15.2     18.4  17.7     47.6  50.2
//   512 x 4096 x 4096   33.6  40.2     16.3  16.5     20.0  17.7     48.7  51.4
//   1024 x 4096 x 4096  64.5  76.8     27.1  28.6     25.2  26.0     50.8  53.9
//   4096 x 4096 x 4096  246   297      94.0  101      77.3  84.3     69.9  68.8
//   512 x 8192 x 8192   138   136      47.6  49.0     41.1  42.3     86.2  91.8
//   8192 x 1000 x 1000  94.3  61.7     26.3  21.9     20.7  20.8     32.8  26.7
//   300 x 3000 x 300    11.1  8.1      7.2   5.8      9.4   7.8      23.0  19.3
//   64 x 28672 x 8192   76.7  61.4     56.8  25.9     59.8  37.9     87.9  99.3
//   256 x 28672 x 8192  258   235      108   82.5     80.9  69.2     98.5  99.3
// Of 49 sizes from 8 x 300 x 5000 to 1024 x 28672 x 8192 none took over 1.2 times the
// quickest kernel's time (1000 x 8192 x 301 1.18, 32 x 28672 x 8192 1.16, 8192 x 4096 x 256 1.12),
// the others at most 1.05.
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
