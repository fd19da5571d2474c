// gemm.hip -- which kernel a packed product takes.
#include "nvfp4_launch.h"

namespace nvfp4 {

// What 32-bit offsets within a tile and the launch grids hold.
bool gemm_supported(int64_t M, int64_t N, int64_t K, bool gated) {
  return K <= ((int64_t)1 << 23) && N <= ((int64_t)1 << 26) &&
         M <= ((int64_t)1 << 31) && gemm_tiles(M, N, gated) <= ((int64_t)1 << 23);
}

// Both kernels take any sizes; the quicker one runs, by a model of their times
// in ns. A few-lines workgroup is counted as 64 lines of A by 64 of B in 8.5 us
// and 1.7 ns a k, 256 at a time (512 x 8192 x 8192: 90 us, measured 93-100; 4096 x
// 2816 x 256: 98 us, 91); a round of 256 tiles of 256 x 256 takes 20 us and 18.5 ns
// a k, however few of its lines and of the CUs are in use (512 x 8192 x 8192: 172
// us, measured 155-162; 4096 x 2816 x 2816: 72 us, 70-77). The model is coarse: 32
// lines and fewer take narrower tiles and half the time it says, odd k nearly
// twice. Where the two are near each other it decides well: of 26 sizes from 16 x
// 4096 x 4096 to 8192 x 4096 x 256 none took over 1.07 times the quicker kernel (2048
// x 2048 x 1024, the nearest: 32.5 against 33.7 us).
static bool few_lines(const GemmArgs& a) {
  const bool gated = a.act == 4;
  const double groups =
      (double)((a.M + 63) / 64) * (double)(((gated ? 2 * a.N : a.N) + 63) / 64), K = (double)a.K;
  // a launch holds fewer than 2^32 threads: of the few-lines kernel's narrowest
  // tiles, 64 (or all) lines by 16 outputs with 512 threads, 2^22
  if (4 * groups > (double)(1 << 22)) return false;
  const double rounds = (double)((gemm_tiles(a.M, a.N, gated) + 255) / 256);
  return (groups > 256 ? groups / 256 : 1.0) * (8500 + 1.7 * K) < rounds * (20000 + 18.5 * K);
}

int launch_gemm(const GemmArgs& a, hipStream_t s) {
  if (few_lines(a)) launch_gemm_rows(a, s);
  else launch_gemm_tile(a, s);
  return hipGetLastError() == hipSuccess ? 0 : -3;
}

}  // namespace nvfp4
