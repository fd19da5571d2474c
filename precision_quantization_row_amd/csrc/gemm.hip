// gemm.hip -- which kernel a packed product takes.
#include "nvfp4_launch.h"

namespace nvfp4 {

// What 32-bit offsets within a tile and the launch grids hold.
bool gemm_supported(int64_t M, int64_t N, int64_t K, bool gated) {
  return K <= ((int64_t)1 << 23) && N <= ((int64_t)1 << 26) &&
         M <= ((int64_t)1 << 31) && gemm_tiles(M, N, gated) <= ((int64_t)1 << 23);
}

// Both kernels take any sizes; the quicker one runs. The few-lines kernel does
// about 700 TFLOP/s once it is bound by its decode (256 x 8192 x 8192: 48 us);
// a round of 256 tiles takes 18.3 ns a k and 12 us around them, however few of
// its 256 lines and of the 256 CUs are in use (512 x 8192 x 8192: 162 us against
// 97; 1024 x 8192 x 8192: 162 against 196). In units of a product and a sum:
static bool few_lines(const GemmArgs& a) {
  const bool gated = a.act == 4;
  const double lines = (double)((a.M + 63) / 64 * 64), nb = (double)(gated ? 2 * a.N : a.N), K = (double)a.K;
  // a launch holds fewer than 2^32 threads; the few-lines kernel's tiles are
  // at least 64 (or all) lines by 16 outputs and have 512
  if ((lines / 64) * (nb / 16 + 1) > (double)(1 << 22)) return false;
  const double rounds = (double)((gemm_tiles(a.M, a.N, gated) + 255) / 256);
  return lines * nb * K < rounds * (6.4e6 * K + 4.2e9);
}

int launch_gemm(const GemmArgs& a, hipStream_t s) {
  if (few_lines(a)) launch_gemm_rows(a, s);
  else launch_gemm_tile(a, s);
  return hipGetLastError() == hipSuccess ? 0 : -3;
}

}  // namespace nvfp4
