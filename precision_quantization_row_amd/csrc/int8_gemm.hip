// int8_gemm.hip -- which kernel a product of 8-bit integer lines takes.
#include "nvfp4_launch.h"

namespace nvfp4 {

// Sums of K products of two 8-bit integers (2^14 at most) in 32 bits; 32-bit
// offsets within a tile; the launch grids.
bool int8_gemm_supported(int64_t M, int64_t N, int64_t K, bool gated) {
  return K < ((int64_t)1 << 17) && N <= ((int64_t)1 << 26) && M <= ((int64_t)1 << 31) &&
         gemm_tiles(M, N, gated) <= ((int64_t)1 << 23);
}

static bool few_lines(const GemmArgs& a) {
  const bool gated = a.act == 4;
  const double groups =
      (double)((a.M + 63) / 64) * (double)(((gated ? 2 * a.N : a.N) + 63) / 64), K = (double)a.K;
  // a launch holds fewer than 2^32 threads: of the few-lines kernel's narrowest
  // tiles, 64 (or all) lines by 16 outputs with 512 threads, 2^22
  if (4 * groups > (double)(1 << 22)) return false;
  const double rounds = (double)((gemm_tiles(a.M, a.N, gated) + 255) / 256);
  return (groups > 256 ? groups / 256 : 1.0) * (8500 + 1.0 * K) < rounds * (15000 + 9.0 * K);
}

int launch_int8_gemm(const GemmArgs& a, hipStream_t s) {
  if (few_lines(a)) launch_int8_rows_gemm(a, s);
  else launch_int8_tile(a, s);
  return hipGetLastError() == hipSuccess ? 0 : -3;
}

}  // namespace nvfp4
