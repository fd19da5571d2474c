// act.hip -- backward pass of the product's epilogue (gfx950).
//
//   dz_ij    = dy_ij * act'(z_ij)
//   gated:     z = [g | u], dz = [dy u silu'(g) | dy silu(g)]
//   dbias_j  = sum_i dz_ij   (of the FP32 dz, before it is rounded)
// Bound by HBM: dy and z are read once, dz is written once. A workgroup owns
// 512 columns (8 a lane) and a run of rows, every fourth of them a wave; the
// bias gradient's sums stay in registers, meet in LDS, go to one workspace row
// per run, and are added in order by a second kernel (no atomics). 8192 x
// (2 x 28672) BF16, gated: 446 us, 5.3 TB/s; 4097 x 2881 FP32 with a bias: 34 + 4 us
// from HBM, 25 + 4 where the 142 MB are still in the memory-side cache.
#include "nvfp4_launch.h"
#include "nvfp4_vec.h"

#include <algorithm>

namespace nvfp4 {

template <typename T, int ACT>
__global__ void __launch_bounds__(256) act_bwd_kernel(const ActBwdArgs p, int64_t rows) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr bool GATED = ACT == ACT_SWIGLU;
  constexpr int H = GATED ? 2 : 1;
  __shared__ float sums[4][H][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t N = p.N, NB = H * N;
  const int64_t c = 512 * (int64_t)blockIdx.x + 8 * lane, n = N - c;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = min(p.M, r0 + rows);
  float b[H][8] = {};
  // 2 lines of a wave on their way at a time
  for (int64_t r = r0 + wave; r < r1 && n > 0; r += 8) {
    Raw8<T> ry[2], rz[2], ru[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int64_t q = r + 4 * v;
      if (q < r1) {
        load8_raw<true>(static_cast<const T*>(p.dy) + q * N + c, n, ry[v]);
        load8_raw<true>(static_cast<const T*>(p.z) + q * NB + c, n, rz[v]);
        if constexpr (GATED) load8_raw<true>(static_cast<const T*>(p.z) + q * NB + N + c, n, ru[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int64_t q = r + 4 * v;
      if (q >= r1) break;
      T* dzr = static_cast<T*>(p.dz) + q * NB + c;
      float dy[8], z[8], d[8];
      unpack8(ry[v], dy);
      unpack8(rz[v], z);
      if constexpr (GATED) {
        float u[8], du[8];
        unpack8(ru[v], u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float s = sigmoid_f(z[k]);
          const float ds = s == 0.0f ? 0.0f : dsilu_f(z[k], s);
          d[k] = dy[k] * u[k] * ds;
          du[k] = dy[k] * (z[k] * s);
          b[0][k] += d[k];
          b[H - 1][k] += du[k];
        }
        store8<true>(dzr, n, d);
        store8<true>(dzr + N, n, du);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          d[k] = dy[k] * dact_f(ACT, z[k]);
          b[0][k] += d[k];
        }
        store8<true>(dzr, n, d);
      }
    }
  }
  if (!p.dbias) return;
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[wave][h][k * 64 + lane] = b[h][k];
  __syncthreads();
  if (wave != 0 || n <= 0) return;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int at = k * 64 + lane;
      t[k] = sums[0][h][at] + sums[1][h][at] + sums[2][h][at] + sums[3][h][at];
    }
    store8(p.part + (int64_t)blockIdx.y * NB + h * N + c, n, t);
  }
}

// Lines a workgroup: about six workgroups a CU, 8 lines at least; a function of
// the sizes alone, so that the sums' order is.
int64_t act_bwd_rows(int64_t M, int64_t N) {
  const int64_t strips = (N + 511) / 512;
  const int64_t want = std::max<int64_t>(1, 1536 / strips);
  return std::max<int64_t>(8, ((M + want - 1) / want + 7) / 8 * 8);
}
int64_t act_bwd_parts(int64_t M, int64_t N) {
  const int64_t rows = act_bwd_rows(M, N);
  return (M + rows - 1) / rows;
}

template <typename T>
static int launch_act_bwd_t(ActBwdArgs a, hipStream_t s) {
  if (act_bwd_parts(a.M, a.N) == 1) a.part = a.dbias;  // one run: its sums are the result
  const int64_t rows = act_bwd_rows(a.M, a.N);
  const dim3 g((unsigned)((a.N + 511) / 512), (unsigned)act_bwd_parts(a.M, a.N)), b(256);
  switch (a.act) {
    case ACT_GELU: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_GELU>), g, b, 0, s, a, rows); break;
    case ACT_SILU: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_SILU>), g, b, 0, s, a, rows); break;
    case ACT_RELU2: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_RELU2>), g, b, 0, s, a, rows); break;
    case ACT_SWIGLU: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_SWIGLU>), g, b, 0, s, a, rows); break;
    default: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_NONE>), g, b, 0, s, a, rows); break;
  }
  if (hipGetLastError() != hipSuccess) return -3;
  if (!a.dbias || a.part == a.dbias) return 0;
  return launch_colsum(a.part, act_bwd_parts(a.M, a.N), a.act == ACT_SWIGLU ? 2 * a.N : a.N, a.dbias,
                       a.noop, s);
}

int launch_act_bwd(const ActBwdArgs& a, hipStream_t s) {
  return a.dtype == 0 ? launch_act_bwd_t<uint16_t>(a, s) : launch_act_bwd_t<float>(a, s);
}

}  // namespace nvfp4
