// act.hip -- backward pass of the product's epilogue (gfx950).
//
//   dz_ij    = dy_ij * act'(z_ij)
//   gated:     z = [g | u], dz = [dy u silu'(g) | dy silu(g)]
//   dbias_j  = sum_i dz_ij   (of the FP32 dz, before it is rounded)
// Bound by HBM: dy and z are read once, dz is written once. A workgroup owns
// 2048 columns (8 a lane) and a run of rows; the bias gradient's partial sums
// stay in the lane's registers, go to one workspace row per run, and
// are added in order by a second kernel (no atomics).
#include "nvfp4_launch.h"
#include "nvfp4_vec.h"

#include <algorithm>

namespace nvfp4 {

template <typename T, int ACT>
__global__ void __launch_bounds__(256) act_bwd_kernel(const ActBwdArgs p, int64_t rows) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr bool GATED = ACT == ACT_SWIGLU;
  const int64_t N = p.N, NB = GATED ? 2 * N : N;
  const int64_t c = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x), n = N - c;
  if (n <= 0) return;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = min(p.M, r0 + rows);
  float b0[8] = {}, b1[8] = {};
  for (int64_t r = r0; r < r1; ++r) {
    const T* zr = static_cast<const T*>(p.z) + r * NB + c;
    T* dzr = static_cast<T*>(p.dz) + r * NB + c;
    float dy[8], z[8], d[8];
    load8<T, true>(static_cast<const T*>(p.dy) + r * N + c, n, dy);
    load8<T, true>(zr, n, z);
    if constexpr (GATED) {
      float u[8], du[8];
      load8<T, true>(zr + N, n, u);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float s = sigmoid_f(z[k]);
        const float ds = s == 0.0f ? 0.0f : dsilu_f(z[k], s);
        d[k] = dy[k] * u[k] * ds;
        du[k] = dy[k] * (z[k] * s);
        b0[k] += d[k];
        b1[k] += du[k];
      }
      store8<true>(dzr, n, d);
      store8<true>(dzr + N, n, du);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        d[k] = dy[k] * dact_f(ACT, z[k]);
        b0[k] += d[k];
      }
      store8<true>(dzr, n, d);
    }
  }
  if (p.dbias) {
    float* part = p.part + (int64_t)blockIdx.y * NB + c;
    store8(part, n, b0);
    if constexpr (GATED) store8(part + N, n, b1);
  }
}

// Runs of rows: enough workgroups for the device (a function of the sizes
// alone, see act_bwd_parts), at least 8 rows a run.
int64_t act_bwd_rows(int64_t M, int64_t N) {
  const int64_t strips = (N + 2047) / 2048;
  const int64_t want = std::max<int64_t>(1, 4096 / strips);
  return std::max<int64_t>(std::min<int64_t>(8, M), (M + want - 1) / want);
}
int64_t act_bwd_parts(int64_t M, int64_t N) {
  const int64_t rows = act_bwd_rows(M, N);
  return (M + rows - 1) / rows;
}

template <typename T>
static int launch_act_bwd_t(const ActBwdArgs& a, hipStream_t s) {
  const int64_t rows = act_bwd_rows(a.M, a.N);
  const dim3 g((unsigned)((a.N + 2047) / 2048), (unsigned)act_bwd_parts(a.M, a.N)), b(256);
  switch (a.act) {
    case ACT_GELU: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_GELU>), g, b, 0, s, a, rows); break;
    case ACT_SILU: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_SILU>), g, b, 0, s, a, rows); break;
    case ACT_RELU2: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_RELU2>), g, b, 0, s, a, rows); break;
    case ACT_SWIGLU: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_SWIGLU>), g, b, 0, s, a, rows); break;
    default: hipLaunchKernelGGL((act_bwd_kernel<T, ACT_NONE>), g, b, 0, s, a, rows); break;
  }
  if (hipGetLastError() != hipSuccess) return -3;
  if (!a.dbias) return 0;
  return launch_colsum(a.part, act_bwd_parts(a.M, a.N), a.act == ACT_SWIGLU ? 2 * a.N : a.N, a.dbias,
                       a.noop, s);
}

int launch_act_bwd(const ActBwdArgs& a, hipStream_t s) {
  return a.dtype == 0 ? launch_act_bwd_t<uint16_t>(a, s) : launch_act_bwd_t<float>(a, s);
}

}  // namespace nvfp4
