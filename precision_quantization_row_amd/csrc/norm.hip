// norm.hip -- root-mean-square norm of the residual stream, quantized on the
// way out, and its backward pass (gfx950).
//
// Forward, per row:
//   h_k = x_k + residual_k          (kept in FP32; h is stored rounded)
//   r   = 1 / sqrt(sum_k h_k^2 / K + eps)
//   y_k = (h_k * r) * w_k
//   a   = max_k |y_k|
//   E4M3:  code_k = E4M3_RNE(clamp(RN(y_k * S), -448, 448)),
//          S = a == 0 ? 1 : min(RN(448 / a), FLT_MAX)
//   NVFP4: codes and block scales of the FP32 y under the row amax a, as the
//          rowwise copy of nvfp4_quantize_transpose has them
// Backward, per row, with xh_k = h_k * r and g_k = dy_k * w_k:
//   dx_k = r (g_k - xh_k * sum_j(g_j xh_j) / K) + dres_k
//   dw_k = sum over rows of dy_k * xh_k
//
// Both are bound by HBM: a row is read once into registers, reduced there and
// written once. 16384 x 4096 BF16 with the residual: forward 71 us (6.6 TB/s, partly
// from the memory-side cache), backward 95 us and 4.5 for its column sums
// (5.3 TB/s); 4097 x 2881 FP32 backward 35 + 5 us from HBM (27 + 5 from the
// memory-side cache); one row of 8192 forward 3.9 us.
#include "nvfp4_launch.h"
#include "nvfp4_vec.h"

#include <algorithm>

namespace nvfp4 {

// Sum / max over a workgroup of NT threads; every thread gets the result.
// `red` holds NT / 64 entries; consecutive calls use different ones.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += red[i];
  }
  return v;
}
template <int NT>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = wave_max_u32(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0u;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v = max(v, red[i]);
  }
  return v;
}

// Writes one lane's 8 values of a row as codes. NaN clamps to 448 in 8 bits: the
// row's amax, NaN as well, is what carries it. c: first column (a multiple
// of 8), n: elements of the row from c on. The lane pair (2i, 2i + 1) holds
// one 16-element block; both lanes are active (lanes past the row hold zeros).
__device__ __forceinline__ void write_codes(const NormArgs& p, int64_t row, int64_t c, int64_t n,
                                            const float (&y)[8], float a, float enc8,
                                            float s_enc) {
  if (p.q_fmt == 1) {  // E4M3
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = fmaxf(fminf(y[k] * enc8, kE4M3Max), -kE4M3Max);
    uint32_t w0 = 0u, w1 = 0u;
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], w0, false);
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], w0, true);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], w1, false);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], w1, true);
    uint8_t* q = p.q + row * p.K + c;
    if (n >= 8) {
      const u32x2 w = {w0, w1};
      *reinterpret_cast<u32x2_a1*>(q) = w;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) q[k] = (uint8_t)((k < 4 ? w0 : w1) >> (8 * (k & 3)));
    }
  } else {  // NVFP4
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(y[k]) & kAbsF32);
    m = max(m, dpp_swap1(m));
    uint32_t byte;
    float enc;
    block_scale(__uint_as_float(m), a, s_enc, p.F_inv, &byte, &enc);
    uint32_t code = e2m1_pack8(y[0] * enc, y[1] * enc, y[2] * enc, y[3] * enc, y[4] * enc,
                               y[5] * enc, y[6] * enc, y[7] * enc);
    if (n > 0 && (c & 8) == 0) p.s[row * ((p.K + 15) / 16) + c / 16] = (uint8_t)byte;
    uint8_t* q = p.q + row * ((p.K + 1) / 2) + c / 2;
    if (n >= 8) {
      *reinterpret_cast<u32_a1*>(q) = code;
    } else {
      if (n > 0) code &= (1u << (4 * n)) - 1u;  // a missing last high nibble is 0
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (2 * k < n) q[k] = (uint8_t)(code >> (8 * k));
    }
  }
}

// One row per workgroup, 8 * NT * V columns at most, held in registers.
template <typename T, typename W, int NT, int V>
__global__ void __launch_bounds__(NT) norm_kernel(const NormArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  __shared__ float red[NT / 64 + 1];
  __shared__ uint32_t redm[NT / 64 + 1];
  const int64_t row = p.row0 + blockIdx.x, K = p.K;
  const T* x = static_cast<const T*>(p.x) + row * K;
  const T* res = static_cast<const T*>(p.residual) + (p.residual ? row * K : 0);
  const W* w = static_cast<const W*>(p.w);
  Raw8<T> rx[V], rr[V];
  Raw8<W> rw[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * ((int64_t)threadIdx.x + j * NT), n = K - c;
    load8_raw<true>(x + c, n, rx[j]);
    if (p.residual) load8_raw<true>(res + c, n, rr[j]);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * ((int64_t)threadIdx.x + j * NT);
    load8_raw(w + c, K - c, rw[j]);
  }
  float h[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * ((int64_t)threadIdx.x + j * NT), n = K - c;
    unpack8(rx[j], h[j]);
    if (p.residual) {
      float t[8];
      unpack8(rr[j], t);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[j][k] += t[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = __builtin_fmaf(h[j][k], h[j][k], ss);
    if (p.h) store8<true>(static_cast<T*>(p.h) + row * K + c, n, h[j]);
  }
  ss = block_sum<NT>(ss, red);
  const float rstd = 1.0f / sqrtf(ss / (float)K + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * ((int64_t)threadIdx.x + j * NT), n = K - c;
    float wv[8];
    unpack8(rw[j], wv);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[j][k] = (h[j][k] * rstd) * wv[k];
      m = max(m, __float_as_uint(h[j][k]) & kAbsF32);
    }
    if (p.y) {
      if (p.y_dtype == 0) store8(static_cast<uint16_t*>(p.y) + row * K + c, n, h[j]);
      else store8(static_cast<float*>(p.y) + row * K + c, n, h[j]);
    }
  }
  if (!p.row_amax) return;
  const float a = __uint_as_float(block_max<NT>(m, redm));
  if (threadIdx.x == 0) p.row_amax[row] = a;
  if (!p.q_fmt) return;
  const float enc8 = global_encode_scale(a, kE4M3Max), s_enc = global_encode_scale(a, p.F);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * ((int64_t)threadIdx.x + j * NT);
    write_codes(p, row, c, K - c, h[j], a, enc8, s_enc);
  }
}

// Rows too long for the registers: the same steps, x and the residual read
// once for each of the three loops (the second and third from L2).
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int NT = 1024;
  __shared__ float red[NT / 64 + 1];
  __shared__ uint32_t redm[NT / 64 + 1];
  const int64_t row = p.row0 + blockIdx.x, K = p.K, step = 8 * NT;
  const T* x = static_cast<const T*>(p.x) + row * K;
  const T* res = static_cast<const T*>(p.residual) + (p.residual ? row * K : 0);
  const W* w = static_cast<const W*>(p.w);
  auto load_h = [&](int64_t c, float (&h)[8]) {
    load8(x + c, K - c, h);
    if (p.residual) {
      float t[8];
      load8(res + c, K - c, t);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] += t[k];
    }
  };
  float ss = 0.0f;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
    float h[8];
    load_h(c, h);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = __builtin_fmaf(h[k], h[k], ss);
  }
  ss = block_sum<NT>(ss, red);
  const float rstd = 1.0f / sqrtf(ss / (float)K + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  uint32_t m = 0u;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
    float h[8], wv[8];
    load_h(c, h);
    load8(w + c, K - c, wv);
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint((h[k] * rstd) * wv[k]) & kAbsF32);
  }
  const float a = __uint_as_float(block_max<NT>(m, redm));
  if (p.row_amax && threadIdx.x == 0) p.row_amax[row] = a;
  const float enc8 = global_encode_scale(a, kE4M3Max), s_enc = global_encode_scale(a, p.F);
  // every lane of a wave takes part in each turn (write_codes joins lane pairs)
  for (int64_t c0 = 8 * (int64_t)(threadIdx.x & ~63); c0 < K; c0 += step) {
    const int64_t c = c0 + 8 * (threadIdx.x & 63), n = K - c;
    float h[8] = {}, y[8], wv[8] = {};
    if (n > 0) {
      load_h(c, h);
      load8(w + c, n, wv);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = (h[k] * rstd) * wv[k];
    // h may be x's or the residual's own buffer: the row is read for the last
    // time above, by the lane that writes it here
    if (p.h) store8(static_cast<T*>(p.h) + row * K + c, n, h);
    if (p.y) {
      if (p.y_dtype == 0) store8(static_cast<uint16_t*>(p.y) + row * K + c, n, y);
      else store8(static_cast<float*>(p.y) + row * K + c, n, y);
    }
    if (p.q_fmt) write_codes(p, row, c, n, y, a, enc8, s_enc);
  }
}

// A launch holds fewer than 2^32 threads: taller inputs take several.
template <typename F>
static int go_rows(NormArgs a, F launch) {
  for (int64_t r = 0; r < a.M; r += 1 << 20) {
    a.row0 = r;
    launch(a, (unsigned)std::min<int64_t>(a.M - r, 1 << 20));
    if (hipGetLastError() != hipSuccess) return -3;
  }
  return 0;
}

template <typename T, typename W, int NT, int V>
static int go_norm(const NormArgs& a, hipStream_t s) {
  return go_rows(a, [s](const NormArgs& p, unsigned rows) {
    hipLaunchKernelGGL((norm_kernel<T, W, NT, V>), dim3(rows), dim3(NT), 0, s, p);
  });
}

template <typename T, typename W>
static int launch_norm_t(const NormArgs& a, hipStream_t s) {
  const int64_t chunks = (a.K + 7) / 8;
  if (chunks <= 64) return go_norm<T, W, 64, 1>(a, s);
  if (chunks <= 256) return go_norm<T, W, 256, 1>(a, s);
  if (chunks <= 512) return go_norm<T, W, 256, 2>(a, s);
  if (chunks <= 1024) return go_norm<T, W, 1024, 1>(a, s);
  if (chunks <= 2048) return go_norm<T, W, 1024, 2>(a, s);
  if (chunks <= 4096) return go_norm<T, W, 1024, 4>(a, s);
  return go_rows(a, [s](const NormArgs& p, unsigned rows) {
    hipLaunchKernelGGL((norm_long_kernel<T, W>), dim3(rows), dim3(1024), 0, s, p);
  });
}

int launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.in_dtype == 0)
    return a.w_dtype == 0 ? launch_norm_t<uint16_t, uint16_t>(a, s) : launch_norm_t<uint16_t, float>(a, s);
  return a.w_dtype == 0 ? launch_norm_t<float, uint16_t>(a, s) : launch_norm_t<float, float>(a, s);
}

// ---------------------------------------------------------------- backward
// A workgroup takes rows blockIdx.x, blockIdx.x + gridDim.x, ... and keeps
// the part of dw that they give in registers; it goes to row blockIdx.x of the
// workspace, and colsum_kernel adds the rows in order: no atomics, so the
// result does not depend on timing.
template <typename T, typename W, int NT, int V>
__global__ void __launch_bounds__(NT) norm_bwd_kernel(const NormBwdArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  __shared__ float red[2][NT / 64 + 1];
  const int64_t K = p.K;
  float wv[V][8], dw[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * ((int64_t)threadIdx.x + j * NT);
    load8(static_cast<const W*>(p.w) + c, K - c, wv[j]);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[j][k] = 0.0f;
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
    Raw8<T> rdy[V], rh[V], rd[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t c = 8 * ((int64_t)threadIdx.x + j * NT), n = K - c;
      load8_raw<true>(static_cast<const T*>(p.dy) + row * K + c, n, rdy[j]);
      load8_raw<true>(static_cast<const T*>(p.h) + row * K + c, n, rh[j]);
      if (p.dres) load8_raw<true>(static_cast<const T*>(p.dres) + row * K + c, n, rd[j]);
    }
    const float r = p.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float dy[8], h[8];
      unpack8(rdy[j], dy);
      unpack8(rh[j], h);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = h[k] * r;
        dw[j][k] = __builtin_fmaf(dy[k], xh, dw[j][k]);
        dot = __builtin_fmaf(dy[k] * wv[j][k], xh, dot);
      }
    }
    // red[turn]: the other half is still being read by slower waves
    const float mean = block_sum<NT>(dot, red[turn]) / (float)K;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t c = 8 * ((int64_t)threadIdx.x + j * NT), n = K - c;
      float dy[8], h[8], dx[8];
      unpack8(rdy[j], dy);
      unpack8(rh[j], h);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        dx[k] = r * __builtin_fmaf(-(h[k] * r), mean, dy[k] * wv[j][k]);
      if (p.dres) {
        float t[8];
        unpack8(rd[j], t);
#pragma unroll
        for (int k = 0; k < 8; ++k) dx[k] += t[k];
      }
      store8<true>(static_cast<T*>(p.dx) + row * K + c, n, dx);
    }
  }
  if (p.dw) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t c = 8 * ((int64_t)threadIdx.x + j * NT);
      store8(p.part + (int64_t)blockIdx.x * K + c, K - c, dw[j]);
    }
  }
}

// Rows too long for the registers, read twice (the second time from L2). Up to
// SUMS = 32768 columns a workgroup's part of dw stays in LDS, each column with
// the lane that owns it; longer rows (SUMS = 0) take dw by a launch of their
// own (norm_dw_long_kernel), which reads dy and h once more. (4096 x
// 28672 BF16 with dres 225 us; in registers, four runs a lane: spills, 458.)
template <typename T, typename W, int SUMS>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const NormBwdArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int NT = 1024;
  __shared__ float red[2][NT / 64 + 1];
  __shared__ __attribute__((aligned(16))) float sums[SUMS ? SUMS : 4];
  if constexpr (SUMS > 0) {
    const float zero[8] = {};
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < p.K; c += 8 * NT) store8(sums + c, 8, zero);
  }
  const int64_t K = p.K, step = 8 * NT;
  const W* w = static_cast<const W*>(p.w);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
    const T* dyr = static_cast<const T*>(p.dy) + row * K;
    const T* hr = static_cast<const T*>(p.h) + row * K;
    const float r = p.rstd[row];
    float dot = 0.0f;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
      float dy[8], h[8], wv[8];
      load8(dyr + c, K - c, dy);
      load8(hr + c, K - c, h);
      load8(w + c, K - c, wv);
#pragma unroll
      for (int k = 0; k < 8; ++k) dot = __builtin_fmaf(dy[k] * wv[k], h[k] * r, dot);
    }
    const float mean = block_sum<NT>(dot, red[turn]) / (float)K;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
      const int64_t n = K - c;
      float dy[8], h[8], wv[8], dx[8];
      load8(dyr + c, n, dy);
      load8(hr + c, n, h);
      load8(w + c, n, wv);
#pragma unroll
      for (int k = 0; k < 8; ++k) dx[k] = r * __builtin_fmaf(-(h[k] * r), mean, dy[k] * wv[k]);
      if (p.dres) {
        float t[8];
        load8(static_cast<const T*>(p.dres) + row * K + c, n, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) dx[k] += t[k];
      }
      store8(static_cast<T*>(p.dx) + row * K + c, n, dx);
      if constexpr (SUMS > 0) {
        float d[8];
        load8(sums + c, 8, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = __builtin_fmaf(dy[k], h[k] * r, d[k]);
        store8(sums + c, 8, d);
      }
    }
  }
  if constexpr (SUMS > 0) {
    if (p.dw)
      for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
        float d[8];
        load8(sums + c, 8, d);
        store8(p.part + (int64_t)blockIdx.x * K + c, K - c, d);
      }
  }
}
// dx may be dy's own buffer (the norm's arguments allow it), so for long rows
// dw is taken before dx is written. Workgroup (bx, by): 2048 columns from c0
// on, rows by, by + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256) norm_dw_long_kernel(const NormBwdArgs p, int64_t c0) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  const int64_t K = p.K, c = c0 + 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x), n = K - c;
  if (n <= 0) return;
  float dw[8] = {};
  for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y) {
    float dy[8], h[8];
    load8(static_cast<const T*>(p.dy) + row * K + c, n, dy);
    load8(static_cast<const T*>(p.h) + row * K + c, n, h);
    const float r = p.rstd[row];
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[k] = __builtin_fmaf(dy[k], h[k] * r, dw[k]);
  }
  store8(p.part + (int64_t)blockIdx.y * K + c, n, dw);
}

// out[c] = sum over i of part[i][c]: 32 strands of rows, each in order, then the
// strands in order. A workgroup owns 32 columns; a strand keeps 8 loads on
// their way (64 columns, 16 strands and one load: 25 us of norm_bwd's 52 at
// 4097 x 2881). c0: the launch's first column.
__global__ void __launch_bounds__(1024) colsum_kernel(const float* part, int64_t P, int64_t N,
                                                      float* out, const float* noop, int64_t c0) {
  if (noop != nullptr && *noop == 1.0f) return;
  __shared__ float acc[32][33];
  const int col = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int64_t c = c0 + (int64_t)blockIdx.x * 32 + col;
  float s = 0.0f;
  if (c < N) {
    const float* q = part + c;
    int64_t i = strand;
    for (; i + 7 * 32 < P; i += 8 * 32) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = q[(i + k * 32) * N];
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
    for (; i < P; i += 32) s += q[i * N];
  }
  acc[strand][col] = s;
  __syncthreads();
  if (strand == 0 && c < N) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += acc[i][col];
    out[c] = s;
  }
}

// Wider inputs take several launches, too: 2^26 columns are 2^31 threads of
// colsum_kernel (32 a column), and of norm_dw_long_kernel with 256 parts.
template <typename F>
static int go_columns(int64_t N, F launch) {
  for (int64_t c = 0; c < N; c += 1 << 26) {
    launch(c, std::min<int64_t>(N - c, 1 << 26));
    if (hipGetLastError() != hipSuccess) return -3;
  }
  return 0;
}

int launch_colsum(const float* part, int64_t P, int64_t N, float* out, const float* noop,
                  hipStream_t s) {
  return go_columns(N, [=](int64_t c0, int64_t n) {
    hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((n + 31) / 32)), dim3(1024), 0, s, part, P, N, out,
                       noop, c0);
  });
}

// Workgroups of the backward pass, a function of the sizes alone so that the
// workspace and the order of the sums do not depend on the device: as many as
// the BF16 kernels keep resident (126 registers: 4 waves a SIMD). The FP32 ones
// hold 134 and 138, one workgroup a CU fewer, and up to 16384 columns 128 with 9
// spilled; from HBM that does not show (4096 x 8192 82 us, 4096 x 16384 163 us, 4.9
// TB/s, as in BF16).
int64_t norm_bwd_parts(int64_t M, int64_t K) {
  const int64_t per_cu = K <= 4096 ? 4 : (K <= 8192 ? 2 : 1);
  return std::min<int64_t>(M, 256 * per_cu);
}

template <typename T, typename W, int NT, int V>
static int go_norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((norm_bwd_kernel<T, W, NT, V>), dim3((unsigned)norm_bwd_parts(a.M, a.K)),
                     dim3(NT), 0, s, a);
  return hipGetLastError() == hipSuccess ? 0 : -3;
}

template <typename T, typename W>
static int launch_norm_bwd_t(NormBwdArgs a, hipStream_t s) {
  if (norm_bwd_parts(a.M, a.K) == 1) a.part = a.dw;  // one part: it is the result
  const int64_t chunks = (a.K + 7) / 8;
  int rc;
  if (chunks <= 64) rc = go_norm_bwd<T, W, 64, 1>(a, s);
  else if (chunks <= 256) rc = go_norm_bwd<T, W, 256, 1>(a, s);
  else if (chunks <= 512) rc = go_norm_bwd<T, W, 256, 2>(a, s);
  else if (chunks <= 1024) rc = go_norm_bwd<T, W, 512, 2>(a, s);
  else if (chunks <= 2048) rc = go_norm_bwd<T, W, 1024, 2>(a, s);
  else if (a.K <= 32768) {
    hipLaunchKernelGGL((norm_bwd_long_kernel<T, W, 32768>), dim3((unsigned)norm_bwd_parts(a.M, a.K)),
                       dim3(1024), 0, s, a);
    rc = hipGetLastError() == hipSuccess ? 0 : -3;
  } else {
    const int64_t P = norm_bwd_parts(a.M, a.K);
    if (a.dw) {
      rc = go_columns(a.K, [&](int64_t c0, int64_t n) {
        hipLaunchKernelGGL((norm_dw_long_kernel<T>), dim3((unsigned)((n + 2047) / 2048), (unsigned)P),
                           dim3(256), 0, s, a, c0);
      });
      if (rc) return rc;
    }
    hipLaunchKernelGGL((norm_bwd_long_kernel<T, W, 0>), dim3((unsigned)P), dim3(1024), 0, s, a);
    rc = hipGetLastError() == hipSuccess ? 0 : -3;
  }
  if (rc) return rc;
  return a.dw && a.part != a.dw ? launch_colsum(a.part, norm_bwd_parts(a.M, a.K), a.K, a.dw, a.noop, s) : 0;
}

int launch_norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  if (a.in_dtype == 0)
    return a.w_dtype == 0 ? launch_norm_bwd_t<uint16_t, uint16_t>(a, s)
                          : launch_norm_bwd_t<uint16_t, float>(a, s);
  return a.w_dtype == 0 ? launch_norm_bwd_t<float, uint16_t>(a, s)
                        : launch_norm_bwd_t<float, float>(a, s);
}

}  // namespace nvfp4
