// int8_quant.hip -- lines of 8-bit integers with one amax each (gfx950).
//
//   a    = the line's amax
//   code = the integer nearest to RN(x * S), halves to the even one, clamped to
//          +-127;  S = a == 0 ? 1 : min(RN(127 / a), FLT_MAX)
//   value = code * a / 127
// Rows: one pass, the row held in registers between its amax and its codes. Both
// copies: the amax pass first (a column's amax is not known before its last
// row), then one pass that writes the rowwise and the transposed codes.
#include "nvfp4_launch.h"
#include "nvfp4_rows.h"

#include <algorithm>

namespace nvfp4 {

// A row takes L lanes and V runs of 8 L columns.
template <typename T, int L, int V, int NT>
__global__ void __launch_bounds__(NT) int8_rows_kernel(const Int8QuantArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int G = NT / L;
  __shared__ uint32_t redm[NT / 64 + 1];
  const int l = threadIdx.x % L;
  const int64_t at = p.row0 + (int64_t)blockIdx.x * G + threadIdx.x / L;
  const bool live = G == 1 || at < p.M;
  const int64_t row = live ? at : p.M - 1, K = live ? p.K : 0;
  Raw8<T> rx[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * (int64_t)(l + j * L);
    load8_raw<true>(static_cast<const T*>(p.x) + row * p.K + c, K - c, rx[j]);
  }
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    m = amax8_raw(rx[j], m);
  }
  const float a = __uint_as_float(row_max<L>(m, redm));
  if (l == 0 && live) p.row_amax[row] = a;
  const float enc = global_encode_scale(a, kInt8Max);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * (int64_t)(l + j * L);
    float v[8];
    unpack8(rx[j], v);
    store8_bytes(p.q_row + row * p.K + c, K - c, pack8_int8(v, enc));
  }
}

// Rows too long for the registers: read twice (the second time from L2).
template <typename T>
__global__ void __launch_bounds__(1024) int8_rows_long_kernel(const Int8QuantArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int NT = 1024;
  __shared__ uint32_t redm[NT / 64 + 1];
  const int64_t row = p.row0 + blockIdx.x, K = p.K;
  const T* x = static_cast<const T*>(p.x) + row * K;
  uint32_t m = 0u;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += 8 * NT) {
    float v[8];
    load8(x + c, K - c, v);
    m = amax8(v, m);
  }
  const float a = __uint_as_float(block_max<NT>(m, redm));
  if (threadIdx.x == 0) p.row_amax[row] = a;
  const float enc = global_encode_scale(a, kInt8Max);
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += 8 * NT) {
    float v[8];
    load8(x + c, K - c, v);
    store8_bytes(p.q_row + row * K + c, K - c, pack8_int8(v, enc));
  }
}

// Both copies of a 128 x 128 tile: a thread holds 8 columns of 8 rows (2 turns of
// 4 rows), writes their rowwise codes, and puts their columnwise codes, 4 rows
// to a dword, into LDS by columns, from where they leave as 16-byte runs.
template <typename T>
__global__ void __launch_bounds__(256) int8_cast_kernel(const Int8QuantArgs p, int64_t row0, unsigned gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int PITCH = 33;  // dwords of a column's 128 rows, one to spare
  __shared__ uint32_t lds[128 * PITCH];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int64_t M = p.M, K = p.K;
  const int64_t i0 = row0 + 128 * (int64_t)(blockIdx.x / gn), j0 = 128 * (int64_t)(blockIdx.x % gn);
  const int64_t c = j0 + 8 * cg, n = K - c;
  float ce[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) ce[k] = k < n ? global_encode_scale(p.col_amax[c + k], kInt8Max) : 0.0f;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t r = i0 + 64 * t + 4 * rg;
    Raw8<T> rx[4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
      load8_raw(static_cast<const T*>(p.x) + min(r + v, M - 1) * K + c, n, rx[v]);
    uint32_t cc[4][8];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float x[8];
      unpack8(rx[v], x);
      if (r + v < M) {
        const float enc = global_encode_scale(p.row_amax[r + v], kInt8Max);
        store8_bytes(p.q_row + (r + v) * K + c, n, pack8_int8(x, enc));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) cc[v][k] = int8_code(x[k], ce[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      lds[(8 * cg + k) * PITCH + 16 * t + rg] = pack4_low(cc[0][k], cc[1][k], cc[2][k], cc[3][k]);
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int col = 32 * t + tid / 8, at = tid % 8;  // 16 rows of a column
    const int64_t j = j0 + col, i = i0 + 16 * at;
    if (j >= K || i >= M) continue;
    const uint32_t* w = lds + col * PITCH + 4 * at;
    uint8_t* q = p.q_col + j * M + i;
    if (i + 16 <= M) {
      *reinterpret_cast<u32x4_a1*>(q) = u32x4{w[0], w[1], w[2], w[3]};
    } else {
      for (int k = 0; k < (int)(M - i); ++k) q[k] = (uint8_t)(w[k / 4] >> (8 * (k & 3)));
    }
  }
}

template <typename T, int L, int V, int NT>
static int go_rows(const Int8QuantArgs& a, hipStream_t s) {
  return rows_in_launches(a.M, [&](int64_t r, int64_t rows) {
    Int8QuantArgs p = a;
    p.row0 = r;
    constexpr int G = NT / L;
    hipLaunchKernelGGL((int8_rows_kernel<T, L, V, NT>), dim3((unsigned)((rows + G - 1) / G)), dim3(NT), 0, s, p);
  });
}

template <typename T>
static int launch_rows_t(const Int8QuantArgs& a, hipStream_t s) {
  const int64_t chunks = (a.K + 7) / 8;
  if (chunks <= 16) return go_rows<T, 16, 1, 256>(a, s);
  if (chunks <= 64) return go_rows<T, 64, 1, 256>(a, s);
  if (chunks <= 256) return go_rows<T, 256, 1, 256>(a, s);
  if (chunks <= 512) return go_rows<T, 256, 2, 256>(a, s);
  if (chunks <= 1024) return go_rows<T, 1024, 1, 1024>(a, s);
  if (chunks <= 2048) return go_rows<T, 1024, 2, 1024>(a, s);
  if (chunks <= 4096) return go_rows<T, 1024, 4, 1024>(a, s);
  return rows_in_launches(a.M, [&](int64_t r, int64_t rows) {
    Int8QuantArgs p = a;
    p.row0 = r;
    hipLaunchKernelGGL((int8_rows_long_kernel<T>), dim3((unsigned)rows), dim3(1024), 0, s, p);
  });
}

int launch_int8_rows(const Int8QuantArgs& a, hipStream_t s) {
  return a.in_dtype == 0 ? launch_rows_t<uint16_t>(a, s) : launch_rows_t<float>(a, s);
}

int launch_int8_rowcol(const Int8QuantArgs& a, hipStream_t s) {
  const int64_t gn = (a.K + 127) / 128, gm = (a.M + 127) / 128;
  // a launch holds fewer than 2^32 threads
  const int64_t step = std::max<int64_t>(1, ((int64_t)1 << 23) / gn);
  for (int64_t i = 0; i < gm; i += step) {
    const dim3 g((unsigned)(std::min(step, gm - i) * gn)), b(256);
    if (a.in_dtype == 0) hipLaunchKernelGGL((int8_cast_kernel<uint16_t>), g, b, 0, s, a, 128 * i, (unsigned)gn);
    else hipLaunchKernelGGL((int8_cast_kernel<float>), g, b, 0, s, a, 128 * i, (unsigned)gn);
    if (hipGetLastError() != hipSuccess) return -3;
  }
  return 0;
}

}  // namespace nvfp4
