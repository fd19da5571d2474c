// int8_quant.hip -- lines of 8-bit integers with one amax each (gfx950).
//
//   a    = the line's amax
//   code = the integer nearest to RN(x * S), halves to the even one, clamped to
//          +-127;  S = a == 0 ? 1 : min(RN(127 / a), FLT_MAX)
//   value = code * a / 127
// (a NaN or infinite: codes of zero)
// Rows: one pass, the row held in registers between its amax and its codes. Both
// copies: the amax pass first (a column's amax is not known before its last
// row), then one pass that writes the rowwise and the transposed codes.
#include "nvfp4_launch.h"
#include "nvfp4_rows.h"

#include <algorithm>
#include <type_traits>

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
  const uint32_t keep = keep_finite(a);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * (int64_t)(l + j * L);
    float v[8];
    unpack8(rx[j], v);
    store8_bytes(p.q_row + row * p.K + c, K - c, pack8_int8(v, enc, keep));
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
  const uint32_t keep = keep_finite(a);
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += 8 * NT) {
    float v[8];
    load8(x + c, K - c, v);
    store8_bytes(p.q_row + row * K + c, K - c, pack8_int8(v, enc, keep));
  }
}

// Row and column amaxes joined to what row_amax and col_amax hold: a tile of `tr` rows and
// 32 runs of 16 bytes, 16 lanes to a row. A maximum may take an element twice, so the runs
// and rows that pass the end of x are moved down to end with it: any K from a run up and
// any address, without branches. Maxima leave as atomics (of bits of magnitudes: in any
// order the same). Atomics of many tiles to the same few lines queue: tiles are tall, and
// few enough for three workgroups to a CU. Measured, 4097 x 2881 FP32 with 64 runs by 64
// rows 43 us, 32 runs by 128 rows 13.6, 16 by 256 12.6; 16384 x 8192 BF16 with 64 runs by
// 256 rows 68 us, 32 by 512 63, 16 by 512 72.
// Of a tile's rows the first half is read past the caches, the second through them: the
// cast reads all of x again right after, and finds what was read last. 16384 x 8192 BF16,
// one call after another: 63 to 70 us by the card, 3.9 TB/s (53 where nothing before it is
// still being written out of the caches).
constexpr int kAmaxRuns = 2, kAmaxRows = 512;
template <typename T>
__global__ void __launch_bounds__(256) int8_amax_kernel(const Int8QuantArgs p, int64_t row0, unsigned gn, int tr) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int E = 16 / sizeof(T), D = 4;  // elements and dwords of a run
  constexpr int NC = kAmaxRuns, U = 8 / NC;  // runs of a lane and row, and rows: 8 loads on their way
  __shared__ uint32_t colmax[16][16 * NC * D + 1];
  __shared__ uint32_t rowmax[kAmaxRows];
  const int tid = threadIdx.x, l = tid & 15, slot = tid >> 4;
  const int64_t r0 = row0 + (int64_t)tr * (blockIdx.x / gn);
  const int64_t c0 = (int64_t)(blockIdx.x % gn) * 16 * NC * E;
  const T* x = static_cast<const T*>(p.x);
  auto column = [&](int run) { return min(c0 + (int64_t)E * run, p.K - E); };
  int64_t col[NC];
  uint32_t cm[NC][D] = {};
#pragma unroll
  for (int j = 0; j < NC; ++j) col[j] = column(16 * j + l);
  auto joined = [](uint32_t m, uint32_t w) __attribute__((always_inline)) {
    if constexpr (sizeof(T) == 2) return pk_max_u16(m, w & kAbsBf16x2);
    else return max(m, w & kAbsF32);
  };
  auto rows = [&](int i, auto past) __attribute__((always_inline)) {
    Piece<T, E> v[U][NC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const T* at = x + min(r0 + i + 16 * u, p.M - 1) * p.K;
#pragma unroll
      for (int j = 0; j < NC; ++j) v[u][j].template load<decltype(past)::value>(at + col[j]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t m = 0u;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          cm[j][d] = joined(cm[j][d], v[u][j].d[d]);
          m = joined(m, v[u][j].d[d]);
        }
      }
      if constexpr (sizeof(T) == 2) m = max(m << 16, m & 0xFFFF0000u);
      m = row_max<16>(m, nullptr);
      if (l == 0) rowmax[i + 16 * u] = m;
    }
  };
  int i = slot;
  for (; i < tr / 2; i += 16 * U) rows(i, std::true_type{});
  for (; i < tr; i += 16 * U) rows(i, std::false_type{});
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int d = 0; d < D; ++d) colmax[slot][D * (16 * j + l) + d] = cm[j][d];
  __syncthreads();
  auto publish = [](float* to, uint32_t m) __attribute__((always_inline)) {
    atomicMax(reinterpret_cast<uint32_t*>(to), m);
  };
  for (int r = tid; r < tr && r0 + r < p.M; r += 256) publish(p.row_amax + r0 + r, rowmax[r]);
  if (tid >= 16 * NC * D) return;
  uint32_t m = 0u;
#pragma unroll
  for (int s = 0; s < 16; ++s) m = joined(m, colmax[s][tid]);
  float* to = p.col_amax + column(tid / D) + E / D * (tid % D);
  if constexpr (sizeof(T) == 2) {
    publish(to, m << 16);
    publish(to + 1, m & 0xFFFF0000u);
  } else {
    publish(to, m);
  }
}

// Both copies of a 128 x 128 tile: a thread holds 8 columns of 8 rows (2 turns of
// 4 rows), writes their rowwise codes, and puts their columnwise codes, 4 rows
// to a dword, into LDS by columns, from where they leave as 16-byte runs. 16384 x 8192
// BF16: 95 us, 5.7 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) int8_cast_kernel(const Int8QuantArgs p, int64_t row0, unsigned gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int PITCH = 33;  // dwords of a column's 128 rows, one to spare
  __shared__ uint32_t lds[128 * PITCH];
  __shared__ uint32_t ckeep[128];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int64_t M = p.M, K = p.K;
  const int64_t i0 = row0 + 128 * (int64_t)(blockIdx.x / gn), j0 = 128 * (int64_t)(blockIdx.x % gn);
  const int64_t c = j0 + 8 * cg, n = K - c;
  // Lines of whole 16-byte runs leave past the caches; what is written in pieces meets there
  // first (16384 x 8192 BF16: 105 -> 94 us; 4097 x 2881 FP32 would go from 19 to 23).
  const bool whole = ((M | K) & 15) == 0;
  float ce[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float a = k < n ? p.col_amax[c + k] : 0.0f;
    ce[k] = global_encode_scale(a, kInt8Max);
    if (rg == 0) ckeep[8 * cg + k] = keep_finite(a);
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t r = i0 + 64 * t + 4 * rg;
    Raw8<T> rx[4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
      load8_raw<true>(static_cast<const T*>(p.x) + min(r + v, M - 1) * K + c, n, rx[v]);
    uint32_t cc[4][8];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float x[8];
      unpack8(rx[v], x);
      if (r + v < M) {
        const float a = p.row_amax[r + v], enc = global_encode_scale(a, kInt8Max);
        const u32x2 codes = pack8_int8(x, enc, keep_finite(a));
        uint8_t* q = p.q_row + (r + v) * K + c;
        if (whole && n >= 8) __builtin_nontemporal_store(codes, reinterpret_cast<u32x2_a1*>(q));
        else store8_bytes(q, n, codes);
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
    const uint32_t *l = lds + col * PITCH + 4 * at, keep = ckeep[col];
    const uint32_t w[4] = {l[0] & keep, l[1] & keep, l[2] & keep, l[3] & keep};
    uint8_t* q = p.q_col + j * M + i;
    if (i + 16 <= M) {
      if (whole) __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4_a1*>(q));
      else *reinterpret_cast<u32x4_a1*>(q) = u32x4{w[0], w[1], w[2], w[3]};
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

// The tallest tiles (fewer maxima to publish) that give 3 workgroups to a CU.
template <typename T>
static int launch_amax_t(const Int8QuantArgs& a, hipStream_t s) {
  constexpr int64_t TC = 16 * kAmaxRuns * 16 / sizeof(T);
  const int64_t gn = (a.K + TC - 1) / TC;
  int64_t tr = kAmaxRows;
  while (tr > 128 && (a.M + tr - 1) / tr * gn < 3 * (int64_t)num_cus()) tr /= 2;
  const int64_t gm = (a.M + tr - 1) / tr, step = std::max<int64_t>(1, ((int64_t)1 << 23) / gn);
  for (int64_t i = 0; i < gm; i += step) {
    hipLaunchKernelGGL((int8_amax_kernel<T>), dim3((unsigned)(std::min(step, gm - i) * gn)), dim3(256), 0, s, a,
                       tr * i, (unsigned)gn, (int)tr);
    if (hipGetLastError() != hipSuccess) return -3;
  }
  return 0;
}

int launch_int8_rowcol(const Int8QuantArgs& a, hipStream_t s) {
  int rc = launch_amax_init(a.row_amax, a.M, a.col_amax, a.K, nullptr, a.noop, s);
  if (rc) return rc;
  if (a.K < 8) rc = launch_row_col_amax(a.x, a.in_dtype, a.M, a.K, a.row_amax, a.col_amax, a.noop, s);
  else rc = a.in_dtype == 0 ? launch_amax_t<uint16_t>(a, s) : launch_amax_t<float>(a, s);
  if (rc) return rc;
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
