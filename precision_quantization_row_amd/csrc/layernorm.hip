// layernorm.hip -- layer norm of the residual stream, quantized on the way
// out, and its backward pass (gfx950).
//
// Forward, per row:
//   h_k = x_k + residual_k                    (kept in FP32; h is stored rounded)
//   mu  = sum_k h_k / K,  var = sum_k (h_k - mu)^2 / K,  r = 1 / sqrt(var + eps)
//   y_k = ((h_k - mu) * r) * w_k + b_k
// and y's row amax and codes as in the root-mean-square norm, or as 8-bit integers.
// The sums are taken twice over the row's registers: mu0 from the first, then
// sum (h - mu0) and sum (h - mu0)^2, which give the mean its low bits back (what
// rounding the first sum to 24 bits took) and the variance without the
// cancellation of sum h^2 - K mu^2.
// Backward, per row, with xh_k = (h_k - mu) * r and g_k = dy_k * w_k:
//   dx_k = r (g_k - sum_j(g_j) / K - xh_k * sum_j(g_j xh_j) / K) + dres_k
//   dw_k = sum over rows of dy_k * xh_k,   db_k = sum over rows of dy_k
//
// Both are bound by HBM: a row is read once into registers, reduced there and
// written once. Forward, 16384 x 4096 BF16 with the residual: 95 to 98 us, 5.5 TB/s, into
// 8-bit lines 81; one row of 8192 4.6 us, a load's latency and the meetings of its waves.
#include "nvfp4_launch.h"
#include "nvfp4_rows.h"

#include <algorithm>

namespace nvfp4 {

// A row takes L lanes (a power of two up to 64, several rows to a wave; or a
// whole workgroup) and V runs of 8 L columns, held in registers.
template <typename T, typename W, int L, int V, int NT>
__global__ void __launch_bounds__(NT) ln_kernel(const LayerNormArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  static_assert(L <= 64 || L == NT, "a row is a part of a wave or a workgroup");
  constexpr int G = NT / L;  // rows of a workgroup
  __shared__ float red[3 * (NT / 64) + 1];
  __shared__ uint32_t redm[NT / 64 + 1];
  const int l = threadIdx.x % L;
  const int64_t at = p.row0 + (int64_t)blockIdx.x * G + threadIdx.x / L;
  const bool live = G == 1 || at < p.M;
  const int64_t row = live ? at : p.M - 1, K = live ? p.K : 0, pitch = p.K;
  const T* x = static_cast<const T*>(p.x) + row * pitch;
  const T* res = static_cast<const T*>(p.residual) + (p.residual ? row * pitch : 0);
  const W *w = static_cast<const W*>(p.w), *b = static_cast<const W*>(p.b);
  // w and b beside the row where the registers have room, after its sums elsewhere
  constexpr bool EARLY = V * sizeof(W) <= 4;
  Raw8<T> rx[V], rr[V];
  Raw8<W> rw[V], rb[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * (int64_t)(l + j * L), n = K - c;
    load8_raw<true>(x + c, n, rx[j]);
    if (p.residual) load8_raw<true>(res + c, n, rr[j]);
  }
  auto load_wb = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t c = 8 * (int64_t)(l + j * L);
      load8_raw(w + c, K - c, rw[j]);
      if (p.b) load8_raw(b + c, K - c, rb[j]);
    }
  };
  if constexpr (EARLY) load_wb();
  float h[V][8];
  float s0 = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * (int64_t)(l + j * L), n = K - c;
    unpack8(rx[j], h[j]);
    if (p.residual) {
      float t[8];
      unpack8(rr[j], t);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[j][k] += t[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s0 += h[j][k];
    if (p.h) store8<true>(static_cast<T*>(p.h) + row * pitch + c, n, h[j]);
  }
  const float mu0 = row_sum<L>(s0, red) / (float)pitch;
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t n = K - 8 * (int64_t)(l + j * L);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[j][k] = k < n ? h[j][k] - mu0 : 0.0f;
      s1 += h[j][k];
      s2 = __builtin_fmaf(h[j][k], h[j][k], s2);
    }
  }
  row_sum2<L>(s1, s2, red + NT / 64);
  const float dm = s1 / (float)pitch, mean = mu0 + dm;
  float var = s2 / (float)pitch - dm * dm;
  var = var < 0.0f ? 0.0f : var;  // (a constant row; NaN stays NaN)
  const float rstd = 1.0f / sqrtf(var + p.eps);
  if (l == 0 && live) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  if constexpr (!EARLY) load_wb();
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * (int64_t)(l + j * L), n = K - c;
    float wv[8], bv[8] = {};
    unpack8(rw[j], wv);
    if (p.b) unpack8(rb[j], bv);
#pragma unroll
    for (int k = 0; k < 8; ++k) h[j][k] = k < n ? __builtin_fmaf((h[j][k] - dm) * rstd, wv[k], bv[k]) : 0.0f;
    m = amax8(h[j], m);
    if (p.y) {
      if (p.y_dtype == 0) store8(static_cast<uint16_t*>(p.y) + row * pitch + c, n, h[j]);
      else store8(static_cast<float*>(p.y) + row * pitch + c, n, h[j]);
    }
  }
  if (!p.row_amax) return;
  const float a = __uint_as_float(row_max<L>(m, redm));
  if (l == 0 && live) p.row_amax[row] = a;
  if (!p.q_fmt) return;
  const float enc = global_encode_scale(a, line_top(p.q_fmt, p.F));
  uint8_t* q = p.q + row * (p.q_fmt == FMT_NVFP4 ? (pitch + 1) / 2 : pitch);
  uint8_t* s = p.s + row * ((pitch + 15) / 16);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = 8 * (int64_t)(l + j * L);
    write_codes<true>(p.q_fmt, q, s, c, K - c, h[j], a, enc, p.F_inv);
  }
}

// Rows too long for the registers: the same steps, x and the residual read
// once for each of the four loops (from L2 after the first).
template <typename T, typename W>
__global__ void __launch_bounds__(1024) ln_long_kernel(const LayerNormArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int NT = 1024;
  __shared__ float red[3 * (NT / 64) + 1];
  __shared__ uint32_t redm[NT / 64 + 1];
  const int64_t row = p.row0 + blockIdx.x, K = p.K, step = 8 * NT;
  const T* x = static_cast<const T*>(p.x) + row * K;
  const T* res = static_cast<const T*>(p.residual) + (p.residual ? row * K : 0);
  const W *w = static_cast<const W*>(p.w), *b = static_cast<const W*>(p.b);
  auto load_h = [&](int64_t c, float (&h)[8]) {
    load8(x + c, K - c, h);
    if (p.residual) {
      float t[8];
      load8(res + c, K - c, t);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] += t[k];
    }
  };
  float s0 = 0.0f;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
    float h[8];
    load_h(c, h);
#pragma unroll
    for (int k = 0; k < 8; ++k) s0 += h[k];
  }
  const float mu0 = block_sum<NT>(s0, red) / (float)K;
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
    float h[8];
    load_h(c, h);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = k < K - c ? h[k] - mu0 : 0.0f;
      s1 += d;
      s2 = __builtin_fmaf(d, d, s2);
    }
  }
  row_sum2<NT>(s1, s2, red + NT / 64);
  const float dm = s1 / (float)K, mean = mu0 + dm;
  float var = s2 / (float)K - dm * dm;
  var = var < 0.0f ? 0.0f : var;
  const float rstd = 1.0f / sqrtf(var + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  // the row's y from its h (zeros past the row)
  auto finish = [&](int64_t c, const float (&h)[8], float (&y)[8]) {
    float wv[8], bv[8] = {};
    load8(w + c, K - c, wv);
    if (p.b) load8(b + c, K - c, bv);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      y[k] = k < K - c ? __builtin_fmaf(((h[k] - mu0) - dm) * rstd, wv[k], bv[k]) : 0.0f;
  };
  float a = 0.0f, enc = 0.0f;
  if (p.row_amax) {
    uint32_t m = 0u;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
      float h[8], y[8];
      load_h(c, h);
      finish(c, h, y);
      m = amax8(y, m);
    }
    a = __uint_as_float(block_max<NT>(m, redm));
    if (threadIdx.x == 0) p.row_amax[row] = a;
    enc = global_encode_scale(a, line_top(p.q_fmt, p.F));
  }
  uint8_t* q = p.q + row * (p.q_fmt == FMT_NVFP4 ? (K + 1) / 2 : K);
  uint8_t* s = p.s + row * ((K + 15) / 16);
  // every lane of a wave takes part in each turn (write_codes joins lane pairs)
  for (int64_t c0 = 8 * (int64_t)(threadIdx.x & ~63); c0 < K; c0 += step) {
    const int64_t c = c0 + 8 * (threadIdx.x & 63), n = K - c;
    float h[8] = {}, y[8] = {};
    if (n > 0) {
      load_h(c, h);
      finish(c, h, y);
    }
    // h may be x's or the residual's own buffer: the row is read for the last
    // time above, by the lane that writes it here
    if (p.h) store8(static_cast<T*>(p.h) + row * K + c, n, h);
    if (p.y) {
      if (p.y_dtype == 0) store8(static_cast<uint16_t*>(p.y) + row * K + c, n, y);
      else store8(static_cast<float*>(p.y) + row * K + c, n, y);
    }
    if (p.q_fmt) write_codes<true>(p.q_fmt, q, s, c, n, y, a, enc, p.F_inv);
  }
}

template <typename T, typename W, int L, int V, int NT>
static int go_ln(const LayerNormArgs& a, hipStream_t s) {
  return rows_in_launches(a.M, [&](int64_t r, int64_t rows) {
    LayerNormArgs p = a;
    p.row0 = r;
    constexpr int G = NT / L;
    hipLaunchKernelGGL((ln_kernel<T, W, L, V, NT>), dim3((unsigned)((rows + G - 1) / G)), dim3(NT), 0, s, p);
  });
}

template <typename T, typename W>
static int launch_ln_t(const LayerNormArgs& a, hipStream_t s) {
  const int64_t chunks = (a.K + 7) / 8;
  if (chunks <= 16) return go_ln<T, W, 16, 1, 256>(a, s);
  if (chunks <= 64) return go_ln<T, W, 64, 1, 256>(a, s);
  if (chunks <= 256) return go_ln<T, W, 256, 1, 256>(a, s);
  if (chunks <= 512) return go_ln<T, W, 256, 2, 256>(a, s);
  if (chunks <= 1024) return go_ln<T, W, 1024, 1, 1024>(a, s);
  if (chunks <= 2048) return go_ln<T, W, 1024, 2, 1024>(a, s);
  if (chunks <= 4096) return go_ln<T, W, 1024, 4, 1024>(a, s);
  return rows_in_launches(a.M, [&](int64_t r, int64_t rows) {
    LayerNormArgs p = a;
    p.row0 = r;
    hipLaunchKernelGGL((ln_long_kernel<T, W>), dim3((unsigned)rows), dim3(1024), 0, s, p);
  });
}

int launch_layernorm(const LayerNormArgs& a, hipStream_t s) {
  if (a.in_dtype == 0)
    return a.w_dtype == 0 ? launch_ln_t<uint16_t, uint16_t>(a, s) : launch_ln_t<uint16_t, float>(a, s);
  return a.w_dtype == 0 ? launch_ln_t<float, uint16_t>(a, s) : launch_ln_t<float, float>(a, s);
}

// ---------------------------------------------------------------- backward
// A workgroup takes G rows at a time, blockIdx.x G, (blockIdx.x + gridDim.x) G,
// ..., and keeps the parts of dw and db that they give in registers; its row
// groups join theirs in LDS, in order, and the sums go to row blockIdx.x of the
// workspace, whose rows colsum_kernel adds in order: no atomics, so the result
// does not depend on timing. A workspace row holds dw, then db (those asked for).
// 16384 x 4096 BF16 with dres: 94 to 97 us, 5.6 TB/s, and 5 us for the joining; 4097 x 2881
// FP32 without: 29 to 31 us, 4.7 TB/s, and 5.2 us. Rows of 8193 to 16384 spill: 45 and 48
// registers of FP32, 5 of BF16 with BF16 weights.
template <typename T, typename W, int L, int V, int NT>
__global__ void __launch_bounds__(NT) ln_bwd_kernel(const LayerNormBwdArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  static_assert(L <= 64 || L == NT, "a row is a part of a wave or a workgroup");
  constexpr int G = NT / L, E = 16 / sizeof(T), R = 8 * V / E;
  // HOLD: w stays in registers, elsewhere it is read again (from L2) for every row. AHEAD:
  // the next rows are read while these are worked on: BF16, 16384 x 4096 (512 threads to a
  // row) 107 -> 94 us; FP32 has the bytes on their way without, and not the registers.
  constexpr bool HOLD = V == 1, AHEAD = HOLD && sizeof(T) == 2;
  __shared__ float red[2][2 * (NT / 64) + 1];
  const int l = threadIdx.x % L;
  const int K = (int)p.K;  // 8 at least
  const float Kf = (float)K;
  const T *dy_ = static_cast<const T*>(p.dy), *h_ = static_cast<const T*>(p.h), *d_ = static_cast<const T*>(p.dres);
  const W* w_ = static_cast<const W*>(p.w);
  Piece<W, E> rw[R];
  float dw[R][E], db[R][E];
  // A lane's runs of 16 bytes, the row's last one moved down to end with the row: every
  // lane reads whole runs, without branches, and takes the first `twice` of its columns,
  // which are another lane's too, as zeros.
  uint32_t col[R];  // (unsigned: a row's base stays in scalar registers)
  int twice[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int c = E * (l + j * L);
    col[j] = (uint32_t)min(c, K - E);
    twice[j] = c - (int)col[j];
    if (HOLD) {
      rw[j].load(w_ + col[j]);
      rw[j].clear_first(twice[j]);
    }
#pragma unroll
    for (int k = 0; k < E; ++k) dw[j][k] = db[j][k] = 0.0f;
  }
  struct Row {
    Piece<T, E> dy[R], h[R], d[R];
    float r, mu;
  };
  // G rows from r0 on; a group behind the last row reads the last one
  auto load = [&](int64_t r0, Row& a) __attribute__((always_inline)) {
    const int64_t at = r0 + (G == 1 ? 0 : (int)threadIdx.x / L);
    const int64_t row = G == 1 || at < p.M ? at : p.M - 1;
    const T *dy = dy_ + row * K, *h = h_ + row * K, *d = d_ + row * K;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      a.dy[j].template load<true>(dy + col[j]);
      a.h[j].template load<true>(h + col[j]);
      if (d_) a.d[j].template load<true>(d + col[j]);
    }
    a.r = p.rstd[row];
    a.mu = p.mean[row];
  };
  auto step = [&](int64_t r0, Row& a, float* rd) __attribute__((always_inline)) {
    const int64_t row = r0 + (G == 1 ? 0 : (int)threadIdx.x / L);
    const bool live = G == 1 || row < p.M;
    const float r = live ? a.r : 0.0f, mu = live ? a.mu : 0.0f;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float dy[E], h[E], w[E];
      const int t = live ? twice[j] : E;
      if (!HOLD) rw[j].load(w_ + col[j]);
      // What is taken as zeros: dy and w (an infinity times zero is none), but not h: it is another
      // lane's element of this row, so that xh is finite if the row's are ((0 - mu) r need not be).
      if (t > 0) {
        a.dy[j].clear_first(t);
        if (!HOLD) rw[j].clear_first(t);
      }
      if (!live) a.h[j].clear_first(E);  // (mu and r are zeros as well)
      a.dy[j].get(dy);
      a.h[j].get(h);
      rw[j].get(w);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float xh = (h[k] - mu) * r, g = dy[k] * w[k];
        dw[j][k] = __builtin_fmaf(dy[k], xh, dw[j][k]);
        db[j][k] += dy[k];
        s1 += g;
        s2 = __builtin_fmaf(g, xh, s2);
      }
    }
    row_sum2<L>(s1, s2, rd);
    const float m1 = s1 / Kf, m2 = s2 / Kf;
    T* out = static_cast<T*>(p.dx) + row * K;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float dy[E], h[E], w[E], dx[E];
      a.dy[j].get(dy);
      a.h[j].get(h);
      if (!HOLD) rw[j].load(w_ + col[j]);
      rw[j].get(w);
#pragma unroll
      for (int k = 0; k < E; ++k)
        dx[k] = r * (__builtin_fmaf(-((h[k] - mu) * r), m2, dy[k] * w[k]) - m1);
      if (d_) {
        float t[E];
        a.d[j].get(t);
#pragma unroll
        for (int k = 0; k < E; ++k) dx[k] += t[k];
      }
      if (!live) continue;
      if (twice[j] == 0) {
        Piece<T, E>::store(out + col[j], dx);
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (k >= twice[j]) store1(out + col[j] + k, dx[k]);
      }
    }
  };
  // two halves of red: the other one may still be read by slower waves
  const int64_t stride = (int64_t)gridDim.x * G;
  int64_t r0 = (int64_t)blockIdx.x * G;
  if constexpr (AHEAD) {
    Row a, b;
    load(r0, a);
    for (;;) {
      const int64_t r1 = r0 + stride, r2 = r1 + stride;
      if (r1 < p.M) load(r1, b);
      step(r0, a, red[0]);
      if (r1 >= p.M) break;
      if (r2 < p.M) load(r2, a);
      step(r1, b, red[1]);
      if (r2 >= p.M) break;
      r0 = r2;
    }
  } else {
    for (int turn = 0; r0 < p.M; r0 += stride, turn ^= 1) {
      Row a;
      load(r0, a);
      step(r0, a, red[turn]);
    }
  }
  if (!p.dw && !p.db) return;
  float* part = p.part + (int64_t)blockIdx.x * K * ((p.dw ? 1 : 0) + (p.db ? 1 : 0));
  float *pw = p.dw ? part : nullptr, *pb = p.db ? part + (p.dw ? K : 0) : nullptr;
  if constexpr (G > 1) {
    __shared__ float sums[2][G][8 * L];
    const int grp = threadIdx.x / L;
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if (k < twice[j]) continue;
        sums[0][grp][col[j] + k] = dw[j][k];
        sums[1][grp][col[j] + k] = db[j][k];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < K; c += NT) {
      float u = 0.0f, v = 0.0f;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        u += sums[0][i][c];
        v += sums[1][i][c];
      }
      if (pw) pw[c] = u;
      if (pb) pb[c] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (twice[j] == 0) {
        if (pw) Piece<float, E>::store(pw + col[j], dw[j]);
        if (pb) Piece<float, E>::store(pb + col[j], db[j]);
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k) {
          if (k < twice[j]) continue;
          if (pw) pw[col[j] + k] = dw[j][k];
          if (pb) pb[col[j] + k] = db[j][k];
        }
      }
    }
  }
}

// Rows too long for the registers (or shorter than a run), read twice (the second time from L2); dw and
// db by a launch of their own (ln_sums_long_kernel), before dx, which may be dy's
// buffer, is written.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) ln_bwd_long_kernel(const LayerNormBwdArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int NT = 1024;
  __shared__ float red[2][2 * (NT / 64) + 1];
  const int64_t K = p.K, step = 8 * NT;
  const W* w = static_cast<const W*>(p.w);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
    const T* dyr = static_cast<const T*>(p.dy) + row * K;
    const T* hr = static_cast<const T*>(p.h) + row * K;
    const float r = p.rstd[row], mu = p.mean[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
      float dy[8], h[8], wv[8];
      load8(dyr + c, K - c, dy);
      load8(hr + c, K - c, h);
      load8(w + c, K - c, wv);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // (past the row's end g is zero, and -mu r may be infinite)
        const float g = dy[k] * wv[k], xh = k < K - c ? (h[k] - mu) * r : 0.0f;
        s1 += g;
        s2 = __builtin_fmaf(g, xh, s2);
      }
    }
    row_sum2<NT>(s1, s2, red[turn]);
    const float m1 = s1 / (float)K, m2 = s2 / (float)K;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < K; c += step) {
      const int64_t n = K - c;
      float dy[8], h[8], wv[8], dx[8];
      load8(dyr + c, n, dy);
      load8(hr + c, n, h);
      load8(w + c, n, wv);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        dx[k] = r * (__builtin_fmaf(-((h[k] - mu) * r), m2, dy[k] * wv[k]) - m1);
      if (p.dres) {
        float t[8];
        load8(static_cast<const T*>(p.dres) + row * K + c, n, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) dx[k] += t[k];
      }
      store8(static_cast<T*>(p.dx) + row * K + c, n, dx);
    }
  }
}
// Workgroup (bx, by): 2048 columns from c0 on, rows by, by + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256) ln_sums_long_kernel(const LayerNormBwdArgs p, int64_t c0) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  const int64_t K = p.K, c = c0 + 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x), n = K - c;
  if (n <= 0) return;
  float dw[8] = {}, db[8] = {};
  for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y) {
    float dy[8], h[8];
    load8(static_cast<const T*>(p.dy) + row * K + c, n, dy);
    load8(static_cast<const T*>(p.h) + row * K + c, n, h);
    const float r = p.rstd[row], mu = p.mean[row];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      dw[k] = __builtin_fmaf(dy[k], (h[k] - mu) * r, dw[k]);
      db[k] += dy[k];
    }
  }
  float* part = p.part + (int64_t)blockIdx.y * K * ((p.dw ? 1 : 0) + (p.db ? 1 : 0)) + c;
  if (p.dw) store8(part, n, dw);
  if (p.db) store8(part + (p.dw ? K : 0), n, db);
}

// Rows of a workgroup, and workgroups of the backward pass: functions of the
// sizes alone, so that the workspace and the order of the sums do not depend
// on the device.
static int64_t ln_bwd_group(int64_t K) { return K <= 128 ? 16 : (K <= 512 ? 4 : 1); }
int64_t layernorm_bwd_parts(int64_t M, int64_t K) {
  const int64_t per_cu = K <= 2048 ? 4 : (K <= 4096 ? 2 : 1), G = ln_bwd_group(K);
  return std::min<int64_t>((M + G - 1) / G, 256 * per_cu);
}

template <typename T, typename W, int L, int V, int NT>
static int go_ln_bwd(const LayerNormBwdArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((ln_bwd_kernel<T, W, L, V, NT>), dim3((unsigned)layernorm_bwd_parts(a.M, a.K)), dim3(NT),
                     0, s, a);
  return hipGetLastError() == hipSuccess ? 0 : -3;
}

template <typename T, typename W>
static int launch_ln_bwd_t(const LayerNormBwdArgs& a, hipStream_t s) {
  const int64_t chunks = (a.K + 7) / 8, P = layernorm_bwd_parts(a.M, a.K);
  int rc;
  if (a.K >= 8 && chunks <= 16) rc = go_ln_bwd<T, W, 16, 1, 256>(a, s);
  else if (a.K >= 8 && chunks <= 64) rc = go_ln_bwd<T, W, 64, 1, 256>(a, s);
  else if (a.K >= 8 && chunks <= 256) rc = go_ln_bwd<T, W, 256, 1, 256>(a, s);
  else if (a.K >= 8 && chunks <= 512) rc = go_ln_bwd<T, W, 512, 1, 512>(a, s);
  else if (a.K >= 8 && chunks <= 1024) rc = go_ln_bwd<T, W, 1024, 1, 1024>(a, s);
  else if (a.K >= 8 && chunks <= 2048) rc = go_ln_bwd<T, W, 1024, 2, 1024>(a, s);
  else {
    if (a.dw || a.db) {
      rc = columns_in_launches(a.K, [&](int64_t c0, int64_t n) {
        hipLaunchKernelGGL((ln_sums_long_kernel<T>), dim3((unsigned)((n + 2047) / 2048), (unsigned)P),
                           dim3(256), 0, s, a, c0);
      });
      if (rc) return rc;
    }
    hipLaunchKernelGGL((ln_bwd_long_kernel<T, W>), dim3((unsigned)P), dim3(1024), 0, s, a);
    rc = hipGetLastError() == hipSuccess ? 0 : -3;
  }
  if (rc || (!a.dw && !a.db)) return rc;
  const int64_t N = a.dw && a.db ? 2 * a.K : a.K;
  return launch_colsum(a.part, P, N, a.dw ? a.dw : a.db, a.noop, s, a.dw ? a.db : nullptr, a.K);
}

int launch_layernorm_bwd(const LayerNormBwdArgs& a, hipStream_t s) {
  if (a.in_dtype == 0)
    return a.w_dtype == 0 ? launch_ln_bwd_t<uint16_t, uint16_t>(a, s)
                          : launch_ln_bwd_t<uint16_t, float>(a, s);
  return a.w_dtype == 0 ? launch_ln_bwd_t<float, uint16_t>(a, s)
                        : launch_ln_bwd_t<float, float>(a, s);
}

}  // namespace nvfp4
