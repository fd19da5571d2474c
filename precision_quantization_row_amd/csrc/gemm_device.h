// gemm_device.h -- product of two packed operands with bias, activation and
// residual in its epilogue (gfx950): what its kernels share.
//
//   z_ij = (a_i f_A)(b_j f_B) sum_k u_ik v_jk + bias_j
//   y_ij = act(z_ij) + residual_ij
// u_ik = e2m1(code) * e4m3(block byte) (NVFP4) or e4m3(byte) (8-bit lines),
// v_jk the NVFP4 value of the other operand; a_i, b_j are the lines'
// second-level amaxes and f the factor 1 / (bound * 6) or 1 / 448. Both
// operands are stored line by line along k, so the three products of training
// are this one: forward (rowwise X, rowwise W), data gradient (rowwise dY,
// columnwise W), weight gradient (columnwise dY, columnwise X).
//
// Arithmetic. e2m1 has 2 significant bits and e4m3 has 4: u and v have at
// most 6 and lie in [2^-10, 2688], so binary16 holds them exactly and the
// matrix instructions take them as they are; products and sums are FP32. The
// second-level factors (amaxes and f) are applied once per output: their
// mantissas are multiplied and their exponents added, so that neither a huge
// times a tiny one nor an intermediate product leaves the FP32 range on the way.
#pragma once

#include "nvfp4_launch.h"
#include "nvfp4_vec.h"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace nvfp4 {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int... I, typename F>
__device__ __forceinline__ void static_for_(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(0), f(1), ..., f(N - 1) with the index a constant
template <int N, typename F>
__device__ __forceinline__ void static_for(F f) {
  static_for_(std::make_integer_sequence<int, N>{}, f);
}

// ------------------------------------------------------------------ decode
// Pair P of a dword's 4 pairs of codes (of its 2 pairs of E4M3 bytes).
template <int P>
__device__ __forceinline__ h2 cvt_fp4(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, P);
}
template <int P>
__device__ __forceinline__ h2 cvt_fp8(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, P != 0);
}
// 8 codes (one dword) times their block scale (both halves of sc).
__device__ __forceinline__ h8 decode8_fp4(uint32_t w, h2 sc) {
  const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * sc;
  const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * sc;
  const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * sc;
  const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * sc;
  return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
// 8 E4M3 bytes (two dwords).
__device__ __forceinline__ h8 decode8_fp8(uint32_t w0, uint32_t w1) {
  const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false);
  const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true);
  const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false);
  const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true);
  return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// ---------------------------------------------------------------- epilogue
struct LineScale {
  float m;  // mantissas of the amax and of f, multiplied: [1/4, 1)
  int e;    // exponents, added
};
__device__ __forceinline__ LineScale line_scale(const GemmOperand& o, int64_t line) {
  const float a = o.amax[o.mode == 0 ? 0 : line];
  return {__builtin_amdgcn_frexp_mantf(a) * o.f_m, __builtin_amdgcn_frexp_expf(a) + o.f_e};
}
__device__ __forceinline__ float apply_scale(float acc, const LineScale& x, const LineScale& w) {
  return __builtin_amdgcn_ldexpf(acc * (x.m * w.m), x.e + w.e);
}
__device__ __forceinline__ float load_bias(const GemmArgs& p, int64_t j) {
  return p.bias == nullptr ? 0.0f
         : p.bias_dtype == 0 ? load1(static_cast<const uint16_t*>(p.bias) + j)
                             : static_cast<const float*>(p.bias)[j];
}
// 8 consecutive outputs, from column j on, of each of the lines i, i + STEP,
// .., i + (NL - 1) STEP; nj columns (8 or more: all) and the lines below M
// are in the matrix. z0: pre-activations (the gate's, if gated), z1: the up
// lines'; both with their bias.
// res: the residual, from load_residual.
template <typename T, int NL, int STEP>
__device__ __forceinline__ void load_residual(const GemmArgs& p, int64_t i, int64_t j, int64_t nj,
                                              Raw8<T> (&res)[NL]) {
  if (!p.residual || nj <= 0) return;
#pragma unroll
  for (int v = 0; v < NL; ++v)
    if (i + v * STEP < p.M)
      load8_raw(static_cast<const T*>(p.residual) + (i + v * STEP) * p.N + j, nj, res[v]);
}
template <typename T, bool GATED, int NL, int STEP>
__device__ __forceinline__ void finish_lines(const GemmArgs& p, int64_t i, int64_t j, int64_t nj,
                                             float (&z0)[NL][8], float (&z1)[NL][8],
                                             const Raw8<T> (&res)[NL]) {
  if (nj <= 0) return;
  if (p.z) {
#pragma unroll
    for (int v = 0; v < NL; ++v)
      if (i + v * STEP < p.M) {
        T* z = static_cast<T*>(p.z) + (i + v * STEP) * (GATED ? 2 * p.N : p.N) + j;
        store8(z, nj, z0[v]);
        if constexpr (GATED) store8(z + p.N, nj, z1[v]);
      }
  }
  if constexpr (GATED) {
#pragma unroll
    for (int v = 0; v < NL; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) z0[v][e] = silu_f(z0[v][e]) * z1[v][e];
  } else if (p.act != ACT_NONE) {
#pragma unroll
    for (int v = 0; v < NL; ++v) act8(p.act, z0[v]);
  }
  if (p.residual) {
#pragma unroll
    for (int v = 0; v < NL; ++v) {
      float r[8];
      unpack8(res[v], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) z0[v][e] += r[e];
    }
  }
#pragma unroll
  for (int v = 0; v < NL; ++v)
    if (i + v * STEP < p.M) store8(static_cast<T*>(p.y) + (i + v * STEP) * p.N + j, nj, z0[v]);
}

// 4 bytes of a packed line from byte `off` on; bytes past the line's end read
// as zero. Only bytes of the line are touched: a dword that would cross the
// end is read from the line's last 4 bytes and shifted down (lines of 4 bytes
// and more; shorter ones byte by byte).
__device__ __forceinline__ uint32_t tail_dword(const uint8_t* line, int pitch, int off) {
  if (pitch >= 4) {
    const int o = min(off, pitch - 4), sh = off - o;
    const uint32_t w = *reinterpret_cast<const u32_a1*>(line + o);
    return sh < 4 ? w >> (8 * sh) : 0u;
  }
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (off + i < pitch) w |= (uint32_t)line[off + i] << (8 * i);
  return w;
}
// keeps the first n of 8 nibbles (n may be below 0 or above 8)
__device__ __forceinline__ uint32_t keep_nibbles(uint32_t w, int n) {
  return n >= 8 ? w : n <= 0 ? 0u : w & ((1u << (4 * n)) - 1u);
}
__device__ __forceinline__ uint32_t keep_bytes(uint32_t w, int n) {
  return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u);
}

}  // namespace nvfp4
