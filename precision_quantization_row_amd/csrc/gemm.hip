// gemm.hip -- product of two packed operands with bias, activation and
// residual in its epilogue (gfx950).
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
// second-level factors are applied once per output: their mantissas are
// multiplied and their exponents added, so that neither a huge times a tiny
// amax nor an intermediate product leaves the FP32 range on the way.
#include "nvfp4_launch.h"
#include "nvfp4_vec.h"

#include <algorithm>

namespace nvfp4 {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------------ decode
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
  float m;  // mantissa of the amax times f_inv
  int e;    // its exponent
};
__device__ __forceinline__ LineScale line_scale(const GemmOperand& o, int64_t line) {
  const float a = o.amax[o.mode == 0 ? 0 : line];
  return {__builtin_amdgcn_frexp_mantf(a) * o.f_inv, __builtin_amdgcn_frexp_expf(a)};
}
__device__ __forceinline__ float apply_scale(float acc, const LineScale& x, const LineScale& w) {
  return __builtin_amdgcn_ldexpf(acc * (x.m * w.m), x.e + w.e);
}
__device__ __forceinline__ float load_bias(const GemmArgs& p, int64_t j) {
  return p.bias == nullptr ? 0.0f
         : p.bias_dtype == 0 ? load1(static_cast<const uint16_t*>(p.bias) + j)
                             : static_cast<const float*>(p.bias)[j];
}
__device__ __forceinline__ float load_out(const void* t, int dtype, int64_t i) {
  return dtype == 0 ? load1(static_cast<const uint16_t*>(t) + i) : static_cast<const float*>(t)[i];
}
__device__ __forceinline__ void store_out(void* t, int dtype, int64_t i, float v) {
  if (dtype == 0) store1(static_cast<uint16_t*>(t) + i, v);
  else static_cast<float*>(t)[i] = v;
}
// One output, scalar accesses. z0: its pre-activation (the gate's, if gated),
// z1: the up line's, if gated; both with their bias.
__device__ __forceinline__ void finish1(const GemmArgs& p, int64_t i, int64_t j, float z0, float z1) {
  const bool gated = p.act == ACT_SWIGLU;
  if (p.z) {
    const int64_t NB = gated ? 2 * p.N : p.N;
    store_out(p.z, p.out_dtype, i * NB + j, z0);
    if (gated) store_out(p.z, p.out_dtype, i * NB + p.N + j, z1);
  }
  float y = gated ? silu_f(z0) * z1 : act_f(p.act, z0);
  if (p.residual) y += load_out(p.residual, p.out_dtype, i * p.N + j);
  store_out(p.y, p.out_dtype, i * p.N + j, y);
}

// ------------------------------------------------------------- tile kernel
// 128 lines of A by 128 lines of B a workgroup, 64 along k a turn; 4 waves of
// 64 x 64. Each turn the threads decode the operands' next slabs into LDS as
// binary16 and the waves read them as matrix fragments.
constexpr int BM = 128, BN = 128, BK = 64, LDT = BK + 8;

// 32 elements of a line from k on (k a multiple of 32): the bytes that lie in
// the line, zeros past it.
__device__ __forceinline__ void load_bytes(const uint8_t* p, int64_t have, uint32_t (&w)[4]) {
  if (have >= 16) {
    const u32x4 v = *reinterpret_cast<const u32x4_a1*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < have) w[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
  }
}
template <bool FP8>
__device__ __forceinline__ void load_slab(const GemmOperand& o, int64_t line, int64_t k, int64_t K,
                                          _Float16* dst) {
  if constexpr (FP8) {
    uint32_t w0[4], w1[4];
    load_bytes(o.q + line * K + k, K - k, w0);
    load_bytes(o.q + line * K + k + 16, K - k - 16, w1);
    h8* d = reinterpret_cast<h8*>(dst);
    d[0] = decode8_fp8(w0[0], w0[1]);
    d[1] = decode8_fp8(w0[2], w0[3]);
    d[2] = decode8_fp8(w1[0], w1[1]);
    d[3] = decode8_fp8(w1[2], w1[3]);
  } else {
    const int64_t qp = (K + 1) / 2, sp = (K + 15) / 16;
    uint32_t w[4];
    load_bytes(o.q + line * qp + k / 2, qp - k / 2, w);
    // a line of odd length: its last high nibble is no element
    const int64_t n = K - k;
    if (n < 32 && n > 0 && (n & 1)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((n >> 3) == i) w[i] &= (1u << (4 * (n & 7))) - 1u;
    }
    const uint32_t s0 = k < K ? o.s[line * sp + k / 16] : 0u;
    const uint32_t s1 = k + 16 < K ? o.s[line * sp + k / 16 + 1] : 0u;
    const h2 s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s0 | (s1 << 8), 1.0f, false);
    h8* d = reinterpret_cast<h8*>(dst);
    d[0] = decode8_fp4(w[0], s.xx);
    d[1] = decode8_fp4(w[1], s.xx);
    d[2] = decode8_fp4(w[2], s.yy);
    d[3] = decode8_fp4(w[3], s.yy);
  }
}

template <bool A8, bool GATED>
__global__ void __launch_bounds__(256) gemm_tile_kernel(const GemmArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  __shared__ _Float16 sa[BM * LDT], sb[BN * LDT];
  constexpr int OUT = GATED ? BN / 2 : BN;  // output columns of a tile
  const int64_t i0 = (int64_t)blockIdx.y * BM, j0 = (int64_t)blockIdx.x * OUT;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1, l32 = lane & 31, g = lane >> 5;
  // the line of B behind row r of the tile; gated: every 64 rows hold 32 gate
  // lines, then the up lines of the same outputs
  auto b_line = [&](int r) -> int64_t {
    if constexpr (GATED) {
      const int64_t j = j0 + (r >> 6) * 32 + (r & 31);
      return min(j, p.N - 1) + ((r & 32) ? p.N : 0);
    }
    return min(j0 + r, p.N - 1);
  };
  const int lr = tid >> 1, lk = 32 * (tid & 1);
  const int64_t la = min(i0 + lr, p.M - 1), lb = b_line(lr);
  f32x16 acc[2][2] = {};
  for (int64_t k = 0; k < p.K; k += BK) {
    load_slab<A8>(p.a, la, k + lk, p.K, sa + lr * LDT + lk);
    load_slab<false>(p.b, lb, k + lk, p.K, sb + lr * LDT + lk);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BK; kk += 16) {
      h8 fa[2], fb[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        fa[t] = *reinterpret_cast<const h8*>(sa + (wm * 64 + t * 32 + l32) * LDT + kk + 8 * g);
        fb[t] = *reinterpret_cast<const h8*>(sb + (wn * 64 + t * 32 + l32) * LDT + kk + 8 * g);
      }
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int ni = 0; ni < 2; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[ni], fa[mi], acc[mi][ni], 0, 0, 0);
    }
    __syncthreads();
  }
  // register r of a 32 x 32 result: line l32 of A, line 8 (r / 4) + 4 g + r % 4 of B
#pragma unroll
  for (int mi = 0; mi < 2; ++mi) {
    const int64_t i = i0 + wm * 64 + mi * 32 + l32;
    if (i >= p.M) continue;
    const LineScale x = line_scale(p.a, i);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int n = 8 * (r >> 2) + 4 * g + (r & 3);
      if constexpr (GATED) {
        const int64_t j = j0 + wn * 32 + n;
        if (j < p.N) {
          const float z0 = apply_scale(acc[mi][0][r], x, line_scale(p.b, j)) + load_bias(p, j);
          const float z1 =
              apply_scale(acc[mi][1][r], x, line_scale(p.b, p.N + j)) + load_bias(p, p.N + j);
          finish1(p, i, j, z0, z1);
        }
      } else {
#pragma unroll
        for (int ni = 0; ni < 2; ++ni) {
          const int64_t j = j0 + wn * 64 + ni * 32 + n;
          if (j < p.N)
            finish1(p, i, j, apply_scale(acc[mi][ni][r], x, line_scale(p.b, j)) + load_bias(p, j),
                    0.0f);
        }
      }
    }
  }
}

int64_t gemm_workspace(int a_fmt, int64_t M, int64_t N, int64_t K, int act) { return 0; }

int launch_gemm(const GemmArgs& a, hipStream_t s) {
  const bool gated = a.act == ACT_SWIGLU;
  const int out = gated ? BN / 2 : BN;
  const dim3 grid((unsigned)((a.N + out - 1) / out), (unsigned)((a.M + BM - 1) / BM)), b(256);
  const bool a8 = a.a.s == nullptr;
  if (a8 && gated) hipLaunchKernelGGL((gemm_tile_kernel<true, true>), grid, b, 0, s, a);
  else if (a8) hipLaunchKernelGGL((gemm_tile_kernel<true, false>), grid, b, 0, s, a);
  else if (gated) hipLaunchKernelGGL((gemm_tile_kernel<false, true>), grid, b, 0, s, a);
  else hipLaunchKernelGGL((gemm_tile_kernel<false, false>), grid, b, 0, s, a);
  return hipGetLastError() == hipSuccess ? 0 : -3;
}

}  // namespace nvfp4
