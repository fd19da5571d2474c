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
// 8 consecutive outputs of line i from column j on, nj of them (8 or more:
// all) in the matrix. z0: pre-activations (the gate's, if gated), z1: the up
// lines'; both with their bias.
template <typename T, bool GATED>
__device__ __forceinline__ void finish8_t(const GemmArgs& p, int64_t i, int64_t j, int64_t nj,
                                          const float (&z0)[8], const float (&z1)[8]) {
  if (p.z) {
    T* z = static_cast<T*>(p.z) + i * (GATED ? 2 * p.N : p.N) + j;
    store8(z, nj, z0);
    if constexpr (GATED) store8(z + p.N, nj, z1);
  }
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if constexpr (GATED) y[k] = silu_f(z0[k]) * z1[k];
    else y[k] = act_f(p.act, z0[k]);
  }
  if (p.residual) {
    float r[8];
    load8(static_cast<const T*>(p.residual) + i * p.N + j, nj, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] += r[k];
  }
  store8(static_cast<T*>(p.y) + i * p.N + j, nj, y);
}
template <bool GATED>
__device__ __forceinline__ void finish8(const GemmArgs& p, int64_t i, int64_t j, int64_t nj,
                                        const float (&z0)[8], const float (&z1)[8]) {
  if (p.out_dtype == 0) finish8_t<uint16_t, GATED>(p, i, j, nj, z0, z1);
  else finish8_t<float, GATED>(p, i, j, nj, z0, z1);
}

// 16 bytes of a packed line from byte `off` on; bytes past the line's end read
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

// ------------------------------------------------------------- tile kernel
// 256 lines of A by 256 lines of B a workgroup of 4 waves, 128 x 128 a wave
// (its FP32 sums take 256 of the 512 registers a lane has at one wave a SIMD).
// A stage is 128 along k. Its codes go to LDS as they are, 64 bytes a line
// (128 for E4M3), and its block scales, 8 bytes a line; every wave decodes its own
// fragments in registers: a 16-byte read holds 32 codes, four matrix
// instructions' worth of k, so LDS moves a quarter of the bytes that binary16
// tiles would, and the decode (one convert and one multiply for two elements)
// runs beside the matrix pipe.
constexpr int TM = 256, TN = 256, TK = 128;

// LDS of a stage: B codes, A codes, B scales, A scales.
template <bool A8>
struct Stage {
  static constexpr int ALINE = A8 ? 128 : 64;
  static constexpr int B0 = 0, A0 = TN * 64, SB0 = A0 + TM * ALINE, SA0 = SB0 + TN * 8;
  static constexpr int BYTES = SA0 + (A8 ? 0 : TM * 8);
};
// Position of 16-byte chunk c of a line within its row of LDS: rotated by the
// row so that the lanes of a read, one row each, spread over the banks.
__device__ __forceinline__ int swz4(int row, int c) { return c ^ ((row >> 1) & 3); }
__device__ __forceinline__ int swz8(int row, int c) { return c ^ (row & 7); }

template <bool A8>
struct RawUnit {  // one lane's codes of 64 k: 32 k of each of its lines
  u32x4 b[4], a[4][A8 ? 2 : 1];
  uint32_t sb[4], sa[4];
};

template <bool A8, bool GATED>
__global__ void __launch_bounds__(256, 1) gemm_tile_kernel(const GemmArgs p, int gm, int gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  using S = Stage<A8>;
  constexpr int EPI = 4 * 32 * 132 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * S::BYTES > EPI ? 2 * S::BYTES : EPI];
  constexpr int OUT = GATED ? TN / 2 : TN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1, l32 = lane & 31, g = lane >> 5;
  // Workgroups go round the 8 XCDs; each XCD takes a run of tiles so that its
  // L2 serves neighbours: runs walk columns of 8 row tiles.
  const int total = gm * gn;
  int t = blockIdx.x;
  {
    const int per = total / 8, rem = total % 8, x = t % 8, i = t / 8;
    t = x * per + min(x, rem) + i;
  }
  const int band = t / (8 * gn), hb = min(8, gm - band * 8), tb = t - band * 8 * gn;
  const int64_t i0 = (int64_t)(band * 8 + tb % hb) * TM, j0 = (int64_t)(tb / hb) * OUT;

  const int K = (int)p.K, qp = (K + 1) / 2, sp = (K + 15) / 16, ap = A8 ? K : qp;
  // the line of B behind row r of the tile; gated: every 128 rows hold 64 gate
  // lines, then the up lines of the same outputs
  auto b_line = [&](int r) -> int64_t {
    if constexpr (GATED) {
      const int64_t j = j0 + (r >> 7) * 64 + (r & 63);
      return min(j, p.N - 1) + ((r & 64) ? p.N : 0);
    } else {
      return min(j0 + r, p.N - 1);
    }
  };
  auto a_line = [&](int r) -> int64_t { return min(i0 + r, p.M - 1); };

  // what this thread fetches of a stage: 16-byte chunk `bc` of 4 lines of B,
  // chunk `ac` of 4 (8) lines of A, 8 scale bytes of one line of each
  constexpr int NA = A8 ? 8 : 4;
  const uint8_t *bp[4], *apt[NA];
  int bc[4], ac[NA];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 64 + tid / 4;
    bp[i] = p.b.q + b_line(r) * qp;
    bc[i] = swz4(r, tid & 3);
  }
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int r = A8 ? i * 32 + tid / 8 : i * 64 + tid / 4;
    apt[i] = p.a.q + a_line(r) * ap;
    ac[i] = A8 ? swz8(r, tid & 7) : swz4(r, tid & 3);
  }
  const uint8_t* sbp = p.b.s + b_line(tid) * sp;
  const uint8_t* sap = A8 ? nullptr : p.a.s + a_line(tid) * sp;

  u32x4 rb[4], ra[NA];
  u32x2 rsb, rsa;
  auto fetch = [&](int k) {
    if (k + TK <= K) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rb[i] = *reinterpret_cast<const u32x4_a1*>(bp[i] + k / 2 + 16 * bc[i]);
#pragma unroll
      for (int i = 0; i < NA; ++i)
        ra[i] = *reinterpret_cast<const u32x4_a1*>(apt[i] + (A8 ? k : k / 2) + 16 * ac[i]);
      rsb = *reinterpret_cast<const u32x2_a1*>(sbp + k / 16);
      if constexpr (!A8) rsa = *reinterpret_cast<const u32x2_a1*>(sap + k / 16);
    } else {  // the last stage of a line that ends inside it
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int d = 0; d < 4; ++d)
          rb[i][d] = keep_nibbles(tail_dword(bp[i], qp, k / 2 + 16 * bc[i] + 4 * d),
                                  K - k - 32 * bc[i] - 8 * d);
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          if constexpr (A8)
            ra[i][d] = keep_bytes(tail_dword(apt[i], ap, k + 16 * ac[i] + 4 * d),
                                  K - k - 16 * ac[i] - 4 * d);
          else
            ra[i][d] = keep_nibbles(tail_dword(apt[i], ap, k / 2 + 16 * ac[i] + 4 * d),
                                    K - k - 32 * ac[i] - 8 * d);
        }
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        rsb[d] = keep_bytes(tail_dword(sbp, sp, k / 16 + 4 * d), sp - k / 16 - 4 * d);
        if constexpr (!A8)
          rsa[d] = keep_bytes(tail_dword(sap, sp, k / 16 + 4 * d), sp - k / 16 - 4 * d);
      }
    }
  };
  auto put = [&](int buf) {
    uint8_t* l = lds + buf * S::BYTES;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<u32x4*>(l + S::B0 + i * 4096 + tid * 16) = rb[i];
#pragma unroll
    for (int i = 0; i < NA; ++i)
      *reinterpret_cast<u32x4*>(l + S::A0 + i * 4096 + tid * 16) = ra[i];
    *reinterpret_cast<u32x2*>(l + S::SB0 + tid * 8) = rsb;
    if constexpr (!A8) *reinterpret_cast<u32x2*>(l + S::SA0 + tid * 8) = rsa;
  };
  // unit u of a stage: chunk 2 u + g of every line, 32 k of it a lane
  auto get = [&](int buf, int u, RawUnit<A8>& r) {
    const uint8_t* l = lds + buf * S::BYTES;
    const int c = 2 * u + g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int br = wn * 128 + i * 32 + l32, ar = wm * 128 + i * 32 + l32;
      r.b[i] = *reinterpret_cast<const u32x4*>(l + S::B0 + br * 64 + 16 * swz4(br, c));
      r.sb[i] = *reinterpret_cast<const uint16_t*>(l + S::SB0 + br * 8 + 2 * c);
      if constexpr (A8) {
        r.a[i][0] = *reinterpret_cast<const u32x4*>(l + S::A0 + ar * 128 + 16 * swz8(ar, 2 * c));
        r.a[i][1] = *reinterpret_cast<const u32x4*>(l + S::A0 + ar * 128 + 16 * swz8(ar, 2 * c + 1));
      } else {
        r.a[i][0] = *reinterpret_cast<const u32x4*>(l + S::A0 + ar * 64 + 16 * swz4(ar, c));
        r.sa[i] = *reinterpret_cast<const uint16_t*>(l + S::SA0 + ar * 8 + 2 * c);
      }
    }
  };

  f32x16 acc[4][4] = {};
  h8 fb[2][4], fa[2][4];
  // fragments of k-slice d (0..3) of a unit
  auto decode = [&](const RawUnit<A8>& r, int d, h8 (&ob)[4], h8 (&oa)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const h2 sb = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.sb[i], 1.0f, false);
      ob[i] = decode8_fp4(r.b[i][d], d < 2 ? sb.xx : sb.yy);
      if constexpr (A8) {
        oa[i] = decode8_fp8(r.a[i][d >> 1][(2 * d) & 3], r.a[i][d >> 1][(2 * d + 1) & 3]);
      } else {
        const h2 sa = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.sa[i], 1.0f, false);
        oa[i] = decode8_fp4(r.a[i][0][d], d < 2 ? sa.xx : sa.yy);
      }
    }
  };
  auto multiply = [&](const h8 (&b)[4], const h8 (&a)[4]) {
#pragma unroll
    for (int mi = 0; mi < 4; ++mi)
#pragma unroll
      for (int ni = 0; ni < 4; ++ni)
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b[ni], a[mi], acc[mi][ni], 0, 0, 0);
  };

  const int ns = (K + TK - 1) / TK;
  RawUnit<A8> r0, r1;
  fetch(0);
  put(0);
  if (ns > 1) fetch(TK);
  __syncthreads();
  get(0, 0, r0);
  decode(r0, 0, fb[0], fa[0]);
  for (int s = 0; s < ns; ++s) {
    const int buf = s & 1;
    // unit 0: the other buffer's last readers passed the previous barrier
    get(buf, 1, r1);
    if (s + 1 < ns) put(buf ^ 1);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (d < 3) decode(r0, d + 1, fb[(d + 1) & 1], fa[(d + 1) & 1]);
      else decode(r1, 0, fb[0], fa[0]);
      multiply(fb[d & 1], fa[d & 1]);
    }
    __syncthreads();
    // unit 1
    if (s + 1 < ns) get(buf ^ 1, 0, r0);
    if (s + 2 < ns) fetch((s + 2) * TK);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (d < 3) decode(r1, d + 1, fb[(d + 1) & 1], fa[(d + 1) & 1]);
      else decode(r0, 0, fb[0], fa[0]);
      multiply(fb[d & 1], fa[d & 1]);
    }
  }
  __syncthreads();  // the last stage's readers are done: LDS becomes the epilogue's

  // Epilogue, 32 lines of A at a time through LDS, so that a lane ends up with
  // 8 consecutive outputs of one line. Register r of a 32 x 32 result: line
  // l32 of A, line 8 (r / 4) + 4 g + r % 4 of B.
  float* sc = reinterpret_cast<float*>(lds) + wave * 32 * 132;
  constexpr int LPR = GATED ? 8 : 16;  // lanes to a line
  const int cl = 8 * (lane % LPR);
  const int64_t j = j0 + wn * (GATED ? 64 : 128) + cl, nj = p.N - j;
  LineScale w0[8], w1[8];
  float b0[8], b1[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t jj = min(j + k, p.N - 1);
    w0[k] = line_scale(p.b, jj);
    b0[k] = load_bias(p, jj);
    if constexpr (GATED) {
      w1[k] = line_scale(p.b, p.N + jj);
      b1[k] = load_bias(p, p.N + jj);
    }
  }
#pragma unroll
  for (int mi = 0; mi < 4; ++mi) {
#pragma unroll
    for (int ni = 0; ni < 4; ++ni)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16& c = acc[mi][ni];
        *reinterpret_cast<float4*>(sc + l32 * 132 + ni * 32 + 8 * q + 4 * g) =
            make_float4(c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]);
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int r = lane / LPR; r < 32; r += 64 / LPR) {
      const int64_t i = i0 + wm * 128 + mi * 32 + r;
      if (i < p.M && nj > 0) {
        const LineScale x = line_scale(p.a, i);
        float z0[8], z1[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          z0[k] = apply_scale(sc[r * 132 + cl + k], x, w0[k]) + b0[k];
          if constexpr (GATED) z1[k] = apply_scale(sc[r * 132 + 64 + cl + k], x, w1[k]) + b1[k];
        }
        finish8<GATED>(p, i, j, nj, z0, z1);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

int64_t gemm_workspace(int a_fmt, int64_t M, int64_t N, int64_t K, int act) {
  const int64_t gm = (M + TM - 1) / TM, gn = (N + TN / 2 - 1) / (TN / 2);
  if (K > ((int64_t)1 << 28) || gm * gn > ((int64_t)1 << 23)) return -1;
  return 0;
}

int launch_gemm(const GemmArgs& a, hipStream_t s) {
  const bool gated = a.act == ACT_SWIGLU;
  const int out = gated ? TN / 2 : TN;
  const int gm = (int)((a.M + TM - 1) / TM), gn = (int)((a.N + out - 1) / out);
  const dim3 grid((unsigned)(gm * gn)), b(256);
  const bool a8 = a.a.s == nullptr;
  if (a8 && gated) hipLaunchKernelGGL((gemm_tile_kernel<true, true>), grid, b, 0, s, a, gm, gn);
  else if (a8) hipLaunchKernelGGL((gemm_tile_kernel<true, false>), grid, b, 0, s, a, gm, gn);
  else if (gated) hipLaunchKernelGGL((gemm_tile_kernel<false, true>), grid, b, 0, s, a, gm, gn);
  else hipLaunchKernelGGL((gemm_tile_kernel<false, false>), grid, b, 0, s, a, gm, gn);
  return hipGetLastError() == hipSuccess ? 0 : -3;
}

}  // namespace nvfp4
