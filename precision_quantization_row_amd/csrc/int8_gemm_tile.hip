// int8_gemm_tile.hip -- the product of 8-bit integer lines for many lines of A
// (gfx950).
#include "gemm_device.h"

namespace nvfp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// 256 lines of A by 256 lines of B a workgroup of 4 waves, 128 x 128 a wave: its
// sums take 256 of the lane's 512 registers. A stage is 128 bytes along k of all
// 512 lines, 64 KB of LDS; two of them take turns.
constexpr int TM = 256, TN = 256, TK = 128;
constexpr int SIDE = TM * TK, STAGE = 2 * SIDE;
// 16-byte slot s of line r, rotated by the line so that 16 lanes that read one
// slot of 16 neighbouring lines touch all 64 banks once (a line is half of them).
__device__ __forceinline__ int rotate(int r) {
  return ((r >> 1) & 1) << 2 | ((r ^ (r >> 3)) & 1) << 1 | ((r >> 2) & 1);
}

// 16 bytes a lane from base + off straight into LDS, at m0 + 16 lane; the caller
// waits for vmcnt. (M0 is the compiler's, which has no use for it in these
// kernels; the compiler's own form of this load makes every later LDS read wait.)
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t off, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(m0)
               : "memory");
}

template <bool DIRECT, bool GATED>
__global__ void __launch_bounds__(256, 1) int8_tile_kernel(const GemmArgs p, int gm, int gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE];
  constexpr int OUT = GATED ? TN / 2 : TN;
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave & 1, wn = wave >> 1;
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

  const int K = (int)p.K;
  const int am = (int)min(p.M - i0, (int64_t)TM) - 1, bm = (int)min(p.N - j0, (int64_t)OUT) - 1;
  const uint8_t *qa = p.a.q + i0 * K, *qb = p.b.q + j0 * K;
  // This thread moves chunk c (16 bytes) of lines wave * 64 + 8 i + lane / 8 of each
  // side. DIRECT: the lane's place in LDS is its own, so the chunk is rotated.
  // Lines past the matrix repeat its last one (their products are not stored).
  // Gated: a wave's 128 lines of B are 64 gate lines and their up lines.
  uint32_t aoff[8], boff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = wave * 64 + 8 * i + lane / 8, c = DIRECT ? (lane % 8) ^ rotate(r) : lane % 8;
    aoff[i] = (uint32_t)min(r, am) * K + 16 * c;
    boff[i] = (uint32_t)min(GATED ? (r / 128) * 64 + r % 64 : r, bm) * K + 16 * c;
  }
  // (gated: a wave moves gate lines or up lines)
  const uint8_t* qu = GATED && (wave & 1) ? qb + p.N * K : qb;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  u32x4 ra[DIRECT ? 1 : 8], rb[DIRECT ? 1 : 8];
  // the whole stage at k, which lies inside the lines, on its way to `buf`
  auto fetch = [&](int k, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (DIRECT) {
        const uint32_t at = lds0 + buf * STAGE + wave * 8192 + i * 1024;
        load_to_lds(qa + k, aoff[i], at);
        load_to_lds(qu + k, boff[i], at + SIDE);
      } else {
        ra[DIRECT ? 0 : i] = *reinterpret_cast<const u32x4_a1*>(qa + k + aoff[i]);
        rb[DIRECT ? 0 : i] = *reinterpret_cast<const u32x4_a1*>(qu + k + boff[i]);
      }
    }
  };
  auto put = [&](int buf) __attribute__((always_inline)) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = wave * 64 + 8 * i + lane / 8;
        uint8_t* d = lds + buf * STAGE + r * TK + 16 * ((lane % 8) ^ rotate(r));
        *reinterpret_cast<u32x4*>(d) = ra[DIRECT ? 0 : i];
        *reinterpret_cast<u32x4*>(d + SIDE) = rb[DIRECT ? 0 : i];
      }
    }
  };
  // a stage that reaches past the lines' end: zeros there
  auto tail = [&](int k, int buf) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const int r = wave * 64 + 8 * (i & 7) + lane / 8, c = lane % 8;
      const uint8_t* line = i < 8 ? qa + (uint32_t)min(r, am) * K
                                  : qu + (uint32_t)min(GATED ? (r / 128) * 64 + r % 64 : r, bm) * K;
      u32x4 w;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int at = k + 16 * c + 4 * d;
        w[d] = keep_bytes(tail_dword(line, K, at), K - at);
      }
      *reinterpret_cast<u32x4*>(lds + buf * STAGE + (i < 8 ? 0 : SIDE) + r * TK + 16 * (c ^ rotate(r))) = w;
    }
  };

  i32x16 acc[4][4] = {};
  auto frag = [&](int buf, int side, int line, int s) __attribute__((always_inline)) {
    return *reinterpret_cast<const i32x4*>(lds + buf * STAGE + side * SIDE + line * TK + 16 * (s ^ rotate(l32)));
  };
  auto compute = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      i32x4 fa[4], fb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fa[i] = frag(buf, 0, wm * 128 + 32 * i + l32, 2 * d + g);
        fb[i] = frag(buf, 1, wn * 128 + 32 * i + l32, 2 * d + g);
      }
#pragma unroll
      for (int mi = 0; mi < 4; ++mi)
#pragma unroll
        for (int ni = 0; ni < 4; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[ni], fa[mi], acc[mi][ni], 0, 0, 0);
    }
  };
  auto arrive = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0);  // (the loads into LDS are not the compiler's)
    __syncthreads();
  };
  const int nu = (K + TK - 1) / TK;
  auto begin = [&](int u) __attribute__((always_inline)) {
    if ((u + 1) * TK <= K) fetch(u * TK, u & 1);
    else tail(u * TK, u & 1);
  };
  begin(0);
  if (TK <= K) put(0);
  arrive();
#pragma unroll 1
  for (int u = 0; u < nu; ++u) {
    if (u + 1 < nu) begin(u + 1);
    compute(u & 1);
    if ((u + 2) * TK <= K) put((u + 1) & 1);
    arrive();
  }

  // Epilogue, 32 lines of A at a time through LDS, so that a lane ends up with
  // 8 consecutive outputs of a line. Register r of a 32 x 32 result: line l32
  // of A, line 8 (r / 4) + 4 g + r % 4 of B.
  constexpr int PITCH = 132;  // floats: 128 sums, the line's scale, bank padding
  float* ep = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
  constexpr int LPR = GATED ? 8 : 16, RPL = 64 / LPR;  // lanes to a line, lines to a wave's access
  constexpr int NL = 4;                                // of these at a time
  const int cl = 8 * (lane % LPR);
  const int64_t j = j0 + wn * (GATED ? 64 : 128) + cl, nj = p.N - j;
  LineScale w0[8], w1[8];
  float b0[8], b1[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int64_t jj = min(j + q, p.N - 1);
    w0[q] = line_scale(p.b, jj);
    b0[q] = load_bias(p, jj);
    if constexpr (GATED) {
      w1[q] = line_scale(p.b, p.N + jj);
      b1[q] = load_bias(p, p.N + jj);
    }
  }
  LineScale x[4];
#pragma unroll
  for (int mi = 0; mi < 4; ++mi) x[mi] = line_scale(p.a, min(i0 + wm * 128 + mi * 32 + l32, p.M - 1));
  auto finish = [&](auto type_) __attribute__((always_inline)) {
    using T = decltype(type_);
    static_for<4>([&](auto m_) __attribute__((always_inline)) {
      constexpr int m = decltype(m_)::value;
      float* e = ep + l32 * PITCH;
#pragma unroll
      for (int ni = 0; ni < 4; ++ni)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const i32x16& v = acc[m][ni];
          *reinterpret_cast<float4*>(e + ni * 32 + 8 * q + 4 * g) =
              make_float4((float)v[4 * q], (float)v[4 * q + 1], (float)v[4 * q + 2], (float)v[4 * q + 3]);
        }
      if (g == 0) *reinterpret_cast<float2*>(e + 128) = make_float2(x[m].m, __int_as_float(x[m].e));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll 1
      for (int h = 0; h < 32; h += NL * RPL) {
        const int64_t i = i0 + wm * 128 + m * 32 + h + lane / LPR;
        Raw8<T> res[NL];
        load_residual<T, NL, RPL>(p, i, j, nj, res);
        float z0[NL][8], z1[NL][8];
#pragma unroll
        for (int v = 0; v < NL; ++v) {
          const float* row = ep + (h + lane / LPR + v * RPL) * PITCH;
          const float2 xs = *reinterpret_cast<const float2*>(row + 128);
          const LineScale xr = {xs.x, __float_as_int(xs.y)};
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            z0[v][q] = apply_scale(row[cl + q], xr, w0[q]) + b0[q];
            if constexpr (GATED) z1[v][q] = apply_scale(row[64 + cl + q], xr, w1[q]) + b1[q];
          }
        }
        finish_lines<T, GATED, NL, RPL>(p, i, j, nj, z0, z1, res);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    });
  };
  if (p.out_dtype == 0) finish(uint16_t{});
  else finish(float{});
}

template <bool DIRECT, bool GATED>
static void go_tile(const GemmArgs& a, hipStream_t s) {
  constexpr int out = GATED ? TN / 2 : TN;
  const int gm = (int)((a.M + TM - 1) / TM), gn = (int)((a.N + out - 1) / out);
  hipLaunchKernelGGL((int8_tile_kernel<DIRECT, GATED>), dim3((unsigned)(gm * gn)), dim3(256), 0, s, a, gm, gn);
}

void launch_int8_tile(const GemmArgs& a, hipStream_t s) {
  const bool gated = a.act == ACT_SWIGLU;
  const bool direct = a.K % 16 == 0 &&
                      ((reinterpret_cast<uintptr_t>(a.a.q) | reinterpret_cast<uintptr_t>(a.b.q)) & 15) == 0;
  if (direct && gated) go_tile<true, true>(a, s);
  else if (direct) go_tile<true, false>(a, s);
  else if (gated) go_tile<false, true>(a, s);
  else go_tile<false, false>(a, s);
}

}  // namespace nvfp4
