// gemm_tile.hip -- the packed product for many lines of A (gfx950).
#include "gemm_device.h"

namespace nvfp4 {

// ------------------------------------------------------------- tile kernel
// 256 lines of A by 256 lines of B a workgroup of 4 waves, one wave a SIMD,
// 256 x 64 a wave: its FP32 sums take 256 of the lane's 512 registers.
//
// Every code is decoded once a workgroup. B's lines belong to one wave each,
// which decodes them straight from the registers they are loaded into; A's
// lines are shared, so each wave decodes a quarter of them into LDS as
// binary16 and reads all of them as matrix fragments. A stage is 64 along k,
// 64 matrix instructions of 32 cycles a wave. Beside each of them go about two
// vector instructions of decode (a convert and a multiply for two elements),
// half an LDS read and an eighth of an LDS write; they are placed one by one,
// because the compiler's own order left the matrix pipe idle a third of the
// time. LDS decides the shape: it reads 16 bytes a lane at 230 bytes a cycle
// but writes at 75, so 128 x 128 a wave with both operands in LDS spent 850 +
// 560 of a stage's 2048 cycles there; this shape spends 430 + 560.
//
// Bound by the matrix pipe and, with real data, by power: 8192 x 8192 x 28672
// takes 2790-2970 us, by card and codes (1.30-1.38 PFLOP/s; a library product of
// dense bf16 matrices 2617), and 2111 on zeros; 8192^3 842-874 us, the pipe busy
// 73 % of the cycles. Around its products a round of tiles spends 20 us (4096 x
// 2816 x 256: 21-24 us, 13 of them the stores of 46 MB).
//
// k order. Stage u is the chunks 2 u and 2 u + 1 of 32 k; slice d of it takes
// codes 8 d .. 8 d + 7 of both, the two halves of the wave one chunk each. Both
// operands alike, so the sum covers every k once.
constexpr int TM = 256, TN = 256, TK = 64;
constexpr int STAGE_BYTES = TM * 128;  // 64 binary16 a line
// 16-byte slot s of line r, rotated by the line so that 16 lanes that read one
// slot of 16 neighbouring lines touch all 64 banks once (a line is half of
// them), and 8 lanes that write 2 neighbouring slots of 4 lines touch 8
// different ones.
__device__ __forceinline__ int slot(int r, int s) {
  return r * 128 + 16 * (s ^ (((r >> 1) & 1) << 2 | ((r ^ (r >> 3)) & 1) << 1 | ((r >> 2) & 1)));
}

template <bool A8, bool GATED>
__global__ void __launch_bounds__(256, 1) gemm_tile_kernel(const GemmArgs p, int gm, int gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int EPI_BYTES = 4 * 2 * 32 * 68 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE_BYTES > EPI_BYTES ? 2 * STAGE_BYTES : EPI_BYTES];
  constexpr int OUT = GATED ? TN / 2 : TN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l32 = lane & 31, g = lane >> 5;
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
  // Lines past the matrix repeat its last one (their products are not stored);
  // offsets are from the tile's first line, which 32 bits hold.
  // A: this thread decodes lines tid / 2 + 128 i, chunk tid % 2 of a stage.
  // B: this lane holds lines wave * 64 + 32 i + l32 (gated: the gate line and
  // the up line of output wave * 32 + l32), chunk g of a stage.
  const int am = (int)min(p.M - i0, (int64_t)TM) - 1, bm = (int)min(p.N - j0, (int64_t)OUT) - 1;
  const int ga = tid & 1;
  uint32_t aoff[2], asoff[2], boff[2], bsoff[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int la = min((tid >> 1) + 128 * i, am);
    const int lb = min(GATED ? wave * 32 + l32 : wave * 64 + 32 * i + l32, bm);
    aoff[i] = (uint32_t)la * ap + (A8 ? 32 : 16) * ga;
    asoff[i] = (uint32_t)la * sp;
    boff[i] = (uint32_t)lb * qp + 16 * g;
    bsoff[i] = (uint32_t)lb * sp;
  }
  const uint8_t *qa = p.a.q + i0 * ap, *sa = A8 ? nullptr : p.a.s + i0 * sp;
  const uint8_t *qb = p.b.q + j0 * qp, *sb = p.b.s + j0 * sp;
  const uint8_t *qu = GATED ? qb + p.N * qp : qb, *su = GATED ? sb + p.N * sp : sb;

  // Codes on their way, a set for each of SETS stages: a line of L2 that has to
  // come from HBM takes longer than one stage.
  constexpr int SETS = 4;
  u32x4 ra[SETS][2] = {}, ra8[A8 ? SETS : 1][2] = {}, rb[SETS][2] = {};  // ra8: the second half of an E4M3 chunk
  // Block scales, 16 bytes of a line for the SETS stages of a quad: this quad's
  // and the next one's. (2 bytes a stage cost as much of the memory pipe, whose
  // rate is lines of memory touched, as the codes' 16.)
  u32x4 csa[2] = {}, csb[2] = {}, nsa[2] = {}, nsb[2] = {};
  // set S, line i of the stage at k, which lies inside the line
  auto fetch_a = [&](auto set_, auto line_, int k) {
    constexpr int S = decltype(set_)::value, i = decltype(line_)::value;
    // (the empty asm keeps the offset a 32-bit one added by the load itself)
    uint32_t o = aoff[i];
    asm volatile("" : "+v"(o));
    const uint8_t* q = qa + (A8 ? k : k / 2);
    ra[S][i] = *reinterpret_cast<const u32x4_a1*>(q + o);
    if constexpr (A8) ra8[S][i] = *reinterpret_cast<const u32x4_a1*>(q + 16 + o);
  };
  auto fetch_b = [&](auto set_, auto line_, int k) {
    constexpr int S = decltype(set_)::value, i = decltype(line_)::value;
    uint32_t o = boff[i];
    asm volatile("" : "+v"(o));
    rb[S][i] = *reinterpret_cast<const u32x4_a1*>((i ? qu : qb) + k / 2 + o);
  };
  // the scales of the quad at k (a multiple of SETS TK): line i of A, i - 2 of B
  auto fetch_s = [&](auto line_, int k) {
    constexpr int i = decltype(line_)::value & 1;
    constexpr bool b = decltype(line_)::value >= 2;
    if constexpr (A8 && !b) return;
    uint32_t o = b ? bsoff[i] : asoff[i];
    asm volatile("" : "+v"(o));
    const u32x4 v = *reinterpret_cast<const u32x4_a1*>((b ? (i ? su : sb) : sa) + k / 16 + o);
    if constexpr (b) nsb[i] = v;
    else nsa[i] = v;
  };
  auto load_s = [&](int k) {
    if (k + 4 * TK <= K) {
      static_for<4>([&](auto i) { fetch_s(i, k); });
    } else if (k < K) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int at = k / 16 + 4 * d;
          if constexpr (!A8) nsa[i][d] = keep_bytes(tail_dword(sa + asoff[i], sp, at), sp - at);
          nsb[i][d] = keep_bytes(tail_dword((i ? su : sb) + bsoff[i], sp, at), sp - at);
        }
    }
  };
  // the same for a stage that reaches past the line's end, or lies past it:
  // zeros there
  auto tail_a = [&](auto set_, int k) {
    constexpr int S = decltype(set_)::value;
    const int kc = k + 32 * ga;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* q = qa + aoff[i] - (A8 ? 32 : 16) * ga;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if constexpr (A8) {
          ra[S][i][d] = keep_bytes(tail_dword(q, ap, kc + 4 * d), K - kc - 4 * d);
          ra8[S][i][d] = keep_bytes(tail_dword(q, ap, kc + 16 + 4 * d), K - kc - 16 - 4 * d);
        } else {
          ra[S][i][d] = keep_nibbles(tail_dword(q, qp, kc / 2 + 4 * d), K - kc - 8 * d);
        }
      }
    }
  };
  auto tail_b = [&](auto set_, int k) {
    constexpr int S = decltype(set_)::value;
    const int kc = k + 32 * g;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* q = (i ? qu : qb) + boff[i] - 16 * g;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        rb[S][i][d] = keep_nibbles(tail_dword(q, qp, kc / 2 + 4 * d), K - kc - 8 * d);
    }
  };

  // any stage; one past the end leaves the set as it is
  auto load_a = [&](auto set_, int k) {
    if (k + TK <= K) static_for<2>([&](auto i) { fetch_a(set_, i, k); });
    else if (k < K) tail_a(set_, k);
  };
  auto load_b = [&](auto set_, int k) {
    if (k + TK <= K) static_for<2>([&](auto i) { fetch_b(set_, i, k); });
    else if (k < K) tail_b(set_, k);
  };

  // Step Z of the decode of line I of A, set S, into its stage's buffer: 16 pairs, a
  // convert running one pair ahead of its multiply.
  constexpr int A_STEPS = A8 ? 16 : 33, B_STEPS = 9;
  h2 cva[2], ova[4], ascale;
  auto step_a = [&](auto set_, auto line_, auto step_) {
    constexpr int S = decltype(set_)::value, I = decltype(line_)::value, Z = decltype(step_)::value;
    constexpr int CV = A8 ? Z : Z == 1 ? 0 : Z >= 2 && Z < 32 && Z % 2 == 0 ? Z / 2 : -1;
    constexpr int MU = A8 ? Z : Z == 32 ? 15 : Z >= 3 && Z % 2 == 1 ? (Z - 3) / 2 : -1;
    if constexpr (!A8 && Z == 0)
      ascale = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((S ? csa[I][S] : nsa[I][0]) >> (16 * ga), 1.0f, false);
    if constexpr (CV >= 0) {
      if constexpr (A8)
        ova[CV & 3] = cvt_fp8<CV & 1>((CV < 8 ? ra[S][I] : ra8[A8 ? S : 0][I])[(CV >> 1) & 3]);
      else
        cva[CV & 1] = cvt_fp4<CV & 3>(ra[S][I][CV >> 2]);
    }
    if constexpr (MU >= 0) {
      if constexpr (!A8) ova[MU & 3] = cva[MU & 1] * (MU < 8 ? ascale.xx : ascale.yy);
      if constexpr ((MU & 3) == 3)
        *reinterpret_cast<h8*>(lds + (S & 1) * STAGE_BYTES +
                               slot((tid >> 1) + 128 * I, 2 * (MU >> 2) + ga)) =
            h8{ova[0].x, ova[0].y, ova[1].x, ova[1].y, ova[2].x, ova[2].y, ova[3].x, ova[3].y};
    }
  };
  // Step Z of the decode of slice D of line I of B, set S, into fragment `out`.
  h2 cvb[2], ovb[4], bscale[2];
  auto step_b = [&](auto set_, auto d_, auto line_, auto step_, h8& out) {
    constexpr int S = decltype(set_)::value, D = decltype(d_)::value, I = decltype(line_)::value,
                  Z = decltype(step_)::value;
    constexpr int CV = Z == 1 ? 0 : Z >= 2 && Z < 8 && Z % 2 == 0 ? Z / 2 : -1;
    constexpr int MU = Z == 8 ? 3 : Z >= 3 && Z % 2 == 1 ? (Z - 3) / 2 : -1;
    if constexpr (Z == 0 && D == 0)
      bscale[I] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((S ? csb[I][S] : nsb[I][0]) >> (16 * g), 1.0f, false);
    if constexpr (CV >= 0) cvb[CV & 1] = cvt_fp4<CV>(rb[S][I][D]);
    if constexpr (MU >= 0) {
      ovb[MU] = cvb[MU & 1] * (D < 2 ? bscale[I].xx : bscale[I].yy);
      if constexpr (MU == 3)
        out = h8{ovb[0].x, ovb[0].y, ovb[1].x, ovb[1].y, ovb[2].x, ovb[2].y, ovb[3].x, ovb[3].y};
    }
  };

  f32x16 acc[8][2] = {};
  h8 fa[2][8], fb[2][2];
  auto read_a = [&](int buf, int d, int mi) {
    return *reinterpret_cast<const h8*>(lds + buf * STAGE_BYTES + slot(mi * 32 + l32, 2 * d + g));
  };
  // Slice D of the stage at k, of set S, whose fragments are in fa, fb[D & 1]:
  // 16 matrix instructions, and beside them the next slice's fragments (D = 3:
  // those of the next stage) and, for D < 3, a third of the next stage's A. The
  // last slice holds the barrier between this stage's LDS traffic and the next's;
  // it stands a few matrix instructions in, when the writes before it are done.
  // FAST: the stages fetched in the last slice lie inside the lines.
  auto slice = [&](auto set_, auto d_, int k, auto fast_) {
    constexpr int S = decltype(set_)::value, D = decltype(d_)::value, BAR = 4, S1 = (S + 1) % SETS;
    constexpr int ND = (D + 1) & 3, NS = D == 3 ? S1 : S, CUR = D & 1, NXT = CUR ^ 1;
    static_for<16>([&](auto n_) {
      constexpr int n = decltype(n_)::value, mi = n / 2, ni = n % 2;
      acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[CUR][ni], fa[CUR][mi], acc[mi][ni], 0, 0, 0);
      if constexpr (D == 3 && n == BAR) __syncthreads();
      constexpr int rd = D == 3 ? n - BAR : n;
      if constexpr (rd >= 0 && rd < 8) fa[NXT][rd] = read_a(NS & 1, ND, rd);
      constexpr int B0 = n * 2 * B_STEPS / 16, B1 = (n + 1) * 2 * B_STEPS / 16;
      static_for<B1 - B0>([&](auto z_) {
        constexpr int z = B0 + decltype(z_)::value, I = z / B_STEPS;
        step_b(std::integral_constant<int, NS>{}, std::integral_constant<int, ND>{},
               std::integral_constant<int, I>{}, std::integral_constant<int, z - I * B_STEPS>{},
               fb[NXT][I]);
      });
      if constexpr (D < 3) {
        constexpr int T0 = 2 * A_STEPS * D / 3, T1 = 2 * A_STEPS * (D + 1) / 3;
        constexpr int A0 = T0 + n * (T1 - T0) / 16, A1 = T0 + (n + 1) * (T1 - T0) / 16;
        static_for<A1 - A0>([&](auto z_) {
          constexpr int z = A0 + decltype(z_)::value, I = z / A_STEPS;
          step_a(std::integral_constant<int, S1>{}, std::integral_constant<int, I>{},
                 std::integral_constant<int, z - I * A_STEPS>{});
        });
      } else if constexpr (decltype(fast_)::value) {
        if constexpr (n == 9 || n == 11)
          fetch_b(set_, std::integral_constant<int, n == 11>{}, k + SETS * TK);
        if constexpr (S == 0 && n >= 8 && n % 2 == 0)
          fetch_s(std::integral_constant<int, (n - 8) / 2>{}, k + SETS * TK);
        if constexpr (n == 13 || n == 15)
          fetch_a(std::integral_constant<int, S1>{}, std::integral_constant<int, n == 15>{},
                  k + (SETS + 1) * TK);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;
  auto stage = [&](auto set_, int k, auto fast_) {
    constexpr int S = decltype(set_)::value;
    if constexpr (S == 0) {  // the next quad's first stage has used its scales
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        csa[i] = nsa[i];
        csb[i] = nsb[i];
      }
    }
    slice(set_, C0{}, k, fast_);
    slice(set_, C1{}, k, fast_);
    slice(set_, C2{}, k, fast_);
    // set S of B and the next set of A are used up
    if constexpr (!decltype(fast_)::value) {
      constexpr int S1 = (S + 1) % SETS;
      load_b(set_, k + SETS * TK);
      if constexpr (S == 0) load_s(k + SETS * TK);
      load_a(std::integral_constant<int, S1>{}, k + (SETS + 1) * TK);
    }
    slice(set_, C3{}, k, fast_);
  };

  load_s(0);
  static_for<SETS>([&](auto i) {
    load_a(i, decltype(i)::value * TK);
    load_b(i, decltype(i)::value * TK);
  });
  static_for<2>([&](auto i) {
    static_for<A_STEPS>([&](auto z) { step_a(C0{}, i, z); });
  });
  load_a(C0{}, SETS * TK);
  __syncthreads();
  static_for<8>([&](auto i) { fa[0][i] = read_a(0, 0, i); });
  static_for<2>([&](auto i) {
    static_for<B_STEPS>([&](auto z) { step_b(C0{}, C0{}, i, z, fb[0][i]); });
  });
  int k = 0;
#pragma unroll 1
  for (; k + (2 * SETS + 1) * TK <= K; k += SETS * TK)
    static_for<SETS>([&](auto i) { stage(i, k + decltype(i)::value * TK, std::true_type{}); });
#pragma unroll 1
  for (; k < K; k += SETS * TK)  // past the end the decode works on old codes
    static_for<SETS>([&](auto i) {
      const int ki = k + decltype(i)::value * TK;
      if (ki < K) stage(i, ki, std::false_type{});
    });
  __syncthreads();  // the last stage's readers are done: LDS becomes the epilogue's

  // Epilogue, 32 lines of A at a time through LDS, so that a lane ends up with
  // 8 consecutive outputs of a line. Register r of a 32 x 32 result: line l32
  // of A, line 8 (r / 4) + 4 g + r % 4 of B.
  constexpr int PITCH = 68;  // floats: 64 sums, the line's scale, bank padding
  float* ep = reinterpret_cast<float*>(lds) + wave * 2 * 32 * PITCH;
  constexpr int LPR = GATED ? 4 : 8, RPL = 64 / LPR;  // lanes to a line, lines to a wave's access
  constexpr int NL = 32 / RPL;
  const int cl = 8 * (lane % LPR);
  const int64_t j = j0 + wave * (GATED ? 32 : 64) + cl, nj = p.N - j;
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
  LineScale x[8];
#pragma unroll
  for (int mi = 0; mi < 8; ++mi) x[mi] = line_scale(p.a, min(i0 + mi * 32 + l32, p.M - 1));
  auto finish = [&](auto type_) __attribute__((always_inline)) {
    using T = decltype(type_);
#pragma unroll 1
    for (int mi = 0; mi < 8; mi += 2) {
      const int64_t i = i0 + mi * 32 + lane / LPR;
      Raw8<T> res[2][NL];
      static_for<2>([&](auto h) __attribute__((always_inline)) {
        constexpr int H = decltype(h)::value;
        load_residual<T, NL, RPL>(p, i + 32 * H, j, nj, res[H]);
      });
      // (one copy of this loop's body: only the choice of registers is unrolled)
      static_for<8>([&](auto m_) __attribute__((always_inline)) {
        constexpr int m = decltype(m_)::value;
        if ((mi | 1) == (m | 1)) {
          float* e = ep + (m & 1) * 32 * PITCH + l32 * PITCH;
#pragma unroll
          for (int ni = 0; ni < 2; ++ni)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x16& v = acc[m][ni];
              *reinterpret_cast<float4*>(e + ni * 32 + 8 * q + 4 * g) =
                  make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
          if (g == 0) *reinterpret_cast<float2*>(e + 64) = make_float2(x[m].m, __int_as_float(x[m].e));
        }
      });
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      static_for<2>([&](auto h) __attribute__((always_inline)) {
        constexpr int H = decltype(h)::value;
        float z0[NL][8], z1[NL][8];
#pragma unroll
        for (int v = 0; v < NL; ++v) {
          const float* row = ep + (32 * H + lane / LPR + v * RPL) * PITCH;
          const float2 xs = *reinterpret_cast<const float2*>(row + 64);
          const LineScale xr = {xs.x, __float_as_int(xs.y)};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            z0[v][e] = apply_scale(row[cl + e], xr, w0[e]) + b0[e];
            if constexpr (GATED) z1[v][e] = apply_scale(row[32 + cl + e], xr, w1[e]) + b1[e];
          }
        }
        finish_lines<T, GATED, NL, RPL>(p, i + 32 * H, j, nj, z0, z1, res[H]);
      });
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  };
  if (p.out_dtype == 0) finish(uint16_t{});
  else finish(float{});
}

int64_t gemm_tiles(int64_t M, int64_t N, bool gated) {
  const int out = gated ? TN / 2 : TN;
  return ((M + TM - 1) / TM) * ((N + out - 1) / out);
}

void launch_gemm_tile(const GemmArgs& a, hipStream_t s) {
  const bool gated = a.act == ACT_SWIGLU, a8 = a.a.s == nullptr;
  const int out = gated ? TN / 2 : TN;
  const int gm = (int)((a.M + TM - 1) / TM), gn = (int)((a.N + out - 1) / out);
  const dim3 grid((unsigned)(gm * gn)), b(256);
  if (a8 && gated) hipLaunchKernelGGL((gemm_tile_kernel<true, true>), grid, b, 0, s, a, gm, gn);
  else if (a8) hipLaunchKernelGGL((gemm_tile_kernel<true, false>), grid, b, 0, s, a, gm, gn);
  else if (gated) hipLaunchKernelGGL((gemm_tile_kernel<false, true>), grid, b, 0, s, a, gm, gn);
  else hipLaunchKernelGGL((gemm_tile_kernel<false, false>), grid, b, 0, s, a, gm, gn);
}

}  // namespace nvfp4
