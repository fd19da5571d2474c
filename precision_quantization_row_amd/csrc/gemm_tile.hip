// gemm_tile.hip -- the packed product for many lines of A (gfx950).
#include "gemm_device.h"

namespace nvfp4 {

// ------------------------------------------------------------- tile kernel
// 256 lines of A by 256 lines of B a workgroup of 4 waves, 128 x 128 a wave
// (its FP32 sums take 256 of the 512 registers a lane has at one wave a SIMD).
//
// Every code is decoded once a workgroup: a thread holds 16-byte chunks of
// packed lines (32 codes, two scale blocks) in registers, turns one block of
// each into binary16 a stage and puts it into LDS, from where the waves read
// matrix fragments. A stage is 64 along k and its products cost a wave 64
// matrix instructions of 32 cycles; beside them go the decode of the next
// stage (about two vector instructions for each: a convert and a multiply for
// two elements), its LDS writes and the loads of the codes after that.
// Decoding each wave's own fragments from packed LDS stages instead moves a
// quarter of the LDS bytes but decodes everything twice: five vector
// instructions beside each matrix instruction, more than fit (1271 against
// MEASURED_HERE TFLOP/s at 8192 x 8192 x 28672).
//
// k order. A block is 128 along k: lane chunk c (0..3) holds 32 c .. 32 c + 31
// of it. Stage 0 of the block takes the first 16 of every chunk, stage 1 the
// last 16; both operands alike, so the sum covers every k once.
constexpr int TM = 256, TN = 256, TK = 128;
constexpr int TILE_BYTES = (TM + TN) * 128;  // one stage in LDS: 64 binary16 a line
// 16-byte slot of chunk c of line r, rotated by the line: 16 lanes that read one
// chunk of 16 neighbouring lines touch all 64 banks once (a line is half of
// them), and 8 lanes that write 4 chunks of 2 lines touch 8 different slots.
// Rotated by r & 7 alone, reads took two passes (counted).
__device__ __forceinline__ int slot(int r, int c) {
  return r * 128 + 16 * (c ^ ((r >> 1) & 7) ^ (r & 1));
}

template <bool A8, bool GATED>
__global__ void __launch_bounds__(256, 1) gemm_tile_kernel(const GemmArgs p, int gm, int gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * TILE_BYTES];
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
  // Row r of the tile is line j0 + r of B; gated: every 128 rows hold 64 gate
  // lines, then the up lines of the same outputs. Lines past the matrix repeat
  // its last one (their products are not stored). This thread holds chunk c of
  // rows row0 + 64 i of B (i = 0..3; gated: odd i are up lines) and of A
  // (i = 4..7): offsets from the tile's first line, which 32 bits hold.
  const int row0 = tid >> 2, c = tid & 3;
  const int am = (int)min(p.M - i0, (int64_t)TM) - 1, bm = (int)min(p.N - j0, (int64_t)OUT) - 1;
  uint32_t qoff[8], soff[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lb = min(GATED ? row0 + 64 * (i >> 1) : row0 + 64 * i, bm);
    const int la = min(row0 + 64 * i, am);
    qoff[i] = (uint32_t)lb * qp + 16 * c;
    soff[i] = (uint32_t)lb * sp + 2 * c;
    qoff[i + 4] = (uint32_t)la * ap + (A8 ? 32 : 16) * c;
    soff[i + 4] = (uint32_t)la * sp + 2 * c;
  }
  const uint8_t *qb = p.b.q + j0 * qp, *sb = p.b.s + j0 * sp;
  const uint8_t *qu = GATED ? qb + p.N * qp : qb, *su = GATED ? sb + p.N * sp : sb;
  const uint8_t *qa = p.a.q + i0 * ap, *sa = A8 ? nullptr : p.a.s + i0 * sp;
  u32x4 raw[8], raw8[A8 ? 4 : 1];  // raw8: the second 16 bytes of an E4M3 chunk
  uint32_t sc[8];
  // chunk i of the block at k; WHOLE: the block lies inside the line
  auto fetch = [&](int i, int k, auto whole) {
    const bool e4m3 = A8 && i >= 4;
    const uint8_t* q = i >= 4 ? qa : (i & 1) ? qu : qb;
    const uint8_t* s = i >= 4 ? sa : (i & 1) ? su : sb;
    if constexpr (decltype(whole)::value) {
      // (the empty asm keeps the offset a 32-bit one added by the load itself)
      uint32_t qo = qoff[i], so = soff[i];
      asm volatile("" : "+v"(qo), "+v"(so));
      q += e4m3 ? k : k / 2;
      raw[i] = *reinterpret_cast<const u32x4_a1*>(q + qo);
      if (e4m3) raw8[A8 ? i - 4 : 0] = *reinterpret_cast<const u32x4_a1*>(q + 16 + qo);
      else sc[i] = *reinterpret_cast<const u16_a1*>(s + k / 16 + so);
    } else {
      const int kc = k + 32 * c;
      q += qoff[i] - (e4m3 ? 32 : 16) * c;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if (e4m3) {
          raw[i][d] = keep_bytes(tail_dword(q, ap, kc + 4 * d), K - kc - 4 * d);
          raw8[A8 ? i - 4 : 0][d] =
              keep_bytes(tail_dword(q, ap, kc + 16 + 4 * d), K - kc - 16 - 4 * d);
        } else {
          raw[i][d] = keep_nibbles(tail_dword(q, qp, kc / 2 + 4 * d), K - kc - 8 * d);
        }
      }
      if (!e4m3)
        sc[i] = keep_bytes(tail_dword(s + soff[i] - 2 * c, sp, kc / 16), sp - kc / 16);
    }
  };
  // half h of chunk i into stage buffer h
  auto expand = [&](int i, int h) {
    uint8_t* l = lds + h * TILE_BYTES + (i >= 4 ? TN * 128 : 0);
    const int r = row0 + 64 * (i & 3);
    h8 lo, hi;
    if (A8 && i >= 4) {
      const u32x4 w = h ? raw8[A8 ? i - 4 : 0] : raw[i];
      lo = decode8_fp8(w[0], w[1]);
      hi = decode8_fp8(w[2], w[3]);
    } else {
      const h2 s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc[i], 1.0f, false);
      lo = decode8_fp4(raw[i][2 * h], h ? s.yy : s.xx);
      hi = decode8_fp4(raw[i][2 * h + 1], h ? s.yy : s.xx);
    }
    *reinterpret_cast<h8*>(l + slot(r, 2 * c)) = lo;
    *reinterpret_cast<h8*>(l + slot(r, 2 * c + 1)) = hi;
  };

  f32x16 acc[4][4] = {};
  h8 fb[2][4], fa[2][4];
  auto frags = [&](int buf, int kk, h8 (&b)[4], h8 (&a)[4]) {
    const uint8_t* l = lds + buf * TILE_BYTES;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = *reinterpret_cast<const h8*>(l + slot(wn * 128 + i * 32 + l32, 2 * kk + g));
      a[i] = *reinterpret_cast<const h8*>(l + TN * 128 + slot(wm * 128 + i * 32 + l32, 2 * kk + g));
    }
  };
  // Stage H of a block: its products, from buffer H; the next stage (half
  // H ^ 1 of the registers) goes to the other buffer, whose last readers passed
  // the previous barrier. NEXT: 0 no stage follows, 1 one does, 2 and the block
  // after this one is fetched, 3 and lies inside the line.
  // Slice KK of it: 16 matrix instructions, and beside them, in this order, the
  // reads of the next slice's fragments and a share of the decode: chunks
  // 3 KK .. of the thread, one vector instruction after the other as listed by
  // Steps (a convert runs one pair ahead of its multiply).
  h2 cv[8], ov[8];
  h2 scale;
  auto decode_step = [&](auto h_, auto chunk_, auto step_, int k, auto next_) {
    constexpr int H = decltype(h_)::value ^ 1, I = decltype(chunk_)::value, Z = decltype(step_)::value;
    constexpr bool E4M3 = A8 && I >= 4;
    constexpr int CV = E4M3 ? Z : Z == 0 ? -1 : Z == 1 ? 0 : Z == 16 ? -1 : Z % 2 == 0 ? Z / 2 : -1;
    constexpr int MU = E4M3 ? Z : Z == 16 ? 7 : Z >= 3 && Z % 2 == 1 ? (Z - 3) / 2 : -1;
    if constexpr (!E4M3 && Z == 0) scale = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc[I], 1.0f, false);
    if constexpr (CV >= 0) {
      if constexpr (E4M3) {
        const u32x4 w = H ? raw8[A8 ? I - 4 : 0] : raw[I];
        ov[CV] = cvt_fp8<CV & 1>(w[CV >> 1]);
      } else {
        cv[CV] = cvt_fp4<CV & 3>(raw[I][2 * H + (CV >> 2)]);
      }
    }
    if constexpr (MU >= 0) {
      if constexpr (!E4M3) ov[MU] = cv[MU] * (H ? scale.yy : scale.xx);
      if constexpr ((MU & 3) == 3) {
        const int r = row0 + 64 * (I & 3);
        uint8_t* l = lds + H * TILE_BYTES + (I >= 4 ? TN * 128 : 0);
        *reinterpret_cast<h8*>(l + slot(r, 2 * c + (MU >> 2))) =
            h8{ov[MU - 3].x, ov[MU - 3].y, ov[MU - 2].x, ov[MU - 2].y,
               ov[MU - 1].x, ov[MU - 1].y, ov[MU].x, ov[MU].y};
      }
      if constexpr (MU == 7 && decltype(next_)::value == 3) fetch(I, k + TK, std::true_type{});
    }
  };
  auto slice = [&](auto h_, auto kk_, int k, auto next_) {
    constexpr int H = decltype(h_)::value, KK = decltype(kk_)::value, NEXT = decltype(next_)::value;
    constexpr int BAR = 4;
    constexpr int FIRST = 3 * KK, CHUNKS = KK == 2 ? 2 : KK == 3 ? 0 : 3;
    constexpr int S0 = A8 && FIRST >= 4 ? 8 : 17, S1 = A8 && FIRST + 1 >= 4 ? 8 : 17,
                  S2 = A8 && FIRST + 2 >= 4 ? 8 : 17;
    constexpr int TOTAL = (CHUNKS > 0 ? S0 : 0) + (CHUNKS > 1 ? S1 : 0) + (CHUNKS > 2 ? S2 : 0);
    h8(&nb)[4] = fb[(KK + 1) & 1];
    h8(&na)[4] = fa[(KK + 1) & 1];
    constexpr int RB = KK == 3 ? H ^ 1 : H, RK = (KK + 1) & 3;  // the next slice's buffer and place
    const uint8_t* lf = lds + RB * TILE_BYTES;
    static_for<16>([&](auto n_) {
      constexpr int n = decltype(n_)::value, mi = n / 4, ni = n % 4;
      acc[mi][ni] =
          __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[KK & 1][ni], fa[KK & 1][mi], acc[mi][ni], 0, 0, 0);
      // The reads come in the order of their use. In the last slice they follow
      // the barrier, which stands a few matrix instructions in, when the LDS
      // writes before it have long been done.
      if constexpr (KK == 3 && n == BAR) __syncthreads();
      constexpr int rd = KK == 3 ? n - BAR : n;
      if constexpr ((NEXT > 0 || KK < 3) && rd >= 0 && rd < 8) {
        if constexpr (rd >= 1 && rd < 5)
          nb[rd - 1] = *reinterpret_cast<const h8*>(lf + slot(wn * 128 + (rd - 1) * 32 + l32, 2 * RK + g));
        else {
          constexpr int i = rd == 0 ? 0 : rd - 4;
          na[i] = *reinterpret_cast<const h8*>(lf + TN * 128 + slot(wm * 128 + i * 32 + l32, 2 * RK + g));
        }
      }
      if constexpr (NEXT > 0 && CHUNKS > 0) {
        constexpr int Z0 = n * TOTAL / 16, Z1 = (n + 1) * TOTAL / 16;
        static_for<Z1 - Z0>([&](auto z_) {
          constexpr int z = Z0 + decltype(z_)::value;
          constexpr int I = FIRST + (z >= S0) + (z >= S0 + S1);
          constexpr int Z = z - (z >= S0 ? S0 : 0) - (z >= S0 + S1 ? S1 : 0);
          decode_step(h_, std::integral_constant<int, I>{}, std::integral_constant<int, Z>{}, k, next_);
        });
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  auto stage = [&](auto h_, int k, auto next_) {
    constexpr int NEXT = decltype(next_)::value;
    slice(h_, std::integral_constant<int, 0>{}, k, next_);
    slice(h_, std::integral_constant<int, 1>{}, k, next_);
    slice(h_, std::integral_constant<int, 2>{}, k, next_);
    if constexpr (NEXT == 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) fetch(i, k + TK, std::false_type{});
    }
    slice(h_, std::integral_constant<int, 3>{}, k, next_);
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;
  if (TK <= K) {
#pragma unroll
    for (int i = 0; i < 8; ++i) fetch(i, 0, std::true_type{});
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) fetch(i, 0, std::false_type{});
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) expand(i, 0);
  __syncthreads();
  frags(0, 0, fb[0], fa[0]);
  int k = 0;
#pragma unroll 1
  for (; k + 2 * TK <= K; k += TK) {
    stage(C0{}, k, C3{});
    stage(C1{}, k, C1{});
  }
  if (k + TK < K) {  // a last block that ends inside the line's end follows
    stage(C0{}, k, C2{});
    stage(C1{}, k, C1{});
    k += TK;
  }
  stage(C0{}, k, C1{});
  stage(C1{}, k, C0{});
  __syncthreads();  // the last stage's readers are done: LDS becomes the epilogue's

  // Epilogue, 32 lines of A at a time through LDS, so that a lane ends up with
  // 8 consecutive outputs of one line. Register r of a 32 x 32 result: line
  // l32 of A, line 8 (r / 4) + 4 g + r % 4 of B.
  float* ep = reinterpret_cast<float*>(lds) + wave * 32 * 132;
  constexpr int LPR = GATED ? 8 : 16, RPL = 64 / LPR;  // lanes to a line, lines to a wave's access
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
  for (int mi = 0; mi < 4; ++mi)
    x[mi] = line_scale(p.a, min(i0 + wm * 128 + mi * 32 + l32, p.M - 1));
#pragma unroll
  for (int mi = 0; mi < 4; ++mi) {
#pragma unroll
    for (int ni = 0; ni < 4; ++ni)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16& v = acc[mi][ni];
        *reinterpret_cast<float4*>(ep + l32 * 132 + ni * 32 + 8 * q + 4 * g) =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      }
    if (g == 0)
      *reinterpret_cast<float2*>(ep + l32 * 132 + 128) = make_float2(x[mi].m, __int_as_float(x[mi].e));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int q = 0; q < 32 / RPL; q += 4) {  // 4 lines of a lane at a time
      float z0[4][8], z1[4][8];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float* row = ep + (lane / LPR + (q + v) * RPL) * 132;
        const float2 xs = *reinterpret_cast<const float2*>(row + 128);
        const LineScale xr = {xs.x, __float_as_int(xs.y)};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          z0[v][e] = apply_scale(row[cl + e], xr, w0[e]) + b0[e];
          if constexpr (GATED) z1[v][e] = apply_scale(row[64 + cl + e], xr, w1[e]) + b1[e];
        }
      }
      const int64_t i = i0 + wm * 128 + mi * 32 + lane / LPR + q * RPL;
      if (p.out_dtype == 0) finish_lines<uint16_t, GATED, 4, RPL>(p, i, j, nj, z0, z1);
      else finish_lines<float, GATED, 4, RPL>(p, i, j, nj, z0, z1);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
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
