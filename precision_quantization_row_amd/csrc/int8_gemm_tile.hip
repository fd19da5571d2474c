// int8_gemm_tile.hip -- the product of 8-bit integer lines for many lines of A
// (gfx950).
#include "gemm_device.h"

namespace nvfp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// 256 lines of A by 256 lines of B a workgroup of 4 waves, one wave a SIMD, 128 x
// 128 a wave: its sums take 256 of the lane's 512 registers. A stage is 128 bytes
// along k of all 512 lines, 64 KB of LDS; two of them take turns. A slice of a
// stage is 32 k: 16 matrix instructions of 32 cycles from 8 fragments (64 bytes of
// LDS a cycle for the CU), and beside them, one by one, the next slice's
// fragments, the next stage's chunks from registers into LDS and the loads of the
// stage after that. The last slice of a stage holds the barrier: by then
// everything of this stage is in registers and the next one is in LDS. (Loads
// straight into LDS, which aligned rows would allow, take longer: 8192^3 of zeros,
// where power does not count, 385 us against 360; half as long stages, four in
// turn, 381.)
constexpr int TM = 256, TN = 256, TK = 128;
constexpr int SIDE = TM * TK;  // A's two halves, then B's
// 16-byte slot s of line r, rotated by the line so that 16 lanes that read one
// slot of 16 neighbouring lines touch all 64 banks once (a line is half of them).
__device__ __forceinline__ int rotate(int r) {
  return ((r >> 1) & 1) << 2 | ((r ^ (r >> 3)) & 1) << 1 | ((r >> 2) & 1);
}

template <bool GATED>
__global__ void __launch_bounds__(256, 1) int8_tile_kernel(const GemmArgs p, int gm, int gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * SIDE];
  __shared__ float2 factors[2][TM];  // of the tile's lines of A and of B: mantissa, exponent
  __shared__ float biases[TN];
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
  // This thread moves chunk lane % 8 (16 bytes) of lines wave * 64 + 8 i + lane / 8 of
  // each side. Lines past the matrix repeat its last one (their products are not stored).
  // Gated: a wave's 128 lines of B are 64 gate lines and their up lines.
  uint32_t aoff[8], boff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = wave * 64 + 8 * i + lane / 8, c = lane % 8;
    aoff[i] = (uint32_t)min(r, am) * K + 16 * c;
    boff[i] = (uint32_t)min(GATED ? (r / 128) * 64 + r % 64 : r, bm) * K + 16 * c;
  }
  // (gated: a wave moves gate lines or up lines)
  const uint8_t* qu = GATED && (wave & 1) ? qb + p.N * K : qb;
  // chunk i of this thread: 0 .. 7 of A, 8 .. 15 of B, of the stage at k, which lies
  // inside the lines
  u32x4 ring[16];
  auto fetch = [&](auto i_, int k) __attribute__((always_inline)) {
    constexpr int i = decltype(i_)::value;
    // (the empty asm keeps the offset a 32-bit one added by the load itself)
    uint32_t o = i < 8 ? aoff[i & 7] : boff[i & 7];
    asm volatile("" : "+v"(o));
    ring[i] = *reinterpret_cast<const u32x4_a1*>((i < 8 ? qa : qu) + k + o);
  };
  auto put = [&](auto i_, int half) __attribute__((always_inline)) {
    constexpr int i = decltype(i_)::value;
    const int r = wave * 64 + 8 * (i & 7) + lane / 8;
    *reinterpret_cast<u32x4*>(lds + (i < 8 ? 0 : 2 * SIDE) + half * SIDE + r * TK + 16 * ((lane % 8) ^ rotate(r))) =
        ring[i];
  };
  const int nu = (K + TK - 1) / TK;
  // Any stage on its way into the registers; one that reaches past the lines' end has
  // zeros there, nothing comes of one that lies past it.
  auto begin = [&](int u) __attribute__((always_inline)) {
    const int k = u * TK;
    if (k + TK <= K) {
      static_for<16>([&](auto i) __attribute__((always_inline)) { fetch(i, k); });
    } else if (u < nu) {
      const int at = k + 16 * (lane % 8);
      static_for<16>([&](auto i_) __attribute__((always_inline)) {
        constexpr int i = decltype(i_)::value;
        const uint8_t* line = (i < 8 ? qa + aoff[i & 7] : qu + boff[i & 7]) - 16 * (lane % 8);
#pragma unroll
        for (int d = 0; d < 4; ++d) ring[i][d] = keep_bytes(tail_dword(line, K, at + 4 * d), K - at - 4 * d);
      });
    }
  };

  // where this lane's fragments of slice d begin, of A's and B's first lines and halves
  uint32_t pa[4], pb[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t o = l32 * TK + 16 * ((2 * d + g) ^ rotate(l32));
    pa[d] = wm * 128 * TK + o;
    pb[d] = 2 * SIDE + wn * 128 * TK + o;
  }
  i32x16 acc[4][4] = {};
  i32x4 fa[2][4], fb[2][4];
  // fragment f of a slice, in the order that its products need them
  auto read = [&](auto f_, auto d_, auto half_, i32x4 (&a)[4], i32x4 (&b)[4]) __attribute__((always_inline)) {
    constexpr int F = decltype(f_)::value, D = decltype(d_)::value, H = decltype(half_)::value;
    constexpr bool of_a = F == 0 || F > 4;
    constexpr int i = F == 0 ? 0 : of_a ? F - 4 : F - 1;
    const i32x4 v = *reinterpret_cast<const i32x4*>(lds + (of_a ? pa[D] : pb[D]) + H * SIDE + i * 32 * TK);
    if constexpr (of_a) a[i] = v;
    else b[i] = v;
  };
  // Slice D of stage u, which lies in half H. FAST: stage u + 2 lies inside the lines.
  // (From product to product one of the two operands stays.)
  auto slice = [&](auto half_, auto d_, int u, auto fast_) __attribute__((always_inline)) {
    constexpr int H = decltype(half_)::value, D = decltype(d_)::value, BAR = 3, CUR = D & 1, NXT = CUR ^ 1;
    constexpr bool FAST = decltype(fast_)::value;
    static_for<16>([&](auto n_) __attribute__((always_inline)) {
      constexpr int n = decltype(n_)::value, mi = n / 4, ni = mi & 1 ? 3 - n % 4 : n % 4;
      acc[mi][ni] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[CUR][ni], fa[CUR][mi], acc[mi][ni], 0, 0, 0);
      if constexpr (D == 3 && n == BAR) __syncthreads();
      constexpr int rd = D == 3 ? n - BAR - 1 : n;
      if constexpr (rd >= 0 && rd < 8)
        read(std::integral_constant<int, rd>{}, std::integral_constant<int, (D + 1) & 3>{},
             std::integral_constant<int, D == 3 ? H ^ 1 : H>{}, fa[NXT], fb[NXT]);
      if constexpr (D < 3 && n % 3 == 2) {
        constexpr int i = 5 * D + n / 3;  // 5 chunks a slice, the last one below
        put(std::integral_constant<int, i>{}, H ^ 1);
        if constexpr (FAST) fetch(std::integral_constant<int, i>{}, (u + 2) * TK);
        if constexpr (i == 14) {
          put(std::integral_constant<int, 15>{}, H ^ 1);
          if constexpr (FAST) fetch(std::integral_constant<int, 15>{}, (u + 2) * TK);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  auto stage = [&](auto half_, int u, auto fast_) __attribute__((always_inline)) {
    slice(half_, std::integral_constant<int, 0>{}, u, fast_);
    slice(half_, std::integral_constant<int, 1>{}, u, fast_);
    slice(half_, std::integral_constant<int, 2>{}, u, fast_);
    if constexpr (!decltype(fast_)::value) begin(u + 2);
    slice(half_, std::integral_constant<int, 3>{}, u, fast_);
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  // the lines' factors and biases, for the epilogue
  const int fb_line = GATED ? (tid / 128) * 64 + tid % 64 : tid;
  const int64_t jf = (GATED && (tid & 64) ? p.N : 0) + j0 + min(fb_line, bm);
  const LineScale xf = line_scale(p.a, i0 + min(tid, am)), wf = line_scale(p.b, jf);
  const float bf = load_bias(p, jf);
  begin(0);
  factors[0][tid] = make_float2(xf.m, __int_as_float(xf.e));
  factors[1][tid] = make_float2(wf.m, __int_as_float(wf.e));
  biases[tid] = bf;
  static_for<16>([&](auto i) __attribute__((always_inline)) { put(i, 0); });
  begin(1);
  __syncthreads();
  static_for<8>([&](auto f) __attribute__((always_inline)) { read(f, C0{}, C0{}, fa[0], fb[0]); });
  int u = 0;
#pragma unroll 1
  for (; (u + 4) * TK <= K; u += 2) {
    stage(C0{}, u, std::true_type{});
    stage(C1{}, u + 1, std::true_type{});
  }
#pragma unroll 1
  for (; u < nu; u += 2) {  // past the end the puts move old chunks
    stage(C0{}, u, std::false_type{});
    if (u + 1 < nu) stage(C1{}, u + 1, std::false_type{});
  }

  // Epilogue, 32 lines of A at a time through LDS, so that a lane ends up with
  // 8 consecutive outputs of a line. Register r of a 32 x 32 result: line l32
  // of A, line 8 (r / 4) + 4 g + r % 4 of B. The sums go as they are; the
  // residual's next lines are on their way meanwhile.
  constexpr int PITCH = 132;  // dwords: 128 sums, the line's scale, bank padding
  int* ep = reinterpret_cast<int*>(lds) + wave * 32 * PITCH;
  constexpr int LPR = GATED ? 8 : 16, RPL = 64 / LPR;  // lanes to a line, lines to a wave's access
  constexpr int NL = 32 / RPL;                         // accesses to 32 lines
  const int cl = 8 * (lane % LPR);
  const int64_t j = j0 + wn * (GATED ? 64 : 128) + cl, nj = p.N - j;
  const int64_t i00 = i0 + wm * 128 + lane / LPR;
  LineScale w0[8], w1[GATED ? 8 : 1], x[4];
  float b0[8], b1[GATED ? 8 : 1];
  // Factors whose exponents are ordinary are multiplied as they are; it gives the
  // same bits as mantissas and exponents on their own, since no step leaves the
  // normal numbers: |sum| < 2^31, factors within 2^+-41.
  bool plain = true;
  auto check = [&](const LineScale& v) { plain = plain && v.e > -40 && v.e < 40; };
  auto factor = [&](int side, int line) {
    const float2 v = factors[side][line];
    return LineScale{v.x, __float_as_int(v.y)};
  };
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int line = wn * 128 + cl + q;
    check(w0[q] = factor(1, line));
    b0[q] = biases[line];
    if constexpr (GATED) {
      check(w1[q] = factor(1, line + 64));
      b1[q] = biases[line + 64];
    }
  }
#pragma unroll
  for (int mi = 0; mi < 4; ++mi) check(x[mi] = factor(0, wm * 128 + mi * 32 + l32));
  const bool all_plain = __ballot(!plain) == 0;
  if (all_plain) {
    auto whole = [](LineScale& v) { v.m = __builtin_amdgcn_ldexpf(v.m, v.e); };
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      whole(w0[q]);
      if constexpr (GATED) whole(w1[q]);
    }
#pragma unroll
    for (int mi = 0; mi < 4; ++mi) whole(x[mi]);
  }
  // (One copy of the loop's body, only the choice of registers is unrolled: code runs
  // once a tile, and comes from L2 where it does not fit the instruction cache.)
  auto finish = [&](auto type_) __attribute__((always_inline)) {
    using T = decltype(type_);
    constexpr int PARTS = 2, PL = NL / PARTS;  // parts of 32 lines, accesses to one
    Raw8<T> res[PL];
    load_residual<T, PL, RPL>(p, i00, j, nj, res);
#pragma unroll 1
    for (int part = 0; part < 4 * PARTS; ++part) {
      if (part % PARTS == 0) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        static_for<4>([&](auto m_) __attribute__((always_inline)) {
          constexpr int m = decltype(m_)::value;
          if (part / PARTS == m) {
            int* e = ep + l32 * PITCH;
#pragma unroll
            for (int ni = 0; ni < 4; ++ni)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const i32x16& v = acc[m][ni];
                *reinterpret_cast<i32x4*>(e + ni * 32 + 8 * q + 4 * g) =
                    i32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
              }
            if (g == 0) *reinterpret_cast<float2*>(e + 128) = make_float2(x[m].m, __int_as_float(x[m].e));
          }
        });
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      const int line = part * PL * RPL;  // of the wave's 128
      // (every read of the part is on its way before the first is used)
      i32x4 s0[PL][2], s1[GATED ? PL : 1][2];
      LineScale xr[PL];
      Raw8<T> now[PL];
#pragma unroll
      for (int v = 0; v < PL; ++v) {
        const int* row = ep + (line % 32 + lane / LPR + v * RPL) * PITCH;
        const float2 xs = *reinterpret_cast<const float2*>(row + 128);
        xr[v] = {xs.x, __float_as_int(xs.y)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s0[v][h] = *reinterpret_cast<const i32x4*>(row + cl + 4 * h);
          if constexpr (GATED) s1[v][h] = *reinterpret_cast<const i32x4*>(row + 64 + cl + 4 * h);
        }
        now[v] = res[v];
      }
      float z0[PL][8], z1[PL][8];
      if (all_plain) {
#pragma unroll
        for (int v = 0; v < PL; ++v)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            z0[v][q] = (float)s0[v][q / 4][q % 4] * (xr[v].m * w0[q].m) + b0[q];
            if constexpr (GATED) z1[v][q] = (float)s1[v][q / 4][q % 4] * (xr[v].m * w1[q].m) + b1[q];
          }
      } else {
#pragma unroll
        for (int v = 0; v < PL; ++v)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            z0[v][q] = apply_scale((float)s0[v][q / 4][q % 4], xr[v], w0[q]) + b0[q];
            if constexpr (GATED) z1[v][q] = apply_scale((float)s1[v][q / 4][q % 4], xr[v], w1[q]) + b1[q];
          }
      }
      if (part + 1 < 4 * PARTS) load_residual<T, PL, RPL>(p, i00 + line + PL * RPL, j, nj, res);
      finish_lines<T, GATED, PL, RPL>(p, i00 + line, j, nj, z0, z1, now);
    }
  };
  __syncthreads();  // the last fragments are read: LDS becomes the epilogue's
  if (p.out_dtype == 0) finish(uint16_t{});
  else finish(float{});
}

template <bool GATED>
static void go_tile(const GemmArgs& a, hipStream_t s) {
  constexpr int out = GATED ? TN / 2 : TN;
  const int gm = (int)((a.M + TM - 1) / TM), gn = (int)((a.N + out - 1) / out);
  hipLaunchKernelGGL((int8_tile_kernel<GATED>), dim3((unsigned)(gm * gn)), dim3(256), 0, s, a, gm, gn);
}

void launch_int8_tile(const GemmArgs& a, hipStream_t s) {
  if (a.act == ACT_SWIGLU) go_tile<true>(a, s);
  else go_tile<false>(a, s);
}

}  // namespace nvfp4
