// int8_gemm_tile.hip -- the product of 8-bit integer lines for many lines of A
// (gfx950).
#include "int8_device.h"

namespace nvfp4 {

// 64 WM lines of A by 64 WN lines of B a workgroup of 4 waves, 32 WM x 32 WN a wave.
// 4 x 4: one wave a SIMD, its sums take 256 of the lane's 512 registers. 2 x 2 and 1 x 2,
// for products that have too few such tiles: two workgroups a CU and more. A stage
// is 128 bytes along k of all lines, 8 KB of LDS for 64 of them; two stages take
// turns. A slice of a stage is 32 k: WM WN matrix instructions of 32 cycles from WM +
// WN fragments (4 x 4: 64 bytes of LDS a cycle for the CU), and beside them, one by
// one, the next slice's fragments, the next stage's chunks from registers into LDS
// and the loads of the stage after that. The last slice of a stage holds the
// barrier: by then everything of this stage is in registers and the next one is in
// LDS. (Loads straight into LDS, which aligned rows would allow, take longer: 8192^3
// of zeros, where power does not count, 385 us against 360; half as long stages, four
// in turn, 381. Two groups of waves with every other stage each gain nothing: what
// bounds few tiles is a CU's share of L2, 40 bytes a cycle.)
// 8192 x 8192 x 28672 of ordinary codes with the residual: 1514 to 1596 us by the card, 2.41 to
// 2.54 PO/s, the matrix pipe busy for 77 % of the cycles (counted), and power.
// The compiler spills 16 registers of <false, 4, 4> and 14 of <true, 4, 4>, read in the loop of
// the last stages (all stages of a product of fewer than four), and 11 of <false, 2, 2>, in
// its epilogue; none in the loop of the others.
constexpr int TK = 128;
template <bool GATED, int WM, int WN>
__global__ void __launch_bounds__(256, WM == 4 ? 1 : 2) int8_tile_kernel(const GemmArgs p, int gm, int gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int TM = 64 * WM, TN = 64 * WN, LM = 32 * WM, LN = 32 * WN;  // lines: a workgroup's, a wave's
  constexpr int SIDE_A = TM * TK, SIDE_B = TN * TK, B0 = 2 * SIDE_A;     // A's two halves, then B's
  constexpr int CA = 2 * WM, CH = CA + 2 * WN;                           // a thread's chunks: A's, all
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * (SIDE_A + SIDE_B)];
  __shared__ float2 factors[TM + TN];  // of the tile's lines of A, of B: mantissa, exponent
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
  // This thread moves chunk lane % 8 (16 bytes) of every 8th line of its wave's quarter of
  // a side, from line lane / 8 on. Lines past the matrix repeat its last one (their
  // products are not stored). Gated: a wave's 32 WN lines of B are 16 WN gate lines and
  // their up lines.
  auto out_of = [&](int r) { return GATED ? r / LN * (LN / 2) + r % (LN / 2) : r; };
  auto line_of = [&](int i) { return i < CA ? wave * (TM / 4) + 8 * i + lane / 8 : wave * (TN / 4) + 8 * (i - CA) + lane / 8; };
  uint32_t off[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i)
    off[i] = (uint32_t)(i < CA ? min(line_of(i), am) : min(out_of(line_of(i)), bm)) * K + 16 * (lane % 8);
  // (gated: a wave moves gate lines or up lines)
  const uint8_t* qu = GATED && (wave & 1) ? qb + p.N * K : qb;
  // chunk i of this thread, A's before B's, of the stage at k, which lies inside the
  // lines
  u32x4 ring[CH];
  auto fetch = [&](auto i_, int k) __attribute__((always_inline)) {
    constexpr int i = decltype(i_)::value;
    // (the empty asm keeps the offset a 32-bit one added by the load itself)
    uint32_t o = off[i];
    asm volatile("" : "+v"(o));
    ring[i] = *reinterpret_cast<const u32x4_a1*>((i < CA ? qa : qu) + k + o);
  };
  auto put = [&](auto i_, int half) __attribute__((always_inline)) {
    constexpr int i = decltype(i_)::value;
    const int r = line_of(i);
    *reinterpret_cast<u32x4*>(lds + (i < CA ? half * SIDE_A : B0 + half * SIDE_B) + r * TK + 16 * ((lane % 8) ^ rotate(r))) =
        ring[i];
  };
  const int nu = (K + TK - 1) / TK;
  // Any stage on its way into the registers; zeros where it reaches past the lines' end.
  auto begin = [&](int u) __attribute__((always_inline)) {
    const int k = u * TK;
    if (k + TK <= K) {
      static_for<CH>([&](auto i) __attribute__((always_inline)) { fetch(i, k); });
    } else if (u < nu) {
      static_for<CH>([&](auto i_) __attribute__((always_inline)) {
        constexpr int i = decltype(i_)::value;
        ring[i] = tail_chunk((i < CA ? qa : qu) + off[i] - 16 * (lane % 8), K, k + 16 * (lane % 8));
      });
    }
  };

  // where this lane's fragments of slice d begin, of A's and B's first lines and halves
  uint32_t pa[4], pb[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t o = l32 * TK + 16 * ((2 * d + g) ^ rotate(l32));
    pa[d] = wm * LM * TK + o;
    pb[d] = B0 + wn * LN * TK + o;
  }
  i32x16 acc[WM][WN] = {};
  i32x4 fa[2][WM], fb[2][WN];
  // fragment f of a slice, in the order that its products need them
  auto read = [&](auto f_, auto d_, auto half_, i32x4 (&a)[WM], i32x4 (&b)[WN]) __attribute__((always_inline)) {
    constexpr int F = decltype(f_)::value, D = decltype(d_)::value, H = decltype(half_)::value;
    constexpr bool of_a = F == 0 || F > WN;
    constexpr int i = F == 0 ? 0 : of_a ? F - WN : F - 1;
    const i32x4 v = *reinterpret_cast<const i32x4*>(lds + (of_a ? pa[D] + H * SIDE_A : pb[D] + H * SIDE_B) + i * 32 * TK);
    if constexpr (of_a) a[i] = v;
    else b[i] = v;
  };
  // Slice D of stage u, which lies in half H. FAST: stage u + 2 lies inside the lines.
  // (From product to product one of the two operands stays.)
  auto slice = [&](auto half_, auto d_, int u, auto fast_) __attribute__((always_inline)) {
    constexpr int H = decltype(half_)::value, D = decltype(d_)::value, CUR = D & 1, NXT = CUR ^ 1;
    constexpr int N = WM * WN, BAR = WM == 4 ? 3 : 0;
    constexpr bool FAST = decltype(fast_)::value;
    static_for<N>([&](auto n_) __attribute__((always_inline)) {
      constexpr int n = decltype(n_)::value, mi = n / WN, ni = mi & 1 ? WN - 1 - n % WN : n % WN;
      acc[mi][ni] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[CUR][ni], fa[CUR][mi], acc[mi][ni], 0, 0, 0);
      if constexpr (D == 3 && n == BAR) __syncthreads();
      // the next slice's fragments: one a product, or as many as it takes
      constexpr int F = WM + WN, room = D == 3 ? N - BAR : N, m = D == 3 ? n - BAR : n;
      constexpr int per = (F + room - 1) / room, f0 = m < 0 ? 0 : m * per, f1 = m < 0 ? 0 : (m + 1) * per;
      static_for<(f1 < F ? f1 : F) - (f0 < F ? f0 : F)>([&](auto f) __attribute__((always_inline)) {
        read(std::integral_constant<int, f0 + decltype(f)::value>{}, std::integral_constant<int, (D + 1) & 3>{},
             std::integral_constant<int, D == 3 ? H ^ 1 : H>{}, fa[NXT], fb[NXT]);
      });
      // the thread's chunks, spread over the first three slices
      constexpr int at = D * N + n, c0 = at * CH / (3 * N), c1 = (at + 1) * CH / (3 * N);
      if constexpr (D < 3)
        static_for<c1 - c0>([&](auto c) __attribute__((always_inline)) {
          put(std::integral_constant<int, c0 + decltype(c)::value>{}, H ^ 1);
          if constexpr (FAST) fetch(std::integral_constant<int, c0 + decltype(c)::value>{}, (u + 2) * TK);
        });
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
  LineScale xf = {}, wf = {};
  float bf = 0.0f;
  if (tid < TM) xf = line_scale(p.a, i0 + min(tid, am));
  if (tid < TN) {
    const int64_t jf = (GATED && tid % LN >= LN / 2 ? p.N : 0) + j0 + min(out_of(tid), bm);
    wf = line_scale(p.b, jf);
    bf = load_bias(p, jf);
  }
  begin(0);
  if (tid < TM) factors[tid] = make_float2(xf.m, __int_as_float(xf.e));
  if (tid < TN) {
    factors[TM + tid] = make_float2(wf.m, __int_as_float(wf.e));
    biases[tid] = bf;
  }
  static_for<CH>([&](auto i) __attribute__((always_inline)) { put(i, 0); });
  begin(1);
  __syncthreads();
  static_for<WM + WN>([&](auto f) __attribute__((always_inline)) { read(f, C0{}, C0{}, fa[0], fb[0]); });
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
  constexpr int PITCH = LN + 4;  // dwords: a line's sums, its scale, bank padding
  int* ep = reinterpret_cast<int*>(lds) + wave * 32 * PITCH;
  constexpr int LPR = (GATED ? LN / 2 : LN) / 8, RPL = 64 / LPR;  // lanes to a line, lines to a wave's access
  constexpr int NL = 32 / RPL;                         // accesses to 32 lines
  const int cl = 8 * (lane % LPR);
  const int64_t j = j0 + wn * (GATED ? LN / 2 : LN) + cl, nj = p.N - j;
  const int64_t i00 = i0 + wm * LM + lane / LPR;
  LineScale w0[8], w1[GATED ? 8 : 1], x[WM];
  float b0[8], b1[GATED ? 8 : 1];
  // Factors whose exponents are ordinary are multiplied as they are; it gives the
  // same bits as mantissas and exponents on their own, since no step leaves the
  // normal numbers: |sum| < 2^31, factors within 2^+-41.
  bool plain = true;
  auto check = [&](const LineScale& v) { plain = plain && v.e > -40 && v.e < 40; };
  auto factor = [&](int line) {
    const float2 v = factors[line];
    return LineScale{v.x, __float_as_int(v.y)};
  };
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int line = wn * LN + cl + q;
    check(w0[q] = factor(TM + line));
    b0[q] = biases[line];
    if constexpr (GATED) {
      check(w1[q] = factor(TM + line + LN / 2));
      b1[q] = biases[line + LN / 2];
    }
  }
#pragma unroll
  for (int mi = 0; mi < WM; ++mi) check(x[mi] = factor(wm * LM + mi * 32 + l32));
  const bool all_plain = __ballot(!plain) == 0;
  if (all_plain) {
    auto whole = [](LineScale& v) { v.m = __builtin_amdgcn_ldexpf(v.m, v.e); };
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      whole(w0[q]);
      if constexpr (GATED) whole(w1[q]);
    }
#pragma unroll
    for (int mi = 0; mi < WM; ++mi) whole(x[mi]);
  }
  // (One copy of the loop's body, only the choice of registers is unrolled: code runs
  // once a tile, and comes from L2 where it does not fit the instruction cache.)
  auto finish = [&](auto type_) __attribute__((always_inline)) {
    using T = decltype(type_);
    constexpr int PARTS = WN == 4 ? 2 : 1, PL = NL / PARTS;  // parts of 32 lines, accesses to one
    Raw8<T> res[PL];
    load_residual<T, PL, RPL>(p, i00, j, nj, res);
#pragma unroll 1
    for (int part = 0; part < WM * PARTS; ++part) {
      if (part % PARTS == 0) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        static_for<WM>([&](auto m_) __attribute__((always_inline)) {
          constexpr int m = decltype(m_)::value;
          if (part / PARTS == m) {
            int* e = ep + l32 * PITCH;
#pragma unroll
            for (int ni = 0; ni < WN; ++ni)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const i32x16& v = acc[m][ni];
                *reinterpret_cast<i32x4*>(e + ni * 32 + 8 * q + 4 * g) =
                    i32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
              }
            if (g == 0) *reinterpret_cast<float2*>(e + LN) = make_float2(x[m].m, __int_as_float(x[m].e));
          }
        });
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      const int line = part * PL * RPL;  // of the wave's
      // (every read of the part is on its way before the first is used)
      i32x4 s0[PL][2], s1[GATED ? PL : 1][2];
      LineScale xr[PL];
      Raw8<T> now[PL];
#pragma unroll
      for (int v = 0; v < PL; ++v) {
        const int* row = ep + (line % 32 + lane / LPR + v * RPL) * PITCH;
        const float2 xs = *reinterpret_cast<const float2*>(row + LN);
        xr[v] = {xs.x, __float_as_int(xs.y)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s0[v][h] = *reinterpret_cast<const i32x4*>(row + cl + 4 * h);
          if constexpr (GATED) s1[v][h] = *reinterpret_cast<const i32x4*>(row + LN / 2 + cl + 4 * h);
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
      if (part + 1 < WM * PARTS) load_residual<T, PL, RPL>(p, i00 + line + PL * RPL, j, nj, res);
      finish_lines<T, GATED, PL, RPL>(p, i00 + line, j, nj, z0, z1, now);
    }
  };
  __syncthreads();  // the last fragments are read: LDS becomes the epilogue's
  if (p.out_dtype == 0) finish(uint16_t{});
  else finish(float{});
}

template <bool GATED, int WM, int WN>
static void go_tile(const GemmArgs& a, hipStream_t s) {
  constexpr int tm = 64 * WM, out = GATED ? 32 * WN : 64 * WN;
  const int gm = (int)((a.M + tm - 1) / tm), gn = (int)((a.N + out - 1) / out);
  hipLaunchKernelGGL((int8_tile_kernel<GATED, WM, WN>), dim3((unsigned)(gm * gn)), dim3(256), 0, s, a, gm, gn);
}
template <bool GATED>
static void launch_tile_t(const GemmArgs& a, int WM, hipStream_t s) {
  if (WM == 4) go_tile<GATED, 4, 4>(a, s);
  else if (WM == 2) go_tile<GATED, 2, 2>(a, s);
  else go_tile<GATED, 1, 2>(a, s);
}

// WM: 4 (256 x 256 tiles), 2 (128 x 128) or 1 (64 x 128)
void launch_int8_tile(const GemmArgs& a, int WM, hipStream_t s) {
  if (a.act == ACT_SWIGLU) launch_tile_t<true>(a, WM, s);
  else launch_tile_t<false>(a, WM, s);
}

}  // namespace nvfp4
