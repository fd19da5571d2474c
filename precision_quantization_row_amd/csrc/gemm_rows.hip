// gemm_rows.hip -- the packed product for few lines of A (gfx950).
#include "gemm_device.h"

namespace nvfp4 {

// ---------------------------------------------------------- few-lines kernel
// For few lines of A (tokens) the product is bound by reading B. A workgroup
// owns 16 NT lines of B and 16 MT lines of A; its 8 waves split k into runs of
// whole quads, so that a launch of a few hundred workgroups has all of B's
// bytes on their way at once and no workspace is needed: the waves' sums meet
// in LDS, in a fixed order. Codes go straight from memory into the lanes that
// hold them as matrix fragments (lane l: line l % 16, chunk l / 16 of the 64
// bytes, or 128, that a unit of 128 k takes). A quad is 4 units: a lane would
// load its block scales 2 bytes at a time, which costs the memory pipe as much
// as the codes' 16 (3.0 against 4.6 TB/s at 1 x 8192 x 28672 without them), so
// the wave loads the 32 scale bytes of each line of a quad in whole and hands
// them out through its own piece of LDS. Measured: 1 x 57344 x 8192 (E4M3 A) 53-56
// us, 4.7-5.0 TB/s; 16 lines, gated, the same size 74 us, where each workgroup's
// own read of A costs 10; 1 x 4096 x 4096 5.6 us, which is latency; 128 x 4096 x 4096
// 11.3 us, two latencies one after the other, as a wave has 4 units of k and 2 on
// their way; 256 x 8192 x 8192 49 us, which is decode (702 TFLOP/s).

// The block scales of 16 T lines for one quad, as one wave loads them: 8 bytes
// a lane (T = 1) or T / 2 times 16.
constexpr int RW = 8;  // waves

template <int T>
struct QuadScales {
  static constexpr int PIECES = T == 1 ? 1 : T / 2, DW = T == 1 ? 2 : 4, PER = 8 / DW;
  uint32_t off[PIECES];  // of this lane's line, from the tile's first
  bool up[PIECES];       // it is one of the up lines
  uint32_t w[2][PIECES][DW];  // of even and odd quads
  // line(r): offset of the tile's row r; whether it is an up line
  template <typename F>
  __device__ __forceinline__ void init(int lane, F line) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) off[i] = line(i * (64 / PER) + lane / PER, up[i]);
  }
  template <int H>
  __device__ __forceinline__ void load(const uint8_t* s, const uint8_t* su, int lane, int q, int sp) {
    const int at = 32 * q + 4 * DW * (lane % PER);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const uint8_t* l = (up[i] ? su : s) + off[i];
      if (32 * (q + 1) <= sp) {
        if constexpr (DW == 2) {
          const u32x2 v = *reinterpret_cast<const u32x2_a1*>(l + at);
          w[H][i][0] = v.x; w[H][i][1] = v.y;
        } else {
          const u32x4 v = *reinterpret_cast<const u32x4_a1*>(l + at);
          w[H][i][0] = v.x; w[H][i][1] = v.y; w[H][i][2] = v.z; w[H][i][3] = v.w;
        }
      } else {
#pragma unroll
        for (int d = 0; d < DW; ++d) w[H][i][d] = keep_bytes(tail_dword(l, sp, at + 4 * d), sp - at - 4 * d);
      }
    }
  }
  template <int H>
  __device__ __forceinline__ void put(uint8_t* lds, int lane) const {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      uint8_t* d = lds + (i * (64 / PER) + lane / PER) * 32 + 4 * DW * (lane % PER);
      if constexpr (DW == 2) *reinterpret_cast<u32x2*>(d) = u32x2{w[H][i][0], w[H][i][1]};
      else *reinterpret_cast<u32x4*>(d) = u32x4{w[H][i][0], w[H][i][1], w[H][i][2], w[H][i][3]};
    }
  }
};

template <bool A8, bool GATED, int MT, int NT>
__global__ void __launch_bounds__(RW * 64) gemm_rows_kernel(const GemmArgs p, unsigned gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int PITCH = NT * 16 + 4, OT = GATED ? NT / 2 : NT, PD = MT == 1 ? 4 : 2;
  constexpr int SROWS = 16 * (A8 ? NT : NT + MT);  // lines with scales
  constexpr int PART = RW * MT * 16 * PITCH * 4, SCALES = RW * SROWS * 32;
  __shared__ __attribute__((aligned(16))) uint8_t lds[PART > SCALES ? PART : SCALES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const int64_t i0 = (int64_t)(blockIdx.x / gn) * (16 * MT), j0 = (int64_t)(blockIdx.x % gn) * (16 * OT);
  const int K = (int)p.K, qp = (K + 1) / 2, sp = (K + 15) / 16, ap = A8 ? K : qp;
  const int am = (int)min(p.M - i0, (int64_t)(16 * MT)) - 1, bm = (int)min(p.N - j0, (int64_t)(16 * OT)) - 1;
  const uint8_t *qa = p.a.q + i0 * ap, *sa = A8 ? nullptr : p.a.s + i0 * sp;
  const uint8_t *qb = p.b.q + j0 * qp, *sb = p.b.s + j0 * sp;
  const uint8_t *qu = GATED ? qb + p.N * qp : qb, *su = GATED ? sb + p.N * sp : sb;
  // this lane's lines, from the tile's first (lines past the matrix repeat its
  // last one; their products are not stored)
  uint32_t ao[MT], bo[NT];
#pragma unroll
  for (int t = 0; t < MT; ++t) ao[t] = (uint32_t)min(16 * t + l16, am) * ap + (A8 ? 32 : 16) * g;
#pragma unroll
  for (int t = 0; t < NT; ++t) bo[t] = (uint32_t)min(16 * (t % OT) + l16, bm) * qp + 16 * g;
  QuadScales<NT> qsb;
  QuadScales<A8 ? 1 : MT> qsa;
  qsb.init(lane, [&](int r, bool& up) {
    up = GATED && r >= 16 * OT;
    return (uint32_t)min(r % (16 * OT), bm) * sp;
  });
  if constexpr (!A8)
    qsa.init(lane, [&](int r, bool& up) {
      up = false;
      return (uint32_t)min(r, am) * sp;
    });
  struct Unit {
    u32x4 a[MT][A8 ? 2 : 1], b[NT];
  } ring[PD];
  // Unit u; past the lines' end zeros. (The offsets include 16 g, 32 g.)
  auto fetch = [&](Unit& r, int u) __attribute__((always_inline)) {
    const int k = 128 * u;
    if (k + 128 <= K) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        r.b[t] = *reinterpret_cast<const u32x4_a1*>((GATED && t >= OT ? qu : qb) + k / 2 + bo[t]);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint8_t* q = qa + (A8 ? k : k / 2);
        r.a[t][0] = *reinterpret_cast<const u32x4_a1*>(q + ao[t]);
        if constexpr (A8) r.a[t][A8] = *reinterpret_cast<const u32x4_a1*>(q + 16 + ao[t]);
      }
    } else {
      const int kc = k + 32 * g;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          r.b[t][d] = keep_nibbles(
              tail_dword((GATED && t >= OT ? qu : qb) + bo[t] - 16 * g, qp, kc / 2 + 4 * d), K - kc - 8 * d);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const uint8_t* q = qa + ao[t] - (A8 ? 32 : 16) * g;
          if constexpr (A8) {
            r.a[t][0][d] = keep_bytes(tail_dword(q, ap, kc + 4 * d), K - kc - 4 * d);
            r.a[t][A8][d] = keep_bytes(tail_dword(q, ap, kc + 16 + 4 * d), K - kc - 16 - 4 * d);
          } else {
            r.a[t][0][d] = keep_nibbles(tail_dword(q, qp, kc / 2 + 4 * d), K - kc - 8 * d);
          }
        }
      }
    }
  };
  f32x4 acc[MT][NT] = {};
  uint8_t* ls = lds + wave * SROWS * 32;  // B's scales, then A's
  auto multiply = [&](const Unit& r, int u) __attribute__((always_inline)) {  // u: unit of its quad
    h2 bsc[NT], asc[MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
      bsc[t] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(
          *reinterpret_cast<const uint16_t*>(ls + (16 * t + l16) * 32 + 8 * u + 2 * g), 1.0f, false);
#pragma unroll
    for (int t = 0; t < MT; ++t)
      if constexpr (!A8)
        asc[t] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(
            *reinterpret_cast<const uint16_t*>(ls + (16 * (NT + t) + l16) * 32 + 8 * u + 2 * g), 1.0f, false);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      h8 a[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if constexpr (A8) a[t] = decode8_fp8(r.a[t][d >> 1 ? A8 : 0][(2 * d) & 3], r.a[t][d >> 1 ? A8 : 0][(2 * d + 1) & 3]);
        else a[t] = decode8_fp4(r.a[t][0][d], d < 2 ? asc[t].xx : asc[t].yy);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const h8 b = decode8_fp4(r.b[n][d], d < 2 ? bsc[n].xx : bsc[n].yy);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a[m], acc[m][n], 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);  // (decoded ahead, fragments would cost waves)
    }
  };
  // This wave's units u0 .. u1 - 1: whole quads, or, with PD 2, pairs where k is
  // too short for quads to reach all waves.
  const int nu = (K + 127) / 128, nq = (nu + 3) / 4, per = (nq + RW - 1) / RW;
  const bool pairs = PD < 4 && nu <= 2 * RW;
  const int q0 = pairs ? wave / 2 : wave * per, u0 = pairs ? 2 * wave : 4 * q0;
  const int u1 = min(nu, pairs ? u0 + 2 : 4 * (q0 + per));
  static_for<2>([&](auto i) __attribute__((always_inline)) {
    constexpr int h = decltype(i)::value;
    if ((PD >= 4 || u0 < u1) && 4 * (q0 + h) < u1) {
      qsb.template load<h>(sb, su, lane, q0 + h, sp);
      if constexpr (!A8) qsa.template load<h>(sa, sa, lane, q0 + h, sp);
    }
  });
  static_for<PD>([&](auto i) __attribute__((always_inline)) {
    if (u0 + decltype(i)::value < u1) fetch(ring[decltype(i)::value], u0 + decltype(i)::value);
  });
#pragma unroll 1
  for (int q2 = q0; (PD >= 4 || u0 < u1) && 4 * q2 < u1; q2 += 2)
    static_for<2>([&](auto h_) __attribute__((always_inline)) {
      constexpr int h = decltype(h_)::value;
      const int q = q2 + h;
      if (4 * q < u1) {
        // (a wave's LDS accesses are done in order: the last quad's reads precede)
        qsb.template put<h>(ls, lane);
        if constexpr (!A8) qsa.template put<h>(ls + NT * 512, lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (4 * (q + 2) < u1) {
          qsb.template load<h>(sb, su, lane, q + 2, sp);
          if constexpr (!A8) qsa.template load<h>(sa, sa, lane, q + 2, sp);
        }
        static_for<4>([&](auto i) __attribute__((always_inline)) {
          constexpr int s = decltype(i)::value, r = (4 * h + s) % PD;
          const int u = 4 * q + s;
          if ((PD >= 4 || u >= u0) && u < u1) {  // (PD 4: u0 begins a quad)
            multiply(ring[r], s);
            if (u + PD < u1) fetch(ring[r], u + PD);
          }
        });
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
    });
  __syncthreads();  // the scales' LDS becomes the sums'
  float(*part)[MT * 16 * PITCH] = reinterpret_cast<float(*)[MT * 16 * PITCH]>(lds);
  // register r of a 16 x 16 result: line l16 of A, line 4 g + r of B
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<f32x4*>(&part[wave][(16 * m + l16) * PITCH + 16 * n + 4 * g]) = acc[m][n];
  // 8 consecutive outputs a thread; their factors and biases are loaded while
  // the waves meet
  constexpr int LPR = 2 * OT;
  static_assert(16 * MT * LPR <= RW * 64, "one run of outputs a thread");
  const int r = tid / LPR, cl = 8 * (tid % LPR);
  const int64_t i = i0 + r, j = j0 + cl, nj = p.N - j;
  const bool live = r < 16 * MT && i < p.M && nj > 0;
  LineScale xs, w0[8], w1[8];
  float b0[8], b1[8];
  if (live) {
    xs = line_scale(p.a, i);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int64_t jj = min(j + x, p.N - 1);
      w0[x] = line_scale(p.b, jj);
      b0[x] = load_bias(p, jj);
      if constexpr (GATED) {
        w1[x] = line_scale(p.b, p.N + jj);
        b1[x] = load_bias(p, p.N + jj);
      }
    }
  }
  __syncthreads();
  if (!live) return;
  float z0[1][8] = {}, z1[1][8] = {};
#pragma unroll 4  // (all sums in flight would cost the main loop its waves)
  for (int w = 0; w < RW; ++w) {
    const f32x4* q = reinterpret_cast<const f32x4*>(&part[w][r * PITCH + cl]);
#pragma unroll
    for (int x = 0; x < 8; ++x) z0[0][x] += q[x / 4][x % 4];
    if constexpr (GATED) {
      const f32x4* qg = reinterpret_cast<const f32x4*>(&part[w][r * PITCH + 16 * OT + cl]);
#pragma unroll
      for (int x = 0; x < 8; ++x) z1[0][x] += qg[x / 4][x % 4];
    }
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    z0[0][x] = apply_scale(z0[0][x], xs, w0[x]) + b0[x];
    if constexpr (GATED) z1[0][x] = apply_scale(z1[0][x], xs, w1[x]) + b1[x];
  }
  auto finish = [&](auto type_) __attribute__((always_inline)) {
    using T = decltype(type_);
    Raw8<T> res[1];
    load_residual<T, 1, 0>(p, i, j, nj, res);
    finish_lines<T, GATED, 1, 0>(p, i, j, nj, z0, z1, res);
  };
  if (p.out_dtype == 0) finish(uint16_t{});
  else finish(float{});
}

template <bool A8, bool GATED, int MT, int NT>
static void go_rows(const GemmArgs& a, hipStream_t s) {
  constexpr int OT = GATED ? NT / 2 : NT;
  const unsigned gn = (unsigned)((a.N + 16 * OT - 1) / (16 * OT));
  const unsigned gm = (unsigned)((a.M + 16 * MT - 1) / (16 * MT));  // (few_lines bounds gm gn)
  hipLaunchKernelGGL((gemm_rows_kernel<A8, GATED, MT, NT>), dim3(gm * gn), dim3(RW * 64), 0, s, a, gn);
}

// The tile of a few-lines launch. Up to 16 lines of A: 32 lines of B, or 16 if
// that leaves CUs without a workgroup (1 x 57344 x 8192: 32 lines with 4 units on
// their way 54 us, 64 with 2 64 us, 64 with 4 73 us: the registers cost it the
// second workgroup of a CU). Up to 32: 32 by 32. More: 64 by 64, or by 32 if 64
// leaves CUs without a workgroup.
template <bool A8, bool GATED>
static void launch_rows_t(const GemmArgs& a, hipStream_t s) {
  const int64_t mt = (a.M + 15) / 16;
  auto groups = [&](int m, int n) {
    const int ot = GATED ? n / 2 : n;
    return ((mt + m - 1) / m) * ((a.N + 16 * ot - 1) / (16 * ot));
  };
  if (mt <= 1) {
    if (GATED || groups(1, 2) >= 256) return go_rows<A8, GATED, 1, 2>(a, s);
    return go_rows<A8, GATED, 1, GATED ? 2 : 1>(a, s);
  }
  if (mt <= 2) return go_rows<A8, GATED, 2, 2>(a, s);
  if (groups(4, 4) >= 256) return go_rows<A8, GATED, 4, 4>(a, s);
  return go_rows<A8, GATED, 4, 2>(a, s);
}

void launch_gemm_rows(const GemmArgs& a, hipStream_t s) {
  const bool gated = a.act == ACT_SWIGLU, a8 = a.a.s == nullptr;
  if (a8 && gated) launch_rows_t<true, true>(a, s);
  else if (a8) launch_rows_t<true, false>(a, s);
  else if (gated) launch_rows_t<false, true>(a, s);
  else launch_rows_t<false, false>(a, s);
}

}  // namespace nvfp4
