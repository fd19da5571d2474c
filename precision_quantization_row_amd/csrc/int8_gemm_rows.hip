// int8_gemm_rows.hip -- the product of 8-bit integer lines for few lines of A
// (gfx950).
#include "gemm_device.h"

namespace nvfp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// For few lines of A (tokens) the product is bound by reading B. A workgroup
// owns 16 NT lines of B and 16 MT lines of A; its 8 waves take the units of 128
// k in turn, so that the workgroup reads runs of 1 KB of each line and no
// workspace is needed: the waves' sums, exact integers, meet in LDS. Bytes go
// straight from memory into the lanes that hold them as matrix fragments: lane
// l has line l % 16 and bytes 32 (l / 16) .. + 31 of the unit, both operands
// alike, so the sum covers every k once.
constexpr int RW = 8;  // waves

template <bool GATED, int MT, int NT>
__global__ void __launch_bounds__(RW * 64) int8_few_kernel(const GemmArgs p, unsigned gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int PITCH = NT * 16 + 4, OT = GATED ? NT / 2 : NT, PD = MT == 1 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) int part[RW][MT * 16 * PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const int64_t i0 = (int64_t)(blockIdx.x / gn) * (16 * MT), j0 = (int64_t)(blockIdx.x % gn) * (16 * OT);
  const int K = (int)p.K;
  const int am = (int)min(p.M - i0, (int64_t)(16 * MT)) - 1, bm = (int)min(p.N - j0, (int64_t)(16 * OT)) - 1;
  const uint8_t *qa = p.a.q + i0 * K, *qb = p.b.q + j0 * K;
  const uint8_t* qu = GATED ? qb + p.N * K : qb;
  // this lane's lines, from the tile's first (lines past the matrix repeat its
  // last one; their products are not stored)
  uint32_t ao[MT], bo[NT];
#pragma unroll
  for (int t = 0; t < MT; ++t) ao[t] = (uint32_t)min(16 * t + l16, am) * K + 32 * g;
#pragma unroll
  for (int t = 0; t < NT; ++t) bo[t] = (uint32_t)min(16 * (t % OT) + l16, bm) * K + 32 * g;
  struct Unit {
    u32x4 a[MT][2], b[NT][2];
  } ring[PD];
  // Unit u; past the lines' end zeros.
  auto fetch = [&](Unit& r, int u) __attribute__((always_inline)) {
    const int k = 128 * u;
    if (k + 128 <= K) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          r.b[t][h] = *reinterpret_cast<const u32x4_a1*>((GATED && t >= OT ? qu : qb) + k + 16 * h + bo[t]);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) r.a[t][h] = *reinterpret_cast<const u32x4_a1*>(qa + k + 16 * h + ao[t]);
    } else {
      const int kc = k + 32 * g;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const int at = kc + 4 * d;
#pragma unroll
        for (int t = 0; t < NT; ++t)
          r.b[t][d / 4][d & 3] =
              keep_bytes(tail_dword((GATED && t >= OT ? qu : qb) + bo[t] - 32 * g, K, at), K - at);
#pragma unroll
        for (int t = 0; t < MT; ++t)
          r.a[t][d / 4][d & 3] = keep_bytes(tail_dword(qa + ao[t] - 32 * g, K, at), K - at);
      }
    }
  };
  i32x4 acc[MT][NT] = {};
  auto multiply = [&](const Unit& r) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, r.b[n][h]),
                                                            __builtin_bit_cast(i32x4, r.a[m][h]), acc[m][n], 0, 0, 0);
  };
  const int nu = (K + 127) / 128;
  static_for<PD>([&](auto i) __attribute__((always_inline)) {
    constexpr int I = decltype(i)::value;
    if (wave + RW * I < nu) fetch(ring[I], wave + RW * I);
  });
#pragma unroll 1
  for (int u = wave; u < nu; u += RW * PD)
    static_for<PD>([&](auto i) __attribute__((always_inline)) {
      constexpr int I = decltype(i)::value;
      if (u + RW * I < nu) {
        multiply(ring[I]);
        if (u + RW * (I + PD) < nu) fetch(ring[I], u + RW * (I + PD));
      }
    });
  // register r of a 16 x 16 result: line l16 of A, line 4 g + r of B
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<i32x4*>(&part[wave][(16 * m + l16) * PITCH + 16 * n + 4 * g]) = acc[m][n];
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
  int s0[8] = {}, s1[8] = {};
#pragma unroll 4  // (all sums in flight would cost the main loop its waves)
  for (int w = 0; w < RW; ++w) {
    const i32x4* q = reinterpret_cast<const i32x4*>(&part[w][r * PITCH + cl]);
#pragma unroll
    for (int x = 0; x < 8; ++x) s0[x] += q[x / 4][x % 4];
    if constexpr (GATED) {
      const i32x4* qg = reinterpret_cast<const i32x4*>(&part[w][r * PITCH + 16 * OT + cl]);
#pragma unroll
      for (int x = 0; x < 8; ++x) s1[x] += qg[x / 4][x % 4];
    }
  }
  float z0[1][8] = {}, z1[1][8] = {};
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    z0[0][x] = apply_scale((float)s0[x], xs, w0[x]) + b0[x];
    if constexpr (GATED) z1[0][x] = apply_scale((float)s1[x], xs, w1[x]) + b1[x];
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

template <bool GATED, int MT, int NT>
static void go_rows(const GemmArgs& a, hipStream_t s) {
  constexpr int OT = GATED ? NT / 2 : NT;
  const unsigned gn = (unsigned)((a.N + 16 * OT - 1) / (16 * OT));
  const unsigned gm = (unsigned)((a.M + 16 * MT - 1) / (16 * MT));  // (few_lines bounds gm gn)
  hipLaunchKernelGGL((int8_few_kernel<GATED, MT, NT>), dim3(gm * gn), dim3(RW * 64), 0, s, a, gn);
}

// The tile of a few-lines launch: narrower ones where wide ones leave CUs without
// a workgroup.
template <bool GATED>
static void launch_rows_t(const GemmArgs& a, hipStream_t s) {
  const int64_t mt = (a.M + 15) / 16;
  auto groups = [&](int m, int n) {
    const int ot = GATED ? n / 2 : n;
    return ((mt + m - 1) / m) * ((a.N + 16 * ot - 1) / (16 * ot));
  };
  if (mt <= 1) {
    if (GATED || groups(1, 2) >= 256) return go_rows<GATED, 1, 2>(a, s);
    return go_rows<GATED, 1, GATED ? 2 : 1>(a, s);
  }
  if (mt <= 2) return go_rows<GATED, 2, 2>(a, s);
  if (groups(4, 4) >= 256) return go_rows<GATED, 4, 4>(a, s);
  return go_rows<GATED, 4, 2>(a, s);
}

void launch_int8_rows_gemm(const GemmArgs& a, hipStream_t s) {
  if (a.act == ACT_SWIGLU) launch_rows_t<true>(a, s);
  else launch_rows_t<false>(a, s);
}

}  // namespace nvfp4
