// int8_gemm_rows.hip -- the product of 8-bit integer lines for few lines of A
// (gfx950).
#include "int8_device.h"

namespace nvfp4 {

// For few lines of A (tokens) the product is bound by reading B. Up to four lines take
// int8_vec_kernel, more int8_few_kernel:
// A workgroup owns 16 NT lines of B and 16 MT lines of A; its 8 waves take the units of 128
// k in turn, so that the workgroup reads runs of 1 KB of each line and no
// workspace is needed: the waves' sums, exact integers, meet in LDS. A matrix
// fragment has 16 lines side by side in a wave's lanes; loaded so, each lane's 16
// bytes are a request of their own (16 bytes a cycle and CU). So 8 lanes load 128 bytes of a
// line, and the unit changes its order in the wave's own piece of LDS, where
// nothing but the wave itself has to be waited for (128 x 4096 x 4096 14.0 -> 10.3 us,
// 8 x 8191 x 8191 41 -> 17, 16 x 28672 x 8192 gated 102 -> 81, past the caches 72:
// 6.5 TB/s).
constexpr int RW = 8;  // waves

// The factors and biases of 8 consecutive outputs of a line, and the outputs from their sums.
template <bool GATED>
struct Factors {
  LineScale xs, w0[8], w1[8];
  float b0[8], b1[8];
  __device__ __forceinline__ void load(const GemmArgs& p, int64_t i, int64_t j) {
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
};
template <bool GATED>
__device__ __forceinline__ void finish_run(const GemmArgs& p, int64_t i, int64_t j, int64_t nj, const Factors<GATED>& f,
                                           const int (&s0)[8], const int (&s1)[8]) {
  float z0[1][8] = {}, z1[1][8] = {};
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    z0[0][x] = apply_scale((float)s0[x], f.xs, f.w0[x]) + f.b0[x];
    if constexpr (GATED) z1[0][x] = apply_scale((float)s1[x], f.xs, f.w1[x]) + f.b1[x];
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

template <bool GATED, int MT, int NT, bool PAST>
__global__ void __launch_bounds__(RW * 64) int8_few_kernel(const GemmArgs p, unsigned gn) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int PITCH = NT * 16 + 4, OT = GATED ? NT / 2 : NT, PD = 2;
  constexpr int UNIT = (NT + MT) * 16 * 128, PART = MT * 16 * PITCH * 4;  // bytes a wave
  __shared__ __attribute__((aligned(16))) uint8_t lds[RW * (UNIT > PART ? UNIT : PART)];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const int64_t i0 = (int64_t)(blockIdx.x / gn) * (16 * MT), j0 = (int64_t)(blockIdx.x % gn) * (16 * OT);
  const int K = (int)p.K;
  const int am = (int)min(p.M - i0, (int64_t)(16 * MT)) - 1, bm = (int)min(p.N - j0, (int64_t)(16 * OT)) - 1;
  const uint8_t *qa = p.a.q + i0 * K, *qb = p.b.q + j0 * K;
  const uint8_t* qu = GATED ? qb + p.N * K : qb;
  // Access t of a unit: this lane's chunk of line 8 t + lane / 8. Offsets are from the
  // tile's first line; lines past the matrix repeat its last one (their products are not
  // stored).
  auto line_at = [&](int t) { return 8 * t + lane / 8; };
  const int byte = 16 * (lane % 8);
  uint32_t ao[2 * MT], bo[2 * NT];
#pragma unroll
  for (int t = 0; t < 2 * MT; ++t) ao[t] = (uint32_t)min(line_at(t), am) * K + byte;
#pragma unroll
  for (int t = 0; t < 2 * NT; ++t) bo[t] = (uint32_t)min(line_at(t % (2 * OT)), bm) * K + byte;
  struct Unit {
    u32x4 a[2 * MT], b[2 * NT];
  } ring[PD];
  // Unit u; past the lines' end zeros.
  auto fetch = [&](Unit& r, int u) __attribute__((always_inline)) {
    const int k = 128 * u;
    if (k + 128 <= K) {
#pragma unroll
      for (int t = 0; t < 2 * NT; ++t) {
        const u32x4_a1* q = reinterpret_cast<const u32x4_a1*>((GATED && t >= 2 * OT ? qu : qb) + k + bo[t]);
        r.b[t] = PAST ? __builtin_nontemporal_load(q) : *q;
      }
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t)
        r.a[t] = *reinterpret_cast<const u32x4_a1*>(qa + k + ao[t]);
    } else {
#pragma unroll
      for (int t = 0; t < 2 * NT; ++t)
        r.b[t] = tail_chunk((GATED && t >= 2 * OT ? qu : qb) + bo[t] - byte, K, k + byte);
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) r.a[t] = tail_chunk(qa + ao[t] - byte, K, k + byte);
    }
  };
  i32x4 acc[MT][NT] = {};
  uint8_t* own = lds + wave * UNIT;  // B's lines, then A's
  uint8_t* to = own + (lane / 8) * 128;
  const uint8_t* from = own + l16 * 128;
  auto multiply = [&](const Unit& r) __attribute__((always_inline)) {
    // (a wave's LDS accesses are done in order: the last unit's reads precede)
#pragma unroll
    for (int t = 0; t < 2 * (NT + MT); ++t)
      *reinterpret_cast<u32x4*>(to + t * 1024 + 16 * ((lane % 8) ^ rotate(8 * t + lane / 8))) =
          t < 2 * NT ? r.b[t < 2 * NT ? t : 0] : r.a[t < 2 * NT ? 0 : t - 2 * NT];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 b[NT], a[MT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        b[n] = *reinterpret_cast<const i32x4*>(from + n * 2048 + 16 * ((4 * h + g) ^ rotate(l16)));
#pragma unroll
      for (int m = 0; m < MT; ++m)
        a[m] = *reinterpret_cast<const i32x4*>(from + (NT + m) * 2048 + 16 * ((4 * h + g) ^ rotate(l16)));
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[n], a[m], acc[m][n], 0, 0, 0);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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
  __syncthreads();  // the units' LDS becomes the sums'
  int(*part)[MT * 16 * PITCH] = reinterpret_cast<int(*)[MT * 16 * PITCH]>(lds);
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
  Factors<GATED> f;
  if (live) f.load(p, i, j);
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
  finish_run<GATED>(p, i, j, nj, f, s0, s1);
}

// For one to MV lines of A, a token or a few: a wave reads R lines of B as they lie, 1 KB
// of each at a time, and multiplies on the vector units, four products an instruction:
// no matrix fragment, so nothing has to change its order. A workgroup owns 4 R lines of
// B (gated: half of them up lines); four of its waves take the units of 1024 k that are
// even, four the others. A lane's sums are of its own 16 bytes in every KB; the lanes'
// sums meet by DPP, the two waves' in LDS. 28672 x 8192: one line 42 us, 5.6 TB/s, two 38,
// four 43 (the matrix kernel 54 for any; eight lines here 68); 8191 x 8191, one line: 13.6.
template <bool GATED, int MV, int R, bool NT>
__global__ void __launch_bounds__(512) int8_vec_kernel(const GemmArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int OUT = GATED ? 2 * R : 4 * R, KW = 1024, PD = MV > 2 ? 1 : 2;
  __shared__ int part[2][MV][4 * R];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lw = wave & 3, kw = wave >> 2, K = (int)p.K, M = (int)p.M;
  const int64_t j0 = (int64_t)blockIdx.x * OUT;
  const uint8_t* line[R];  // past the matrix: its last line (its product is not stored)
#pragma unroll
  for (int n = 0; n < R; ++n) {
    const int at = R * lw + n;
    const bool up = GATED && at >= OUT;
    line[n] = p.b.q + ((up ? p.N : 0) + min(j0 + (up ? at - OUT : at), p.N - 1)) * K;
  }
  struct Unit {
    u32x4 a[MV], b[R];
  } ring[PD];
  auto fetch = [&](Unit& r, int u) __attribute__((always_inline)) {
    const int k = KW * u;
    const uint32_t at = 16 * lane;
    if (k + KW <= K) {
#pragma unroll
      for (int n = 0; n < R; ++n)
        r.b[n] = NT ? __builtin_nontemporal_load(reinterpret_cast<const u32x4_a1*>(line[n] + k + at))
                    : *reinterpret_cast<const u32x4_a1*>(line[n] + k + at);
#pragma unroll
      for (int m = 0; m < MV; ++m)
        r.a[m] = *reinterpret_cast<const u32x4_a1*>(p.a.q + (int64_t)min(m, M - 1) * K + k + at);
    } else {
#pragma unroll
      for (int n = 0; n < R; ++n) r.b[n] = tail_chunk(line[n], K, k + at);
#pragma unroll
      for (int m = 0; m < MV; ++m) r.a[m] = tail_chunk(p.a.q + (int64_t)min(m, M - 1) * K, K, k + at);
    }
  };
  int acc[MV][R] = {};
  const int nu = (K + KW - 1) / KW;
  static_for<PD>([&](auto i) __attribute__((always_inline)) {
    constexpr int I = decltype(i)::value;
    if (kw + 2 * I < nu) fetch(ring[I], kw + 2 * I);
  });
#pragma unroll 1
  for (int u = kw; u < nu; u += 2 * PD)
    static_for<PD>([&](auto i) __attribute__((always_inline)) {
      constexpr int I = decltype(i)::value;
      if (u + 2 * I < nu) {
#pragma unroll
        for (int m = 0; m < MV; ++m)
#pragma unroll
          for (int n = 0; n < R; ++n)
#pragma unroll
            for (int d = 0; d < 4; ++d)
              acc[m][n] = __builtin_amdgcn_sdot4((int)ring[I].b[n][d], (int)ring[I].a[m][d], acc[m][n], false);
        if (u + 2 * (I + PD) < nu) fetch(ring[I], u + 2 * (I + PD));
      }
    });
  const int r = tid / (OUT / 8), cl = 8 * (tid % (OUT / 8));
  const int64_t j = j0 + cl, nj = p.N - j;
  const bool live = r < MV && r < M && nj > 0;
  Factors<GATED> f;
  if (live) f.load(p, r, j);
#pragma unroll
  for (int m = 0; m < MV; ++m)
#pragma unroll
    for (int n = 0; n < R; ++n) {
      const int s = lanes_sum_int(acc[m][n]);
      if (lane == 0) part[kw][m][R * lw + n] = s;
    }
  __syncthreads();
  if (!live) return;
  int s0[8], s1[8] = {};
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    s0[x] = part[0][r][cl + x] + part[1][r][cl + x];
    if constexpr (GATED) s1[x] = part[0][r][OUT + cl + x] + part[1][r][OUT + cl + x];
  }
  finish_run<GATED>(p, r, j, nj, f, s0, s1);
}

// B of 128 MB, half the memory-side cache, and more is read past the caches: what a model
// reads once a token is not there any more when the next token comes. (Taken side
// by side: 1 x 28672 x 8192 40 -> 38 us, gated 80 -> 71; 8 lines, gated, 79 -> 70; but
// 1 x 4096 x 14336, 59 MB and read again soon, 11 -> 13.)
static bool past_caches(const GemmArgs& a) { return (a.act == ACT_SWIGLU ? 2 : 1) * a.N * a.K >= (int64_t)128 << 20; }

template <bool GATED, int MT, int NT>
static void go_rows(const GemmArgs& a, hipStream_t s) {
  constexpr int OT = GATED ? NT / 2 : NT;
  const unsigned gn = (unsigned)((a.N + 16 * OT - 1) / (16 * OT));
  const unsigned gm = (unsigned)((a.M + 16 * MT - 1) / (16 * MT));  // (few lines, or few tiles: gm gn is at most 2^22)
  if (past_caches(a)) hipLaunchKernelGGL((int8_few_kernel<GATED, MT, NT, true>), dim3(gm * gn), dim3(RW * 64), 0, s, a, gn);
  else hipLaunchKernelGGL((int8_few_kernel<GATED, MT, NT, false>), dim3(gm * gn), dim3(RW * 64), 0, s, a, gn);
}

template <bool GATED, int MV, int R>
static void go_vec(const GemmArgs& a, hipStream_t s) {
  constexpr int OUT = GATED ? 2 * R : 4 * R;
  const dim3 g((unsigned)((a.N + OUT - 1) / OUT)), b(512);
  if (past_caches(a))
    hipLaunchKernelGGL((int8_vec_kernel<GATED, MV, R, true>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((int8_vec_kernel<GATED, MV, R, false>), g, b, 0, s, a);
}

// The tile of a few-lines launch. 5 to 16 lines, not gated, take 16 lines of B a workgroup
// where 32 leave CUs without one; others always take the widest that their lines of A
// allow, and up to four lines 16 of B.
template <bool GATED>
static void launch_rows_t(const GemmArgs& a, hipStream_t s) {
  const int64_t mt = (a.M + 15) / 16;
  auto groups = [&](int m, int n) {
    const int ot = GATED ? n / 2 : n;
    return ((mt + m - 1) / m) * ((a.N + 16 * ot - 1) / (16 * ot));
  };
  if (a.N <= (int64_t)1 << 25) {  // (a launch holds fewer than 2^32 threads)
    if (a.M == 1) return go_vec<GATED, 1, 4>(a, s);
    if (a.M == 2) return go_vec<GATED, 2, 4>(a, s);
    if (a.M <= 4) return go_vec<GATED, 4, 4>(a, s);
  }
  if (mt <= 1) {
    if (GATED || groups(1, 2) >= 256) return go_rows<GATED, 1, 2>(a, s);
    return go_rows<GATED, 1, GATED ? 2 : 1>(a, s);
  }
  if (mt <= 2) return go_rows<GATED, 2, 2>(a, s);
  return go_rows<GATED, 4, 2>(a, s);
}

void launch_int8_rows_gemm(const GemmArgs& a, hipStream_t s) {
  if (a.act == ACT_SWIGLU) launch_rows_t<true>(a, s);
  else launch_rows_t<false>(a, s);
}

}  // namespace nvfp4
