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
#include <type_traits>
#include <utility>

namespace nvfp4 {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int... I, typename F>
__device__ __forceinline__ void static_for_(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(0), f(1), ..., f(N - 1) with the index a constant
template <int N, typename F>
__device__ __forceinline__ void static_for(F f) {
  static_for_(std::make_integer_sequence<int, N>{}, f);
}

// ------------------------------------------------------------------ decode
// Pair P of a dword's 4 pairs of codes (of its 2 pairs of E4M3 bytes).
template <int P>
__device__ __forceinline__ h2 cvt_fp4(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, P);
}
template <int P>
__device__ __forceinline__ h2 cvt_fp8(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, P != 0);
}
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
// 8 consecutive outputs, from column j on, of each of the lines i, i + STEP,
// .., i + (NL - 1) STEP; nj columns (8 or more: all) and the lines below M
// are in the matrix. z0: pre-activations (the gate's, if gated), z1: the up
// lines'; both with their bias.
template <typename T, bool GATED, int NL, int STEP>
__device__ __forceinline__ void finish_lines(const GemmArgs& p, int64_t i, int64_t j, int64_t nj,
                                             float (&z0)[NL][8], float (&z1)[NL][8]) {
  if (nj <= 0) return;
  Raw8<T> res[NL];
  if (p.residual) {
#pragma unroll
    for (int v = 0; v < NL; ++v)
      if (i + v * STEP < p.M)
        load8_raw(static_cast<const T*>(p.residual) + (i + v * STEP) * p.N + j, nj, res[v]);
  }
  if (p.z) {
#pragma unroll
    for (int v = 0; v < NL; ++v)
      if (i + v * STEP < p.M) {
        T* z = static_cast<T*>(p.z) + (i + v * STEP) * (GATED ? 2 * p.N : p.N) + j;
        store8(z, nj, z0[v]);
        if constexpr (GATED) store8(z + p.N, nj, z1[v]);
      }
  }
  if constexpr (GATED) {
#pragma unroll
    for (int v = 0; v < NL; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) z0[v][e] = silu_f(z0[v][e]) * z1[v][e];
  } else if (p.act != ACT_NONE) {
#pragma unroll
    for (int v = 0; v < NL; ++v) act8(p.act, z0[v]);
  }
  if (p.residual) {
#pragma unroll
    for (int v = 0; v < NL; ++v) {
      float r[8];
      unpack8(res[v], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) z0[v][e] += r[e];
    }
  }
#pragma unroll
  for (int v = 0; v < NL; ++v)
    if (i + v * STEP < p.M) store8(static_cast<T*>(p.y) + (i + v * STEP) * p.N + j, nj, z0[v]);
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
// them out through its own piece of LDS.
constexpr int RW = 8;  // waves

// The block scales of 16 T lines for one quad, as one wave loads them: 8 bytes
// a lane (T = 1) or T / 2 times 16.
template <int T>
struct QuadScales {
  static constexpr int PIECES = T == 1 ? 1 : T / 2, DW = T == 1 ? 2 : 4, PER = 8 / DW;
  uint32_t off[PIECES];  // of this lane's line, from the tile's first
  bool up[PIECES];       // it is one of the up lines
  uint32_t w[PIECES][DW];
  // line(r): offset of the tile's row r; whether it is an up line
  template <typename F>
  __device__ __forceinline__ void init(int lane, F line) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) off[i] = line(i * (64 / PER) + lane / PER, up[i]);
  }
  __device__ __forceinline__ void load(const uint8_t* s, const uint8_t* su, int lane, int q, int sp) {
    const int at = 32 * q + 4 * DW * (lane % PER);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const uint8_t* l = (up[i] ? su : s) + off[i];
      if (32 * (q + 1) <= sp) {
        if constexpr (DW == 2) {
          const u32x2 v = *reinterpret_cast<const u32x2_a1*>(l + at);
          w[i][0] = v.x; w[i][1] = v.y;
        } else {
          const u32x4 v = *reinterpret_cast<const u32x4_a1*>(l + at);
          w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
        }
      } else {
#pragma unroll
        for (int d = 0; d < DW; ++d) w[i][d] = keep_bytes(tail_dword(l, sp, at + 4 * d), sp - at - 4 * d);
      }
    }
  }
  __device__ __forceinline__ void put(uint8_t* lds, int lane) const {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      uint8_t* d = lds + (i * (64 / PER) + lane / PER) * 32 + 4 * DW * (lane % PER);
      if constexpr (DW == 2) *reinterpret_cast<u32x2*>(d) = u32x2{w[i][0], w[i][1]};
      else *reinterpret_cast<u32x4*>(d) = u32x4{w[i][0], w[i][1], w[i][2], w[i][3]};
    }
  }
};

template <bool A8, bool GATED, int MT, int NT>
__global__ void __launch_bounds__(RW * 64) gemm_rows_kernel(const GemmArgs p) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int PITCH = NT * 16 + 4, OT = GATED ? NT / 2 : NT, PD = MT >= 2 ? 2 : NT >= 4 ? 2 : 4;
  constexpr int SROWS = 16 * (A8 ? NT : NT + MT);  // lines with scales
  constexpr int PART = RW * MT * 16 * PITCH * 4, SCALES = RW * SROWS * 32;
  __shared__ __attribute__((aligned(16))) uint8_t lds[PART > SCALES ? PART : SCALES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const int64_t i0 = (int64_t)blockIdx.y * (16 * MT), j0 = (int64_t)blockIdx.x * (16 * OT);
  const int K = (int)p.K, qp = (K + 1) / 2, sp = (K + 15) / 16, ap = A8 ? K : qp;
  const int am = (int)min(p.M - i0, (int64_t)(16 * MT)) - 1, bm = (int)min(p.N - j0, (int64_t)(16 * OT)) - 1;
  const uint8_t *qa = p.a.q + i0 * ap, *sa = A8 ? nullptr : p.a.s + i0 * sp;
  const uint8_t *qb = p.b.q + j0 * qp, *sb = p.b.s + j0 * sp;
  const uint8_t *qu = GATED ? qb + p.N * qp : qb, *su = GATED ? sb + p.N * sp : sb;
  // this lane's lines, from the tile's first (lines past the matrix repeat its
  // last one; their products are not stored)
  uint32_t ao[MT], bo[NT];
#pragma unroll
  for (int t = 0; t < MT; ++t) ao[t] = (uint32_t)min(16 * t + l16, am) * ap;
#pragma unroll
  for (int t = 0; t < NT; ++t) bo[t] = (uint32_t)min(16 * (t % OT) + l16, bm) * qp;
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
  auto fetch = [&](Unit& r, int u) {
    const int k = 128 * u, c = 32 * g;
    if (k + 128 <= K) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        r.b[t] = *reinterpret_cast<const u32x4_a1*>((GATED && t >= OT ? qu : qb) + k / 2 + (bo[t] + 16 * g));
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint8_t* q = qa + (A8 ? k : k / 2);
        if constexpr (A8) {
          r.a[t][0] = *reinterpret_cast<const u32x4_a1*>(q + (ao[t] + 32 * g));
          r.a[t][A8] = *reinterpret_cast<const u32x4_a1*>(q + (ao[t] + 32 * g + 16));
        } else {
          r.a[t][0] = *reinterpret_cast<const u32x4_a1*>(q + (ao[t] + 16 * g));
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint8_t* q = (GATED && t >= OT ? qu : qb) + bo[t];
#pragma unroll
        for (int d = 0; d < 4; ++d)
          r.b[t][d] = keep_nibbles(tail_dword(q, qp, (k + c) / 2 + 4 * d), K - k - c - 8 * d);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint8_t* q = qa + ao[t];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          if constexpr (A8) {
            r.a[t][0][d] = keep_bytes(tail_dword(q, ap, k + c + 4 * d), K - k - c - 4 * d);
            r.a[t][A8][d] = keep_bytes(tail_dword(q, ap, k + c + 16 + 4 * d), K - k - c - 16 - 4 * d);
          } else {
            r.a[t][0][d] = keep_nibbles(tail_dword(q, qp, (k + c) / 2 + 4 * d), K - k - c - 8 * d);
          }
        }
      }
    }
  };
  f32x4 acc[MT][NT] = {};
  uint8_t* ls = lds + wave * SROWS * 32;  // B's scales, then A's
  auto multiply = [&](const Unit& r, int u) {  // u: unit of its quad
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
    }
  };
  const int nu = (K + 127) / 128, nq = (nu + 3) / 4, per = (nq + RW - 1) / RW;
  const int q0 = wave * per, u1 = min(nu, 4 * (q0 + per));
  if (4 * q0 < u1) {
    qsb.load(sb, su, lane, q0, sp);
    if constexpr (!A8) qsa.load(sa, sa, lane, q0, sp);
  }
  static_for<PD>([&](auto i) {
    if (4 * q0 + decltype(i)::value < u1) fetch(ring[decltype(i)::value], 4 * q0 + decltype(i)::value);
  });
#pragma unroll 1
  for (int q = q0; 4 * q < u1; ++q) {
    // (a wave's LDS accesses are done in order: the last quad's reads precede)
    qsb.put(ls, lane);
    if constexpr (!A8) qsa.put(ls + NT * 512, lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (4 * (q + 1) < u1) {
      qsb.load(sb, su, lane, q + 1, sp);
      if constexpr (!A8) qsa.load(sa, sa, lane, q + 1, sp);
    }
    static_for<4>([&](auto i) {
      constexpr int s = decltype(i)::value;
      const int u = 4 * q + s;
      if (u < u1) {
        multiply(ring[s % PD], s);
        if (u + PD < u1) fetch(ring[s % PD], u + PD);
      }
    });
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  __syncthreads();  // the scales' LDS becomes the sums'
  float(*part)[MT * 16 * PITCH] = reinterpret_cast<float(*)[MT * 16 * PITCH]>(lds);
  // register r of a 16 x 16 result: line l16 of A, line 4 g + r of B
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<f32x4*>(&part[wave][(16 * m + l16) * PITCH + 16 * n + 4 * g]) = acc[m][n];
  __syncthreads();
  // 8 consecutive outputs a thread
  constexpr int LPR = 2 * OT;
#pragma unroll 1
  for (int e = tid; e < 16 * MT * LPR; e += RW * 64) {
    const int r = e / LPR, cl = 8 * (e % LPR);
    const int64_t i = i0 + r, j = j0 + cl, nj = p.N - j;
    if (i >= p.M || nj <= 0) continue;
    float z0[1][8] = {}, z1[1][8] = {};
#pragma unroll
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
    const LineScale xs = line_scale(p.a, i);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int64_t jj = min(j + x, p.N - 1);
      z0[0][x] = apply_scale(z0[0][x], xs, line_scale(p.b, jj)) + load_bias(p, jj);
      if constexpr (GATED)
        z1[0][x] = apply_scale(z1[0][x], xs, line_scale(p.b, p.N + jj)) + load_bias(p, p.N + jj);
    }
    if (p.out_dtype == 0) finish_lines<uint16_t, GATED, 1, 0>(p, i, j, nj, z0, z1);
    else finish_lines<float, GATED, 1, 0>(p, i, j, nj, z0, z1);
  }
}

template <bool A8, bool GATED, int MT, int NT>
static void go_rows(const GemmArgs& a, hipStream_t s) {
  constexpr int OT = GATED ? NT / 2 : NT;
  const dim3 grid((unsigned)((a.N + 16 * OT - 1) / (16 * OT)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((gemm_rows_kernel<A8, GATED, MT, NT>), grid, dim3(RW * 64), 0, s, a);
}

// Few-lines launch: 16 MT lines of A a workgroup, and the most lines of B that
// leave at least WG workgroups.
template <bool A8, bool GATED>
static void launch_rows(const GemmArgs& a, hipStream_t s) {
  const int64_t mt = (a.M + 15) / 16;
  auto groups = [&](int m, int n) {
    const int ot = GATED ? n / 2 : n;
    return ((mt + m - 1) / m) * ((a.N + 16 * ot - 1) / (16 * ot));
  };
  constexpr int WG = 256;
  if (mt <= 1) {
    if (groups(1, 4) >= WG) return go_rows<A8, GATED, 1, 4>(a, s);
    if (GATED || groups(1, 2) >= WG) return go_rows<A8, GATED, 1, 2>(a, s);
    return go_rows<A8, GATED, 1, GATED ? 2 : 1>(a, s);
  }
  if (mt <= 2) {
    if (groups(2, 4) >= WG) return go_rows<A8, GATED, 2, 4>(a, s);
    return go_rows<A8, GATED, 2, 2>(a, s);
  }
  if (groups(4, 4) >= WG) return go_rows<A8, GATED, 4, 4>(a, s);
  return go_rows<A8, GATED, 4, 2>(a, s);
}

int64_t gemm_workspace(int a_fmt, int64_t M, int64_t N, int64_t K, int act) {
  const int64_t gm = (M + TM - 1) / TM, gn = (N + TN / 2 - 1) / (TN / 2);
  if (K > ((int64_t)1 << 23) || N > ((int64_t)1 << 26) || gm * gn > ((int64_t)1 << 23)) return -1;
  return 0;
}

int launch_gemm(const GemmArgs& a, hipStream_t s) {
  const bool gated = a.act == ACT_SWIGLU, a8 = a.a.s == nullptr;
  if (a.M <= 256) {
    if (a8 && gated) launch_rows<true, true>(a, s);
    else if (a8) launch_rows<true, false>(a, s);
    else if (gated) launch_rows<false, true>(a, s);
    else launch_rows<false, false>(a, s);
    return hipGetLastError() == hipSuccess ? 0 : -3;
  }
  const int out = gated ? TN / 2 : TN;
  const int gm = (int)((a.M + TM - 1) / TM), gn = (int)((a.N + out - 1) / out);
  const dim3 grid((unsigned)(gm * gn)), b(256);
  if (a8 && gated) hipLaunchKernelGGL((gemm_tile_kernel<true, true>), grid, b, 0, s, a, gm, gn);
  else if (a8) hipLaunchKernelGGL((gemm_tile_kernel<true, false>), grid, b, 0, s, a, gm, gn);
  else if (gated) hipLaunchKernelGGL((gemm_tile_kernel<false, true>), grid, b, 0, s, a, gm, gn);
  else hipLaunchKernelGGL((gemm_tile_kernel<false, false>), grid, b, 0, s, a, gm, gn);
  return hipGetLastError() == hipSuccess ? 0 : -3;
}

}  // namespace nvfp4
