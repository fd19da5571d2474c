// nvfp4_rows.h -- rows (lines) held by groups of lanes, 8 elements a lane and
// run: reductions over the group and the codes of its elements (gfx950).
#pragma once

#include "nvfp4_vec.h"

namespace nvfp4 {

enum { FMT_NONE = 0, FMT_E4M3 = 1, FMT_NVFP4 = 2, FMT_INT8 = 3 };
constexpr float kInt8Max = 127.0f;

// Sum over each L lanes (a power of two up to 64), every lane gets it. Partners by DPP,
// in a few cycles each where a shuffle goes through LDS: neighbour, pairs, half-row mirror,
// row mirror, then the other 16 and 32 lanes. (After each step the lanes of a group hold
// the same value, so a mirror joins the same groups as lane ^ 4 and lane ^ 8 would.)
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L >= 2) v = add_dpp<0xB1>(v);
  if constexpr (L >= 4) v = add_dpp<0x4E>(v);
  if constexpr (L >= 8) v = add_dpp<0x141>(v);
  if constexpr (L >= 16) v = add_dpp<0x140>(v);
  if constexpr (L >= 32) {
    const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
  }
  if constexpr (L >= 64) {
    const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
  }
  return v;
}

// The same over a wave, partners 32, 16, 8, 4, 2 and 1 lanes apart in this order: sums of
// floats depend on it. (After each step the lanes whose numbers differ by a multiple
// of the step hold the same value, so that turning a row of 16 lanes by 8, 4, 2 or 1
// joins the same sums as lane ^ 8 and so on.)
__device__ __forceinline__ float wave_sum(float v) {
  const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
  const auto u = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(u[0]) + __uint_as_float(u[1]);
  v = add_dpp<0x128>(v);
  v = add_dpp<0x124>(v);
  v = add_dpp<0x122>(v);
  return add_dpp<0x121>(v);
}

// Integers over a wave.
__device__ __forceinline__ int lanes_sum_int(int v) {
  v += __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, false);
  v += __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, false);
  v += __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, false);
  v += __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, false);
  const auto t = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
  v = (int)(t[0] + t[1]);
  const auto w = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
  return (int)(w[0] + w[1]);
}

// Sum / max over a workgroup of NT threads; every thread gets the result.
// `red` holds NT / 64 entries; consecutive calls use different ones. FAR_FIRST: lanes
// join as in wave_sum, else as in lanes_sum; the waves join in their order.
template <int NT, bool FAR_FIRST = false>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = FAR_FIRST ? wave_sum(v) : lanes_sum<64>(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += red[i];
  }
  return v;
}
template <int NT>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = wave_max_u32(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0u;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v = max(v, red[i]);
  }
  return v;
}

// The same over a row's L lanes: a power of two up to 64 (rows side by side in
// a wave; `red` unused), or a whole workgroup of L threads.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* red) {
  if constexpr (L <= 64) {
    return lanes_sum<L>(v);
  } else {
    return block_sum<L>(v, red);
  }
}
// two sums at once (red: 2 L / 64 entries)
template <int L>
__device__ __forceinline__ void row_sum2(float& u, float& v, float* red) {
  constexpr int P = L < 64 ? L : 64;
  u = lanes_sum<P>(u);
  v = lanes_sum<P>(v);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) {
      red[2 * (threadIdx.x >> 6)] = u;
      red[2 * (threadIdx.x >> 6) + 1] = v;
    }
    __syncthreads();
    u = v = 0.0f;
#pragma unroll
    for (int i = 0; i < L / 64; ++i) {
      u += red[2 * i];
      v += red[2 * i + 1];
    }
  }
}
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  if constexpr (L <= 64) {
    // DPP: neighbour, pairs, half-row mirror, row mirror; the rest by shuffles
    if constexpr (L >= 2) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));
    if constexpr (L >= 4) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));
    if constexpr (L >= 8) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
    if constexpr (L >= 16) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));
    if constexpr (L >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    if constexpr (L >= 64) v = max(v, (uint32_t)__shfl_xor((int)v, 32));
    return v;
  } else {
    return block_max<L>(v, red);
  }
}

// E elements as they lie in memory, at any element's address
template <typename T, int E>
struct Piece {
  static constexpr int D = E * sizeof(T) / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(D)));
  typedef Words Any __attribute__((aligned(sizeof(T))));
  Words d;
  template <bool NT = false>
  __device__ __forceinline__ void load(const T* p) {
    const Any* q = reinterpret_cast<const Any*>(p);
    d = NT ? __builtin_nontemporal_load(q) : *q;
  }
  __device__ __forceinline__ void clear_first(int t) {
#pragma unroll
    for (int i = 0; i < D; ++i) {
      if constexpr (sizeof(T) == 4) d[i] = i < t ? 0u : d[i];
      else d[i] = 2 * i + 1 < t ? 0u : (2 * i < t ? d[i] & 0xFFFF0000u : d[i]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[E]) {
    Words w;
#pragma unroll
    for (int i = 0; i < D; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
      else w[i] = bf16x2_rne(v[2 * i], v[2 * i + 1]);
    }
    __builtin_nontemporal_store(w, reinterpret_cast<Any*>(p));
  }
  __device__ __forceinline__ void get(float (&v)[E]) const {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      if constexpr (sizeof(T) == 4) v[k] = __uint_as_float(d[k]);
      else v[k] = __uint_as_float(k & 1 ? d[k / 2] & 0xFFFF0000u : d[k / 2] << 16);
    }
  }
};

// The second-level amax bits of 8 values joined to m. A NaN's bits lie above
// every number's, so a line that holds one has a NaN amax.
__device__ __forceinline__ uint32_t amax8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & kAbsF32);
  return m;
}

// The same of 8 elements as they lie in memory. (Two BF16 to an instruction.)
__device__ __forceinline__ uint32_t amax8_raw(const Raw8<float>& r, uint32_t m) {
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, r.d[k] & kAbsF32);
  return m;
}
__device__ __forceinline__ uint32_t amax8_raw(const Raw8<uint16_t>& r, uint32_t m) {
  uint32_t p = r.d[0] & kAbsBf16x2;
#pragma unroll
  for (int k = 1; k < 4; ++k) p = pk_max_u16(p, r.d[k] & kAbsBf16x2);
  return max(m, max(p << 16, p & 0xFFFF0000u));
}

// All ones for a line whose amax is a number, else zero: the codes of a line that holds a
// NaN or an infinity are zeros, and its amax makes whatever is decoded from them NaN.
__device__ __forceinline__ uint32_t keep_finite(float a) { return __float_as_uint(a) < 0x7F800000u ? ~0u : 0u; }

// 8 values as E4M3 bytes: RN(v enc) clamped to 448 with the sign kept, to nearest
// even; a NaN's byte is a number, too. CLAMP false: enc is RN(448 / a) of an a that
// no |v| passes, so that RN(v enc) is at most 448 (1 + 2^-23), which rounds to 448; of
// an a that is no number, bytes may be NaNs: keep_finite clears them. (The clamp in
// the cache's write: 32768 lines of 576, 17.6 -> 18.8 us.)
template <bool CLAMP = true>
__device__ __forceinline__ u32x2 pack8_e4m3(const float (&v)[8], float enc) {
  float t[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    t[k] = v[k] * enc;
    if (CLAMP) t[k] = fmaxf(fminf(t[k], kE4M3Max), -kE4M3Max);
  }
  uint32_t w0 = 0u, w1 = 0u;
  w0 = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], w0, false);
  w0 = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], w0, true);
  w1 = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], w1, false);
  w1 = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], w1, true);
  return u32x2{w0, w1};
}

// The integer nearest to RN(v enc), halves to the even one, in the low byte. 1.5 *
// 2^23 has steps of one and is even: adding it rounds so, and the sum's low byte is
// the integer's two's complement. enc is RN(127 / a) of an a that no |v| passes:
// RN(v enc) is at most 127 (1 + 2^-23), which rounds to 127. Of an a that is no
// number, the low byte is any: keep_finite clears it.
__device__ __forceinline__ uint32_t int8_code(float v, float enc) {
  return __float_as_uint(v * enc + 12582912.0f);
}
// the low bytes of four dwords, a first
__device__ __forceinline__ uint32_t pack4_low(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0C0C0400u);
  const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x0C0C0400u);
  return __builtin_amdgcn_perm(cd, ab, 0x05040100u);
}
__device__ __forceinline__ u32x2 pack8_int8(const float (&v)[8], float enc, uint32_t keep) {
  uint32_t t[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) t[k] = int8_code(v[k], enc);
  return u32x2{pack4_low(t[0], t[1], t[2], t[3]) & keep, pack4_low(t[4], t[5], t[6], t[7]) & keep};
}

// 8 bytes, or the first n of them
__device__ __forceinline__ void store8_bytes(uint8_t* q, int64_t n, u32x2 w) {
  if (n >= 8) {
    *reinterpret_cast<u32x2_a1*>(q) = w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) q[k] = (uint8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
  }
}

// What a format maps a line's amax to, before its block scales if it has any.
__device__ __forceinline__ float line_top(int fmt, float F) {
  return fmt == FMT_E4M3 ? kE4M3Max : fmt == FMT_INT8 ? kInt8Max : F;
}

// Writes one lane's 8 values of a line as codes. q, s: the line's
// first code and block scale; c: first element (a multiple of 8), n: elements
// of the line from c on; a: the line's amax, enc: its encode scale. The lane
// pair (2i, 2i + 1) holds one 16-element block; both lanes are active (lanes
// past the line hold zeros). I8: the format may be INT8.
template <bool I8>
__device__ __forceinline__ void write_codes(int fmt, uint8_t* q, uint8_t* s, int64_t c, int64_t n,
                                            const float (&y)[8], float a, float enc, float F_inv) {
  if (I8 && fmt == FMT_INT8) {
    store8_bytes(q + c, n, pack8_int8(y, enc, keep_finite(a)));
  } else if (fmt == FMT_E4M3) {
    store8_bytes(q + c, n, pack8_e4m3(y, enc));
  } else {  // NVFP4
    uint32_t m = amax8(y, 0u);
    m = max(m, dpp_swap1(m));
    uint32_t byte;
    float e;
    block_scale(__uint_as_float(m), a, enc, F_inv, &byte, &e);
    uint32_t code = e2m1_pack8(y[0] * e, y[1] * e, y[2] * e, y[3] * e, y[4] * e, y[5] * e, y[6] * e,
                               y[7] * e);
    if (n > 0 && (c & 8) == 0) s[c / 16] = (uint8_t)byte;
    q += c / 2;
    if (n >= 8) {
      *reinterpret_cast<u32_a1*>(q) = code;
    } else {
      if (n > 0) code &= (1u << (4 * n)) - 1u;  // a missing last high nibble is 0
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (2 * k < n) q[k] = (uint8_t)(code >> (8 * k));
    }
  }
}

// A launch holds fewer than 2^32 threads: taller inputs take several.
// launch(first row, rows)
template <typename F>
static int rows_in_launches(int64_t M, F launch) {
  for (int64_t r = 0; r < M; r += 1 << 20) {
    launch(r, M - r < (1 << 20) ? M - r : (int64_t)(1 << 20));
    if (hipGetLastError() != hipSuccess) return -3;
  }
  return 0;
}

// Wider inputs take several launches, too: 2^26 columns are 2^31 threads at 32
// threads a column, and with 256 parts at 8 columns a thread.
// launch(first column, columns)
template <typename F>
static int columns_in_launches(int64_t N, F launch) {
  for (int64_t c = 0; c < N; c += 1 << 26) {
    launch(c, N - c < (1 << 26) ? N - c : (int64_t)(1 << 26));
    if (hipGetLastError() != hipSuccess) return -3;
  }
  return 0;
}

}  // namespace nvfp4
