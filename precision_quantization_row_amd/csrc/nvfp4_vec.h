// nvfp4_vec.h -- runs of 8 elements in memory (gfx950).
//
// A lane of the norm, activation and product kernels holds 8 consecutive
// elements of a row. Rows are packed, so with odd lengths a run may start at
// any element: the vector types below carry the element's own alignment, and
// the compiler emits one 16-byte access for them (gfx950 global memory takes
// any alignment; an aligned run costs the same instruction). Runs that end a
// row are moved element by element, so nothing outside the row is touched.
#pragma once

#include "nvfp4_device.h"

namespace nvfp4 {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
// BF16: round to nearest even
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)bf16x2_rne(v, v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// The raw dwords of 8 elements: what a kernel keeps in flight before use.
template <typename T>
struct Raw8 {
  static constexpr int DW = 2 * sizeof(T);  // 4 (BF16) or 8 (FP32)
  uint32_t d[DW];
};

// n >= 8: the whole run; else its first n elements, the rest read as zero.
template <bool NT = false>
__device__ __forceinline__ void load8_raw(const uint16_t* p, int64_t n, Raw8<uint16_t>& r) {
  if (n >= 8) {
    const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p);
    const u32x4 w = NT ? __builtin_nontemporal_load(q) : *q;
    r.d[0] = w.x; r.d[1] = w.y; r.d[2] = w.z; r.d[3] = w.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = 2 * k < n ? p[2 * k] : 0u, hi = 2 * k + 1 < n ? p[2 * k + 1] : 0u;
      r.d[k] = lo | (hi << 16);
    }
  }
}
// (FP32: a lane's run is two accesses, each half of a wave's 2 KB; past the
// caches, NT, the halves would move on their own)
template <bool NT = false>
__device__ __forceinline__ void load8_raw(const float* p, int64_t n, Raw8<float>& r) {
  if (n >= 8) {
    const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(p);
    const u32x4 a = q[0], b = q[1];
    r.d[0] = a.x; r.d[1] = a.y; r.d[2] = a.z; r.d[3] = a.w;
    r.d[4] = b.x; r.d[5] = b.y; r.d[6] = b.z; r.d[7] = b.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) r.d[k] = k < n ? __float_as_uint(p[k]) : 0u;
  }
}
__device__ __forceinline__ void unpack8(const Raw8<uint16_t>& r, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = bf16_lo(r.d[k]);
    v[2 * k + 1] = bf16_hi(r.d[k]);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r.d[k]);
}
template <typename T, bool NT = false>
__device__ __forceinline__ void load8(const T* p, int64_t n, float (&v)[8]) {
  Raw8<T> r;
  load8_raw<NT>(p, n, r);
  unpack8(r, v);
}

// n >= 8: the whole run; else its first n elements only.
template <bool NT = false>
__device__ __forceinline__ void store8(uint16_t* p, int64_t n, const float (&v)[8]) {
  if (n >= 8) {
    const u32x4 w = {bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]),
                     bf16x2_rne(v[6], v[7])};
    u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p);
    if (NT) __builtin_nontemporal_store(w, q);
    else *q = w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) store1(p + k, v[k]);
  }
}
template <bool NT = false>
__device__ __forceinline__ void store8(float* p, int64_t n, const float (&v)[8]) {
  if (n >= 8) {
    const u32x4 a = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3])};
    const u32x4 b = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                     __float_as_uint(v[7])};
    u32x4_a4* q = reinterpret_cast<u32x4_a4*>(p);
    q[0] = a;
    q[1] = b;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = v[k];
  }
}

// ------------------------------------------------------------- activations
// The exponentials go through the hardware's exp2 (1 ulp): e^x = 2^(x log2 e)
// carries the rounding of x log2 e, a relative error near |x| 2^-24, which
// only matters where e^-x is large and the sigmoid below is tiny.
constexpr float kLog2e = 1.442695040888963f;
constexpr float kGeluA = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

enum { ACT_NONE = 0, ACT_GELU = 1, ACT_SILU = 2, ACT_RELU2 = 3, ACT_SWIGLU = 4 };

// 1 / (1 + e^-x): e^-x = +inf gives 0, as it should; NaN stays NaN. The
// reciprocal is the hardware's (1 ulp); it flushes results below 2^-126, so for
// x < -87.3 silu and its slope are 0 where they should be up to 1e-36.
__device__ __forceinline__ float sigmoid_f(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}
// x * sigmoid(x); like the formula, x = -inf gives NaN
__device__ __forceinline__ float silu_f(float x) { return x * sigmoid_f(x); }

// gelu in the tanh form: 0.5 z (1 + tanh u) = z sigmoid(2 u),
// u = sqrt(2/pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu_2u(float z) {
  return 2.0f * kGeluA * z * __builtin_fmaf(kGeluB * z, z, 1.0f);
}
__device__ __forceinline__ float act_f(int act, float z) {
  switch (act) {
    case ACT_GELU: return z * sigmoid_f(gelu_2u(z));
    case ACT_SILU: return silu_f(z);
    case ACT_RELU2: {
      const float r = z < 0.0f ? 0.0f : z;  // NaN passes
      return r * r;
    }
    default: return z;
  }
}
// the activation of 8 values: one branch for all
__device__ __forceinline__ void act8(int act, float (&z)[8]) {
  if (act == ACT_GELU) {
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = act_f(ACT_GELU, z[k]);
  } else if (act == ACT_SILU) {
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = act_f(ACT_SILU, z[k]);
  } else if (act == ACT_RELU2) {
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = act_f(ACT_RELU2, z[k]);
  }
}
// d silu / dz = s (1 + z (1 - s)); 1 - s = sigmoid(-z) without cancellation
__device__ __forceinline__ float dsilu_f(float z, float s) {
  return s * __builtin_fmaf(z, sigmoid_f(-z), 1.0f);
}
__device__ __forceinline__ float dact_f(int act, float z) {
  switch (act) {
    case ACT_GELU: {
      const float u2 = gelu_2u(z), s = sigmoid_f(u2), c = sigmoid_f(-u2);
      const float du = 2.0f * kGeluA * __builtin_fmaf(3.0f * kGeluB * z, z, 1.0f);
      const float t = s * c;  // 0 where |z| is large: z du may overflow there
      return t == 0.0f ? s : __builtin_fmaf(z * t, du, s);
    }
    case ACT_SILU: {
      const float s = sigmoid_f(z);
      return s == 0.0f ? 0.0f : dsilu_f(z, s);
    }
    case ACT_RELU2: return z < 0.0f ? 0.0f : 2.0f * z;
    default: return 1.0f;
  }
}

// ------------------------------------------------------------- reductions
// Sum over the 64 lanes of a wave; every lane gets it. The order is fixed.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = row16_max(v);
  v = max(v, (uint32_t)__shfl_xor((int)v, 16));
  return max(v, (uint32_t)__shfl_xor((int)v, 32));
}

}  // namespace nvfp4
