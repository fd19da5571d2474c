// cache_read.hip -- the cached tokens of sequences, back as values (gfx950).
#include "cache_device.h"

namespace nvfp4 {

// A lane's 8 codes as they lie: 4 bytes (NVFP4) or 8.
template <int FMT, bool EVEN>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* q, int c, int n) {
  u32x2 w = {0u, 0u};
  if constexpr (FMT == FMT_NVFP4) {
    if (EVEN || n >= 8) {
      w.x = *reinterpret_cast<const u32_a1*>(q + (EVEN && n <= 0 ? 0 : c / 2));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (2 * k < n) w.x |= (uint32_t)q[c / 2 + k] << (8 * k);
    }
  } else {
    if (EVEN || n >= 8) {
      w = *reinterpret_cast<const u32x2_a1*>(q + (EVEN && n <= 0 ? 0 : c));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) {
          if (k < 4) w.x |= (uint32_t)q[c + k] << (8 * k);
          else w.y |= (uint32_t)q[c + k] << (8 * (k - 4));
        }
    }
  }
  return w;
}
template <int FMT>
__device__ __forceinline__ void decode_codes(u32x2 w, float d, float (&v)[8]) {
  if constexpr (FMT == FMT_NVFP4) {
    const f32x2 e[4] = {fp4x2_decode<0>(w.x), fp4x2_decode<1>(w.x), fp4x2_decode<2>(w.x), fp4x2_decode<3>(w.x)};
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = e[k / 2][k & 1] * d;
  } else if constexpr (FMT == FMT_E4M3) {
    const f32x2 e[4] = {__builtin_amdgcn_cvt_pk_f32_fp8(w.x, false), __builtin_amdgcn_cvt_pk_f32_fp8(w.x, true),
                        __builtin_amdgcn_cvt_pk_f32_fp8(w.y, false), __builtin_amdgcn_cvt_pk_f32_fp8(w.y, true)};
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = e[k / 2][k & 1] * d;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = (float)(int8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3))) * d;
  }
}

// Lines that a group of lanes has on their way at once. 131072 tokens, 8 x 128, NVFP4,
// BF16 out: 1 160 us, 2 159, 4 138, 8 126.
template <int V>
constexpr int lines_at_once() { return V == 1 ? 8 : 4; }

// EVEN: D is a multiple of 8, so that a lane has a whole run or none: its loads
// need no branch (which would wait for the ones before it).
template <typename T, int L, int V, int FMT, bool EVEN>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheArgs p, int tb) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int G = 256 / L, N = lines_at_once<V>();
  __shared__ Place places[TB_MAX];
  const int l = threadIdx.x % L, grp = threadIdx.x / L, which = blockIdx.y;
  const int64_t t0 = p.t0 + (int64_t)blockIdx.x * tb;
  const int nt = (int)min((int64_t)tb, p.T - t0), D = (int)p.D;
  const uint32_t lines = nt * (uint32_t)p.H;
  T* dst = static_cast<T*>(p.dst[which]) + t0 * p.stride[which];
  const uint32_t pq = FMT == FMT_NVFP4 ? (D + 1) / 2 : D, ps = (D + 15) / 16;
  const float f8 = FMT == FMT_E4M3 ? 1.0f / kE4M3Max : 1.0f / kInt8Max;
  find_places(p, t0, nt, places);
  for (uint32_t i0 = 0; i0 < lines; i0 += N * G) {
    float am[N];
    u32x2 w[N][V];
    uint32_t sc[N][V];
    // (lines without a page load the cache's first: their values are not used)
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (i0 + u * G >= lines) break;
      const Line at = line_of(p, min(i0 + u * G + grp, lines - 1));
      const Place from = places[at.t];
      const uint8_t *q = p.q[which] + from.q + __umul24(at.h, pq), *s = p.s[which] + from.s + __umul24(at.h, ps);
      am[u] = p.amax[which][max(from.line, (int64_t)0) + at.h];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = 8 * (l + j * L);
        w[u][j] = load_codes<FMT, EVEN>(q, c, D - c);
        if constexpr (FMT == FMT_NVFP4) sc[u][j] = s[c < D ? c / 16 : 0];
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const uint32_t i = i0 + u * G + grp;
      if (i >= lines) break;
      const Line at = line_of(p, i);
      const Place from = places[at.t];
      if (from.line == kNoToken) continue;  // rows of no sequence stay as they are
      T* y = dst + from.row + __umul24(at.h, (uint32_t)D);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = 8 * (l + j * L), n = D - c;
        if (n <= 0) continue;
        float v[8];
        decode_codes<FMT>(w[u][j], FMT == FMT_NVFP4 ? (__builtin_amdgcn_cvt_f32_fp8((int)sc[u][j], 0) * am[u]) * p.F_inv : am[u] * f8, v);
        if (from.line < 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        }
        store8<true>(y + c, EVEN ? 8 : n, v);
      }
    }
  }
}

template <typename T>
static int launch_t(const CacheArgs& a, hipStream_t s) {
  return by_line(a, [&](auto l, auto v, auto f, auto e) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value, FMT = decltype(f)::value;
    constexpr bool EVEN = decltype(e)::value;
    return launch_tokens(a, L, lines_at_once<V>(), [&](const CacheArgs& p, dim3 g, int tb) {
      hipLaunchKernelGGL((cache_read_kernel<T, L, V, FMT, EVEN>), g, dim3(256), 0, s, p, tb);
    });
  });
}

int launch_cache_read(const CacheArgs& a, hipStream_t s) {
  return a.dtype == 0 ? launch_t<uint16_t>(a, s) : launch_t<float>(a, s);
}

}  // namespace nvfp4
