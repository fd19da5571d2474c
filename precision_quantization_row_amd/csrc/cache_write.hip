// cache_write.hip -- keys and values quantized into the pages of a cache as their
// tokens come (gfx950).
#include "cache_device.h"

namespace nvfp4 {

// Lines that a group of lanes has on their way at once, of the TURNS times as many
// it takes. 16384 tokens, 8 x 128, keys and values to E4M3: 1 and 4 25.4 us, 2 and 4 26.6, 4
// and 1 27.7, 4 and 2 25.6, 8 and 1 27.1.
template <int V>
constexpr int lines_at_once() { return V == 1 ? 4 : 2; }
constexpr int TURNS = 2;

// EVEN: D is a multiple of 8, so that a lane has a whole run or none: its loads
// need no branch (which would wait for the ones before it).
template <typename T, int L, int V, int FMT, bool EVEN>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheArgs p, int tb) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int G = 256 / L, N = lines_at_once<V>();
  __shared__ Place places[TB_MAX];
  const int l = threadIdx.x % L, grp = threadIdx.x / L, which = blockIdx.y;
  const int64_t t0 = p.t0 + (int64_t)blockIdx.x * tb;
  const int nt = (int)min((int64_t)tb, p.T - t0), D = (int)p.D;
  const uint32_t lines = nt * (uint32_t)p.H;
  const T* src = static_cast<const T*>(p.src[which]) + t0 * p.stride[which];
  const uint32_t pq = FMT == FMT_NVFP4 ? (D + 1) / 2 : D, ps = (D + 15) / 16;
  for (uint32_t i0 = 0; i0 < lines; i0 += N * G) {
    Raw8<T> rx[N][V];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (i0 + u * G >= lines) break;
      const Line at = line_of(p, min(i0 + u * G + grp, lines - 1));
      const T* x = src + at.t * (uint32_t)p.stride[which] + __umul24(at.h, (uint32_t)D);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = 8 * (l + j * L);
        if constexpr (EVEN) load8_raw<true>(x + (c < D ? c : 0), 8, rx[u][j]);
        else load8_raw<true>(x + c, D - c, rx[u][j]);
      }
    }
    if (i0 == 0) find_places(p, t0, nt, places);  // (the first lines are on their way)
    // every lane of a wave takes part in each turn (lines are joined over lanes)
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const uint32_t i = i0 + u * G + grp;
      if (i0 + u * G >= lines) break;
      const Line at = line_of(p, min(i, lines - 1));
      float v[V][8];
      uint32_t m = 0u;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (EVEN && 8 * (l + j * L) >= D) {
#pragma unroll
          for (int k = 0; k < Raw8<T>::DW; ++k) rx[u][j].d[k] = 0u;
        }
        m = amax8_raw(rx[u][j], m);
        unpack8(rx[u][j], v[j]);
      }
      const float a = __uint_as_float(row_max<L>(m, nullptr));
      const float enc = global_encode_scale(a, line_top(FMT, p.F));
      const Place to = places[at.t];
      const bool live = i < lines && to.line >= 0;
      if (live && l == 0) p.amax[which][to.line + at.h] = a;
      uint8_t *q = p.q[which] + to.q + __umul24(at.h, pq), *s = p.s[which] + to.s + __umul24(at.h, ps);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = 8 * (l + j * L);
        const int64_t n = !live ? 0 : EVEN ? (c < D ? 8 : 0) : D - c;
        if constexpr (FMT == FMT_E4M3) store8_bytes(q + c, n, pack8_e4m3<false>(v[j], enc) & keep_finite(a));
        else write_codes<true>(FMT, q, s, c, n, v[j], a, enc, p.F_inv);
      }
    }
  }
}

template <typename T>
static int launch_t(const CacheArgs& a, hipStream_t s) {
  return by_line(a, [&](auto l, auto v, auto f, auto e) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value, FMT = decltype(f)::value;
    constexpr bool EVEN = decltype(e)::value;
    return launch_tokens(a, L, TURNS * lines_at_once<V>(), [&](const CacheArgs& p, dim3 g, int tb) {
      hipLaunchKernelGGL((cache_write_kernel<T, L, V, FMT, EVEN>), g, dim3(256), 0, s, p, tb);
    });
  });
}

int launch_cache_write(const CacheArgs& a, hipStream_t s) {
  return a.dtype == 0 ? launch_t<uint16_t>(a, s) : launch_t<float>(a, s);
}

}  // namespace nvfp4
