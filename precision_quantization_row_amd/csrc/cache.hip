// cache.hip -- quantized keys and values in pages: written as tokens come, and
// read back (gfx950).
//
// A line is what one head of one token holds, D elements with one amax:
//   q    [pages][page_size][H][ceil(D/2) (NVFP4) or D (E4M3, INT8)]
//   s    [pages][page_size][H][ceil(D/16)]   (NVFP4)
//   amax [pages][page_size][H]
// so a token's lines lie together, in the cache as in the rows they come from.
// Token t of a call belongs to the sequence b with starts[b] <= t < starts[b + 1]
// and has position first[b] + t - starts[b] there; position n lies at place
// n mod page_size of page table[b][n / page_size].
//
// Bound by HBM where tokens are many, by latency where they are few. A line
// takes L lanes (a power of two) and V runs of 8 L elements. A workgroup takes
// TB tokens of the keys (blockIdx.y 0) or of the values (1): its waves look up
// the tokens' places, 64 sequences at a time, and leave them in LDS; then
// groups of L lanes take the lines in turn.
#include "nvfp4_launch.h"
#include "nvfp4_rows.h"

#include <algorithm>

namespace nvfp4 {

constexpr int64_t kNoToken = -1;  // no sequence's token: nothing is done
constexpr int64_t kBadPage = -2;  // a token whose page does not exist

// The cache's row (page * page_size + place) of token t; a wave, all lanes alike.
// Every index is bounded whatever starts, first and table hold.
__device__ __forceinline__ int64_t token_slot(const CacheArgs& p, int64_t t, int lane) {
  // how many of starts[0 .. B] are at most t: 64 probes at a time
  int64_t lo = 0, n = p.B + 1;
  while (n > 64) {
    const int64_t step = (n + 63) / 64, at = min((lane + 1) * step, n) - 1;
    const int64_t full = __builtin_popcountll(__ballot(p.starts[lo + at] <= t)) * step;
    // (the last probe is the last entry: past t, but for tokens behind the last sequence)
    if (full >= n) return kNoToken;
    lo += full;
    n = min(step, n - full);
  }
  const bool below = lane < n && p.starts[lo + min((int64_t)lane, n - 1)] <= t;
  const int64_t b = lo + __builtin_popcountll(__ballot(below)) - 1;
  if (b < 0 || b >= p.B) return kNoToken;
  const int64_t pos = (p.first ? (int64_t)p.first[b] : 0) + t - p.starts[b];
  if (pos < 0 || pos > 0x7FFFFFFF) return kBadPage;
  const uint32_t size = (uint32_t)min(p.page_size, (int64_t)0xFFFFFFFFu);
  const uint32_t col = (uint32_t)pos / size;
  if (col >= p.cols) return kBadPage;
  const int64_t page = p.table[b * p.cols + col];
  if (page < 0 || page >= p.pages) return kBadPage;
  return page * p.page_size + ((uint32_t)pos - col * size);
}

constexpr int TB_MAX = 64;

template <typename T, int L, int V>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheArgs p, int tb) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int G = 256 / L;
  __shared__ int64_t slots[TB_MAX];
  const int tid = threadIdx.x, lane = tid & 63, l = tid % L, which = blockIdx.y;
  const int64_t t0 = p.t0 + (int64_t)blockIdx.x * tb, D = p.D;
  const int nt = (int)min((int64_t)tb, p.T - t0);
  const uint32_t H = (uint32_t)p.H, lines = nt * H;
  const T* src = static_cast<const T*>(p.src[which]) + t0 * p.stride[which];
  const int64_t stride = p.stride[which];
  // (the first lines are on their way while the places are looked up)
  Raw8<T> rx[V];
  auto load = [&](uint32_t i) __attribute__((always_inline)) {
    const uint32_t t = i / H, h = i - t * H;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t c = 8 * (int64_t)(l + j * L);
      load8_raw(src + t * stride + h * D + c, i < lines ? D - c : 0, rx[j]);
    }
  };
  load(min((uint32_t)(tid / L), lines - 1));
  for (int i = tid >> 6; i < nt; i += 4) {
    const int64_t s = token_slot(p, t0 + i, lane);
    if (lane == 0) slots[i] = s;
  }
  __syncthreads();
  const int64_t pq = p.fmt == FMT_NVFP4 ? (D + 1) / 2 : D, ps = (D + 15) / 16;
  // every lane of a wave takes part in each turn (lines are joined over lanes)
  for (uint32_t i0 = 0; i0 < lines; i0 += G) {
    const uint32_t i = i0 + tid / L, ic = min(i, lines - 1);
    float v[V][8];
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      unpack8(rx[j], v[j]);
      m = amax8(v[j], m);
    }
    load(min(i + G, lines - 1));
    const int64_t slot = slots[ic / H];
    const bool live = i < lines && slot >= 0;
    const int64_t line = live ? slot * H + ic % H : 0;
    const float a = __uint_as_float(row_max<L>(m, nullptr));
    const float enc = global_encode_scale(a, line_top(p.fmt, p.F));
    if (live && l == 0) p.amax[which][line] = a;
    uint8_t *q = p.q[which] + line * pq, *s = p.s[which] + line * ps;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t c = 8 * (int64_t)(l + j * L);
      write_codes<true>(p.fmt, q, s, c, live ? D - c : 0, v[j], a, enc, p.F_inv);
    }
  }
}

template <typename T, int L, int V>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheArgs p, int tb) {
  if (p.noop != nullptr && *p.noop == 1.0f) return;
  constexpr int G = 256 / L;
  __shared__ int64_t slots[TB_MAX];
  const int tid = threadIdx.x, lane = tid & 63, l = tid % L, which = blockIdx.y;
  const int64_t t0 = p.t0 + (int64_t)blockIdx.x * tb, D = p.D;
  const int nt = (int)min((int64_t)tb, p.T - t0);
  const uint32_t H = (uint32_t)p.H, lines = nt * H;
  T* dst = static_cast<T*>(p.dst[which]) + t0 * p.stride[which];
  const int64_t stride = p.stride[which];
  for (int i = tid >> 6; i < nt; i += 4) {
    const int64_t s = token_slot(p, t0 + i, lane);
    if (lane == 0) slots[i] = s;
  }
  __syncthreads();
  const int64_t pq = p.fmt == FMT_NVFP4 ? (D + 1) / 2 : D, ps = (D + 15) / 16;
  for (uint32_t i = tid / L; i < lines; i += G) {
    const uint32_t t = i / H, h = i - t * H;
    const int64_t slot = slots[t];
    if (slot == kNoToken) continue;  // rows of no sequence stay as they are
    const int64_t line = slot < 0 ? 0 : slot * H + h;
    T* y = dst + t * stride + h * D;
    const float a = p.amax[which][line];
    const uint8_t* q = p.q[which] + line * pq;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t c = 8 * (int64_t)(l + j * L), n = D - c;
      if (n <= 0) continue;
      float v[8];
      if (p.fmt == FMT_NVFP4) {
        const uint32_t byte = p.s[which][line * ps + c / 16];
        uint32_t w = 0u;
        if (n >= 8) {
          w = *reinterpret_cast<const u32_a1*>(q + c / 2);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (2 * k < n) w |= (uint32_t)q[c / 2 + k] << (8 * k);
        }
        const float d = (__builtin_amdgcn_cvt_f32_fp8((int)byte, 0) * a) * p.F_inv;
        f32x2 u[4] = {fp4x2_decode<0>(w), fp4x2_decode<1>(w), fp4x2_decode<2>(w), fp4x2_decode<3>(w)};
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = u[k / 2][k & 1] * d;
      } else {
        u32x2 w = {0u, 0u};
        if (n >= 8) {
          w = *reinterpret_cast<const u32x2_a1*>(q + c);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < n) {
              if (k < 4) w.x |= (uint32_t)q[c + k] << (8 * k);
              else w.y |= (uint32_t)q[c + k] << (8 * (k - 4));
            }
        }
        if (p.fmt == FMT_E4M3) {
          const float d = a / kE4M3Max;
          const f32x2 u[4] = {__builtin_amdgcn_cvt_pk_f32_fp8(w.x, false), __builtin_amdgcn_cvt_pk_f32_fp8(w.x, true),
                              __builtin_amdgcn_cvt_pk_f32_fp8(w.y, false), __builtin_amdgcn_cvt_pk_f32_fp8(w.y, true)};
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = u[k / 2][k & 1] * d;
        } else {
          const float d = a / kInt8Max;
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = (float)(int8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3))) * d;
        }
      }
      if (slot < 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
      }
      store8(y + c, n, v);
    }
  }
}

// Tokens of a workgroup: enough lines for a few turns of its groups, unless
// that leaves the card short of workgroups.
static int tokens_of_block(const CacheArgs& a, int L) {
  const int64_t lines = 4 * (256 / L), fill = (a.T + 1023) / 1024;
  return (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)TB_MAX, lines / a.H, fill}));
}

template <typename F>
static int go_cache(const CacheArgs& a, int L, F launch) {
  const int tb = tokens_of_block(a, L);
  // a launch holds fewer than 2^32 threads
  for (int64_t t = 0; t < a.T; t += (int64_t)tb << 22) {
    CacheArgs p = a;
    p.t0 = t;
    const int64_t blocks = std::min<int64_t>((a.T - t + tb - 1) / tb, 1 << 22);
    launch(p, dim3((unsigned)blocks, a.q[1] ? 2u : 1u), tb);
    if (hipGetLastError() != hipSuccess) return -3;
  }
  return 0;
}

// lanes of a line and its runs of 8 elements a lane (D <= 1024)
template <typename T, bool WRITE>
static int launch_cache_t(const CacheArgs& a, hipStream_t s) {
  const int64_t chunks = (a.D + 7) / 8;
  auto go = [&](auto l_, auto v_) {
    constexpr int L = decltype(l_)::value, V = decltype(v_)::value;
    return go_cache(a, L, [&](const CacheArgs& p, dim3 g, int tb) {
      if constexpr (WRITE) hipLaunchKernelGGL((cache_write_kernel<T, L, V>), g, dim3(256), 0, s, p, tb);
      else hipLaunchKernelGGL((cache_read_kernel<T, L, V>), g, dim3(256), 0, s, p, tb);
    });
  };
  using C1 = std::integral_constant<int, 1>;
  if (chunks <= 8) return go(std::integral_constant<int, 8>{}, C1{});
  if (chunks <= 16) return go(std::integral_constant<int, 16>{}, C1{});
  if (chunks <= 32) return go(std::integral_constant<int, 32>{}, C1{});
  if (chunks <= 64) return go(std::integral_constant<int, 64>{}, C1{});
  return go(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
}

int launch_cache_write(const CacheArgs& a, hipStream_t s) {
  return a.dtype == 0 ? launch_cache_t<uint16_t, true>(a, s) : launch_cache_t<float, true>(a, s);
}
int launch_cache_read(const CacheArgs& a, hipStream_t s) {
  return a.dtype == 0 ? launch_cache_t<uint16_t, false>(a, s) : launch_cache_t<float, false>(a, s);
}

}  // namespace nvfp4
