// cache_device.h -- quantized keys and values in pages: what the write and the
// read of a cache share (gfx950).
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
// TB tokens of the keys (blockIdx.y 0) or of the values (1): its first wave
// looks up the tokens' places and leaves them in LDS; groups of L lanes take a
// few lines each, all of them on their way at once.
#pragma once

#include "nvfp4_launch.h"
#include "nvfp4_rows.h"

#include <algorithm>
#include <type_traits>

namespace nvfp4 {

constexpr int64_t kNoToken = -1;  // no sequence's token: nothing is done
constexpr int64_t kBadPage = -2;  // a token whose page does not exist

// How many of starts[0 .. B] are at most t, 64 probes at a time; a wave, all
// lanes alike. Every index is bounded whatever starts holds.
__device__ __forceinline__ int64_t starts_up_to(const CacheArgs& p, int64_t t, int lane) {
  int64_t lo = 0, n = p.B + 1;
  while (n > 64) {
    const int64_t step = (n + 63) / 64, at = min((lane + 1) * step, n) - 1;
    const int64_t full = __builtin_popcountll(__ballot(p.starts[lo + at] <= t)) * step;
    // (the last probe is the last entry: past t, but for tokens behind the last sequence)
    if (full >= n) return p.B + 1;
    lo += full;
    n = min(step, n - full);
  }
  return lo + __builtin_popcountll(__ballot(lane < n && p.starts[lo + min((int64_t)lane, n - 1)] <= t));
}
// The same, each lane for its own t, by halves.
__device__ __forceinline__ int64_t starts_up_to_lane(const CacheArgs& p, int64_t t) {
  int64_t lo = 0, hi = p.B + 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (p.starts[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// The cache's row (page * page_size + place) of token t of sequence b.
__device__ __forceinline__ int64_t slot_of(const CacheArgs& p, int64_t b, int64_t t) {
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

constexpr int TB_MAX = 64;  // tokens of a workgroup: a lane each

// Where this group's line i0 + u G + grp of the workgroup lies.
struct Line {
  uint32_t t, h;  // token of the workgroup, head
};
// Where a token's lines begin: in the cache and in the caller's rows. (64-bit
// products take a wave 64 cycles and more each: once a token, not once a line.)
struct Place {
  int64_t line;  // kNoToken, kBadPage or the first line's index
  int64_t q, s;  // offsets of its codes and block scales
  int64_t row;   // of its elements, from the workgroup's first token
};

// Looks up a workgroup's tokens, a lane of the first wave each. (All of them in one
// sequence is the rule where tokens are many; a search by a wave for each token
// took 60 us of 131072 tokens' 230.)
__device__ __forceinline__ void find_places(const CacheArgs& p, int64_t t0, int nt, Place* places) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int64_t b = starts_up_to(p, t0, lane) - 1;
    if (lane < nt) {
      const int64_t t = t0 + lane;
      if (b < 0 || (b < p.B && t >= p.starts[b + 1])) b = starts_up_to_lane(p, t) - 1;
      const int64_t slot = slot_of(p, b, t);
      const int64_t pq = p.fmt == FMT_NVFP4 ? (p.D + 1) / 2 : p.D, ps = (p.D + 15) / 16;
      const int64_t line = slot < 0 ? slot : slot * p.H, at = slot < 0 ? 0 : line;
      places[lane] = Place{line, at * pq, at * ps, lane * p.stride[blockIdx.y]};
    }
  }
  __syncthreads();
}
// i / H for i < 2^16, by h_inv = ceil(2^32 / H): i h_inv / 2^32 lies past i / H by less than
// i / 2^32, and i / H at least 1 / H below the next whole number
__device__ __forceinline__ uint32_t over_heads(const CacheArgs& p, uint32_t i) {
  return p.H == 1 ? i : __umulhi(i, p.h_inv);
}

__device__ __forceinline__ Line line_of(const CacheArgs& p, uint32_t i) {
  const uint32_t t = over_heads(p, i);
  return {t, i - __umul24(t, (uint32_t)p.H)};
}

// Tokens of a workgroup whose groups take `of_group` lines each, unless that leaves the
// card short of workgroups, or their rows lie past 32-bit offsets.
inline int tokens_of_block(const CacheArgs& a, int L, int of_group) {
  if (std::max(a.stride[0], a.stride[1]) >= (int64_t)1 << 26) return 1;
  const int64_t lines = of_group * (256 / L), fill = (a.T + 1023) / 1024;
  return (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)TB_MAX, lines / a.H, fill}));
}

template <typename F>
static int launch_tokens(const CacheArgs& a, int L, int of_group, F launch) {
  const int tb = tokens_of_block(a, L, of_group);
  // a launch holds fewer than 2^32 threads
  for (int64_t t = 0; t < a.T; t += (int64_t)tb << 22) {
    CacheArgs p = a;
    p.t0 = t;
    p.h_inv = (uint32_t)((((uint64_t)1 << 32) + a.H - 1) / a.H);
    const int64_t blocks = std::min<int64_t>((a.T - t + tb - 1) / tb, 1 << 22);
    launch(p, dim3((unsigned)blocks, a.q[1] ? 2u : 1u), tb);
    if (hipGetLastError() != hipSuccess) return -3;
  }
  return 0;
}

// launch(lanes of a line, runs of 8 elements a lane, format, D a multiple of 8) as
// constants, D <= 1024
template <typename F>
static int by_line(const CacheArgs& a, F launch) {
  auto even = [&](auto l, auto v, auto f) {
    return a.D % 8 == 0 ? launch(l, v, f, std::true_type{}) : launch(l, v, f, std::false_type{});
  };
  auto fmt = [&](auto l, auto v) {
    if (a.fmt == FMT_E4M3) return even(l, v, std::integral_constant<int, FMT_E4M3>{});
    if (a.fmt == FMT_INT8) return even(l, v, std::integral_constant<int, FMT_INT8>{});
    return even(l, v, std::integral_constant<int, FMT_NVFP4>{});
  };
  using C1 = std::integral_constant<int, 1>;
  const int64_t chunks = (a.D + 7) / 8;
  if (chunks <= 8) return fmt(std::integral_constant<int, 8>{}, C1{});
  if (chunks <= 16) return fmt(std::integral_constant<int, 16>{}, C1{});
  if (chunks <= 32) return fmt(std::integral_constant<int, 32>{}, C1{});
  if (chunks <= 64) return fmt(std::integral_constant<int, 64>{}, C1{});
  return fmt(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
}

}  // namespace nvfp4
