// int8_device.h -- what the kernels of the 8-bit integer product share (gfx950).
#pragma once

#include "gemm_device.h"
#include "nvfp4_rows.h"

namespace nvfp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// LDS holds lines of 128 bytes: 16-byte slot s of line r is at s ^ rotate(r), so that
// 16 lanes that read one slot of 16 neighbouring lines touch all 64 banks once (a
// line is half of them), and 8 lanes that write a line too.
__device__ __forceinline__ int rotate(int r) {
  return ((r >> 1) & 1) << 2 | ((r ^ (r >> 3)) & 1) << 1 | ((r >> 2) & 1);
}

// 16 bytes of a line of K bytes from byte `at` on; bytes past the line's end read as
// zero. Only bytes of the line are touched: a run that would cross the end is read
// from the line's last 16 bytes and shifted down.
__device__ __forceinline__ u32x4 tail_chunk(const uint8_t* line, int K, int at) {
  u32x4 w = {0u, 0u, 0u, 0u};
  if (K >= 16) {
    const int o = min(at, K - 16), sh = at - o;
    const u32x4 v = *reinterpret_cast<const u32x4_a1*>(line + o);
    uint32_t t[5] = {v.x, v.y, v.z, v.w, 0u};
    if (sh & 8) {
      t[0] = t[2];
      t[1] = t[3];
      t[2] = t[3] = 0u;
    }
    if (sh & 4) {
      t[0] = t[1];
      t[1] = t[2];
      t[2] = t[3];
      t[3] = 0u;
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] = sh < 16 ? __builtin_amdgcn_alignbyte(t[d + 1], t[d], sh & 3) : 0u;
  } else {
    for (int i = 0; i < 16; ++i)
      if (at + i < K) w[i / 4] |= (uint32_t)line[at + i] << (8 * (i & 3));
  }
  return w;
}

}  // namespace nvfp4
