"""The library on stand-ins for the runtime's launch calls, in a process of its
own: which kernels a call launches, on which grids. Nothing reaches a GPU, so
addresses are never used."""
import json
import os
import subprocess
import sys

import precision_quantization_row_amd as p

STUB = r"""
#include <stddef.h>
#include <stdint.h>
typedef struct { uint32_t x, y, z; } dim3;
static dim3 grid_, block_;
static size_t shared_;
static void* stream_;
static struct { const void* fn; const char* name; } kernels[4096];
static int nk;
static uint32_t notes[4096][7];
static int count;
static void* module;
void** __hipRegisterFatBinary(const void* d) { return &module; }
void __hipUnregisterFatBinary(void** m) {}
void __hipRegisterFunction(void** m, const void* fn, char* dev, const char* name, unsigned tl, void* tid, void* bid,
                           void* bd, void* gd, int* ws) {
  if (nk < 4096) { kernels[nk].fn = fn; kernels[nk++].name = name; }
}
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t s, void* st) {
  grid_ = g; block_ = b; shared_ = s; stream_ = st;
  return 0;
}
int __hipPopCallConfiguration(dim3* g, dim3* b, size_t* s, void** st) {
  *g = grid_; *b = block_; *s = shared_; *st = stream_;
  return 0;
}
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t s, void* st) {
  if (count < 4096) {
    uint32_t* n = notes[count++];
    int k = 0;
    while (k < nk && kernels[k].fn != f) ++k;
    n[0] = k; n[1] = g.x; n[2] = g.y; n[3] = g.z; n[4] = b.x; n[5] = b.y; n[6] = b.z;
  }
  return 0;
}
int hipGetLastError(void) { return 0; }
int kernel_count(void) { return nk; }
const char* kernel_name(int k) { return kernels[k].name; }
int taken(uint32_t* out) {
  const int n = count;
  for (int i = 0; i < n * 7; ++i) out[i] = notes[i / 7][i % 7];
  count = 0;
  return n;
}
"""

RUN = r"""
import ctypes, json, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)   # found before the runtime's own
lib = ctypes.CDLL(sys.argv[2])
stub.kernel_name.restype = ctypes.c_char_p
names = [stub.kernel_name(k).decode() for k in range(stub.kernel_count())]
conv = {"i": ctypes.c_int, "l": ctypes.c_int64, "f": ctypes.c_float, "p": ctypes.c_void_p}
buf = (ctypes.c_uint32 * (7 * 4096))()
out = []
for fn, kinds, args in json.load(sys.stdin):
    f = getattr(lib, fn)
    f.restype = ctypes.c_int
    rc = f(*[conv[k](a) for k, a in zip(kinds, args)])
    n = stub.taken(buf)
    out.append([rc, [[names[buf[7 * i]]] + list(buf[7 * i + 1:7 * i + 7]) for i in range(n)]])
print(json.dumps([names, out]))
"""

F, W, L = 0x1000, 0x2000, 1 << 40   # (W: the workspace, which is no output)


def gemm(M, N, K, act=0, fmt=2):
    return ["nvfp4_gemm", "ippipfppipflllpiipppipp",
            [fmt, F, F if fmt == 2 else None, 1, F, 448.0, F, F, 1, F, 448.0, M, N, K, None, 0, act, None, None, F, 0, None, None]]


def act(M, N, a=1, dt=0):
    return ["nvfp4_act_backward", "ppillippplpp", [F, F, dt, M, N, a, F, F, W, L, None, None]]


def norm(M, K, dt=0, wd=0):
    return ["nvfp4_rmsnorm", "ppipifllppipipppfpp",
            [F, None, dt, F, wd, 1e-5, M, K, None, F, 0, None, 0, None, None, None, 448.0, None, None]]


def norm_bwd(M, K, dt=0, wd=0):
    return ["nvfp4_rmsnorm_backward", "ppipippllppplpp", [F, F, dt, F, wd, F, None, M, K, F, F, W, L, None, None]]


def launches(calls, folder):
    """(names of the library's kernels, [status, [name, grid, block] of each launch] of each call)."""
    src, lib = os.path.join(folder, "stub.c"), os.path.join(folder, "libstub.so")
    with open(src, "w") as f:
        f.write(STUB)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", src, "-o", lib], check=True)
    p.load_library()
    so = os.path.join(os.path.dirname(p.__file__), "libnvfp4.so")
    r = subprocess.run([sys.executable, "-c", RUN, lib, so], input=json.dumps(calls), capture_output=True, text=True,
                       timeout=100)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)
