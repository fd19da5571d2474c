"""Host side, on stand-ins for the runtime's launch calls: the sizes of the GPU
tests reach every kernel of the 8-bit integer product and quantizers, the layer
norm and the cache; and at the largest sizes that the calls take, every launch
has fewer than 2^32 threads and at most 65535 workgroups along y."""
import pytest

import launch_stub
import precision_quantization_row_amd as p
from launch_stub import F, L, W

COLS = 1 << 27


def gemm(M, N, K, act=0):
    return ["nvfp4_int8_gemm", "pippiplllpiipppipp", [F, 1, F, F, 1, F, M, N, K, None, 0, act, None, None, F, 0, None, None]]


def quant(M, K, dt=0):
    return ["nvfp4_int8_quantize", "pillpppp", [F, dt, M, K, F, F, None, None]]


def rowcol(M, K, dt=0):
    return ["nvfp4_int8_quantize_rowcol", "pillpppppp", [F, dt, M, K, F, F, F, F, None, None]]


def norm(M, K, dt=0, wd=0):
    return ["nvfp4_layernorm", "ppippifllppippippp" + "fpp",
            [F, None, dt, F, F, wd, 1e-5, M, K, None, F, 0, F, F, 0, None, None, None, 448.0, None, None]]


def norm_bwd(M, K, dt=0, wd=0):
    return ["nvfp4_layernorm_backward", "ppipipppllppppl" + "pp", [F, F, dt, F, wd, F, F, None, M, K, F, F, F, W, L, None, None]]


def write(T, H, D, fmt, dt=0, stride=None, v=True):
    s, q = (F if fmt == 2 else None), (F if v else None)
    st = H * D if stride is None else stride
    return ["nvfp4_cache_write", "plplilllifllppppppplipppp".replace("plipppp", "pllpppp"),
            [F, st, q, st if v else 0, dt, T, H, D, fmt, 448.0, 100, 16, F, s, F, q, s if v else None, q, F, 4, 50, F, None, None, None]]


def read(T, H, D, fmt, dt=0, v=True):
    s, q = (F if fmt == 2 else None), (F if v else None)
    return ["nvfp4_cache_read", "ppppppifllpllpplllplplipp",
            [F, s, F, q, s if v else None, q, fmt, 448.0, 100, 16, F, 4, 50, F, None, T, H, D, F, H * D, q, H * D if v else 0, dt, None, None]]


# sizes of the GPU tests
GEMM = [(1, 1, 1), (16, 96, 1000), (2, 130, 1025), (3, 1000, 4097), (1, 1100, 122017), (2, 1100, 122017), (4, 1100, 122017), (7, 1100, 122017),
        (16, 9000, 15001), (30, 1100, 122017), (50, 1100, 122017), (1, 4096, 4096), (16, 9000, 1111), (20, 300, 4097), (129, 300, 31), (512, 512, 2880), (1030, 515, 101), (4099, 2601, 515), (4099, 4101, 101)]
GATED = [(1, 72, 200), (5, 96, 64), (2, 131, 1030), (3, 77, 2049), (1, 560, 122017), (2, 560, 122017), (4, 560, 122017), (7, 560, 122017),
         (30, 560, 122017), (50, 560, 122017), (20, 33, 1000), (40, 66, 321), (1030, 300, 101), (4099, 1403, 515), (4099, 2051, 101)]
ROWS = [(3, 7), (5, 512), (3, 513), (3, 2881), (2, 8192), (2, 16384), (1, 28672), (1, 50001)]
BWD = [(50, 7), (2100, 96), (700, 512), (1100, 2048), (700, 4096), (600, 8192), (300, 16384), (300, 17000), (2, 40001)]
HEADS = [(8, 64), (5, 40), (5, 100), (8, 128), (2, 129), (1, 192), (1, 257), (2, 512), (1, 1023), (2, 1024), (2, 7), (3, 250)]
REACHED = [gemm(*s) for s in GEMM] + [gemm(*s, act=p.NVFP4_ACT_SWIGLU) for s in GATED]
REACHED += [f(*s, dt) for f in (quant, rowcol) for s in ROWS for dt in (0, 1)]
REACHED += [f(*s, dt, wd) for f, sizes in ((norm, ROWS), (norm_bwd, BWD)) for s in sizes for dt in (0, 1) for wd in (0, 1)]
REACHED += [f(50, H, D, fmt, dt) for f in (write, read) for H, D in HEADS for fmt in (1, 2, 3) for dt in (0, 1)]

SIZES = [(1, COLS), (2, COLS), (255, COLS), (300, COLS - 32), (1 << 30, 1), (1 << 30, 600), (1 << 26, 40000), (5, 32768), (1 << 20, 32769)]
LARGEST = [f(M, K) for f in (quant, norm, norm_bwd) for M, K in SIZES] + [norm_bwd(M, K, 1) for M, K in SIZES]
LARGEST += [rowcol(*s) for s in ((1, COLS), (COLS, 1), (COLS, 1 << 10), (1 << 10, COLS), (1 << 18, 1 << 19))]   # (2^37 elements: what the memory holds)
LARGEST += [gemm(*s, act=a) for a in (0, 4)
            for s in ((1, 1 << 26, 128), (1, (1 << 26) - 1, (1 << 17) - 1), (32, 1 << 26, 64), (33, 1 << 26, 64), (64, 1 << 22, 512), ((1 << 31) // 4, 1, 16),
                      (1 << 20, 1 << 17, 64), (1 << 22, 16, 1), (1 << 20, 64, 1 << 16), (1 << 18, 1 << 18, 300))]
LARGEST += [f((1 << 31) - 1, H, D, 1) for f in (write, read) for H, D in ((1, 1), (1, 1024), (8, 128), (65535, 1024))]
LARGEST += [write((1 << 31) - 1, 8, 128, 3, stride=1 << 40)]


@pytest.fixture(scope="module")
def seen(tmp_path_factory):
    return launch_stub.launches(REACHED + LARGEST, tmp_path_factory.mktemp("stub"))


def test_sizes_reach_every_kernel(seen):
    names, out = seen
    ours = {n for n in names if any(k in n for k in ("int8_", "ln_", "cache_"))}
    assert len(ours) > 120
    got = {launch[0] for _, grids in out[:len(REACHED)] for launch in grids}
    assert not ours - got


@pytest.mark.parametrize("i", range(len(LARGEST)), ids=lambda i: f"{i}-{LARGEST[i][0]}")
def test_threads_of_a_launch(seen, i):
    rc, grids = seen[1][len(REACHED) + i]
    assert rc == p.NVFP4_OK and grids, LARGEST[i]
    for _, gx, gy, gz, bx, by, bz in grids:
        assert gz == by == bz == 1 and 1 <= bx <= 1024
        assert gx >= 1 and 1 <= gy <= 65535
        assert gx * gy * bx < 1 << 32, (LARGEST[i], gx, gy, bx)
