"""Host side, on stand-ins for the runtime's launch calls: each size of the 8-bit integer product's kernel tests
launches the kernel that it stands for there."""
import re

import pytest

import launch_stub
import precision_quantization_row_amd as p
from test_gpu_int8_tiles import FEW, FEW_GATED, GATED, PLAIN
from test_int8_norm_cache_launches import gemm

TILES = [(s, gated, tile) for gated, sizes in ((False, PLAIN), (True, GATED)) for tile, group in sizes.items() for s in group]
FEWS = [(s, gated) for gated, group in ((False, FEW), (True, FEW_GATED)) for s in group]


@pytest.fixture(scope="module")
def seen(tmp_path_factory):
    calls = [gemm(*s, act=p.NVFP4_ACT_SWIGLU if gated else 0) for s, gated, *_ in TILES + FEWS]
    return [grids for _, grids in launch_stub.launches(calls, tmp_path_factory.mktemp("stub"))[1]]


@pytest.mark.parametrize("i", range(len(TILES)), ids=lambda i: "x".join(map(str, TILES[i][0])))
def test_tiles(seen, i):
    size, gated, (tm, tn) = TILES[i]
    assert len(seen[i]) == 1
    found = re.search(r"int8_tile_kernelILb([01])ELi(\d+)ELi(\d+)E", seen[i][0][0])
    assert found and (bool(int(found[1])), 64 * int(found[2]), 64 * int(found[3])) == (gated, tm, tn), seen[i]


@pytest.mark.parametrize("i", range(len(FEWS)), ids=lambda i: "x".join(map(str, FEWS[i][0])))
def test_few_lines(seen, i):
    (M, _, _), gated = FEWS[i]
    name = seen[len(TILES) + i][0][0]
    assert ("int8_vec_kernel" if M <= 4 else "int8_few_kernel") in name and f"ILb{int(gated)}E" in name, name
