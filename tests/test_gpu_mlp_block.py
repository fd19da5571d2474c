"""The example's MLP block: every product of a training and a decode step against
its dequantized operands. A BF16 output is within 2^-9 of its value; the
dequantized operands carry FP32 roundings only."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,width,hidden", [(300, 256, 704), (33, 130, 75), (1024, 1024, 2816)])
def test_mlp_block(tokens, width, hidden):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    spec = importlib.util.spec_from_file_location("mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    got = m.main(tokens, width, hidden)
    assert len(got) == 9
    for name, err in got.items():
        if name == "decode against training":
            assert err < 0.2, (name, err)     # 4-bit against 8-bit tokens
        elif "weight" in name:
            assert err < 1e-5, (name, err)    # FP32
        else:
            assert err < 2.0 ** -8, (name, err)
