"""The block-scaled 8-bit block's example runs and stays near the unquantised one.

Rounding to E4M3 leaves a relative error of 2^-4/sqrt(3) times about 0.7 (the spacing is between 1/16 and 1/8 of the value):
0.026 (root mean square).  Weights and activations of two products, each with such an error, add up to between sqrt(2) and
sqrt(4) times that, the gate's slope to a little more: 0.02 to 0.1."""
import os
import runpy

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_blk_layer_example(capsys):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_moe_expert_gb300 import build
    build.build()
    result = runpy.run_path(os.path.join(ROOT, "examples", "blk_layer.py"))["main"]()
    assert set(result) == {512, 1}
    assert all(0.02 < v < 0.1 for v in result.values()), result
    assert "tokens" in capsys.readouterr().out
