"""The MXFP4 layer's example runs and stays near the unquantised layer.

Rounding to MXFP4 leaves a relative error of about 0.11 (root mean square) on normally distributed values: E2M1's spacing
over the range of a block.  Weights and activations of two products, each with such an error, add up to between sqrt(2) and
sqrt(4) times that, the gate's slope to a little more: 0.1 to 0.35."""
import os
import runpy

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_mx_layer_example(capsys):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_moe_expert_gb300 import build
    build.build()
    result = runpy.run_path(os.path.join(ROOT, "examples", "mx_layer.py"))["main"]()
    assert set(result) == {512, 1}
    assert all(0.1 < v < 0.35 for v in result.values()), result
    assert "tokens" in capsys.readouterr().out
