"""One token through a linear layer, by the product that quantises it and by the two launches: which of them a size takes
follows modelled times.  The bound is that of test_gpu_blk.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_moe_expert_gb300 as bm  # noqa: E402
import blk_ref  # noqa: E402
from test_gpu_blk import TYPES, _built  # noqa: E402,F401


def _spread(s, N, K):
    return s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def _linear(N, K, kind):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    x = torch.randn(2, K + 16, device="cuda", generator=gen).to(TYPES[kind])[1:, 16:]   # a row inside a larger tensor
    m = bm.BlkMat.empty(1, N, K)
    m.q.random_(0, 120, generator=gen).bitwise_or_(torch.randint(0, 2, m.q.shape, device="cuda", generator=gen, dtype=torch.uint8) << 7)
    m.s.uniform_(0.5, 1.5, generator=gen)
    ws = bm.workspace(bm.moe_blk_linear_workspace_bytes(1, N, K))
    y = torch.full((2, N), 7.0, dtype=torch.float32, device="cuda")
    bm.moe_blk_linear(x, m, y[:1], ws)
    assert bm.moe_check_status(ws) == 0 and (y[1] == 7).all()
    a = torch.from_numpy(blk_ref.rounded(x.double().cpu().numpy())).cuda()
    w = m.q[0].view(torch.float8_e4m3fn).double() * _spread(m.s[0], N, K)
    want = a @ w.t()
    bound = (4 * 2.0 ** -22 + (K / 128 + 18) * 2.0 ** -24) * (a.abs() @ w.abs().t())
    assert ((y[:1] >= (want - bound).float()) & (y[:1] <= (want + bound).float())).all()
    return x, m, y[:1], ws


@pytest.mark.parametrize("N,K", [(128, 65536), (1024, 16384), (256, 16384), (8193, 16400), (1, 32768)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_long_sums_take_the_product_of_codes(N, K, kind):
    """Eight warps through all of K take far longer there (16384 -> 1024 14 us, the two launches 10)."""
    x, m, y, ws = _linear(N, K, kind)
    a, z = bm.BlkAct.empty(1, K), torch.empty_like(y)
    bm.moe_blk_quantize(x, a)
    bm.moe_blk_matmul(a, m, z, ws)
    assert torch.equal(y, z)


@pytest.mark.parametrize("N,K", [(512, 8192), (24576, 2048), (16, 4096), (17, 1040)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_short_sums_take_one_launch(N, K, kind):
    _linear(N, K, kind)


def test_both_ways_in_one_graph():
    """Captured and replayed with a new row in the same memory."""
    runs = [_linear(N, K, "bf16") for N, K in ((128, 65536), (2048, 512), (1024, 16384))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for x, m, y, ws in runs:
            bm.moe_blk_linear(x, m, y, ws)
    for x, _, y, _ in runs:
        x.copy_(x.flip(1))
    g.replay()
    torch.cuda.synchronize()
    for x, m, y, ws in runs:
        z = torch.empty_like(y)
        bm.moe_blk_linear(x, m, z, ws)
        assert torch.equal(y, z) and y.abs().max() > 0
