"""RMS norm: the stated error of y in each type, and values at the ends of fp32's range.

y is off by less than 2^-21 of itself before it is rounded to its type, which adds half a step of what is there by then:
|y - y64| <= |y64| (2^-21 + (1 + 2^-21) eps / 2), and in fp16, whose subnormals the drawn values reach, half of their step
(2^-25) more; bf16 and fp32 have none there."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_moe_expert_gb300 as bm  # noqa: E402
import blk_ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_moe_expert_gb300 import build
    build.build()
    bm.lib()


@pytest.mark.parametrize("T,d", [(1, 16), (3, 48), (33, 272), (777, 2816), (600, 8192), (3, 16400), (2, 32768)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_y_to_its_own_bound(T, d, kind):
    rng = np.random.default_rng(3 * T + d)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(TYPES[kind]).cuda()
    res = torch.from_numpy((3 * rng.standard_normal((T, d))).astype(np.float32)).cuda()
    gamma = torch.from_numpy((np.exp(2 * rng.standard_normal(d))).astype(np.float32)).cuda()
    r = (x.double() + res.double()).float()
    y64 = blk_ref.norm(r.double().cpu().numpy(), gamma.double().cpu().numpy(), 1e-6)
    for out in TYPES:
        y = torch.empty((T, d), dtype=TYPES[out], device="cuda")
        bm.moe_rmsnorm(x, gamma, 1e-6, residual=res, stream_out=torch.empty_like(res), Y=y)
        rel = 2.0 ** -21 + (1 + 2.0 ** -21) * torch.finfo(y.dtype).eps / 2
        tiny = 2.0 ** -25 if out == "fp16" else 0.0
        assert (np.abs(y.double().cpu().numpy() - y64) <= np.abs(y64) * rel + tiny).all()


@pytest.mark.parametrize("other", [1.75, 1.0])
@pytest.mark.parametrize("swap", [False, True])
def test_a_y_past_fp32_is_its_own_blocks_affair(other, swap):
    """A block with such a y has a NaN scale, also where the other block of the same 256 columns has its maximum where
    the scale steps up (1.75 times a power of two), which is looked at more closely."""
    x = np.ones((1, 256), np.float32)
    x[0, 200] = 2
    inv = 1 / np.sqrt((x.astype(np.float64) ** 2).mean())
    gamma = np.full(256, other / inv, np.float32)
    gamma[128:] = 1
    gamma[200] = 3e38                                            # y = 6e38
    if swap:
        x, gamma = np.roll(x, 128, 1), np.roll(gamma, 128)
    a = bm.BlkAct.empty(1, 256)
    y = torch.empty((1, 256), dtype=torch.float32, device="cuda")
    bm.moe_rmsnorm(torch.from_numpy(x).cuda(), torch.from_numpy(gamma).cuda(), 0.0, Y=y, out=a)
    at = int(swap)
    assert torch.isinf(y).sum() == 1
    s = a.s[:, 0].cpu().numpy()
    assert np.isnan(s[1 - at]) and np.isfinite(s[at])
    values = torch.empty_like(y)
    bm.moe_blk_dequant(a, values)
    values = values.cpu().numpy()[0]
    bad = slice(128, 256) if not swap else slice(0, 128)
    assert np.isnan(values[bad]).all() and np.isfinite(np.delete(values, np.r_[bad])).all()
