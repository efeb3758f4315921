"""RMS norm with the residual's addition against 64 bits.

The residual stream is exact: the sum of two numbers of its type rounds the same from 32 and from 64 bits (fp32's 24 bits
hold it wherever it lies near the middle of two values of a 16-bit type).  y is off by less than 2^-21 of itself before its
own rounding (half a step).  Codes and scales are those of the exact y wherever it is further than 2^-27 of itself from
where the next code or scale begins."""
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


def _to(x, kind):
    return torch.from_numpy(np.asarray(x, np.float32)).to(TYPES[kind]).cuda()


def _check_codes(a, y64):
    rows, d = y64.shape
    v, s = blk_ref.quantise(y64)
    got_s = a.s.cpu().numpy()[:, :rows].T.astype(np.float64)
    near = blk_ref.quantise(y64 * (1 - 2.0 ** -27)), blk_ref.quantise(y64 * (1 + 2.0 ** -27))
    assert ((got_s == s) | (got_s == near[0][1]) | (got_s == near[1][1])).all()
    got = blk_ref.decode(a.q.cpu().numpy())
    same = blk_ref.spread(got_s == s, d)
    assert ((got == v) | (got == near[0][0]) | (got == near[1][0]) | ~same).all()
    assert same.mean() > 0.999


def _check_y(y, y64):
    eps = torch.finfo(y.dtype).eps / 2
    y = y.double().cpu().numpy()
    tiny = float(torch.finfo(torch.float16).smallest_normal) * 2.0 ** -11  # half a step of fp16's subnormals
    assert (np.abs(y - y64) <= np.abs(y64) * (eps + 2.0 ** -21) + tiny).all()


SIZES = [(1, 16), (1, 2048), (3, 48), (5, 128), (2, 1040), (33, 272), (777, 2816), (600, 8192), (2, 8208), (513, 8208),
         (3, 16400), (2, 32768)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("x_kind,r_kind", [("bf16", None), ("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", None),
                                           ("fp16", "fp32"), ("fp32", "fp32"), ("fp32", None)])
def test_rmsnorm(T, d, x_kind, r_kind):
    rng = np.random.default_rng(T + d)
    x = _to(rng.standard_normal((T, d)), x_kind)
    gamma = _to(1 + 0.2 * rng.standard_normal(d), "fp32" if d % 32 else "bf16")
    res = _to(3 * rng.standard_normal((T, d)) * np.exp(0.7 * rng.standard_normal(d)), r_kind) if r_kind else None
    r = x.double()
    if res is not None:
        r = (r + res.double()).to(res.dtype).double()
    y64 = blk_ref.norm(r.cpu().numpy(), gamma.double().cpu().numpy(), 1e-6)
    y, a = torch.empty_like(x), bm.BlkAct.empty(T, d)
    kept = res.clone() if res is not None else None
    stream = torch.empty_like(res) if res is not None else None
    bm.moe_rmsnorm(x, gamma, 1e-6, residual=res, stream_out=stream, Y=y, out=a)
    if res is not None:
        assert torch.equal(stream.double(), r) and torch.equal(res, kept)
    _check_y(y, y64)
    _check_codes(a, y64)
    # one output at a time, the stream in place, another type of y
    b = bm.BlkAct.empty(T, d)
    bm.moe_rmsnorm(x, gamma, 1e-6, residual=res, out=b)
    assert torch.equal(a.q, b.q) and torch.equal(a.s[:, :T], b.s[:, :T])
    if res is not None:
        assert torch.equal(res, stream)
        res.copy_(kept)
    y32 = torch.empty((T, d), dtype=torch.float32, device="cuda")
    bm.moe_rmsnorm(x, gamma, 1e-6, residual=res, Y=y32)
    _check_y(y32, y64)


def test_strided_rows_and_another_stream():
    rng = np.random.default_rng(2)
    x = _to(rng.standard_normal((20, 512)), "bf16")[1:18, 64:320]
    gamma = _to(rng.standard_normal(256), "bf16")
    y, a = torch.empty((17, 256), dtype=torch.bfloat16, device="cuda"), bm.BlkAct.empty(17, 256)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    bm.moe_rmsnorm(x, gamma, 1e-5, Y=y, out=a, stream=st)
    torch.cuda.synchronize()
    y64 = blk_ref.norm(x.double().cpu().numpy(), gamma.double().cpu().numpy(), 1e-5)
    _check_y(y, y64)
    _check_codes(a, y64)


def test_edges():
    """Zeros, tiny and large rows, and rows with a NaN or an infinity, which stay their own."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((8, 256))
    x[1] = 0
    x[2] *= 1e-20
    x[3] *= 1e15
    x[4, 7] = np.nan
    x[5, 200] = np.inf
    x[6, :] = 1e30                      # squares past fp32's range
    x[7, 1:] = 0
    x = _to(x, "fp32")
    gamma = torch.ones(256, device="cuda")
    y, a = torch.empty_like(x), bm.BlkAct.empty(8, 256)
    bm.moe_rmsnorm(x, gamma, 1e-6, Y=y, out=a)
    values = torch.empty_like(x)
    bm.moe_blk_dequant(a, values)
    good = [0, 1, 2, 3, 7]
    y64 = blk_ref.norm(x.double().cpu().numpy()[good], np.ones(256), 1e-6)
    yh = y.double().cpu().numpy()
    assert (np.abs(yh[good] - y64) <= np.abs(y64) * (2.0 ** -21 + 2.0 ** -24)).all()
    assert np.isnan(yh[4:7]).all() and torch.isnan(values[4:7]).all()
    np.testing.assert_array_equal(values.double().cpu().numpy()[good], blk_ref.rounded(y64))


@pytest.mark.parametrize("T,d", [(1, 2048), (300, 512), (4001, 2048), (1300, 8192)])
@pytest.mark.parametrize("x_kind,r_kind", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32")])
def test_norms_in_place_one_after_another(T, d, x_kind, r_kind):
    """Each call reads the stream, and the X, that the one before it wrote where it had read them: the results of a program
    that waits for each."""
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    x0 = torch.randn(T, d, device="cuda", generator=gen).to(TYPES[x_kind])
    res0 = torch.randn(T, d, device="cuda", generator=gen).to(TYPES[r_kind])
    gamma = 1 + 0.1 * torch.randn(d, device="cuda", generator=gen)
    got = {}
    for wait in (True, False):
        x, res, a = x0.clone(), res0.clone(), bm.BlkAct.empty(T, d)
        for _ in range(12):
            bm.moe_rmsnorm(x, gamma, 1e-6, residual=res, Y=x, out=a)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        got[wait] = x, res, a.q, a.s[:, :T]
    assert torch.isfinite(got[True][1]).all()
    assert all(torch.equal(p, q) for p, q in zip(got[True], got[False]))
    # the first call against 64 bits
    x, res = x0.clone(), res0.clone()
    bm.moe_rmsnorm(x, gamma, 1e-6, residual=res, Y=x)
    r = (x0.double() + res0.double()).to(res0.dtype)
    assert torch.equal(res, r)
    _check_y(x, blk_ref.norm(r.double().cpu().numpy(), gamma.double().cpu().numpy(), 1e-6))
