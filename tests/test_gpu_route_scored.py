"""moe_route_scored against the definition in 64 bits: ids and every integer output exactly, weights within the error of
their fp32 evaluation.  A weight takes an exponential (2 units in the last place of 2^-24), a softmax's sum over at most
1024 experts (at most 32 terms in a lane, then 5 levels: 37 roundings at worst), a sum over the selection (5), two divisions,
two products: below 64 roundings of 2^-24, 4e-6.  Rows whose selection hangs on less than 2e-5 are drawn again: their
order has no value in fp32."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_moe_expert_gb300 as bm  # noqa: E402
import mx_ref  # noqa: E402

W_RTOL = 4e-6
GAP = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_moe_expert_gb300 import build
    build.build()
    bm.lib()


def _reference(l, bias, k, kw):
    rows = [mx_ref.route_row(x, kw["score"], bias, k, kw["n_group"], kw["topk_group"], kw["group_top"],
                             kw["renormalize"], kw["scale"]) for x in l]
    return np.array([r[0] for r in rows]).reshape(len(l), k), np.array([r[1] for r in rows]).reshape(len(l), k), \
        np.array([r[2] for r in rows])


def _run(l, bias, k, block_rows, kw, stream=None):
    T, E = l.shape
    out = bm.Routing.empty(T, E, k, block_rows)
    for f in ("ids", "counts", "offsets", "perm", "inv_perm", "block_map"):
        getattr(out, f).fill_(-7)
    ws = bm.workspace(bm.moe_route_workspace_bytes(T, E, k))
    sc = bm.Scoring(bias=torch.from_numpy(bias).cuda() if bias is not None else None, **kw)
    bm.moe_route_scored(torch.from_numpy(l).cuda(), sc, k, block_rows, out, ws, stream)
    torch.cuda.synchronize()
    return out, ws


def _check(out, ids, w, E, block_rows, l1=None):
    got = out.ids.cpu().numpy()
    np.testing.assert_array_equal(got, ids)
    np.testing.assert_allclose(out.w.cpu().numpy(), w, rtol=W_RTOL, atol=1e-38)
    counts, offsets, perm, inv, tiles = mx_ref.tables(ids, E, block_rows)
    A = ids.size
    np.testing.assert_array_equal(out.counts.cpu().numpy(), counts)
    np.testing.assert_array_equal(out.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(out.perm.cpu().numpy()[:A], perm)
    np.testing.assert_array_equal(out.inv_perm.cpu().numpy()[:A], inv)
    n = int(out.num_blocks.item())
    assert n == len(tiles)
    np.testing.assert_array_equal(out.block_map.cpu().numpy()[:n], tiles)
    assert out.block_rows == block_rows


def _kw(score, n_group=1, topk_group=1, group_top=2, renormalize=True, scale=1.0):
    return dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top, renormalize=renormalize,
                scale=scale)


CASES = [  # T, E, k, block_rows, bias, kw
    (1, 256, 8, 16, True, _kw("sigmoid", 8, 4, scale=2.5)),
    (33, 256, 8, 32, True, _kw("softmax", 8, 3)),
    (100, 256, 8, 128, False, _kw("sigmoid", 4, 2, group_top=1, renormalize=False)),
    (64, 130, 6, 64, False, _kw("softmax")),
    (5, 7, 7, 16, True, _kw("sigmoid")),                       # k = E
    (3, 1, 1, 16, False, _kw("softmax", scale=0.5)),           # one expert
    (40, 96, 3, 48, True, _kw("sigmoid", 32, 5)),              # groups of three
    (40, 64, 2, 48, True, _kw("sigmoid", 32, 2, group_top=1)),  # k = topk_group's smallest group share
    (70, 1024, 32, 128, True, _kw("sigmoid", 16, 4)),          # the wide selection
    (20, 300, 9, 100, True, _kw("softmax", 3, 2)),
    (2000, 64, 4, 128, True, _kw("sigmoid", 8, 4)),            # many chunks of tokens
    (30, 1024, 16, 64, True, _kw("sigmoid", 16, 8)),           # more candidates than lanes
    (40, 352, 8, 64, False, _kw("softmax", 4, 2)),             # between the narrow and the wide selection
    (3, 513, 32, 16, True, _kw("sigmoid")),
    (6000, 32, 2, 64, False, _kw("softmax")),                  # chunks that are not resident together
]


@pytest.mark.parametrize("T,E,k,block_rows,with_bias,kw", CASES)
def test_against_the_definition(T, E, k, block_rows, with_bias, kw):
    rng = np.random.default_rng(T * 31 + E)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
    l = rng.standard_normal((T, E)).astype(np.float32)
    ids, w, gap = _reference(l, bias, k, kw)
    for _ in range(20):
        bad = gap < GAP
        if not bad.any():
            break
        l[bad] = rng.standard_normal((int(bad.sum()), E)).astype(np.float32)
        ids[bad], w[bad], gap[bad] = _reference(l[bad], bias, k, kw)
    assert not (gap < GAP).any()
    out, ws = _run(l, bias, k, block_rows, kw)
    _check(out, ids, w, E, block_rows)
    assert bm.moe_check_status(ws) == 0


@pytest.mark.parametrize("mode", ["ticket", "gridsync", ""])
def test_every_way_of_placing_many_chunks(mode, monkeypatch):
    monkeypatch.setenv("MOE_ROUTE_MODE", mode)
    rng = np.random.default_rng(9)
    kw = _kw("softmax", 8, 4)
    T, E, k = 700, 256, 4
    l = rng.standard_normal((T, E)).astype(np.float32)
    out, _ = _run(l, None, k, 32, kw)
    ids = out.ids.cpu().numpy()
    w = np.take_along_axis(mx_ref.scores(l, "softmax"), ids, 1)
    _check(out, ids, w / w.sum(1, keepdims=True), E, 32)


def test_ties_go_to_the_lower_expert_and_the_lower_group():
    E, k = 64, 4
    kw = _kw("sigmoid", 8, 2)
    l = np.zeros((3, E), np.float32)
    l[1, 40:48] = 1.0
    l[2] = np.repeat(np.array([0, 1, 2, 2, 2, 1, 0, 0], np.float32), 8)
    bias = np.full(E, 0.25, np.float32)
    want = [[0, 1, 2, 3], [40, 41, 42, 43], [16, 17, 18, 19]]
    for b in (bias, None):
        out, _ = _run(l, b, k, 16, kw)
        np.testing.assert_array_equal(out.ids.cpu().numpy(), want)
        np.testing.assert_allclose(out.w.cpu().numpy(), 0.25, rtol=W_RTOL)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group", [(64, 1), (64, 4), (512, 8)])
def test_masked_experts(score, E, n_group):
    """-infinity masks: rows with fewer experts than k left, and with none."""
    rng = np.random.default_rng(11)
    k, T = 6, 6
    kw = _kw(score, n_group, max(1, n_group // 2))
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[0, rng.permutation(E)[:E // 2]] = -np.inf
    l[1, :] = -np.inf
    l[2, 3:] = -np.inf                       # three left
    l[3, :-2] = -np.inf                      # the last two
    l[4, E // 2:] = -np.inf
    l[5, :] = -np.inf
    l[5, 0] = -50.0
    for bias in (None, (0.1 * rng.standard_normal(E)).astype(np.float32)):
        ids, w, gap = _reference(l, bias, k, kw)
        assert (gap > 1e-6).all()
        out, ws = _run(l, bias, k, 16, kw)
        _check(out, ids, w, E, 16)
        assert np.isfinite(out.w.cpu().numpy()).all()
        assert bm.moe_check_status(ws) == 0


def test_extreme_logits():
    l = np.zeros((3, 16), np.float32)
    l[0, 5], l[0, 9] = 3e38, -3e38
    l[1, 5], l[1, 9] = 200.0, 100.0
    l[2, :] = -1000.0
    out, ws = _run(l, None, 2, 16, _kw("softmax"))
    np.testing.assert_array_equal(out.ids.cpu().numpy(), [[5, 0], [5, 9], [0, 1]])
    np.testing.assert_allclose(out.w.cpu().numpy(), [[1, 0], [1, np.exp(-100)], [.5, .5]], rtol=1e-5, atol=1e-38)
    assert bm.moe_check_status(ws) == 0


@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_a_non_finite_logit_is_reported_and_counts_as_masked(value):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((40, 32)).astype(np.float32)
    l[7, 4] = value
    kw = _kw("sigmoid")
    out, ws = _run(l, None, 4, 16, kw)
    l[7, 4] = -np.inf
    ids, w, _ = _reference(l, None, 4, kw)
    _check(out, ids, w, 32, 16)
    assert bm.STATUS_NAMES[bm.moe_check_status(ws)] == "MOE_ERR_NONFINITE"
    assert bm.moe_check_status(ws) == 0


def test_agrees_with_moe_route_where_both_say_the_same():
    """Softmax scores, no bias, no groups: moe_route's selection and tables bit for bit."""
    rng = np.random.default_rng(4)
    l = rng.standard_normal((300, 256)).astype(np.float32)
    out, _ = _run(l, None, 8, 64, _kw("softmax"))
    ref = bm.Routing.empty(300, 256, 8, 64)
    bm.moe_route(torch.from_numpy(l).cuda(), 8, 64, ref, bm.workspace(bm.moe_route_workspace_bytes(300, 256, 8)))
    torch.cuda.synchronize()
    for f in ("ids", "counts", "offsets", "perm", "inv_perm", "num_blocks"):
        assert torch.equal(getattr(out, f), getattr(ref, f)), f
    np.testing.assert_allclose(out.w.cpu().numpy(), ref.w.cpu().numpy(), rtol=W_RTOL)


def test_no_tokens_another_stream_and_a_graph():
    kw = _kw("sigmoid", 8, 4)
    out, _ = _run(np.zeros((0, 64), np.float32), None, 4, 16, kw)
    assert int(out.num_blocks.item()) == 0 and int(out.counts.sum()) == 0 and int(out.offsets.abs().sum()) == 0
    rng = np.random.default_rng(5)
    l = rng.standard_normal((50, 64)).astype(np.float32)
    ids, w, _ = _reference(l, None, 4, kw)
    s = torch.cuda.Stream()
    out, _ = _run(l, None, 4, 16, kw, stream=s)
    _check(out, ids, w, 64, 16)
    lg = torch.from_numpy(l).cuda()
    out = bm.Routing.empty(50, 64, 4, 16)
    ws = bm.workspace(bm.moe_route_workspace_bytes(50, 64, 4))
    sc = bm.Scoring(**kw)
    bm.moe_route_scored(lg, sc, 4, 16, out, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bm.moe_route_scored(lg, sc, 4, 16, out, ws)
    out.ids.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    _check(out, ids, w, 64, 16)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 300])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("low,high", [(-95, -88), (-90, -78)])
def test_scores_at_the_end_of_the_range(score, E, renormalize, low, high):
    """Selected scores down to e^-95: weights keep their shares.  A score is off by two units of its last place (2^-149 for
    a subnormal one), a sum of k by as much of each, and the rest is as above."""
    rng = np.random.default_rng(E)
    k = 4
    T = 40
    l = rng.uniform(low, high, (T, E)).astype(np.float32)
    bias = None
    if score == "softmax":  # the largest logit is 0; the bias takes the selection to the small ones
        l[:, 0] = 0.0
        bias = (1 + np.arange(E) / E).astype(np.float32)
        bias[0] = -2.0
    kw = _kw(score, renormalize=renormalize, scale=1.5)
    ids, w, gap = _reference(l, bias, k, kw)
    out, ws = _run(l, bias, k, 16, kw)
    assert bm.moe_check_status(ws) == 0
    got_ids, got = out.ids.cpu().numpy(), out.w.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(got_ids, ids)
    s = np.take_along_axis(mx_ref.scores(l, score), ids, 1)
    unit = 2 * 2.0 ** -149
    if renormalize:
        tol = w * (W_RTOL + unit / s + k * unit / s.sum(1, keepdims=True))
    else:
        tol = w * W_RTOL + (1.5 + 1) * unit
    assert (np.abs(got - w) <= tol).all(), np.max(np.abs(got - w) / tol)


@pytest.mark.parametrize("scored", [True, False])
def test_a_block_map_past_2_31_elements(scored):
    """Tiles of one row, all experts selected: tile b is (b / T, b, 1)."""
    T, E, k = (1 << 31) // 3 // 32 + 9999, 32, 32
    lg = torch.zeros((T, E), dtype=torch.float32, device="cuda")
    out = bm.Routing.empty(T, E, k, 1)
    ws = bm.workspace(bm.moe_route_workspace_bytes(T, E, k))
    if scored:
        bm.moe_route_scored(lg, bm.Scoring(**_kw("softmax")), k, 1, out, ws)
    else:
        bm.moe_route(lg, k, 1, out, ws)
    torch.cuda.synchronize()
    assert bm.moe_check_status(ws) == 0
    n = int(out.num_blocks.item())
    assert n == T * k and 3 * n > 1 << 31
    for b0 in range(0, n, 1 << 26):
        b = torch.arange(b0, min(n, b0 + (1 << 26)), device="cuda")
        want = torch.stack([b // T, b, torch.ones_like(b)], 1).to(torch.int32)
        assert torch.equal(out.block_map[b0:b0 + len(b)], want), b0


def _settled(rng, T, E, k, bias, kw):
    """Logits whose selection hangs on no less than GAP, and the reference."""
    l = rng.standard_normal((T, E)).astype(np.float32)
    ids, w, gap = _reference(l, bias, k, kw)
    for _ in range(20):
        bad = gap < GAP
        if not bad.any():
            break
        l[bad] = rng.standard_normal((int(bad.sum()), E)).astype(np.float32)
        ids[bad], w[bad], gap[bad] = _reference(l[bad], bias, k, kw)
    assert not (gap < GAP).any()
    return l, ids, w


@pytest.mark.parametrize("mode", ["ticket", "gridsync", ""])
@pytest.mark.parametrize("T,E,k,n_group,topk_group", [
    (700, 256, 4, 8, 4),     # bases in shared memory beside the candidates
    (4000, 64, 4, 8, 4),     # between one chunk an SM and half of what is resident: the barrier without being asked
    (700, 300, 6, 3, 2),     # groups that fall on no whole lanes: the widest use of shared memory
])
def test_every_way_of_placing_selects_by_the_definition(T, E, k, n_group, topk_group, mode, monkeypatch):
    monkeypatch.setenv("MOE_ROUTE_MODE", mode)
    rng = np.random.default_rng(T + E)
    kw = _kw("sigmoid", n_group, topk_group, scale=2.5)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    l, ids, w = _settled(rng, T, E, k, bias, kw)
    out, ws = _run(l, bias, k, 32, kw)
    _check(out, ids, w, E, 32)
    assert bm.moe_check_status(ws) == 0


def test_more_chunks_than_the_counts_sums_hold():
    """Past 65,504 tokens the last CTA places everything, with the bases in global memory."""
    rng = np.random.default_rng(12)
    T, E, k = 66000, 16, 2
    kw = _kw("sigmoid", 4, 2)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    l, ids, w = _settled(rng, T, E, k, bias, kw)
    out, ws = _run(l, bias, k, 128, kw)
    _check(out, ids, w, E, 128)
    assert bm.moe_check_status(ws) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [16, 300])
def test_weights_that_have_an_exact_value(score, E):
    """One expert selected, or a power of two of equal ones: exactly scale / k, whatever the scores."""
    rng = np.random.default_rng(E)
    T = 500
    for k in (1, 2, 8):
        l = np.full((T, E), -30.0, np.float32)
        for t in range(T):
            l[t, rng.permutation(E)[:k]] = rng.uniform(-20, 20)
        for scale in (1.0, 2.5):
            out, _ = _run(l, None, k, 16, _kw(score, scale=scale))
            assert (out.w.cpu().numpy() == np.float32(scale / k)).all(), k


@pytest.mark.parametrize("E", [1, 16, 512])
def test_scores_that_have_an_exact_value(E):
    """Without renormalisation: equal shares of a power of two, the logistic function at 0 and far above it."""
    for score, l, want in (("softmax", 3.0, 1 / E), ("sigmoid", 0.0, 0.5), ("sigmoid", 40.0, 1.0)):
        out, _ = _run(np.full((20, E), l, np.float32), None, 1, 16, _kw(score, renormalize=False, scale=2.5))
        assert (out.w.cpu().numpy() == np.float32(2.5 * want)).all(), (score, l)
