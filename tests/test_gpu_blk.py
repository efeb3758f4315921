"""Block-scaled 8-bit floating point: quantisation and its inverse exactly, products and expert layers against 64 bits.

Products: the codes' products are exact, so an error comes from the fp32 accumulation alone.  The tensor cores add 32
products at a time and may drop bits below the last place of the largest: two last places (2^-22) of the sum of
magnitudes for each of the four additions of a block of 128.  Then the two scales' product and its product with the
block's sum (2^-24 each), and one addition (2^-24 of the sum so far) per block, and up to 16 more where the blocks are
added up in shares: |Y - Y64| <= bound = (4 2^-22 + (K/128 + 18) 2^-24) sum_k |a_k w_k|.  Rounding is monotone, so a Y
in fewer bits lies between the values nearest to Y64 - bound and Y64 + bound: exact but for the sum.

Expert layers: the hidden values are rounded to E4M3 from fp32 sums here and from 64 bits in the reference.  They differ
by about 1e-6 of themselves, so about 3e-5 of them (that over the spacing of E4M3, 1/16 to 1/8) land on the other side of
a rounding, by at most 1/8 of themselves: 7e-4 of the norm of h and of Y.  With bf16's own 2^-9/sqrt(3): relative L2 error
below 3e-3.  One such value moves an element of Y by its share of it, about 1/sqrt(I) of the root mean square; a few at
once stay below 3/sqrt(I) + 2^-8."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_moe_expert_gb300 as bm  # noqa: E402
import blk_ref  # noqa: E402
import mx_ref  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_moe_expert_gb300 import build
    build.build()
    bm.lib()


TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _to(x, kind):
    return torch.from_numpy(np.asarray(x, np.float32)).to(TYPES[kind]).cuda()


def _mat(mat):
    return bm.BlkMat(*(torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in mat))


def _act(v, s):
    """E4M3 values [rows][K] and scales [rows][blocks] -> a BlkAct whose padding is NaN."""
    a = bm.BlkAct.empty(*v.shape)
    a.s.fill_(float("nan"))
    a.q.copy_(torch.from_numpy(blk_ref.encode(v)))
    a.s[:, :v.shape[0]] = torch.from_numpy(np.ascontiguousarray(s.T.astype(np.float32)))
    return a


def _check_codes(q, s, v64, s64):
    """Codes (as bytes) and scales [rows][blocks] against the reference's, NaN blocks aside."""
    np.testing.assert_array_equal(s, s64)
    ok = ~np.isnan(blk_ref.spread(s64, v64.shape[-1]))
    np.testing.assert_array_equal(blk_ref.decode(q)[ok], v64[ok])


ROWS = [(1, 16), (1, 2048), (3, 48), (5, 128), (33, 160), (130, 272), (7, 4112), (1000, 528), (2, 20000)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,K", ROWS)
def test_quantise_rows(kind, rows, K):
    rng = np.random.default_rng(rows + K)
    x = _to(rng.standard_normal((rows, K)) * np.exp2(rng.integers(-12, 12, (rows, 1))), kind)
    a = bm.BlkAct.empty(rows, K)
    bm.moe_blk_quantize(x, a)
    x64 = x.double().cpu().numpy()
    v, s = blk_ref.quantise(x64)
    _check_codes(a.q.cpu().numpy(), a.s.cpu().numpy()[:, :rows].T, v, s)
    for out in TYPES:
        y = torch.empty((rows, K), dtype=TYPES[out], device="cuda")
        bm.moe_blk_dequant(a, y)
        want = torch.from_numpy(v * blk_ref.spread(s, K)).to(TYPES[out])
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (1, 128, 128), (3, 131, 416), (2, 704, 272), (1, 257, 2064)])
def test_quantise_weights(kind, E, N, K):
    rng = np.random.default_rng(E + N + K)
    w = _to(rng.standard_normal((E, N, K)) * np.exp2(rng.integers(-9, 9, (E, N, 1))), kind)
    m = bm.BlkMat.empty(E, N, K)
    bm.moe_blk_quantize_weights(w, m)
    v, s = blk_ref.quantise_weights(w.double().cpu().numpy())
    np.testing.assert_array_equal(m.s.cpu().numpy(), s)
    np.testing.assert_array_equal(blk_ref.decode(m.q.cpu().numpy()), v)
    for out in TYPES:
        y = torch.empty((E, N, K), dtype=TYPES[out], device="cuda")
        bm.moe_blk_dequant(m, y)
        want = torch.from_numpy(blk_ref.weights((blk_ref.encode(v), s))).to(TYPES[out])
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("kind", list(TYPES))
def test_quantise_edges(kind):
    """Ties at every scale; magnitudes at and next to 448; zeros; the smallest and largest numbers; NaN and infinity."""
    g = blk_ref.GRID
    ties = np.concatenate([(g[:-1] + g[1:]) / 2, [448.0]])           # 126 midpoints and the largest code
    ties = np.concatenate([ties, [-448.0]]) * np.where(np.arange(128) % 3 == 0, -1, 1)
    info = torch.finfo(TYPES[kind])
    rows = [ties * 2.0 ** e for e in (-6, 0, 5)] if kind != "bf16" else [ties, ties * 2.0 ** -20, ties * 2.0 ** 40]
    for top in (447.0, 448.0, 450.0, 512.0, 224.0):
        rows.append(np.where(np.arange(128) == 5, top, np.arange(128) / 7))
    rows += [np.zeros(128), np.where(np.arange(128) == 3, info.max, 1.0), np.where(np.arange(128) == 3, -info.max, 0.0)]
    rows += [np.full(128, info.tiny), np.where(np.arange(128) % 2, info.smallest_normal / 2, 0.0)]
    rows += [np.where(np.arange(128) == 9, np.nan, ties), np.where(np.arange(128) == 31, -np.inf, ties)]
    x = torch.tensor(np.stack(rows), dtype=torch.float64).to(TYPES[kind]).cuda()
    a = bm.BlkAct.empty(*x.shape)
    bm.moe_blk_quantize(x, a)
    v, s = blk_ref.quantise(x.double().cpu().numpy())
    _check_codes(a.q.cpu().numpy(), a.s.cpu().numpy()[:, :len(rows)].T, v, s)
    y = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    bm.moe_blk_dequant(a, y)
    y = y.cpu().numpy()
    assert np.isnan(y[-2:]).all()
    # bf16's and fp32's largest number is 255 and more 2^120: the nearest code (steps of 16) stands for 256 2^120 = 2^128,
    # which fp32 rounds to infinity
    with np.errstate(over="ignore"):
        np.testing.assert_array_equal(y[:-2], (v * blk_ref.spread(s, 128))[:-2].astype(np.float32))
    m = bm.BlkMat.empty(len(rows), 1, 128)
    bm.moe_blk_quantize_weights(x.view(-1, 1, 128), m)
    _check_codes(m.q.cpu().numpy()[:, 0], m.s.cpu().numpy()[:, 0], v, s)


def test_quantise_strided_rows_and_another_stream():
    rng = np.random.default_rng(1)
    x = _to(rng.standard_normal((40, 512)), "bf16")[3:29, 64:240]
    a = bm.BlkAct.empty(26, 176)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    bm.moe_blk_quantize(x, a, stream=st)
    torch.cuda.synchronize()
    _check_codes(a.q.cpu().numpy(), a.s.cpu().numpy()[:, :26].T, *blk_ref.quantise(x.double().cpu().numpy()))


SIZES = [(1, 1, 16), (1, 2048, 2048), (1, 130, 48), (2, 8, 4112), (3, 33, 160), (8, 200, 1040), (9, 64, 128), (16, 128, 64),
         (17, 200, 272), (63, 129, 512), (128, 513, 288), (129, 129, 512), (200, 31, 1056), (300, 700, 2048), (257, 512, 32),
         (1000, 256, 320), (640, 1000, 4096), (1300, 2080, 400), (2433, 1500, 144), (1000, 2601, 1040), (1537, 4000, 128)]


def _assert_product(y, av, wv, K):
    want = av @ wv.T
    bound = (4 * 2.0 ** -22 + (K / 128 + 18) * 2.0 ** -24) * (np.abs(av) @ np.abs(wv).T)
    low, high = (torch.from_numpy(v).to(y.dtype).double().numpy() for v in (want - bound, want + bound))
    y = y.double().cpu().numpy()
    assert np.isfinite(y).all()
    worst = np.maximum(low - y, y - high)
    assert worst.max() <= 0, (worst.max(), np.argwhere(worst > 0)[:5], len(np.argwhere(worst > 0)))


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("y_kind", list(TYPES))
def test_matmul(M, N, K, y_kind):
    """Operands with any fp32 scales, their padding NaN."""
    rng = np.random.default_rng(M + N + K)
    v, s = blk_ref.quantise(rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1))))
    s = (s * rng.uniform(0.6, 1.7, s.shape)).astype(np.float32)
    mat = blk_ref.draw_matrix(rng, 1, N, K)
    ws = bm.workspace(256)
    y = torch.full((M + 1, N), 7.0, dtype=TYPES[y_kind], device="cuda")
    bm.moe_blk_matmul(_act(v, s), _mat(mat), y[:M], ws)
    assert bm.moe_check_status(ws) == 0
    assert (y[M] == 7).all()                                         # nothing behind the last row
    _assert_product(y[:M], v * blk_ref.spread(s.astype(np.float64), K), blk_ref.weights(mat)[0], K)


@pytest.mark.parametrize("M,N,K", [(8, 8192, 8192), (16, 2049, 8208), (33, 130, 4112), (48, 1000, 1040), (64, 640, 2064), (70, 1001, 1040),
                                   (96, 129, 272), (100, 300, 20016), (333, 1001, 2816), (500, 256, 1168)])
def test_matmul_whose_blocks_several_ctas_share(M, N, K):
    """Few tiles and many blocks of columns, a short last one among them; the same bits in every call."""
    rng = np.random.default_rng(M + N + K)
    v, s = blk_ref.quantise(rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1))))
    s = (s * rng.uniform(0.6, 1.7, s.shape)).astype(np.float32)
    mat = blk_ref.draw_matrix(rng, 1, N, K)
    a, m, ws = _act(v, s), _mat(mat), bm.workspace(256)
    y = torch.full((M + 1, N), 7.0, dtype=torch.float32, device="cuda")
    first = None
    for _ in range(4):
        bm.moe_blk_matmul(a, m, y[:M], ws)
        assert first is None or torch.equal(y, first)
        first = y.clone()
    assert bm.moe_check_status(ws) == 0
    assert (y[M] == 7).all()
    _assert_product(y[:M], v * blk_ref.spread(s.astype(np.float64), K), blk_ref.weights(mat)[0], K)


@pytest.mark.parametrize("T,N,K", [(1, 2048, 2048), (1, 17, 16), (5, 100, 1040), (8, 2048, 512), (9, 300, 272), (333, 1001, 2816)])
@pytest.mark.parametrize("x_kind", list(TYPES))
def test_linear(T, N, K, x_kind):
    rng = np.random.default_rng(T + N + K)
    x = _to(rng.standard_normal((T, K + 16)), x_kind)[:, :K]         # strided rows
    mat = blk_ref.draw_matrix(rng, 1, N, K)
    ws = bm.workspace(bm.moe_blk_linear_workspace_bytes(T, N, K))
    y = torch.empty((T, N), dtype=torch.float32, device="cuda")
    bm.moe_blk_linear(x, _mat(mat), y, ws)
    assert bm.moe_check_status(ws) == 0
    _assert_product(y, blk_ref.rounded(x.double().cpu().numpy()), blk_ref.weights(mat)[0], K)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_nan_stays_in_its_row_and_column(M):
    rng = np.random.default_rng(M)
    v, s = blk_ref.quantise(rng.standard_normal((M, 512)))
    mat = blk_ref.draw_matrix(rng, 1, 300, 512)
    mat[0][0, 77, 400] = 0x7F                                        # a NaN weight
    a = _act(v, s)
    a.q[1, 130] = 0xFF                                               # a NaN code
    a.s[0, 2] = float("nan")                                         # a NaN scale
    y = torch.empty((M, 300), dtype=torch.float32, device="cuda")
    bm.moe_blk_matmul(a, _mat(mat), y, bm.workspace(256))
    bad = torch.isnan(y).cpu().numpy()
    want = np.zeros((M, 300), bool)
    want[1:3] = want[:, 77] = True
    np.testing.assert_array_equal(bad, want)


def test_weights_just_quantised():
    """A product may follow its weights' quantisation directly, whatever was in that memory before."""
    rng = np.random.default_rng(5)
    T, N, K = 4, 4096, 2048
    x = _to(rng.standard_normal((T, K)), "bf16")
    m = bm.BlkMat.empty(1, N, K)
    ws = bm.workspace(bm.moe_blk_linear_workspace_bytes(64, N, K))
    for rows in (T, 64):
        xr = x.repeat(rows // T, 1)
        for i in range(3):
            w = _to(rng.standard_normal((1, N, K)), "bf16")
            m.q.fill_(0x7F)
            torch.cuda.synchronize()
            y = torch.empty((rows, N), dtype=torch.float32, device="cuda")
            bm.moe_blk_quantize_weights(w, m)
            bm.moe_blk_linear(xr, m, y, ws)
            v, s = blk_ref.quantise_weights(w.double().cpu().numpy())
            _assert_product(y, blk_ref.rounded(xr.double().cpu().numpy()), blk_ref.weights((blk_ref.encode(v), s))[0], K)


# ------------------------------------------------------------------ expert layers

def _experts(rng, E, d, I):
    host = [blk_ref.draw_matrix(rng, E, *nk) for nk in ((I, d), (I, d), (d, I))]
    return host, bm.BlkExperts(*(_mat(m) for m in host))


def _routing(ids, w, E, rows):
    T, k = ids.shape
    r = bm.Routing.empty(T, E, k, rows)
    counts, offsets, perm, inv, tiles = mx_ref.tables(ids, E, rows)
    for name, v in (("ids", ids), ("w", w), ("counts", counts), ("offsets", offsets), ("perm", perm), ("inv_perm", inv)):
        getattr(r, name).copy_(torch.from_numpy(np.ascontiguousarray(v)))
    r.block_map[:len(tiles)] = torch.from_numpy(tiles.astype(np.int32)).cuda()
    r.num_blocks.fill_(len(tiles))
    return r


def _draw_routing(rng, T, E, k, rows, hot=0.0):
    """Distinct experts per token; with `hot` some experts are far more popular."""
    p = rng.random((T, E)) + hot * (np.arange(E) < max(1, E // 8))
    ids = np.argsort(-p, axis=1)[:, :k]
    w = rng.random((T, k)).astype(np.float32)
    w /= w.sum(1, keepdims=True)
    return ids, w, _routing(ids, w, E, rows)


def _assert_layer(y, want, I):
    y = y.double().cpu().numpy()
    assert np.isfinite(y).all()
    rel = np.linalg.norm(y - want) / np.linalg.norm(want)
    rms = np.linalg.norm(want) / np.sqrt(want.size)
    assert rel < 3e-3, rel
    assert (np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + 3 / np.sqrt(I) * rms).all()


LAYERS = [(1, 256, 96, 0, 8, 2, 16), (1, 2048, 512, 512, 16, 8, 16), (2, 256, 128, 64, 4, 1, 16), (3, 288, 160, 32, 6, 6, 1),
          (8, 512, 256, 512, 32, 4, 16), (9, 512, 256, 128, 32, 4, 16), (37, 704, 352, 0, 12, 3, 48), (64, 256, 704, 96, 8, 2, 32),
          (130, 512, 128, 256, 4, 2, 128), (300, 256, 256, 0, 64, 8, 33), (517, 384, 224, 224, 5, 2, 96)]


@pytest.mark.parametrize("T,d,I,I_shared,E,k,rows", LAYERS)
@pytest.mark.parametrize("quantised", [False, True])
def test_forward(T, d, I, I_shared, E, k, rows, quantised):
    rng = np.random.default_rng(T + d + I)
    ids, w, r = _draw_routing(rng, T, E, k, rows, hot=0.5)
    routed_host, routed = _experts(rng, E, d, I)
    shared_host, shared = _experts(rng, 1, d, I_shared) if I_shared else (None, None)
    x = _to(rng.standard_normal((T, d)), "bf16")
    v, s = blk_ref.quantise(x.double().cpu().numpy())
    ws = bm.workspace(bm.moe_blk_forward_workspace_bytes(T, d, I, E, k, I_shared, rows))
    y = torch.full((T + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):                                               # the workspace is ready for the next call
        bm.moe_blk_forward(_act(v, s) if quantised else x, routed, shared, r, y[:T], ws)
    assert bm.moe_check_status(ws) == 0
    assert (y[T] == 7).all()
    _assert_layer(y[:T], blk_ref.layer(v * blk_ref.spread(s, d), routed_host, shared_host, ids, w.astype(np.float64)), I)


@pytest.mark.parametrize("T,d,I,I_shared,E,k,rows", [(1, 256, 1184, 0, 12, 8, 16), (2, 256, 608, 96, 8, 8, 33), (2, 320, 1216, 0, 9, 7, 128),
                                                     (8, 256, 96, 0, 16, 1, 16), (5, 2464, 64, 32, 12, 3, 16), (7, 512, 352, 0, 4, 3, 3),
                                                     (1, 2560, 704, 704, 40, 12, 64), (8, 1024, 256, 0, 3, 2, 16),
                                                     (1, 320, 416, 416, 20, 7, 16), (2, 544, 608, 96, 9, 9, 16), (1, 1152, 704, 0, 16, 12, 16)])
@pytest.mark.parametrize("quantised", [False, True])
def test_forward_of_few_tokens(T, d, I, I_shared, E, k, rows, quantised):
    """Either way of computing few tokens, at sizes on both sides of where one follows on the other."""
    test_forward(T, d, I, I_shared, E, k, rows, quantised)


def test_forward_with_experts_that_nobody_takes_and_one_that_all_take():
    rng = np.random.default_rng(8)
    T, d, I, E, k, rows = 100, 256, 128, 9, 2, 32
    ids = np.stack([np.full(T, 4), np.where(np.arange(T) % 2, 0, 8)], 1)
    w = rng.random((T, k)).astype(np.float32)
    w[3] = 0
    r = _routing(ids, w, E, rows)
    host, routed = _experts(rng, E, d, I)
    x = _to(rng.standard_normal((T, d)), "bf16")
    x[5] = 0
    ws = bm.workspace(bm.moe_blk_forward_workspace_bytes(T, d, I, E, k, 0, rows))
    y = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    bm.moe_blk_forward(x, routed, None, r, y, ws)
    assert bm.moe_check_status(ws) == 0
    assert not y[3].any() and not y[5].any()
    _assert_layer(y, blk_ref.layer(blk_ref.rounded(x.double().cpu().numpy()), host, None, ids, w.astype(np.float64)), I)


@pytest.mark.parametrize("T,rows", [(1, 16), (2, 16), (2, 2), (40, 16), (40, 96)])
def test_forward_with_an_expert_that_a_token_takes_twice(T, rows):
    """Tables of the caller's own: both weights count."""
    rng = np.random.default_rng(T + rows)
    d, I, E, k = 256, 160, 4, 3
    ids = np.stack([np.full(T, 2), np.arange(T) % 2, np.full(T, 2)], 1)
    w = rng.random((T, k)).astype(np.float32)
    r = _routing(ids, w, E, rows)
    host, routed = _experts(rng, E, d, I)
    x = _to(rng.standard_normal((T, d)), "bf16")
    ws = bm.workspace(bm.moe_blk_forward_workspace_bytes(T, d, I, E, k, 0, rows))
    y = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    bm.moe_blk_forward(x, routed, None, r, y, ws)
    assert bm.moe_check_status(ws) == 0
    xv = blk_ref.rounded(x.double().cpu().numpy())
    want = sum(blk_ref.layer(xv, host, None, ids[:, j], w[:, j].astype(np.float64)) for j in (slice(0, 2), slice(2, 3)))
    _assert_layer(y, want, I)


def test_more_rows_of_one_expert_than_a_tile_of_few_tokens_takes():
    rng = np.random.default_rng(0)
    T, d, I, E, k = 2, 256, 128, 8, 5
    ids = np.full((T, k), 3)
    _, routed = _experts(rng, E, d, I)
    x = _to(rng.standard_normal((T, d)), "bf16")
    y = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    ws = bm.workspace(bm.moe_blk_forward_workspace_bytes(T, d, I, E, k, 0, 16))
    bm.moe_blk_forward(x, routed, None, _routing(ids, np.ones((T, k), np.float32), E, 16), y, ws)
    assert bm.moe_check_status(ws) == 1


# ------------------------------------------------------------------ calls in a program

def _forward_buffers(T, d, I, E, k, I_shared, rows):
    return (torch.empty((T, d), dtype=torch.bfloat16, device="cuda"),
            bm.workspace(bm.moe_blk_forward_workspace_bytes(T, d, I, E, k, I_shared, rows)))


@pytest.mark.parametrize("T,rows", [(1, 16), (2, 16), (40, 16), (40, 64), (200, 128)])
def test_a_block_of_a_model(T, rows):
    """Residual and norm, router projection from its bf16 output, scored routing and experts from its codes, in one call
    of moe_blk_layer; the next norm adds the result to the stream.  Each step against 64 bits from what the one before
    gave; the layer also equals routing and experts called one after the other, and itself from a captured graph."""
    rng = np.random.default_rng(T + rows)
    d, I, E, k, I_shared = 512, 224, 16, 4, 128
    x, stream = _to(rng.standard_normal((T, d)), "bf16"), _to(3 * rng.standard_normal((T, d)), "bf16")
    gamma = _to(1 + 0.2 * rng.standard_normal(d), "bf16")
    router = _to(rng.standard_normal((E, d)) / np.sqrt(d), "bf16")
    scoring = bm.Scoring("sigmoid", _to(0.1 * rng.standard_normal(E), "fp32"), n_group=4, topk_group=2, scale=1.5)
    routed_host, routed = _experts(rng, E, d, I)
    shared_host, shared = _experts(rng, 1, d, I_shared)
    normed, act = torch.empty_like(x), bm.BlkAct.empty(T, d)
    logits = torch.empty((T, E), dtype=torch.float32, device="cuda")
    r = bm.Routing.empty(T, E, k, rows)
    y = torch.empty_like(x)
    ws = bm.workspace(bm.moe_blk_layer_workspace_bytes(T, d, I, E, k, I_shared, rows))
    before, after = stream.clone(), torch.empty_like(stream)
    out = bm.BlkAct.empty(T, d)

    def block():
        bm.moe_rmsnorm(x, gamma, 1e-6, residual=stream, stream_out=after, Y=normed, out=act)
        bm.moe_router_logits(normed, router, logits)
        bm.moe_blk_layer(logits, scoring, act, routed, shared, k, rows, r, y, ws)
        bm.moe_rmsnorm(y, gamma, 1e-6, residual=after, out=out)          # adds to `after` in place

    block()
    assert bm.moe_check_status(ws) == 0
    res = (x.double() + before.double()).to(torch.bfloat16)
    xq = blk_ref.decode(act.q.cpu().numpy()) * blk_ref.spread(act.s.cpu().numpy()[:, :T].T.astype(np.float64), d)
    want = blk_ref.rounded(blk_ref.norm(res.double().cpu().numpy(), gamma.double().cpu().numpy(), 1e-6))
    np.testing.assert_array_equal(xq, want)
    ids, w = r.ids.cpu().numpy(), r.w.double().cpu().numpy()
    for t in range(T):
        got = mx_ref.route_row(logits[t].double().cpu().numpy(), "sigmoid", scoring.bias.double().cpu().numpy(), k, 4, 2, 2, True, 1.5)
        if got[2] > 1e-5:
            np.testing.assert_array_equal(ids[t], got[0])
            np.testing.assert_allclose(w[t], got[1], rtol=1e-5)
    _assert_layer(y, blk_ref.layer(xq, routed_host, shared_host, ids, w), I)
    assert torch.equal(after, (res.double() + y.double()).to(torch.bfloat16))
    first = [t.clone() for t in (y, after, out.q, out.s[:, :T])]
    # one after the other
    y2, ws2 = _forward_buffers(T, d, I, E, k, I_shared, rows)
    bm.moe_blk_forward(act, routed, shared, r, y2, ws2)
    assert torch.equal(y2, y)
    # from a graph, with other inputs in the same memory in between
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            block()
    torch.cuda.synchronize()
    kept = x.clone()
    x.copy_(_to(rng.standard_normal((T, d)), "bf16"))
    g.replay()
    x.copy_(kept)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip((y, after, out.q, out.s[:, :T]), first):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls with workspaces of their own, side by side, give what they give alone."""
    rng = np.random.default_rng(4)
    d, I, E, k, rows = 1024, 256, 16, 4, 64
    _, routed = _experts(rng, E, d, I)
    m = _mat(blk_ref.draw_matrix(rng, 1, 2080, d))
    jobs = []
    for T in (300, 1):
        x = _to(rng.standard_normal((T, d)), "bf16")
        _, _, r = _draw_routing(rng, T, E, k, rows)
        y, ws = _forward_buffers(T, d, I, E, k, 0, rows)
        z = torch.empty((T, 2080), dtype=torch.float32, device="cuda")
        jobs.append((x, r, y, ws, z, bm.workspace(bm.moe_blk_linear_workspace_bytes(T, 2080, d)), torch.cuda.Stream()))

    def run(job, stream):
        x, r, y, ws, z, ws2, _ = job
        bm.moe_blk_forward(x, routed, None, r, y, ws, stream=stream)
        bm.moe_blk_linear(x, m, z, ws2, stream=stream)

    alone = []
    for j in jobs:
        run(j, None)
        alone.append((j[2].clone(), j[4].clone()))
    torch.cuda.synchronize()
    for _ in range(20):
        for j in jobs:
            run(j, j[6])
    torch.cuda.synchronize()
    for j, (y, z) in zip(jobs, alone):
        assert torch.equal(j[2], y) and torch.equal(j[4], z) and bm.moe_check_status(j[3]) == 0


def test_calls_without_rows():
    a = bm.BlkAct.empty(0, 256)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    m = _mat(blk_ref.draw_matrix(np.random.default_rng(0), 1, 64, 256))
    ws = bm.workspace(256)
    bm.moe_blk_quantize(x, a)
    bm.moe_blk_dequant(a, x)
    bm.moe_blk_matmul(a, m, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), ws)
    bm.moe_blk_linear(x, m, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), ws)
    bm.moe_rmsnorm(x, torch.ones(256, device="cuda"), 1e-6, residual=x, Y=x, out=a)
    assert bm.moe_check_status(ws) == 0


@pytest.mark.parametrize("kind", ["one", "few", "narrow", "wide"])
def test_a_product_right_after_its_weights(kind):
    """moe_blk_quantize_weights, then at once the product with them: the results of a synchronised program."""
    M, N, K = {"one": (1, 2048, 2048), "few": (20, 2048, 2048), "narrow": (300, 2048, 2048), "wide": (2500, 2304, 1040)}[kind]
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = [torch.randn(1, N, K, device="cuda", generator=gen) * 2.0 ** i for i in (0, 3)]
    x = torch.randn(M, K, device="cuda", generator=gen).to(torch.bfloat16)
    m, a = bm.BlkMat.empty(1, N, K), bm.BlkAct.empty(M, K)
    bm.moe_blk_quantize(x, a)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = bm.workspace(bm.moe_blk_linear_workspace_bytes(M, N, K))
    got = {}
    for sync in (True, False):
        got[sync] = []
        for i in range(8):
            bm.moe_blk_quantize_weights(w[i % 2], m)
            if sync:
                torch.cuda.synchronize()
            if kind == "one":
                bm.moe_blk_linear(x, m, y, ws)
            else:
                bm.moe_blk_matmul(a, m, y, ws)
            got[sync].append(y.clone())
        torch.cuda.synchronize()
    assert not torch.equal(got[True][0], got[True][1])
    assert all(torch.equal(p, q) for p, q in zip(got[True], got[False])) and bm.moe_check_status(ws) == 0


@pytest.mark.parametrize("T,rows", [(2, 16), (40, 16), (40, 128)])
@pytest.mark.parametrize("bad", ["expert", "rows", "first", "count"])
def test_a_malformed_routing_is_reported_and_harms_no_later_call(T, rows, bad):
    """Entries that the kernels check: an expert that is not there, more rows than a tile has, rows past the last, no tiles."""
    rng = np.random.default_rng(T)
    d, I, E, k = 256, 128, 8, 2
    _, routed = _experts(rng, E, d, I)
    _, _, r = _draw_routing(rng, T, E, k, rows)
    x = _to(rng.standard_normal((T, d)), "bf16")
    y, ws = _forward_buffers(T, d, I, E, k, 0, rows)
    bm.moe_blk_forward(x, routed, None, r, y, ws)
    good = y.clone()
    assert bm.moe_check_status(ws) == 0
    saved, tiles = r.block_map.clone(), r.num_blocks.clone()
    if bad == "count":
        r.num_blocks.fill_(0)
    else:
        column, value = {"expert": (0, E), "rows": (2, 10 ** 6), "first": (1, T * k + 1)}[bad]
        r.block_map[0, column] = value
    bm.moe_blk_forward(x, routed, None, r, y, ws)
    assert bm.moe_check_status(ws) == 1
    r.block_map.copy_(saved)
    r.num_blocks.copy_(tiles)
    bm.moe_blk_forward(x, routed, None, r, y, ws)
    assert bm.moe_check_status(ws) == 0 and torch.equal(y, good)


def test_new_memory_under_the_same_objects():
    """A BlkMat and a BlkAct whose tensors move are taken as they are now."""
    rng = np.random.default_rng(6)
    M, N, K = 4, 300, 256
    v, s = blk_ref.quantise(rng.standard_normal((M, K)))
    a, m = _act(v, s), _mat(blk_ref.draw_matrix(rng, 1, N, K))
    y, ws = torch.empty((M, N), dtype=torch.float32, device="cuda"), bm.workspace(256)
    bm.moe_blk_matmul(a, m, y, ws)
    first = y.clone()
    for t in (a.q, a.s, m.q, m.s):
        old = t.clone()
        t.set_(old)                                                    # other memory, the same tensor object
    bm.moe_blk_matmul(a, m, y, ws)
    assert torch.equal(y, first)
    m.q = m.q.view(torch.float8_e4m3fn)
    bm.moe_blk_matmul(a, m, y, ws)
    assert torch.equal(y, first)


# ------------------------------------------------------------------ sizes past 2^31 elements

def test_rows_past_2_to_the_31_elements():
    rows, K = 270_000, 8192
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, K, device="cuda", generator=gen, dtype=torch.bfloat16)
    a, b = bm.BlkAct.empty(rows, K), bm.BlkAct.empty(rows, K)
    bm.moe_blk_quantize(x, a)
    some = np.r_[0:5, rows // 2:rows // 2 + 5, rows - 5:rows]
    x64 = x[some].double().cpu().numpy()
    _check_codes(a.q[some].cpu().numpy(), a.s[:, some].cpu().numpy().T, *blk_ref.quantise(x64))
    y = torch.empty_like(x)
    bm.moe_blk_dequant(a, y)
    np.testing.assert_array_equal(y[some].double().cpu().numpy(), blk_ref.rounded(x64))
    gamma = torch.ones(K, device="cuda")
    bm.moe_rmsnorm(x, gamma, 1e-6, residual=x, stream_out=y, out=b)
    res = (2 * x[some].double()).cpu().numpy()                        # exact in bf16
    np.testing.assert_array_equal(y[some].double().cpu().numpy(), res)
    values = blk_ref.decode(b.q[some].cpu().numpy()) * blk_ref.spread(b.s[:, some].cpu().numpy().T.astype(np.float64), K)
    np.testing.assert_array_equal(values, blk_ref.rounded(blk_ref.norm(res, np.ones(K), 1e-6)))


def test_weights_past_2_to_the_31_elements():
    E, N, K = 5, 55_000, 8192
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(E, N, K, device="cuda", generator=gen, dtype=torch.bfloat16)
    m = bm.BlkMat.empty(E, N, K)
    bm.moe_blk_quantize_weights(w, m)
    at = slice(N // 128 * 128, N)                                     # the last block's rows of the last matrix
    v, s = blk_ref.quantise_weights(w[-1:, at].double().cpu().numpy())
    np.testing.assert_array_equal(m.s[-1:, -1:].cpu().numpy(), s)
    np.testing.assert_array_equal(blk_ref.decode(m.q[-1:, at].cpu().numpy()), v)
    bm.moe_blk_dequant(m, w)
    np.testing.assert_array_equal(w[-1:, at].double().cpu().numpy(), blk_ref.weights((blk_ref.encode(v), s)))


@pytest.mark.parametrize("M,N", [(16, 150_000_000), (40, 60_000_000), (70_000, 33_000)])
def test_products_past_2_to_the_31_elements(M, N):
    """Few tokens, narrow tiles, wide tiles: results past 2^31 elements."""
    K = 64
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(M, K, device="cuda", generator=gen, dtype=torch.bfloat16)
    a = bm.BlkAct.empty(M, K)
    bm.moe_blk_quantize(x, a)
    m = bm.BlkMat.empty(1, N, K)
    m.q.copy_(torch.randint(0, 120, (1, N, K), device="cuda", generator=gen, dtype=torch.uint8))
    m.s.copy_(torch.rand(m.s.shape, device="cuda", generator=gen) + 0.5)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = bm.workspace(256)
    bm.moe_blk_matmul(a, m, y, ws)
    assert bm.moe_check_status(ws) == 0
    rows, cols = np.r_[0, M - 1], np.r_[0:40, N // 2:N // 2 + 40, N - 40:N]
    xv = blk_ref.rounded(x[rows].double().cpu().numpy())
    s = m.s[0, cols // 128].double().cpu().numpy()
    _assert_product(y[rows][:, cols], xv, blk_ref.decode(m.q[0, cols].cpu().numpy()) * s, K)


def test_experts_rows_past_2_to_the_31_elements():
    """Rows of the experts' outputs past 2^31 elements: a token's result does not change with the tokens around it."""
    T, d, I, E, k = 34_000, 8192, 32, 8, 8
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    rng = np.random.default_rng(7)
    _, routed = _experts(rng, E, d, I)

    def run(x):
        n = x.shape[0]
        r = bm.Routing.empty(n, E, k, 128)
        ws = bm.workspace(bm.moe_blk_layer_workspace_bytes(n, d, I, E, k, 0, 128))
        y = torch.empty_like(x)
        logits = (x[:, :E].float() * 3).contiguous()
        bm.moe_blk_layer(logits, bm.Scoring("softmax"), x, routed, None, k, 128, r, y, ws)
        assert bm.moe_check_status(ws) == 0
        return y

    y = run(x)
    some = torch.cat([torch.arange(300), torch.arange(T - 300, T)]).cuda()
    assert torch.isfinite(y).all() and torch.equal(y[some], run(x[some].contiguous()))
