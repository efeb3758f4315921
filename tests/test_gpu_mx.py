"""MXFP4: quantisation and its inverse exactly, products and expert layers against 64 bits.

Products: the operands' products are exact, so an error comes from the fp32 accumulation alone.  The tensor cores add
64 products at a time and may drop bits below the last place of the largest; with a bound of two last places (2^-22) of
the sum of magnitudes for each of the K/64 additions, |Y - Y64| <= bound = (K/64 + 2) 2^-22 sum_k |a_k b_k|.  Rounding
is monotone, so a Y in bf16 lies between the bf16 values nearest to Y64 - bound and Y64 + bound: exact but for the sum.

Expert layers: the hidden values are rounded to MXFP4 from fp32 accumulators here and from 64 bits in the reference.  They
differ by about 1e-6 of themselves, so about 1e-5 of them (that over the spacing of E2M1, 1/6 to 1/2, and twice, since
a block's scale can flip too) land on the other side of a rounding, by at most half of themselves: 2e-3 of the norm of h
and of Y.  With bf16's own 2^-9/sqrt(3): relative L2 error below 5e-3.  One such value moves an element of Y by its
share of it: half of 1/sqrt(I) of the root mean square; a few at once stay below 3/sqrt(I) + 2^-8."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_moe_expert_gb300 as bm  # noqa: E402
import mx_ref  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_moe_expert_gb300 import build
    build.build()
    bm.lib()


TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _mat(mat):
    """(codes, bytes) [E]... on the device, scales packed by the library."""
    q, s = (torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in mat)
    m = bm.MxMat.empty(q.shape[0], q.shape[1], 2 * q.shape[2])
    m.sp.fill_(255)
    bm.moe_mx_prepack_scales(s, m.sp)
    m.q = q
    return m


def _quantise(x):
    m = bm.MxMat.empty(1, x.shape[0], x.shape[1])
    m.sp.fill_(255)
    bm.moe_mx_quantize(x, m)
    torch.cuda.synchronize()
    return m


def _check_quantised(m, x64):
    v, s = mx_ref.quantise(x64)
    rows, K = x64.shape
    got = m.sp.cpu().numpy()
    want = mx_ref.pack(s[None])
    n, g = np.meshgrid(np.arange(rows), np.arange(4 * got.shape[2]), indexing="ij")
    at = (0, n // 128, g // 4, 16 * (n % 32) + 4 * (n % 128 // 32) + g % 4)
    np.testing.assert_array_equal(got[at], want[at])           # blocks past K are zeros too
    ok = np.repeat(s != 255, 32, -1)
    np.testing.assert_array_equal(mx_ref.decode(m.q.cpu().numpy()[0])[ok], v[ok])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 2048), (3, 96), (33, 160), (129, 256), (130, 288), (7, 4128), (1000, 544)])
def test_quantise(kind, rows, K):
    rng = np.random.default_rng(rows + K)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-12, 12, (rows, 1)))
    x = torch.from_numpy(x.astype(np.float32)).to(TYPES[kind]).cuda()
    _check_quantised(_quantise(x), x.double().cpu().numpy())


@pytest.mark.parametrize("kind", list(TYPES))
def test_quantise_edges(kind):
    """Ties and saturation at every scale; zeros; the smallest and the largest numbers; NaN and infinity."""
    ties = np.array([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 6.5, 7, 7.9375, .5, 1, 1.5, 2, 3, 4, .2, .3, -.25, -.75,
                     -1.25, -1.75, -2.5, -3.5, -5, -6.5, -7.5, -0., .1, 2.75])
    info = torch.finfo(TYPES[kind])
    rows = [ties * 2.0 ** e for e in (-10, 0, 9)]
    rows += [np.zeros(32), np.where(np.arange(32) == 3, info.max, 1.0), np.where(np.arange(32) == 3, -info.max, 0.0)]
    rows += [np.full(32, info.tiny), np.where(np.arange(32) % 2, info.smallest_normal / 2, 0.0)]
    rows += [np.where(np.arange(32) == 9, np.nan, ties), np.where(np.arange(32) == 31, -np.inf, ties)]
    x = torch.tensor(np.stack(rows), dtype=torch.float64).to(TYPES[kind]).cuda()
    m = _quantise(x)
    _check_quantised(m, x.double().cpu().numpy())
    w = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    bm.moe_mx_dequant(m, w)
    w = w.cpu().numpy()
    assert np.isnan(w[-2:]).all() and np.isfinite(w[:-2]).all()


def test_quantise_strided_rows_and_another_stream():
    rng = np.random.default_rng(1)
    big = torch.from_numpy(rng.standard_normal((40, 512)).astype(np.float32)).to(torch.bfloat16).cuda()
    x = big[3:29, 64:160]
    m = bm.MxMat.empty(1, 26, 96)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bm.moe_mx_quantize(x, m, stream=s)
    torch.cuda.synchronize()
    _check_quantised(m, x.double().cpu().numpy())


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_dequant_of_every_code_and_scale(kind):
    q = np.tile(np.arange(256, dtype=np.uint8), 8).reshape(1, 128, 16)  # 32 codes a row
    s = np.arange(128, dtype=np.uint8).reshape(1, 128, 1)
    for base in (0, 128):
        m = _mat((q, s + np.uint8(base)))
        w = torch.empty((1, 128, 32), dtype=TYPES[kind], device="cuda")
        bm.moe_mx_dequant(m, w)
        want = torch.from_numpy(mx_ref.values(mx_ref.decode(q), s + np.uint8(base))).to(TYPES[kind]).double().numpy()
        np.testing.assert_array_equal(w.double().cpu().numpy(), want)


def test_dequant_of_a_stack_with_odd_rows():
    rng = np.random.default_rng(2)
    mat = mx_ref.draw_matrix(rng, 3, 131, 416)
    w = torch.empty((3, 131, 416), dtype=torch.float32, device="cuda")
    bm.moe_mx_dequant(_mat(mat), w)
    np.testing.assert_array_equal(w.double().cpu().numpy(), mx_ref.weights(mat))


SIZES = [(1, 1, 32), (1, 2048, 2048), (1, 130, 96), (3, 33, 160), (16, 128, 64), (17, 200, 256), (128, 513, 288),
         (129, 129, 512), (200, 31, 1056), (300, 700, 2048), (257, 512, 32), (1000, 256, 320), (640, 1000, 4096)]


def _product_error(y, xv, wv, K, bf16):
    want = xv @ wv.T
    bound = (K / 64 + 2) * 2.0 ** -22 * (np.abs(xv) @ np.abs(wv).T)
    low, high = want - bound, want + bound
    if bf16:
        low, high = (torch.from_numpy(v).to(torch.bfloat16).double().numpy() for v in (low, high))
    assert np.isfinite(y).all()
    return float(np.max(np.maximum(low - y, y - high)))


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("y_kind", ["bf16", "fp32"])
def test_matmul(M, N, K, y_kind):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, w = mx_ref.draw_matrix(rng, 1, M, K), mx_ref.draw_matrix(rng, 1, N, K)
    w[1][...] = w[1] + rng.integers(-3, 4, w[1].shape)          # scales that differ from block to block
    y = torch.full((M + 1, N), 7.0, dtype=TYPES[y_kind], device="cuda")
    ws = bm.workspace(256)
    bm.moe_mx_matmul(_mat(a), _mat(w), y[:M], ws)
    torch.cuda.synchronize()
    assert bm.moe_check_status(ws) == 0
    got = y.double().cpu().numpy()
    assert _product_error(got[:M], mx_ref.weights(a)[0], mx_ref.weights(w)[0], K, y_kind == "bf16") <= 0
    assert (got[M] == 7).all()                                  # nothing past the last row


@pytest.mark.parametrize("M,N,K,x_kind", [(1, 2048, 2048, "bf16"), (5, 100, 96, "fp16"), (128, 96, 256, "fp32"),
                                          (333, 1001, 2816, "fp16"), (140, 64, 416, "fp32"), (32, 300, 1184, "bf16"),
                                          (33, 300, 1184, "bf16"), (3, 40, 12320, "bf16"), (3, 40, 16416, "fp32"),
                                          (1, 40, 12320, "bf16"), (8, 200, 2048, "bf16"), (17, 300, 960, "fp32"),
                                          (32, 130, 512, "fp16")])
def test_linear(M, N, K, x_kind):
    rng = np.random.default_rng(M + N)
    x = torch.from_numpy(rng.standard_normal((M, K + 32)).astype(np.float32)).to(TYPES[x_kind]).cuda()[:, :K]
    w = mx_ref.draw_matrix(rng, 1, N, K)
    y = torch.empty((M, N), dtype=torch.float32, device="cuda")
    ws = bm.workspace(bm.moe_mx_linear_workspace_bytes(M, N, K))
    for _ in range(2):  # the workspace is ready for the next call
        y.fill_(float("nan"))
        bm.moe_mx_linear(x, _mat(w), y, ws)
    torch.cuda.synchronize()
    assert bm.moe_check_status(ws) == 0
    assert _product_error(y.double().cpu().numpy(), mx_ref.rounded(x.double().cpu().numpy()), mx_ref.weights(w)[0], K,
                          False) <= 0


def test_a_nan_stays_in_its_row():
    rng = np.random.default_rng(5)
    for M in (20, 200):
        x = torch.from_numpy(rng.standard_normal((M, 512)).astype(np.float32)).cuda()
        x[7, 100] = float("nan")
        x[11, 511] = float("inf")
        y = torch.zeros((M, 96), dtype=torch.float32, device="cuda")
        bm.moe_mx_linear(x, _mat(mx_ref.draw_matrix(rng, 1, 96, 512)), y, bm.workspace(bm.moe_mx_linear_workspace_bytes(M, 96, 512)))
        bad = torch.isnan(y).cpu().numpy()
        assert bad[[7, 11]].all() and not np.delete(bad, [7, 11], 0).any()


@pytest.mark.parametrize("M,N,K,y_kind", [(4865, 4353, 1312, "fp32"), (5001, 4099, 1056, "bf16"), (2600, 2100, 3392, "fp32")])
def test_large_products(M, N, K, y_kind):
    """Sizes for pairs of CTAs, with last tiles of one row and stages past K: values, a row of NaN, the bits of a row alone."""
    rng = np.random.default_rng(M + N)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).cuda()
    x[M - 2, K - 1] = float("nan")
    wm = mx_ref.draw_matrix(rng, 1, N, K)
    w, y = _mat(wm), torch.full((M + 1, N), 7.0, dtype=TYPES[y_kind], device="cuda")
    ws = bm.workspace(bm.moe_mx_linear_workspace_bytes(M, N, K))
    for _ in range(2):
        bm.moe_mx_linear(x, w, y[:M], ws)
    rows = [0, 127, 128, 256, M - 1]
    alone = [torch.empty((1, N), dtype=TYPES[y_kind], device="cuda") for _ in rows]
    for r, one in zip(rows, alone):
        bm.moe_mx_linear(x[r:r + 1], w, one, ws)
    torch.cuda.synchronize()
    assert bm.moe_check_status(ws) == 0
    assert torch.equal(torch.cat(alone), y[rows]) and torch.isnan(y[M - 2]).all() and (y[M] == 7).all()
    keep = np.delete(np.arange(M), M - 2)
    got, xv = y.double().cpu().numpy()[keep], mx_ref.rounded(x.double().cpu().numpy()[keep])
    assert _product_error(got, xv, mx_ref.weights(wm)[0], K, y_kind == "bf16") <= 0


@pytest.mark.parametrize("K", [32, 1312])
def test_offsets_past_32_bits(K):
    """Elements past 2^31 of Y (one CTA a tile, and pairs): the bits of the same rows alone."""
    M, N = 70001, 32776
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(M, K, device="cuda", generator=gen, dtype=torch.float32).to(torch.bfloat16)
    w = _quantise(torch.randn(N, K, device="cuda", generator=gen, dtype=torch.float32))
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = bm.workspace(bm.moe_mx_linear_workspace_bytes(M, N, K))
    bm.moe_mx_linear(x, w, y, ws)
    some = torch.cat([torch.arange(0, 130), torch.arange(65500, 65630), torch.arange(M - 130, M)])
    alone = torch.empty((len(some), N), dtype=torch.bfloat16, device="cuda")
    bm.moe_mx_linear(x[some].contiguous(), w, alone, ws)
    torch.cuda.synchronize()
    assert bm.moe_check_status(ws) == 0 and torch.equal(alone, y[some])


def test_quantise_offsets_past_32_bits():
    rows, K = 70001, 65536
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    x.view(-1)[:] = 1.0
    x[-200:] = torch.randn(200, K, device="cuda").to(torch.bfloat16)
    m, part = _quantise(x), _quantise(x[rows // 128 * 128 - 128:])  # from a piece's first row on
    n = part.q.shape[1]
    assert n >= 100 and torch.equal(m.q[0, -n:], part.q[0])
    assert torch.equal(m.sp.view(-1)[-part.sp.numel():], part.sp.view(-1))
    back = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    bm.moe_mx_dequant(m, back)
    some = torch.empty((n, K), dtype=torch.bfloat16, device="cuda")
    bm.moe_mx_dequant(part, some)
    torch.cuda.synchronize()
    assert torch.equal(back[-n:], some) and (back[0] == 1).all()


def test_a_row_does_not_depend_on_its_batch():
    """The same bits for a token alone, among few and among many."""
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.standard_normal((300, 1024)).astype(np.float32)).to(torch.bfloat16).cuda()
    w = _mat(mx_ref.draw_matrix(rng, 1, 320, 1024))
    got = []
    for M in (1, 30, 300):
        y = torch.empty((M, 320), dtype=torch.float32, device="cuda")
        bm.moe_mx_linear(x[:M], w, y, bm.workspace(bm.moe_mx_linear_workspace_bytes(M, 320, 1024)))
        got.append(y[0].clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


class _Layer:
    def __init__(self, seed, T, d, I, I_shared, E):
        rng = np.random.default_rng(seed)
        self.E, self.I, self.I_shared, self.d = E, I, I_shared, d
        self.x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(torch.bfloat16).cuda()
        self.logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
        draw = mx_ref.draw_matrix
        self.routed_host = [draw(rng, E, I, d), draw(rng, E, I, d), draw(rng, E, d, I)]
        self.routed = bm.prepare_mx_experts(dict(zip(("gate", "up", "down"), self.routed_host)))
        self.shared_host = self.shared = None
        if I_shared:
            self.shared_host = [draw(rng, 1, I_shared, d), draw(rng, 1, I_shared, d), draw(rng, 1, d, I_shared)]
            self.shared = bm.prepare_mx_experts(dict(zip(("gate", "up", "down"), self.shared_host)))

    def run(self, scoring, k, block_rows, rows=None, runs=1):
        x = self.x if rows is None else self.x[rows].contiguous()
        lg = self.logits if rows is None else self.logits[rows].contiguous()
        T = x.shape[0]
        r = bm.Routing.empty(T, self.E, k, block_rows)
        ws = bm.workspace(bm.moe_mx_layer_workspace_bytes(T, self.d, self.I, self.E, k, self.I_shared, block_rows))
        y = torch.full((T, self.d), float("nan"), dtype=torch.bfloat16, device="cuda")
        for _ in range(runs):
            bm.moe_mx_layer(lg, scoring, x, self.routed, self.shared, k, block_rows, r, y, ws)
        torch.cuda.synchronize()
        assert bm.moe_check_status(ws) == 0
        return y, r

    def check(self, y, r):
        ref = mx_ref.layer(self.x.double().cpu().numpy(), self.routed_host, self.shared_host, r.ids.cpu().numpy(),
                           r.w.double().cpu().numpy())
        y = y.double().cpu().numpy()
        assert np.isfinite(y).all()
        assert np.linalg.norm(y - ref) <= 5e-3 * np.linalg.norm(ref)
        rms = np.sqrt(np.mean(ref ** 2))
        assert np.max(np.abs(y - ref) / np.maximum(rms, np.abs(ref))) <= 3 / np.sqrt(self.I) + 2.0 ** -8


LAYERS = [  # T, d, I, I_shared, E, k, block_rows
    (1, 256, 128, 128, 16, 2, 16),
    (1, 2048, 512, 512, 9, 8, 16),
    (2, 96, 32, 0, 4, 4, 16),            # one block of 32 a row of h
    (40, 288, 160, 96, 8, 3, 32),        # no size a multiple of 64
    (40, 288, 160, 96, 8, 3, 20),        # tiles of a height that is no multiple of 16
    (32, 288, 160, 96, 8, 3, 16),        # several tiles of an expert among few tokens
    (17, 2048, 96, 512, 12, 5, 64),      # a shared expert wider than the routed ones
    (300, 512, 224, 256, 6, 2, 128),     # full tiles, one accumulator
    (300, 512, 224, 0, 6, 2, 96),
    (150, 320, 704, 64, 5, 1, 64),
]


@pytest.mark.parametrize("T,d,I,I_shared,E,k,block_rows", LAYERS)
def test_layer(T, d, I, I_shared, E, k, block_rows):
    layer = _Layer(T + d, T, d, I, I_shared, E)
    scoring = bm.Scoring("sigmoid", scale=1.5) if I_shared else bm.Scoring("softmax")
    y, r = layer.run(scoring, k, block_rows, runs=2)
    layer.check(y, r)


def test_layer_after_moe_route():
    """moe_mx_forward takes any routing, moe_route's as well."""
    layer = _Layer(1, 70, 256, 128, 128, 8)
    r = bm.Routing.empty(70, 8, 2, 32)
    bm.moe_route(layer.logits, 2, 32, r, bm.workspace(bm.moe_route_workspace_bytes(70, 8, 2)))
    ws = bm.workspace(bm.moe_mx_forward_workspace_bytes(70, 256, 128, 8, 2, 128, 32))
    y = torch.empty((70, 256), dtype=torch.bfloat16, device="cuda")
    bm.moe_mx_forward(layer.x, layer.routed, layer.shared, r, y, ws)
    torch.cuda.synchronize()
    assert bm.moe_check_status(ws) == 0
    layer.check(y, r)


def test_layer_does_not_depend_on_tiles_or_batch():
    layer = _Layer(2, 200, 512, 256, 128, 8)
    sc = bm.Scoring("sigmoid")
    y, _ = layer.run(sc, 2, 16)
    for block_rows in (48, 128):
        assert torch.equal(y, layer.run(sc, 2, block_rows)[0])
    for rows in (slice(0, 1), slice(5, 9), slice(100, 200)):
        assert torch.equal(y[rows], layer.run(sc, 2, 32, rows)[0])


def test_layer_without_tokens_with_masked_experts_and_in_a_graph():
    layer = _Layer(3, 30, 256, 96, 64, 6)
    sc = bm.Scoring("softmax")
    y, _ = layer.run(sc, 2, 16, slice(0, 0))
    assert y.shape == (0, 256)
    layer.logits[:, 2:] = -float("inf")      # every token takes the same two experts
    y, r = layer.run(sc, 2, 16)
    assert int(r.counts[:2].sum()) == 60
    layer.check(y, r)
    ws = bm.workspace(bm.moe_mx_layer_workspace_bytes(30, 256, 96, 6, 2, 64, 16))
    z = torch.empty_like(y)
    bm.moe_mx_layer(layer.logits, sc, layer.x, layer.routed, layer.shared, 2, 16, r, z, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bm.moe_mx_layer(layer.logits, sc, layer.x, layer.routed, layer.shared, 2, 16, r, z, ws)
    z.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, z) and bm.moe_check_status(ws) == 0


def test_a_malformed_block_map_is_reported():
    """Tiles outside of the assignments are skipped and recorded, not read."""
    layer = _Layer(4, 20, 256, 96, 0, 4)
    r = bm.Routing.empty(20, 4, 2, 16)
    bm.moe_route(layer.logits, 2, 16, r, bm.workspace(bm.moe_route_workspace_bytes(20, 4, 2)))
    torch.cuda.synchronize()
    r.block_map[1] = torch.tensor([99, 5, 3], dtype=torch.int32)
    ws = bm.workspace(bm.moe_mx_forward_workspace_bytes(20, 256, 96, 4, 2, 0, 16))
    y = torch.empty((20, 256), dtype=torch.bfloat16, device="cuda")
    bm.moe_mx_forward(layer.x, layer.routed, None, r, y, ws)
    torch.cuda.synchronize()
    assert bm.STATUS_NAMES[bm.moe_check_status(ws)] == "MOE_ERR_INVALID_ARG"


@pytest.mark.parametrize("T,E,k,block_rows", [
    (131080, 256, 8, 16),     # more than 2^16 tiles of the routed experts
    (6291560, 2, 1, 96),      # and of the shared expert's tokens
])
def test_layer_of_more_tiles_than_16_bits_count(T, E, k, block_rows):
    """The bits of the same tokens in a smaller batch, those of the last tiles among them."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    d, I, I_shared = 64, 32, 32
    x = torch.randn(T, d, device="cuda", generator=gen, dtype=torch.float32).to(torch.bfloat16)
    logits = torch.randn(T, E, device="cuda", generator=gen, dtype=torch.float32)
    layer = _Layer(T, 1, d, I, I_shared, E)
    sc = bm.Scoring("sigmoid")

    def run(x, logits, block_rows):
        r = bm.Routing.empty(x.shape[0], E, k, block_rows)
        ws = bm.workspace(bm.moe_mx_layer_workspace_bytes(x.shape[0], d, I, E, k, I_shared, block_rows))
        y = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        bm.moe_mx_layer(logits, sc, x, layer.routed, layer.shared, k, block_rows, r, y, ws)
        torch.cuda.synchronize()
        assert bm.moe_check_status(ws) == 0
        return y, r

    y, r = run(x, logits, block_rows)
    assert int(r.num_blocks.item()) > 1 << 16 and torch.isfinite(y).all()
    some = torch.cat([torch.arange(1000), torch.arange(T - 20000, T)]).cuda()
    assert torch.equal(y[some], run(x[some], logits[some], 128)[0])


class _Rewritten:
    """Two fp32 matrices, written in turn into one MxMat that holds the other's codes when it is overwritten."""

    def __init__(self, N, K, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w = [torch.randn(N, K, device="cuda", generator=gen, dtype=torch.float32) * 2.0 ** i for i in (0, 3)]
        self.m = bm.MxMat.empty(1, N, K)

    def results(self, call, sync):
        """call()'s clones after each rewriting, with or without a synchronisation between the two."""
        got = []
        for i in range(8):
            bm.moe_mx_quantize(self.w[i % 2], self.m)
            if sync:
                torch.cuda.synchronize()
            got.append(call().clone())
        torch.cuda.synchronize()
        return torch.stack(got)


@pytest.mark.parametrize("kind", ["linear", "matmul", "pair"])
def test_a_product_right_after_its_weights(kind):
    """moe_mx_quantize into weights, then at once the product with them: the results of a synchronised program."""
    M, N, K = {"linear": (1, 2048, 2048), "matmul": (300, 2048, 2048), "pair": (4096, 4352, 1312)}[kind]
    w = _Rewritten(N, K, 1)
    x = torch.randn(M, K, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    a = _quantise(x)
    ws = bm.workspace(bm.moe_mx_linear_workspace_bytes(M, N, K))

    def call():
        if kind == "linear":
            bm.moe_mx_linear(x, w.m, y, ws)
        else:
            bm.moe_mx_matmul(a, w.m, y, ws)
        return y

    want = w.results(call, True)
    assert not torch.equal(want[0], want[1])
    assert torch.equal(w.results(call, False), want) and bm.moe_check_status(ws) == 0


def test_an_expert_layer_right_after_the_shared_experts_weights():
    layer = _Layer(8, 1, 512, 96, 128, 8)
    w = _Rewritten(128, 512, 2)
    layer.shared.gate = w.m
    r = bm.Routing.empty(1, 8, 2, 16)
    bm.moe_route(layer.logits, 2, 16, r, bm.workspace(bm.moe_route_workspace_bytes(1, 8, 2)))
    ws = bm.workspace(bm.moe_mx_forward_workspace_bytes(1, 512, 96, 8, 2, 128, 16))
    y = torch.empty((1, 512), dtype=torch.bfloat16, device="cuda")

    def call():
        bm.moe_mx_forward(layer.x, layer.routed, layer.shared, r, y, ws)
        return y

    want = w.results(call, True)
    assert not torch.equal(want[0], want[1]) and torch.equal(w.results(call, False), want)


def test_router_logits_right_after_the_routers_weights():
    """moe_mx_dequant writes bf16 weights of another kernel that reads them early."""
    E, d = 256, 2048
    ms = [_quantise(torch.randn(E, d, device="cuda", dtype=torch.float32) * 2.0 ** i) for i in (0, 3)]
    W = torch.empty((E, d), dtype=torch.bfloat16, device="cuda")
    x = torch.randn(1, d, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    logits = torch.empty((1, E), dtype=torch.float32, device="cuda")
    got = {}
    for sync in (True, False):
        got[sync] = []
        for i in range(8):
            bm.moe_mx_dequant(ms[i % 2], W)
            if sync:
                torch.cuda.synchronize()
            bm.moe_router_logits(x, W, logits)
            got[sync].append(logits.clone())
    torch.cuda.synchronize()
    assert not torch.equal(got[True][0], got[True][1]) and torch.equal(torch.stack(got[True]), torch.stack(got[False]))


@pytest.mark.parametrize("T,I_shared", [(2, 0), (2, 64), (40, 0), (40, 64)])  # the products for few tokens, and for more
def test_a_malformed_number_of_tiles_is_reported_and_harms_no_later_call(T, I_shared):
    E, k, br = 8, 2, 16
    layer = _Layer(9, T, 256, 96, I_shared, E)
    sc = bm.Scoring("softmax")
    want, _ = layer.run(sc, k, br)
    r = bm.Routing.empty(T, E, k, br)
    r.block_map.zero_()
    bm.moe_route_scored(layer.logits, sc, k, br, r, bm.workspace(bm.moe_route_workspace_bytes(T, E, k)))
    torch.cuda.synchronize()
    good = int(r.num_blocks.item())
    most = bm.moe_route_max_blocks(T, E, k, br)
    ws = bm.workspace(bm.moe_mx_forward_workspace_bytes(T, 256, 96, E, k, I_shared, br))
    for bad in (0, -1, T * k + 1, most + 1):
        for n, status in ((bad, "MOE_ERR_INVALID_ARG"), (good, "MOE_OK"), (good, "MOE_OK")):
            r.num_blocks.fill_(n)
            y = torch.full((T, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
            bm.moe_mx_forward(layer.x, layer.routed, layer.shared, r, y, ws)
            torch.cuda.synchronize()
            assert bm.STATUS_NAMES[bm.moe_check_status(ws)] == status, (bad, n)
            assert n != good or torch.equal(y, want), (bad, n)


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("entry", [[0, 2 ** 31 - 5, 16], [0, -2 ** 31, 1], [0, 0, -2 ** 31], [0, 0, 2 ** 31 - 1],
                                   [2 ** 31 - 1, 0, 1], [-1, 0, 1]])
def test_a_tile_at_the_ends_of_32_bits_is_reported(T, entry):
    """Such an entry of the block map is skipped: sums of its numbers that wrap do not let it pass."""
    layer = _Layer(4, T, 256, 96, 0, 4)
    r = bm.Routing.empty(T, 4, 2, 16)
    bm.moe_route(layer.logits, 2, 16, r, bm.workspace(bm.moe_route_workspace_bytes(T, 4, 2)))
    torch.cuda.synchronize()
    r.block_map[1] = torch.tensor(entry, dtype=torch.int32)
    ws = bm.workspace(bm.moe_mx_forward_workspace_bytes(T, 256, 96, 4, 2, 0, 16))
    y = torch.empty((T, 256), dtype=torch.bfloat16, device="cuda")
    bm.moe_mx_forward(layer.x, layer.routed, None, r, y, ws)
    torch.cuda.synchronize()
    assert bm.STATUS_NAMES[bm.moe_check_status(ws)] == "MOE_ERR_INVALID_ARG"


def test_new_memory_under_the_same_tensors():
    """Weights, the bias and a routing's buffers that were given other memory: the results of newly made objects."""
    a, b = _Layer(20, 24, 256, 96, 64, 8), _Layer(21, 24, 256, 96, 64, 8)
    bias = [torch.randn(8, device="cuda") for _ in range(2)]

    def run(layer, scoring, r, x, logits):
        y = torch.empty((24, 256), dtype=torch.bfloat16, device="cuda")
        ws = bm.workspace(bm.moe_mx_layer_workspace_bytes(24, 256, 96, 8, 2, 64, 16))
        bm.moe_mx_layer(logits, scoring, x, layer.routed, layer.shared, 2, 16, r, y, ws)
        torch.cuda.synchronize()
        return y, r.ids.clone()

    fresh = run(b, bm.Scoring("sigmoid", bias[1].clone()), bm.Routing.empty(24, 8, 2, 16), a.x, a.logits)
    sc, r = bm.Scoring("sigmoid", bias[0]), bm.Routing.empty(24, 8, 2, 16)
    run(a, sc, r, a.x, a.logits)
    old = []  # kept, so that nothing else gets their memory

    def replace(t, by):
        old.append(t.data)
        t.data = by.clone()

    for name in ("gate", "up", "down"):
        for mine, other in ((a.routed, b.routed), (a.shared, b.shared)):
            replace(getattr(mine, name).q, getattr(other, name).q)
            replace(getattr(mine, name).sp, getattr(other, name).sp)
    replace(sc.bias, bias[1])
    for name in ("ids", "w", "counts", "offsets", "perm", "inv_perm", "block_map", "num_blocks"):
        replace(getattr(r, name), getattr(r, name))
        getattr(r, name).fill_(-1)
    y, ids = run(a, sc, r, a.x, a.logits)
    assert torch.equal(ids, fresh[1]) and torch.equal(y, fresh[0])


@pytest.mark.parametrize("T,d,I,I_shared,E,k,block_rows", [
    (1000, 256, 96, 64, 64, 6, 128),
    (700, 160, 96, 0, 130, 4, 32),
    (2000, 128, 160, 96, 40, 3, 96),
])
def test_layer_of_many_tokens_and_experts(T, d, I, I_shared, E, k, block_rows):
    layer = _Layer(T + E, T, d, I, I_shared, E)
    y, r = layer.run(bm.Scoring("sigmoid", scale=1.5), k, block_rows, runs=2)
    layer.check(y, r)
