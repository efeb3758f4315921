"""Refusals of the scored routing's and the MXFP4 calls, on the host (nothing is launched), and the reference's own
pieces that need no GPU."""
import ctypes as C

import numpy as np
import pytest

import bit_moe_expert_gb300 as bm
import mx_ref
from bit_moe_expert_gb300 import build as bbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x100000


@pytest.fixture(scope="module")
def L():
    bbuild.build()
    return bm.lib()


def _scoring(score=1, bias=0, n_group=1, topk_group=1, group_top=1, renormalize=1, scale=1.0):
    return bm._Scoring(score, bias, n_group, topk_group, group_top, renormalize, scale)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(E=2000), UNSUPPORTED),
    (dict(k=33), UNSUPPORTED), (dict(k=65, E=64), UNSUPPORTED), (dict(block_rows=0), UNSUPPORTED),
    (dict(block_rows=129), UNSUPPORTED), (dict(logits=0), INVALID), (dict(ws=0), WORKSPACE),
    (dict(ws=FAKE + 16), WORKSPACE), (dict(short=1), WORKSPACE), (dict(sc=None), INVALID),
    (dict(sc=_scoring(score=2)), INVALID), (dict(sc=_scoring(score=-1)), INVALID),
    (dict(sc=_scoring(n_group=0)), INVALID), (dict(sc=_scoring(n_group=5)), INVALID),
    (dict(sc=_scoring(n_group=64, topk_group=64)), UNSUPPORTED), (dict(sc=_scoring(n_group=8, topk_group=0)), INVALID),
    (dict(sc=_scoring(n_group=8, topk_group=9)), INVALID), (dict(sc=_scoring(n_group=32, topk_group=1)), INVALID),
    (dict(sc=_scoring(group_top=0)), INVALID), (dict(sc=_scoring(group_top=3)), INVALID),
    (dict(E=32, k=4, sc=_scoring(n_group=32, topk_group=8, group_top=2)), INVALID),
    (dict(sc=_scoring(scale=float("nan"))), INVALID), (dict(sc=_scoring(scale=float("inf"))), INVALID),
    (dict(sc=_scoring(bias=FAKE + 2)), INVALID)])
def test_route_scored_refuses(L, change, want):
    a = dict(T=16, E=64, k=4, block_rows=16, logits=FAKE, ws=FAKE, sc=_scoring(), short=0)
    a.update(change)
    need = bm.moe_route_workspace_bytes(16, a["E"] or 64, a["k"] or 4) - a["short"]
    r = bm._Routing(*([FAKE] * 8), 0)
    sc = C.byref(a["sc"]) if a["sc"] is not None else None
    assert L.moe_route_scored(a["logits"], sc, a["T"], a["E"], a["k"], a["block_rows"], C.byref(r), a["ws"], need,
                              None) == want


def test_scale_bytes(L):
    assert bm.moe_mx_scale_bytes(1, 1, 32) == 512
    assert bm.moe_mx_scale_bytes(3, 129, 160) == 3 * 2 * 2 * 512
    for bad in ((0, 1, 32), (1, 0, 32), (1, 1, 0), (1, 1, 48), (1, 1, -32), (1, 1, (1 << 20) + 32)):
        assert bm.moe_mx_scale_bytes(*bad) == 0


def test_quantise_and_dequant_refuse(L):
    m = bm._MxMat(FAKE, FAKE)
    q = lambda X=FAKE, t=0, rows=4, K=64, ld=64, m=m: L.moe_mx_quantize(X, t, rows, K, ld, C.byref(m), None)
    assert q(rows=0) == OK
    assert q(X=0) == INVALID and q(X=FAKE + 2) == INVALID
    assert q(t=3) == INVALID and q(t=-1) == INVALID
    assert q(rows=-1) == INVALID and q(K=48) == INVALID and q(K=0) == INVALID
    assert q(ld=32) == INVALID and q(ld=68) == INVALID          # rows overlap; the pitch is no multiple of 16 bytes
    assert q(m=bm._MxMat(0, FAKE)) == INVALID and q(m=bm._MxMat(FAKE, FAKE + 4)) == INVALID
    d = lambda E=1, N=4, K=64, t=0, W=FAKE, m=m: L.moe_mx_dequant(C.byref(m), E, N, K, t, W, None)
    assert d(t=1) == UNSUPPORTED
    assert d(E=0) == INVALID and d(N=0) == INVALID and d(K=31) == INVALID and d(W=0) == INVALID and d(W=FAKE + 8) == INVALID
    assert L.moe_mx_prepack_scales(0, 1, 4, 64, FAKE, None) == INVALID
    assert L.moe_mx_prepack_scales(FAKE, 1, 4, 65, FAKE, None) == INVALID
    assert L.moe_mx_prepack_scales(FAKE, 0, 4, 64, FAKE, None) == INVALID


def test_products_refuse(L):
    m = bm._MxMat(FAKE, FAKE)
    bad = bm._MxMat(FAKE, 0)

    def mm(A=m, M=4, W=m, N=8, K=64, Y=FAKE, t=0, ws=FAKE, nb=256):
        return L.moe_mx_matmul(C.byref(A), M, C.byref(W), N, K, Y, t, ws, nb, None)

    assert mm(M=0) == OK
    assert mm(M=-1) == INVALID and mm(N=0) == INVALID and mm(K=33) == INVALID and mm(Y=0) == INVALID
    assert mm(Y=FAKE + 8) == INVALID and mm(A=bad) == INVALID and mm(W=bad) == INVALID
    assert mm(t=1) == UNSUPPORTED and mm(t=7) == INVALID
    assert mm(ws=0) == WORKSPACE and mm(ws=FAKE + 1) == WORKSPACE and mm(nb=255) == WORKSPACE
    need = bm.moe_mx_linear_workspace_bytes(4, 8, 64)
    assert need % 256 == 0 and need >= 256 + 4 * 32 + 512 and bm.moe_mx_linear_workspace_bytes(4, 8, 60) == 0

    def lin(X=FAKE, xt=0, T=4, K=64, ld=64, W=m, N=8, Y=FAKE, t=0, ws=FAKE, nb=need):
        return L.moe_mx_linear(X, xt, T, K, ld, C.byref(W), N, Y, t, ws, nb, None)

    assert lin(T=0) == OK
    assert lin(X=0) == INVALID and lin(xt=4) == INVALID and lin(ld=60) == INVALID and lin(W=bad) == INVALID
    assert lin(t=1) == UNSUPPORTED and lin(nb=need - 1) == WORKSPACE and lin(ws=0) == WORKSPACE


def test_expert_calls_refuse(L):
    m = bm._MxMat(FAKE, FAKE)
    ex, sh = bm._MxExperts(m, m, m, 16), bm._MxExperts(m, m, m, 1)
    need = bm.moe_mx_forward_workspace_bytes(8, 256, 96, 16, 2, 64, 16)
    need_layer = bm.moe_mx_layer_workspace_bytes(8, 256, 96, 16, 2, 64, 16)
    assert need_layer >= max(need, bm.moe_route_workspace_bytes(8, 16, 2))

    def call(T=8, d=256, I=96, k=2, ex=ex, sh=sh, I_sh=64, ws=FAKE, nb=None, X=FAKE, Y=FAKE, br=16, layer=False, w=FAKE):
        r = bm._Routing(FAKE, w, *([FAKE] * 6), br)
        a = (C.byref(ex), C.byref(sh) if sh is not None else None, I_sh, C.byref(r), Y, ws)
        if layer:
            return L.moe_mx_layer(FAKE, C.byref(_scoring()), X, T, d, I, k, br, *a, need_layer if nb is None else nb, None)
        return L.moe_mx_forward(X, T, d, I, k, *a, need if nb is None else nb, None)

    assert call(T=0) == OK
    for layer in (False, True):
        f = lambda **kw: call(layer=layer, **kw)
        assert f(T=-1) == INVALID and f(d=100) == INVALID and f(I=80) == INVALID and f(I_sh=33) == INVALID
        assert f(k=0) == INVALID and f(k=17) == UNSUPPORTED
        assert f(sh=None) == INVALID and f(I_sh=0) == INVALID           # one without the other
        assert f(sh=bm._MxExperts(m, m, m, 2)) == INVALID
        assert f(ex=bm._MxExperts(m, m, bm._MxMat(FAKE + 4, FAKE), 16)) == INVALID
        assert f(ex=bm._MxExperts(m, m, m, 2000)) == UNSUPPORTED
        assert f(X=0) == INVALID and f(Y=FAKE + 2) == INVALID
        assert f(br=0) == UNSUPPORTED and f(br=129) == UNSUPPORTED
        assert f(ws=0) == WORKSPACE and f(ws=FAKE + 128) == WORKSPACE and f(nb=(need_layer if layer else need) - 1) == WORKSPACE
    assert call(w=0) == INVALID
    assert bm.moe_mx_forward_workspace_bytes(8, 256, 90, 16, 2, 0, 16) == 0


@pytest.mark.parametrize("layer", [False, True])
def test_expert_calls_refuse_more_items_than_are_counted(L, layer):
    """Tiles times 128-row tiles of an expert's matrices up to 2^30, of the routed experts and of the shared one."""
    m = bm._MxMat(FAKE, FAKE)

    def call(T, d, k, E, I_sh, br):
        ex, sh = bm._MxExperts(m, m, m, E), bm._MxExperts(m, m, m, 1)
        r = bm._Routing(*([FAKE] * 8), br)
        a = (C.byref(ex), C.byref(sh) if I_sh else None, I_sh, C.byref(r), FAKE, FAKE, 0, None)  # no workspace
        if layer:
            return L.moe_mx_layer(FAKE, C.byref(_scoring()), FAKE, T, d, 32, k, br, *a)
        return L.moe_mx_forward(FAKE, T, d, 32, k, *a)

    # 2^20 columns are 2^13 M tiles; T k + E = 2^17 tiles of them are exactly 2^30
    assert call(T=(1 << 17) - 4, d=1 << 20, k=1, E=4, I_sh=0, br=1) == WORKSPACE
    assert call(T=(1 << 17) - 3, d=1 << 20, k=1, E=4, I_sh=0, br=1) == UNSUPPORTED
    assert call(T=(1 << 17) - 4, d=1 << 20, k=1, E=4, I_sh=32, br=1) == UNSUPPORTED  # the shared expert's tiles
    assert call(T=8193, d=256, k=8, E=256, I_sh=32, br=1) == WORKSPACE               # past 2^16 tiles is fine


def test_binding_refuses_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="score"):
        bm.Scoring("relu")._ref(4)
    with pytest.raises(ValueError, match="CUDA"):
        bm.Scoring(bias=torch.zeros(4))._ref(4)
    with pytest.raises(ValueError, match="float64"):
        bm.Scoring(bias=torch.zeros(4, dtype=torch.float64))._ref(4)
    with pytest.raises(ValueError, match="uint8"):
        bm.MxMat(torch.zeros((1, 4, 16)), torch.zeros((1, 1, 1, 512)))._c()
    with pytest.raises(ValueError, match="CUDA"):
        bm.moe_mx_quantize(torch.zeros((4, 32)), None)
    with pytest.raises(ValueError, match="multiple of 32"):
        bm.MxMat.empty(1, 4, 40, device="cpu")


class _Dtype:
    def __init__(self, name):
        self.name = name

    def __str__(self):
        return "torch." + self.name


_UINT8, _FLOAT32 = _Dtype("uint8"), _Dtype("float32")


class _Tensor:
    """What the binding asks of a CUDA tensor, whose memory can be replaced as by set_ or an assignment to .data."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, at, shape, dtype):
        self.at, self.shape, self.dtype = at, shape, dtype

    def data_ptr(self):
        return self.at

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape))


def _fake_mat(at, E, N, K):
    return bm.MxMat(_Tensor(at, (E, N, K // 2), _UINT8), _Tensor(at + 8, (E, -(-N // 128), -(-K // 128), 512), _UINT8))


def test_structs_follow_their_tensors_memory():
    """A tensor that keeps its identity but not its memory or size: the next call gets the new ones."""
    m = _fake_mat(1024, 1, 128, 64)
    assert m._c().q == 1024 and m._c() is m._c()
    m.q.at = 2048
    assert m._c().q == 2048
    m.sp.at = 4096
    assert m._c().sp == 4096
    m.q.shape = (1, 64, 32)
    assert m._ref_and_shape()[1] == (1, 64, 64)

    ex = bm.MxExperts(_fake_mat(16, 2, 96, 256), _fake_mat(32, 2, 96, 256), _fake_mat(48, 2, 256, 96))
    first = ex._ref_and_sizes()
    assert ex._ref_and_sizes()[0] is first[0] and first[1] == (2, 96, 256)
    for mat, name in ((ex.gate, "gate"), (ex.up, "up"), (ex.down, "down")):
        for field in ("q", "sp"):
            getattr(mat, field).at += 4096
            got = getattr(ex._ref_and_sizes()[0]._obj, name)
            assert getattr(got, field) == getattr(mat, field).at, (name, field)
    ex.up.q.shape = (2, 64, 128)
    with pytest.raises(ValueError, match="expected"):
        ex._ref_and_sizes()

    sc = bm.Scoring(bias=_Tensor(64, (8,), _FLOAT32))
    assert sc._ref(8)._obj.bias == 64
    sc.bias.at = 128
    assert sc._ref(8)._obj.bias == 128

    names = ("ids", "w", "counts", "offsets", "perm", "inv_perm", "block_map", "num_blocks")
    r = bm.Routing(*(_Tensor(16 * i, (4,), None) for i in range(1, 9)), block_rows=16)
    assert r._c().ids == 16 and r._c() is r._c()
    for n in names:
        getattr(r, n).at += 1024
        assert getattr(r._c(), n) == getattr(r, n).at, n
    r.ids = None
    assert r._c().ids is None and r._c().w == r.w.at


def test_reference_rounding():
    """The tests' own MXFP4: the worked values of the E2M1 grid, its ties and its saturation."""
    x = np.zeros((1, 32))
    x[0, :12] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7, -0.75, 0.2, 0.3]
    v, s = mx_ref.quantise(x)
    assert s[0, 0] == 127
    np.testing.assert_array_equal(v[0, :12], [4, 0, 1, 1, 2, 2, 4, 4, 6, -1, 0, 0.5])
    np.testing.assert_array_equal(mx_ref.decode(mx_ref.encode(v)), v)
    assert mx_ref.quantise(np.full((1, 32), 2.0 ** -140))[1][0, 0] == 0
    assert mx_ref.pack(np.arange(8, dtype=np.uint8).reshape(1, 2, 4))[0, 0, 0, 16:20].tolist() == [4, 5, 6, 7]
