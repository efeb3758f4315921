"""Refusals of the block-scaled 8-bit calls and the RMS norm, on the host (nothing is launched), and the reference's own
pieces that need no GPU."""
import ctypes as C

import numpy as np
import pytest

import bit_moe_expert_gb300 as bm
import blk_ref
from bit_moe_expert_gb300 import build as bbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x100000


@pytest.fixture(scope="module")
def L():
    bbuild.build()
    return bm.lib()


M = bm._BlkMat(FAKE, FAKE)
BAD = [bm._BlkMat(0, FAKE), bm._BlkMat(FAKE, 0), bm._BlkMat(FAKE + 8, FAKE), bm._BlkMat(FAKE, FAKE + 4)]


def test_quantise_and_dequant_refuse(L):
    q = lambda X=FAKE, t=0, rows=4, K=64, ld=64, m=M: L.moe_blk_quantize(X, t, rows, K, ld, C.byref(m), None)
    assert q(rows=0) == OK
    assert q(X=0) == INVALID and q(X=FAKE + 2) == INVALID and q(t=3) == INVALID and q(t=-1) == INVALID
    assert q(rows=-1) == INVALID and q(K=40) == INVALID and q(K=0) == INVALID and q(K=(1 << 20) + 16) == INVALID
    assert q(ld=48) == INVALID and q(ld=68) == INVALID               # rows overlap; the pitch is no multiple of 16 bytes
    assert q(rows=(1 << 30) + 1) == UNSUPPORTED
    assert all(q(m=b) == INVALID for b in BAD) and L.moe_blk_quantize(FAKE, 0, 4, 64, 64, None, None) == INVALID
    w = lambda W=FAKE, t=0, E=1, N=4, K=64, m=M: L.moe_blk_quantize_weights(W, t, E, N, K, C.byref(m), None)
    v = lambda W=FAKE, t=0, E=1, N=4, K=64, m=M: L.moe_blk_dequant_weights(C.byref(m), E, N, K, t, W, None)
    for f in (w, v):
        assert f(W=0) == INVALID and f(W=FAKE + 8) == INVALID and f(t=3) == INVALID and f(E=0) == INVALID
        assert f(N=0) == INVALID and f(K=24) == INVALID and all(f(m=b) == INVALID for b in BAD)
        assert f(E=1 << 20, N=1 << 20, K=1 << 20) == UNSUPPORTED
    d = lambda X=FAKE, t=0, rows=4, K=64, m=M: L.moe_blk_dequant(C.byref(m), rows, K, t, X, None)
    assert d(rows=0) == OK and d(X=0) == INVALID and d(K=24) == INVALID and d(t=5) == INVALID and d(rows=-1) == INVALID
    assert all(d(m=b) == INVALID for b in BAD)


def test_products_refuse(L):
    def mm(A=M, m=4, W=M, N=8, K=64, Y=FAKE, t=0, ws=FAKE, nb=256):
        return L.moe_blk_matmul(C.byref(A), m, C.byref(W), N, K, Y, t, ws, nb, None)

    assert mm(m=0) == OK
    assert mm(m=-1) == INVALID and mm(N=0) == INVALID and mm(K=40) == INVALID and mm(Y=0) == INVALID
    assert mm(Y=FAKE + 8) == INVALID and all(mm(A=b) == INVALID and mm(W=b) == INVALID for b in BAD)
    assert mm(t=7) == INVALID and mm(m=(1 << 30) + 1) == UNSUPPORTED and mm(N=(1 << 30) + 1) == UNSUPPORTED
    assert mm(ws=0) == WORKSPACE and mm(ws=FAKE + 1) == WORKSPACE and mm(nb=255) == WORKSPACE
    need = bm.moe_blk_linear_workspace_bytes(4, 8, 64)
    assert need % 256 == 0 and need >= 256 + 4 * 64 + 4 * 4 and bm.moe_blk_linear_workspace_bytes(4, 8, 60) == 0

    def lin(X=FAKE, xt=0, T=4, K=64, ld=64, W=M, N=8, Y=FAKE, t=0, ws=FAKE, nb=need):
        return L.moe_blk_linear(X, xt, T, K, ld, C.byref(W), N, Y, t, ws, nb, None)

    assert lin(T=0) == OK
    assert lin(X=0) == INVALID and lin(xt=4) == INVALID and lin(ld=60) == INVALID and all(lin(W=b) == INVALID for b in BAD)
    assert lin(t=3) == INVALID and lin(nb=need - 1) == WORKSPACE and lin(ws=0) == WORKSPACE


def test_rmsnorm_refuses(L):
    def f(X=FAKE, xt=0, T=4, d=64, ld=64, r=FAKE, ro=FAKE, rt=0, g=FAKE, gt=0, eps=1e-6, Y=FAKE, yt=0, out=M):
        return L.moe_rmsnorm(X, xt, T, d, ld, r, ro, rt, g, gt, eps, Y, yt, C.byref(out) if out else None, None)

    assert f(T=0) == OK and f(T=0, r=0, ro=0, rt=7) == OK and f(T=0, Y=0, yt=9) == OK and f(T=0, out=None) == OK
    assert f(X=0) == INVALID and f(X=FAKE + 4) == INVALID and f(xt=3) == INVALID and f(T=-1) == INVALID
    assert f(d=0) == INVALID and f(d=40) == INVALID and f(ld=48) == INVALID and f(ld=68) == INVALID
    assert f(d=32784, ld=32784) == UNSUPPORTED
    assert f(r=0) == INVALID and f(ro=0) == INVALID and f(r=FAKE + 2) == INVALID and f(ro=FAKE + 2) == INVALID
    assert f(rt=1) == INVALID and f(xt=2, rt=0) == INVALID            # neither X's type nor fp32
    assert f(g=0) == INVALID and f(g=FAKE + 4) == INVALID and f(gt=1) == INVALID
    assert f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID and f(eps=float("inf")) == INVALID
    assert f(Y=0, out=None) == INVALID and f(Y=FAKE + 4) == INVALID and f(yt=3) == INVALID
    assert all(f(out=b) == INVALID for b in BAD)


def _scoring():
    return bm._Scoring(1, 0, 1, 1, 1, 1, 1.0)


def test_expert_calls_refuse(L):
    ex, sh = bm._BlkExperts(M, M, M, 16), bm._BlkExperts(M, M, M, 1)
    need = bm.moe_blk_forward_workspace_bytes(8, 256, 96, 16, 2, 64, 16)
    need_layer = bm.moe_blk_layer_workspace_bytes(8, 256, 96, 16, 2, 64, 16)
    assert need_layer >= max(need, bm.moe_route_workspace_bytes(8, 16, 2))

    def call(T=8, d=256, I=96, k=2, ex=ex, sh=sh, I_sh=64, ws=FAKE, nb=None, X=FAKE, XQ=None, Y=FAKE, br=16, layer=False, w=FAKE):
        r = bm._Routing(FAKE, w, *([FAKE] * 6), br)
        x = (X, C.byref(XQ) if XQ else None)
        a = (C.byref(ex), C.byref(sh) if sh is not None else None, I_sh, C.byref(r), Y, ws)
        if layer:
            return L.moe_blk_layer(FAKE, C.byref(_scoring()), *x, T, d, I, k, br, *a, need_layer if nb is None else nb, None)
        return L.moe_blk_forward(*x, T, d, I, k, *a, need if nb is None else nb, None)

    assert call(T=0) == OK and call(T=0, X=0, XQ=M) == OK
    for layer in (False, True):
        f = lambda **kw: call(layer=layer, **kw)
        assert f(T=-1) == INVALID and f(d=100) == INVALID and f(I=80) == INVALID and f(I_sh=33) == INVALID
        assert f(d=48) == INVALID and f(I=48) == INVALID              # multiples of 16, not of 32
        assert f(k=0) == INVALID and f(k=17) == UNSUPPORTED
        assert f(sh=None) == INVALID and f(I_sh=0) == INVALID and f(I_sh=-32) == INVALID
        assert f(sh=bm._BlkExperts(M, M, M, 2)) == INVALID
        assert all(f(ex=bm._BlkExperts(M, M, b, 16)) == INVALID for b in BAD)
        assert f(ex=bm._BlkExperts(M, M, M, 2000)) == UNSUPPORTED
        assert f(X=0) == INVALID and f(X=FAKE + 2) == INVALID and f(Y=FAKE + 2) == INVALID
        assert f(XQ=M) == INVALID                                     # both forms of X
        assert all(f(X=0, XQ=b) == INVALID for b in BAD)
        assert f(br=0) == UNSUPPORTED and f(br=129) == UNSUPPORTED
        assert f(ws=0) == WORKSPACE and f(ws=FAKE + 128) == WORKSPACE and f(nb=(need_layer if layer else need) - 1) == WORKSPACE
        assert f(X=0, XQ=M, ws=0) == WORKSPACE
    assert call(w=0) == INVALID
    assert bm.moe_blk_forward_workspace_bytes(8, 256, 90, 16, 2, 0, 16) == 0


@pytest.mark.parametrize("layer", [False, True])
def test_expert_calls_refuse_more_items_than_are_counted(L, layer):
    def call(T, d, k, E, I_sh, br):
        ex, sh = bm._BlkExperts(M, M, M, E), bm._BlkExperts(M, M, M, 1)
        r = bm._Routing(*([FAKE] * 8), br)
        a = (C.byref(ex), C.byref(sh) if I_sh else None, I_sh, C.byref(r), FAKE, FAKE, 0, None)  # no workspace
        if layer:
            return L.moe_blk_layer(FAKE, C.byref(_scoring()), FAKE, None, T, d, 32, k, br, *a)
        return L.moe_blk_forward(FAKE, None, T, d, 32, k, *a)

    # 2^20 columns are 2^13 M tiles; T k + E = 2^17 tiles of them are exactly 2^30
    assert call(T=(1 << 17) - 4, d=1 << 20, k=1, E=4, I_sh=0, br=1) == WORKSPACE
    assert call(T=(1 << 17) - 3, d=1 << 20, k=1, E=4, I_sh=0, br=1) == UNSUPPORTED
    assert call(T=(1 << 17) - 4, d=1 << 20, k=1, E=4, I_sh=32, br=1) == UNSUPPORTED  # the shared expert's tiles


@pytest.mark.parametrize("layer", [False, True])
def test_items_of_the_shared_expert_are_counted_in_tiles_of_its_height(L, layer):
    def call(T, I_sh, br):
        ex, sh = bm._BlkExperts(M, M, M, 4), bm._BlkExperts(M, M, M, 1)
        a = (C.byref(ex), C.byref(sh), I_sh, C.byref(bm._Routing(*([FAKE] * 8), br)), FAKE, FAKE, 0, None)  # no workspace
        if layer:
            return L.moe_blk_layer(FAKE, C.byref(_scoring()), FAKE, None, T, 32, 32, 1, br, *a)
        return L.moe_blk_forward(FAKE, None, T, 32, 32, 1, *a)

    # tiles of 16 tokens, 2^13 M tiles each, and ceil(T/16) + 4 routed ones of one M tile: 2^30 - 12, then 2^30 + 8181
    assert call((1 << 21) - 16 * 16, 1 << 20, 16) == WORKSPACE
    assert call((1 << 21) - 16 * 15, 1 << 20, 16) == UNSUPPORTED
    assert call((1 << 21) - 16 * 15, 1 << 20, 1) == UNSUPPORTED
    assert call((1 << 21) - 16 * 15, 1 << 20, 32) == WORKSPACE


def test_binding_refuses_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="CUDA"):
        bm.BlkMat.empty(1, 4, 64, device="cpu")._ref_and_shape()
    with pytest.raises(ValueError, match="expected a 2-D CUDA"):
        bm.moe_blk_quantize(torch.zeros(4, 64), None)
    with pytest.raises(ValueError, match="uint8"):
        bm.BlkAct(torch.zeros(4, 64), torch.zeros(1, 4))._ref_and_shape()
    with pytest.raises(ValueError, match="CUDA"):
        bm.moe_rmsnorm(torch.zeros(4, 64), torch.zeros(64), 1e-6)


def test_reference_quantisation_against_a_search():
    """The tests' own rounding: every candidate scale and code tried out."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 128)) * np.exp2(rng.integers(-8, 8, (6, 1)))
    x[0, :3] = [448 * 2.0 ** -5, -0.3, 17 / 1024]
    v, s = blk_ref.quantise(x)
    grid = np.concatenate([-blk_ref.GRID[::-1], blk_ref.GRID])
    for r in range(6):
        e = min(e for e in range(-40, 40) if np.abs(x[r]).max() <= 448 * 2.0 ** e)
        assert s[r, 0] == 2.0 ** e
        d = np.abs(x[r][:, None] / 2.0 ** e - grid[None])
        assert (np.abs(x[r] / 2.0 ** e - v[r]) == d.min(1)).all()
    q = np.arange(256, dtype=np.uint8)
    ok = (q & 127) != 127
    np.testing.assert_array_equal(blk_ref.encode(blk_ref.decode(q[ok])), q[ok])
    torch = pytest.importorskip("torch")
    np.testing.assert_array_equal(blk_ref.decode(q), torch.from_numpy(q).view(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("d,I,E,k,I_shared,rows", [(32, 4096, 8, 8, 0, 16), (2048, 512, 256, 8, 512, 16), (64, 1024, 4, 1, 8192, 128)])
def test_a_workspace_for_some_tokens_is_one_for_fewer(L, d, I, E, k, I_shared, rows):
    for f in (bm.moe_blk_forward_workspace_bytes, bm.moe_blk_layer_workspace_bytes):
        need = [f(T, d, I, E, k, I_shared, rows) for T in range(200)]
        assert need[0] > 0 and all(a <= b for a, b in zip(need, need[1:]))
        assert f((1 << 30) + 1, d, I, E, k, I_shared, rows) == 0
    need = [bm.moe_blk_linear_workspace_bytes(T, I, d) for T in range(200)]
    assert all(a <= b for a, b in zip(need, need[1:]))
