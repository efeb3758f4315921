"""A Routing whose buffers are too small for a call is refused by the binding, which alone knows their sizes: the library
would read or write past their ends.  Nothing is launched: the tensors are stand-ins, and the library's calls are noted."""
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bit_moe_expert_gb300 as bm  # noqa: E402


class _Tensor:
    is_cuda, device = True, "cuda:0"

    def __init__(self, at, shape, dtype):
        self.at, self.shape, self.dtype = at, tuple(shape), dtype

    def data_ptr(self):
        return self.at

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape))

    def stride(self):
        return tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def element_size(self):
        return self.dtype.itemsize


def _t(*shape, dtype=torch.int32):
    _t.at += 4096
    return _Tensor(_t.at, shape, dtype)


_t.at = 1 << 20
T, E, k, d, I, ROWS = 8, 16, 2, 256, 96, 16
A, TILES = T * k, 1 + E  # ceil(16 / 16) + E
NEED = {"ids": A, "w": A, "perm": A, "inv_perm": A, "block_map": 3 * TILES, "num_blocks": 1, "counts": E, "offsets": E + 1}
STREAM = types.SimpleNamespace(cuda_stream=0)


def _routing(T=T, ROWS=ROWS):
    tiles = -(-T * k // ROWS) + E
    return bm.Routing(ids=_t(T, k), w=_t(T, k, dtype=torch.float32), counts=_t(E), offsets=_t(E + 1), perm=_t(T * k),
                      inv_perm=_t(T * k), block_map=_t(tiles, 3), num_blocks=_t(1), block_rows=ROWS)


@pytest.fixture
def calls(monkeypatch):
    """The names of the library's calls made; every one succeeds."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or 0

    monkeypatch.setattr(bm, "lib", Library)
    return made


def _mx():
    def mat(E, N, K):
        return bm.MxMat(_t(E, N, K // 2, dtype=torch.uint8), _t(E, -(-N // 128), -(-K // 128), 512, dtype=torch.uint8))
    return bm.MxExperts(mat(E, I, d), mat(E, I, d), mat(E, d, I))


def _blk():
    def mat(E, N, K):
        return bm.BlkMat(_t(E, N, K, dtype=torch.uint8), _t(E, -(-N // 128), -(-K // 128), dtype=torch.float32))
    return bm.BlkExperts(mat(E, I, d), mat(E, I, d), mat(E, d, I))


def _affine():
    def mat(E, N, K):
        return bm.QMat(_t(E, K // 64, N, 8), _t(E, K // 64, N))
    return bm.Experts(mat(E, 64, d), mat(E, 64, d), mat(E, d, 64))


X, Y, LOGITS = (lambda: _t(T, d, dtype=torch.bfloat16)), (lambda: _t(T, d, dtype=torch.bfloat16)), (lambda: _t(T, E, dtype=torch.float32))
W_R, WS, SCORING = (lambda: _t(E, d, dtype=torch.bfloat16)), (lambda: _t(1 << 24, dtype=torch.uint8)), bm.Scoring("sigmoid")
ACT = lambda: bm.BlkAct(_t(T, d, dtype=torch.uint8), _t(d // 128, T, dtype=torch.float32))  # noqa: E731
WRITES = {
    "moe_route": lambda r: bm.moe_route(LOGITS(), k, ROWS, r, WS(), STREAM),
    "moe_route_x": lambda r: bm.moe_route_x(X(), W_R(), k, ROWS, r, WS(), LOGITS(), STREAM),
    "moe_route_noalloc": lambda r: bm.moe_route_noalloc(LOGITS(), k, ROWS, r, STREAM),
    "moe_route_scored": lambda r: bm.moe_route_scored(LOGITS(), SCORING, k, ROWS, r, WS(), STREAM),
    "moe_layer": lambda r: bm.moe_layer(LOGITS(), X(), _affine(), None, k, ROWS, r, Y(), WS(), STREAM),
    "moe_layer_x": lambda r: bm.moe_layer_x(X(), W_R(), _affine(), None, k, ROWS, LOGITS(), r, Y(), WS(), STREAM),
    "moe_mx_layer": lambda r: bm.moe_mx_layer(LOGITS(), SCORING, X(), _mx(), None, k, ROWS, r, Y(), WS(), STREAM),
    "moe_blk_layer": lambda r: bm.moe_blk_layer(LOGITS(), SCORING, X(), _blk(), None, k, ROWS, r, Y(), WS(), STREAM),
}
READS = {
    "moe_forward": lambda r: bm.moe_forward(X(), _affine(), None, r, Y(), WS(), STREAM),
    "moe_mx_forward": lambda r: bm.moe_mx_forward(X(), _mx(), None, r, Y(), WS(), STREAM),
    "moe_blk_forward": lambda r: bm.moe_blk_forward(X(), _blk(), None, r, Y(), WS(), STREAM),
    "moe_blk_forward of codes": lambda r: bm.moe_blk_forward(ACT(), _blk(), None, r, Y(), WS(), STREAM),
}
CALLS = {**WRITES, **READS}


def _used(name):
    return [b for b in NEED if name in WRITES or b in ("w", "perm", "inv_perm", "block_map", "num_blocks")
            or b == "ids" and name == "moe_forward"]


@pytest.mark.parametrize("name", CALLS)
def test_buffers_of_the_documented_sizes_are_taken(calls, name):
    for r in (_routing(), _routing(T + 5), _routing(T, ROWS // 2)):
        r.block_rows = ROWS
        CALLS[name](r)
        CALLS[name](r)
    assert [c for c in calls if c != "moe_route_max_blocks"] == 6 * [name.split()[0]]


@pytest.mark.parametrize("name", CALLS)
def test_one_element_too_few_is_refused(calls, name):
    for b in _used(name):
        r = _routing()
        full = getattr(r, b)
        short = _Tensor(full.at, (T, k) if b == "ids" else (NEED[b] - 1,), full.dtype)
        if b == "ids":  # (its columns are the call's k)
            short.numel = lambda: A - 1
        CALLS[name](r)
        setattr(r, b, short)                    # where the other one was
        with pytest.raises(ValueError, match=rf"{b} has {NEED[b] - 1} elements, expected {NEED[b]}"):
            CALLS[name](r)
        setattr(r, b, full)
        CALLS[name](r)
    assert len(calls) == 2 * len(_used(name))


@pytest.mark.parametrize("name", CALLS)
def test_buffers_of_a_decode_step_are_refused_for_a_prompt(calls, name):
    with pytest.raises(ValueError, match="elements"):
        CALLS[name](_routing(1))
    assert not calls


@pytest.mark.parametrize("name", WRITES)
def test_a_lower_tile_than_the_block_map_is_for_is_refused(calls, name):
    r = _routing()
    r.block_map = _t(TILES - 1, 3)
    with pytest.raises(ValueError, match="block_map"):
        CALLS[name](r)
    assert not calls


@pytest.mark.parametrize("name", CALLS)
def test_other_memory_than_32_bit_values_on_the_device_is_refused(calls, name):
    for change in (dict(dtype=torch.int64), dict(is_cuda=False), dict(is_contiguous=lambda: False)):
        r = _routing()
        for field, v in change.items():
            setattr(r.perm, field, v)
        with pytest.raises(ValueError, match="perm .* expected contiguous 32-bit"):
            CALLS[name](r)
    assert not calls


@pytest.mark.parametrize("name", READS)
def test_a_missing_buffer_is_left_to_the_library(calls, name):
    r = _routing()
    r.counts = r.offsets = None
    CALLS[name](r)
    assert calls == [name.split()[0]]
