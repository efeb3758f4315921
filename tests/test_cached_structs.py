"""Matrices whose tensors change their layout in place, at the same address and with as many elements: a call takes them
as they are now, or refuses them.  (CPU tensors that pass for CUDA ones: nothing is launched.)"""
import pytest

torch = pytest.importorskip("torch")

import bit_moe_expert_gb300 as bm  # noqa: E402


class _Tensor(torch.Tensor):
    is_cuda = True


def _t(shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Tensor)


def _blk(E, N, K):
    return bm.BlkMat(_t((E, N, K)), _t((E, -(-N // 128), -(-K // 128)), torch.float32))


def _mx(E, N, K):
    return bm.MxMat(_t((E, N, K // 2)), _t((E, -(-N // 128), -(-K // 128), 512)))


def _act(rows, K):
    return bm.BlkAct(_t((rows, K)), _t((-(-K // 128), (rows + 3) // 4 * 4), torch.float32))


def test_a_new_shape_of_the_same_size_is_the_calls_shape():
    a, m, x = _act(4, 256), _blk(2, 256, 512), _mx(2, 256, 512)
    assert a._ref_and_shape()[1] == (4, 256) and m._ref_and_shape()[1] == x._ref_and_shape()[1] == (2, 256, 512)
    assert m._ref_and_shape() is m._ref_and_shape()
    a.q.resize_(8, 128)
    with pytest.raises(ValueError, match="s: shape"):            # scales for 4 x 256 still
        a._ref_and_shape()
    a.s.resize_(1, 8)
    assert a._ref_and_shape()[1] == (8, 128)
    a.q.resize_(6, 128)                                          # as many rows of scales
    assert a._ref_and_shape()[1] == (6, 128)
    m.q.resize_(2, 512, 256)
    with pytest.raises(ValueError, match="s: shape"):
        m._ref_and_shape()
    m.s.resize_(2, 4, 2)
    assert m._ref_and_shape()[1] == (2, 512, 256)
    x.q.resize_(2, 512, 128)
    x.sp.resize_(2, 4, 2, 512)
    assert x._ref_and_shape()[1] == (2, 512, 256)
    m.q.resize_(1, 512, 512)
    m.s.resize_(1, 4, 4)
    assert m._ref_and_shape()[1] == (1, 512, 512)


def test_sets_follow_their_matrices_shapes():
    for make, cls, scales in ((_blk, bm.BlkExperts, "s"), (_mx, bm.MxExperts, "sp")):
        ex = cls(make(2, 256, 512), make(2, 256, 512), make(2, 512, 256))
        assert ex._ref_and_sizes()[1] == (2, 256, 512)
        up = ex.up
        shape, sshape = up.q.shape, getattr(up, scales).shape
        up.q.resize_(2, 2 * shape[1], shape[2] // 2)
        getattr(up, scales).resize_(2, sshape[2], sshape[1], *sshape[3:])
        with pytest.raises(ValueError, match="expected"):
            ex._ref_and_sizes()


@pytest.mark.parametrize("make,scales", [(lambda: _blk(1, 256, 256), "s"), (lambda: _mx(1, 256, 512), "sp"), (lambda: _act(256, 256), "s")])
def test_a_transposed_matrix_or_a_shorter_table_of_scales_is_refused(make, scales):
    m = make()
    m._ref_and_shape()
    m.q.transpose_(-1, -2)                                       # square: shape, address and size stay
    with pytest.raises(ValueError, match="q: not contiguous"):
        m._ref_and_shape()
    m.q.transpose_(-1, -2)
    m._ref_and_shape()
    s = getattr(m, scales)
    shape = s.shape
    s.resize_(shape[0] - 1, *shape[1:])
    with pytest.raises(ValueError, match=f"{scales}: shape"):
        m._ref_and_shape()
    s.resize_(shape)
    m._ref_and_shape()


def test_scales_of_another_type_at_the_same_address_are_refused():
    for m in (_blk(1, 256, 256), _act(8, 256)):
        m._ref_and_shape()
        m.s.data = m.s.view(torch.int32)
        with pytest.raises(ValueError, match="s: torch.int32"):
            m._ref_and_shape()
