"""Checks of the product operators' C entry points that need no GPU: what is
refused before any CUDA call, and what workspace is asked for."""
import pytest


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__

    __graft_entry__.build_library()
    from lossless_float_tensor_gb300 import ops

    return ops


FAKE = 1 << 40  # aligned, never dereferenced
OK, BAD_ARG, BAD_DTYPE = 0, 1, 2


def _linear(ops, **kw):
    a = ops.LinearArgs(dtype=0, act=0, m=4, n=8, k=16, groups=0, x=FAKE, ldx=16, w=FAKE, ldw=16, y=FAKE, ldy=8)
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def _grad(ops, **kw):
    a = ops.LinearGradArgs(dtype=0, act=0, m=4, n=8, k=16, dy=FAKE, lddy=8, x=FAKE, ldx=16, w=FAKE, ldw=16, dx=FAKE, lddx=16,
                           dw=FAKE, lddw=16, db=FAKE)
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def _loss(ops, **kw):
    a = ops.CrossEntropyArgs(dtype=0, t=4, v=8, d=16, h=FAKE, ldh=16, w=FAKE, ldw=16, targets=FAKE, loss=FAKE, lse=FAKE)
    for name, v in kw.items():
        setattr(a, name, v)
    return a


@pytest.mark.parametrize("change,want", [
    (dict(dtype=1), BAD_DTYPE), (dict(dtype=3), BAD_DTYPE), (dict(dtype=9), BAD_DTYPE), (dict(dtype=-1), BAD_DTYPE),
    (dict(act=4), BAD_ARG), (dict(act=-1), BAD_ARG), (dict(m=-1), BAD_ARG), (dict(n=1 << 31), BAD_ARG),
    (dict(k=1 << 40), BAD_ARG), (dict(groups=2), BAD_ARG), (dict(offsets=FAKE), BAD_ARG), (dict(x=None), BAD_ARG),
    (dict(w=FAKE + 1), BAD_ARG), (dict(ldx=15), BAD_ARG), (dict(ldx=-16), BAD_ARG), (dict(ldx=1 << 40), BAD_ARG),
    (dict(y=None), BAD_ARG),
])
def test_linear_refuses(ops, change, want):
    assert ops.uzip_linear(_linear(ops, **change), None, 0, None, 0) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=1), BAD_DTYPE), (dict(act=7), BAD_ARG), (dict(dy=None), BAD_ARG), (dict(act=3), BAD_ARG),
    (dict(lddw=3), BAD_ARG), (dict(lddx=15), BAD_ARG), (dict(x=None), BAD_ARG), (dict(w=None), BAD_ARG),
])
def test_linear_backward_refuses(ops, change, want):
    assert ops.uzip_linear_backward(_grad(ops, **change), None, 0, None, 0) == want


@pytest.mark.parametrize("change", [
    dict(), dict(groups=2), dict(groups=0, offsets=FAKE), dict(groups=1025, offsets=FAKE, w_group=128),
    dict(groups=2, offsets=FAKE + 4, w_group=128), dict(groups=2, offsets=FAKE, w_group=127),
    dict(groups=2, offsets=FAKE, w_group=0),
])
def test_grouped_refuses(ops, change):
    assert ops.uzip_grouped_linear(_linear(ops, **change), None, 0, None, 0) == BAD_ARG


@pytest.mark.parametrize("change,want", [
    (dict(dtype=1), BAD_DTYPE), (dict(reserved=1), BAD_ARG), (dict(v=0), BAD_ARG), (dict(t=-1), BAD_ARG),
    (dict(targets=None), BAD_ARG), (dict(targets=FAKE + 4), BAD_ARG), (dict(d=1 << 31), BAD_ARG),
])
def test_cross_entropy_refuses(ops, change, want):
    assert ops.uzip_cross_entropy(_loss(ops, **change), None, 0, None, 0) == want
    a = ops.CrossEntropyGradArgs(dtype=0, t=4, v=8, d=16, h=FAKE, ldh=16, w=FAKE, ldw=16, targets=FAKE, lse=FAKE, dloss=FAKE)
    for name, v in change.items():
        setattr(a, name, v)
    assert ops.uzip_cross_entropy_backward(a, None, 0, None, 0) == want


def test_null_arguments(ops):
    lib = ops.library()
    for name in ("linear", "grouped_linear", "linear_backward", "grouped_linear_backward", "cross_entropy",
                 "cross_entropy_backward"):
        assert getattr(lib, f"uzip_{name}")(None, None, 0, None, None) == BAD_ARG
        assert getattr(lib, f"uzip_{name}_workspace_size")(None) == 0


def test_workspace_only_where_something_is_kept(ops):
    """Aligned operands need none; rows off 16-byte boundaries are copied, 256
    bytes at a time."""
    assert ops.uzip_linear_workspace_size(_linear(ops)) == 0
    assert ops.uzip_linear_workspace_size(_linear(ops, m=1, ldx=3)) == 0  # a lone row's stride says nothing
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    assert ops.uzip_linear_workspace_size(_linear(ops, ldx=17)) == up(4 * 16 * 2)
    assert ops.uzip_linear_workspace_size(_linear(ops, x=FAKE + 2)) == up(4 * 16 * 2)
    assert ops.uzip_linear_workspace_size(_linear(ops, k=13, ldx=13, ldw=13)) == up(4 * 16 * 2) + up(8 * 16 * 2)
    g = _linear(ops, groups=3, offsets=FAKE, k=13, ldx=16, ldw=13, w_group=8 * 13)
    assert ops.uzip_grouped_linear_workspace_size(g) == up(3 * 8 * 16 * 2)
    assert ops.uzip_linear_backward_workspace_size(_grad(ops)) == 0
    assert ops.uzip_linear_backward_workspace_size(_grad(ops, act=3, z=FAKE, ldz=8)) == up(4 * 8 * 2)
    # loss statistics for every 128 classes, and the targets' logits
    assert ops.uzip_cross_entropy_workspace_size(_loss(ops, t=100, v=1000)) == up(8 * 100 * 8) + up(100 * 4)


def test_cross_entropy_pieces(ops):
    """The gradient's workspace is a piece of the vocabulary wide, whatever the
    vocabulary, beside a copy of h (2 bytes a value), sums of dh over the
    pieces (4 bytes a value) and 28 bytes a token."""
    def need(t, v, piece=0, dh=FAKE):
        a = ops.CrossEntropyGradArgs(dtype=0, t=t, v=v, d=64, piece=piece, h=FAKE, ldh=64, w=FAKE, ldw=64, targets=FAKE,
                                     lse=FAKE, dloss=FAKE, dh=dh, lddh=64)
        return ops.uzip_cross_entropy_backward_workspace_size(a)

    def most(t, piece):
        return t * (2 * piece + 64 * (2 + 4) + 28) + 10 * 256

    assert need(4096, 128256) <= most(4096, 32768)
    assert need(4096, 1 << 30) == need(4096, 128256)
    assert need(1 << 20, 128256) <= most(1 << 20, 256)
    assert need(4096, 128256, piece=1024) <= most(4096, 1024)
    assert need(100, 1000, piece=10) - need(100, 1000, piece=10, dh=None) == 100 * 64 * 4  # sums over the pieces
