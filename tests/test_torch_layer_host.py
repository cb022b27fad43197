"""What the torch functions refuse before a C entry point is called, as far as
that needs no GPU: tensors stand in for those of a second device."""
import pytest
import torch


@pytest.fixture(scope="module")
def uz():
    import __graft_entry__

    __graft_entry__.build_library()
    import lossless_float_tensor_gb300 as uz

    return uz


class _There:
    """A tensor on another device, of which nobody may take the address."""

    def __init__(self, t, index):
        self._t, self._index = t, index

    def __getattr__(self, name):
        assert name not in ("data_ptr", "nbytes"), "refused before its memory is asked for"
        return getattr(self._t, name)

    def get_device(self):
        return self._index

    device = property(lambda self: torch.device("cuda", self._index))


class _Entry:
    name = "entry"

    def size(self, args):
        return 0

    def call(self, args, workspace, need, status, stream):
        raise AssertionError("called")


@pytest.mark.parametrize("which", ["workspace", "status"])
@pytest.mark.parametrize("layer", ["cache", "ops"])
def test_memory_of_another_device_is_refused(uz, monkeypatch, layer, which):
    from lossless_float_tensor_gb300 import cache, ops

    there = {"workspace": None, "status": None, which: _There(torch.zeros(8, dtype=torch.int32), 1)}
    monkeypatch.setitem(ops._calls, "entry", (lambda ref: 0, _Entry().call))
    monkeypatch.setattr(cache, "_torch", torch)
    with pytest.raises(uz.UzipError, match=f"{which} is on cuda:1, the call runs on cuda:0"):
        if layer == "cache":
            cache._issue(_Entry(), b"", 0, there["workspace"], there["status"], False)
        else:
            ops._run("entry", ops.LinearArgs(), torch.device("cuda", 0), there["workspace"], there["status"], False)


def test_memory_of_this_device_and_of_the_host_is_passed_on(uz):
    from lossless_float_tensor_gb300 import ops

    t = torch.zeros(8, dtype=torch.int32)
    ops._extras(t, t, 0)  # the C entry point refuses host memory that is not mapped
    ops._extras(_There(t, 1), _There(t, 1), 1)
    for bad in ((t[::2], None), (None, t.long()), (None, t[:0])):
        with pytest.raises(uz.UzipError):
            ops._extras(*bad, 0)


# ---- allocation ----------------------------------------------------------------

def _as_it_is(shape, strides, dtype):
    return torch.empty_strided(shape, strides, dtype=dtype)


@pytest.mark.parametrize("change", [
    None, lambda shape, strides, dtype, device: _as_it_is(shape, strides, dtype), lambda shape, dtype, strides: _as_it_is(shape, strides, dtype),
    lambda *a: _as_it_is(a[0], (3, 1), a[2]), lambda *a: _as_it_is(*a[:2], torch.int32), lambda *a: None, lambda *a: 1 / 0,
    lambda *a: _as_it_is(a[0], a[1], a[2])[:1], lambda *a: _There(_as_it_is(*a), 7),
])
def test_an_allocation_of_torchs_own_that_has_changed_is_not_used(uz, monkeypatch, change):
    from lossless_float_tensor_gb300 import cache

    guards = torch._C._dynamo.guards
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # that of tensors without a GPU
    for name in ("_torch", "_empty"):
        monkeypatch.setattr(cache, name, None)
    monkeypatch.setattr(guards, "_empty_strided_cuda", change, raising=False)
    assert cache._load() is torch and cache._empty is not None and cache._empty is not change
    monkeypatch.setattr(guards, "_empty_strided_cuda", _as_it_is, raising=False)
    assert cache._load() is torch and cache._empty is _as_it_is


@pytest.mark.gpu
def test_results_without_torchs_own_allocation(uz, monkeypatch):
    from lossless_float_tensor_gb300 import cache

    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((3, 8, 64), (200, 2, 16, 64), (200, 2, 16, 64)))
    table, lengths = torch.arange(180, dtype=torch.int32, device="cuda").view(3, 60), torch.tensor([900, 1, 300], dtype=torch.int32, device="cuda")
    call = lambda: uz.paged_attention(q, k, v, table, lengths, with_lse=True, check=True)  # noqa: E731
    want = call()
    for name in ("_torch", "_empty"):
        monkeypatch.setattr(cache, name, None)
    monkeypatch.setattr(torch._C._dynamo.guards, "_empty_strided_cuda", None, raising=False)
    got = call()
    assert cache._empty is not None and all(torch.equal(a, b) for a, b in zip(got, want))
