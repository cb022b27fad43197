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
