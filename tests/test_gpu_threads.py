"""Operators as the first CUDA call of a new thread, with everything allocated
before: the thread has no current context then."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _in_a_thread(f):
    got = []

    def work():
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join(60)
    assert len(got) == 1
    if isinstance(got[0], Exception):
        raise got[0]


@pytest.mark.parametrize("name", ["linear", "grouped_linear", "rotary", "rotary_append", "paged_attention", "cut_attention", "reserve", "fork", "compact", "copy", "compress"])
def test_first_call_of_a_thread(name):
    import lossless_float_tensor_gb300 as uz

    bf = dict(dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, w, offsets = rand(4, 64), rand(32, 64), torch.tensor([0, 1, 4], device="cuda")
    q, pool, pool2 = rand(2, 4, 64), rand(60, 2, 16, 64), rand(60, 2, 16, 64)
    table = torch.arange(60, dtype=torch.int32, device="cuda").view(1, 60).expand(2, -1)
    lengths = torch.tensor([900, 3], dtype=torch.int32, device="cuda")
    positions, slots, freqs = torch.arange(2, device="cuda"), torch.arange(2, device="cuda"), uz.rotary_frequencies(64)
    refs, rows, n = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in (60, (3, 20), 3))
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    room = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    outs = torch.empty(4, 32, **bf), torch.empty(2, 4, 64, **bf), torch.empty(2, 4, 64, **bf)
    listed = [torch.empty(3, dtype=torch.int64, device="cuda"), torch.empty(3, dtype=torch.int64, device="cuda"), torch.empty(3, 2, dtype=torch.int32, device="cuda")]
    moves, kids = torch.empty(30, 2, dtype=torch.int32, device="cuda"), torch.tensor([1], dtype=torch.int32, device="cuda")
    size = torch.empty((), dtype=torch.int64, device="cuda")
    calls = {
        "linear": lambda: uz.linear(x, w, out=outs[0]),
        "grouped_linear": lambda: uz.grouped_linear(x, w.view(2, 16, 64), offsets, out=outs[0][:, :16]),
        "rotary": lambda: uz.rotary(q, None, positions, freqs, out=(outs[1], None)),
        "rotary_append": lambda: uz.rotary_append(q, q[:, :2], q[:, 2:], positions, freqs, pool2, pool, slots, out=outs[1]),
        "paged_attention": lambda: uz.paged_attention(q, pool, pool2, table[:, :20], short, out=outs[1]),
        "cut_attention": lambda: uz.paged_attention(q, pool, pool2, table, lengths, out=outs[2], workspace=room),
        "reserve": lambda: uz.cache_reserve(refs, rows, n, one, 3, 16, out=listed, workspace=room),
        "fork": lambda: uz.cache_fork(refs, rows, n, zero, kids, 16, workspace=room),
        "compact": lambda: uz.cache_compact(refs, rows, n, 16, out=moves, workspace=room),
        "copy": lambda: uz.cache_copy(pool, pool2, listed[2]),
        "compress": lambda: uz.compress(x, out=room, out_size=size),
    }
    listed[2].fill_(-1)
    short, zero = lengths.clamp(max=300), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    _in_a_thread(calls[name])
    torch.cuda.synchronize()
    if name == "linear":
        assert torch.equal(outs[0], uz.linear(x, w))
    if name == "cut_attention":
        assert torch.equal(outs[2], uz.paged_attention(q, pool, pool2, table, lengths))
