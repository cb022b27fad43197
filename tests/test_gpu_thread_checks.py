"""What the first CUDA call of a new thread checks: the thread has no current
context then, and a driver call is what knows where an allocation ends.

Each call here is one that has nothing to do (no tokens, no sequences, no
pairs), so that nothing is launched whatever becomes of it; it names an operand
that its checks look at all the same.
"""
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OK, BAD_ARG = 0, 1


def _in_a_thread(f):
    got = []
    t = threading.Thread(target=lambda: got.append(f()))
    t.start()
    t.join(60)
    assert len(got) == 1
    return got[0]


def _calls(at):
    """name -> (entry point, its arguments, a field, its value past any allocation); `at` is the address of 1 MB."""
    from lossless_float_tensor_gb300 import cache, ops

    far = 1 << 30  # of what `at` starts: more than the allocation that holds it
    pool = dict(pages=4, page=4, k_pages=at, kp_page=64, kp_head=64, kp_token=16, v_pages=at + 4096, vp_page=64, vp_head=64, vp_token=16)
    state = dict(pages=4, page=4, seqs=0, width=4, refs=at, table=at, ldt=4, lengths=at, list=at, from_=at, slots=at, positions=at, pairs=at)
    attention = dict(dtype=0, seqs=0, q_heads=2, kv_heads=1, d=16, width=4, q=at, q_row=32, q_head=16, table=at, ldt=4, lengths=at, scale=1.0, out=at,
                     out_row=32, out_head=16, **pool)
    copy = dict(dtype=0, layers=1, heads=1, page=4, d=16, from_pages=4, to_pages=4, pairs=at, n=0)
    for n, name in enumerate(("k", "v")):
        copy |= {name: at + 4096 * n, name + "_page": 64, name + "_head": 64, name + "_token": 16}
        copy |= {name + "_to": at + 4096 * (n + 2), name + "t_page": 64, name + "t_head": 64, name + "t_token": 16}
    rotary = dict(dtype=0, scale=1.0, t=0, d=16, rot=16, positions=at, freqs=at)
    return {
        "rotary": (cache.uzip_rotary, cache.RotaryArgs(**rotary), "t", far),  # no heads: only the positions count
        "rotary_append": (cache.uzip_rotary_append, cache.RotaryArgs(**rotary, kv_heads=1, **pool), "pages", far),
        "paged_attention": (cache.uzip_paged_attention, cache.PagedAttentionArgs(**attention), "pages", far),
        "cache_reserve": (cache.uzip_cache_reserve, cache.CacheArgs(**state), "pages", far),
        "cache_fork": (cache.uzip_cache_fork, cache.CacheArgs(**state), "pages", far),
        "cache_free": (cache.uzip_cache_free, cache.CacheArgs(**state), "pages", far),
        "cache_compact": (cache.uzip_cache_compact, cache.CacheArgs(**(state | dict(pages=0, seqs=1))), "width", far),
        "cache_copy": (cache.uzip_cache_copy, cache.CacheCopyArgs(**copy), "from_pages", far),
        "linear": (ops.uzip_linear, ops.LinearArgs(dtype=0, n=8, k=8, w=at, ldw=8), "n", far),
        "cross_entropy": (ops.uzip_cross_entropy, ops.CrossEntropyArgs(dtype=0, v=8, d=8, w=at, ldw=8), "v", far),
        "cross_entropy_backward": (ops.uzip_cross_entropy_backward, ops.CrossEntropyGradArgs(dtype=0, v=8, d=8, w=at, ldw=8), "v", far),
    }


@pytest.fixture(scope="module")
def room():
    return torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")


NAMES = ("rotary", "rotary_append", "paged_attention", "cache_reserve", "cache_fork", "cache_free", "cache_compact", "cache_copy", "linear",
         "cross_entropy", "cross_entropy_backward")


@pytest.mark.parametrize("new_thread", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_an_operand_that_ends_too_early_is_refused(room, name, new_thread):
    call, args, field, far = _calls(room.data_ptr())[name]
    torch.cuda.synchronize()
    run = _in_a_thread if new_thread else lambda f: f()
    assert run(lambda: call(args, room.data_ptr(), room.numel(), None, 0)) == OK
    setattr(args, field, far)
    assert run(lambda: call(args, room.data_ptr(), room.numel(), None, 0)) == BAD_ARG


@pytest.mark.parametrize("new_thread", [False, True])
def test_a_status_that_is_not_the_devices_is_refused(room, new_thread):
    call, args, _, _ = _calls(room.data_ptr())["cache_fork"]
    torch.cuda.synchronize()
    run = _in_a_thread if new_thread else lambda f: f()
    for status in (torch.zeros(64, dtype=torch.int32).data_ptr(), 1 << 45):
        assert run(lambda: call(args, None, 0, status, 0)) == BAD_ARG
    assert run(lambda: call(args, None, 0, room.data_ptr(), 0)) == OK


_AT_ONCE = """
import threading, torch
from tests.test_gpu_thread_checks import _calls
room = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
call, args, field, far = _calls(room.data_ptr())["paged_attention"]
setattr(args, field, far)
torch.cuda.synchronize()
gate, got = threading.Barrier(16), []
def work():
    gate.wait()
    got.append(call(args, None, 0, None, 0))
threads = [threading.Thread(target=work) for _ in range(16)]
for t in threads:
    t.start()
for t in threads:
    t.join(60)
assert got == [1] * 16, got
"""


def test_the_first_calls_of_a_process_at_once():
    """The driver's functions are looked up by whichever call is first: none goes by an address check that is not there yet."""
    for _ in range(3):
        done = subprocess.run([sys.executable, "-c", _AT_ONCE], cwd=ROOT, timeout=300, capture_output=True, text=True)
        assert done.returncode == 0, done.stderr


# ---- results ----------------------------------------------------------------------

FIRST = ("linear", "grouped_linear", "linear_backward", "cross_entropy", "rotary", "rotary_append", "paged_attention", "cut_attention", "reserve", "fork", "free", "compact",
         "copy", "compress")


def _work(name, seed=1):
    """(call, what it changes or gives) for an operator with everything allocated before."""
    import lossless_float_tensor_gb300 as uz

    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x, w, offsets, targets = rand(4, 64), rand(32, 64), torch.tensor([0, 1, 4], device="cuda"), torch.tensor([0, 5, 31, 2], device="cuda")
    q, k, pool, pool2 = rand(2, 4, 64), rand(2, 2, 64), rand(60, 2, 16, 64), rand(60, 2, 16, 64)
    table, short, long = torch.arange(120, dtype=torch.int32, device="cuda").view(2, 60) % 60, i32(300, 3), i32(900, 3)
    positions, slots, freqs = torch.tensor([5, 1000], device="cuda"), torch.tensor([77, 3], device="cuda"), uz.rotary_frequencies(64)
    refs, rows, n = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in (60, (3, 20), 3))
    state = refs, rows, n
    if name in ("fork", "free", "compact"):
        uz.cache_reserve(*state, i32(40, 0, 50), 90, 16)
    if name == "compact":
        uz.cache_free(*state, i32(0), 16)
    room, size, status = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda"), torch.zeros((), dtype=torch.int64, device="cuda"), i32(9)
    out, y, moves = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"), i32(*[[7, 7]] * 30)
    listed = [torch.full((3,), 7, device="cuda"), torch.full((3,), 7, device="cuda"), i32(*[[7, 7]] * 3)]
    pairs, counts, zero, one = i32([3, 9], [-1, -1], [4, 10]), i32(1, 1, 1), i32(0), i32(1)
    kw = dict(status=status)
    calls = {
        "linear": (lambda: uz.linear(x, w, out=y, workspace=room, **kw), [y]),
        "grouped_linear": (lambda: uz.grouped_linear(x, w.view(2, 16, 64), offsets, out=y[:, :16], workspace=room, **kw), [y]),
        "linear_backward": (lambda: uz.linear_backward(y, x, w, workspace=room, **kw), []),
        "cross_entropy": (lambda: uz.cross_entropy(x, w, targets, workspace=room, **kw), []),
        "rotary": (lambda: uz.rotary(q, None, positions, freqs, out=(out, None), **kw), [out]),
        "rotary_append": (lambda: uz.rotary_append(q, k, k + 0, positions, freqs, pool2, pool, slots, out=out, **kw), [out, pool, pool2]),
        "paged_attention": (lambda: uz.paged_attention(q, pool, pool2, table[:, :20], short, out=out, **kw), [out]),
        "cut_attention": (lambda: uz.paged_attention(q, pool, pool2, table, long, out=out, workspace=room, **kw), [out]),
        "reserve": (lambda: uz.cache_reserve(*state, counts, 3, 16, out=listed, workspace=room, **kw), [*listed, *state]),
        "fork": (lambda: uz.cache_fork(*state, zero, one, 16, workspace=room, **kw), [*state]),
        "free": (lambda: uz.cache_free(*state, zero, 16, workspace=room, **kw), [*state]),
        "compact": (lambda: uz.cache_compact(*state, 16, out=moves, workspace=room, **kw), [moves, *state]),
        "copy": (lambda: uz.cache_copy(pool, pool2, pairs, **kw), [pool, pool2]),
        "compress": (lambda: uz.compress(x, out=room, out_size=size), [size]),
    }
    y.copy_(rand(4, 32))
    call, kept = calls[name]
    return call, kept, status, (room, size)


@pytest.mark.parametrize("name", FIRST)
def test_results_of_a_threads_first_call(name):
    """The same inputs in this thread and as the first call of a new one: the same bits of all that the call gives and changes."""
    def run(where):
        call, kept, status, (room, size) = _work(name)
        before = [t.clone() for t in kept]
        torch.cuda.synchronize()
        got = where(call)
        torch.cuda.synchronize()
        given = [t for t in (got if isinstance(got, (list, tuple)) else [got]) if t is not None]
        if name == "compress":
            given = [room[: int(size)]]
        else:
            assert int(status) == 0
            assert not kept or any(not torch.equal(a, b) for a, b in zip(before, kept))  # something was done
        return given + kept

    here, there = run(lambda f: f()), run(_in_a_thread)
    assert len(here) == len(there) and here
    for a, b in zip(here, there):
        assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))
