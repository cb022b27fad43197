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
