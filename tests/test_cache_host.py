"""Checks of the cache operators' C entry points that need no GPU: what is
refused, what workspace is asked for, and the frequencies.  (Without a GPU no
address is one of a device; the refusals run again on real ones there.)"""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def cache():
    import __graft_entry__

    __graft_entry__.build_library()
    from lossless_float_tensor_gb300 import cache

    return cache


FAKE = 1 << 40  # aligned, never dereferenced
BAD_ARG, BAD_DTYPE = 1, 2


def _set(a, kw):
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def _rotary(cache, **kw):
    return _set(cache.RotaryArgs(dtype=0, scale=1.0, t=4, q_heads=2, kv_heads=1, d=16, rot=16, positions=FAKE, freqs=FAKE, q=FAKE, q_row=32,
                                 q_head=16, k=FAKE, k_row=16, k_head=16, q_out=FAKE, q_out_row=32, q_out_head=16, k_out=FAKE, k_out_row=16,
                                 k_out_head=16), kw)


def _append(cache, **kw):
    a = _rotary(cache, v=FAKE, v_row=16, v_head=16, pages=8, page=4, k_pages=FAKE, kp_page=64, kp_head=64, kp_token=16, v_pages=2 * FAKE, vp_page=64,
                vp_head=64, vp_token=16, slots=FAKE)
    return _set(a, kw)


def _attention(cache, **kw):
    return _set(cache.PagedAttentionArgs(dtype=0, seqs=3, q_heads=4, kv_heads=2, d=16, pages=8, page=4, width=5, q=3 * FAKE, q_row=64, q_head=16,
                                         k_pages=FAKE, kp_page=128, kp_head=64, kp_token=16, v_pages=FAKE, vp_page=128, vp_head=64, vp_token=16,
                                         table=FAKE, ldt=5, lengths=FAKE, scale=0.25, out=FAKE, out_row=64, out_head=16), kw)


def _state(cache, **kw):
    return _set(cache.CacheArgs(pages=8, page=4, seqs=3, width=5, refs=FAKE, table=FAKE, ldt=5, lengths=FAKE, n=2, from_=FAKE, list=FAKE, tokens=6,
                                slots=FAKE, positions=FAKE, pairs=FAKE), kw)


def _copy(cache, **kw):
    a = cache.CacheCopyArgs(dtype=0, layers=2, heads=2, page=4, d=16, from_pages=8, to_pages=8, pairs=FAKE, n=3)
    for pre, at in (("k", FAKE), ("v", 2 * FAKE)):
        _set(a, {pre: at, pre + "_layer": 1024, pre + "_page": 128, pre + "_head": 64, pre + "_token": 16})
        _set(a, {pre + "_to": at, pre + "t_layer": 1024, pre + "t_page": 128, pre + "t_head": 64, pre + "t_token": 16})
    return _set(a, kw)


ROTARY = [
    (dict(dtype=1), BAD_DTYPE), (dict(dtype=3), BAD_DTYPE), (dict(dtype=-1), BAD_DTYPE), (dict(interleaved=2), BAD_ARG), (dict(backward=-1), BAD_ARG),
    (dict(t=-1), BAD_ARG), (dict(t=1 << 31), BAD_ARG), (dict(d=0), BAD_ARG), (dict(d=1025), BAD_ARG), (dict(rot=18), BAD_ARG), (dict(rot=7), BAD_ARG),
    (dict(rot=-2), BAD_ARG), (dict(q_heads=-1), BAD_ARG), (dict(q=None), BAD_ARG), (dict(k=None), BAD_ARG), (dict(q=FAKE + 1), BAD_ARG),
    (dict(q_row=-32), BAD_ARG), (dict(q_row=1 << 50), BAD_ARG), (dict(q_out=None), BAD_ARG), (dict(q_out_row=31), BAD_ARG), (dict(q_out_head=8), BAD_ARG),
    (dict(q_out_row=0), BAD_ARG), (dict(positions=None), BAD_ARG), (dict(positions=FAKE + 4), BAD_ARG), (dict(freqs=FAKE + 4), BAD_ARG),
    (dict(slots=FAKE), BAD_ARG),
]


@pytest.mark.parametrize("change,want", ROTARY)
def test_rotary_refuses(cache, change, want):
    assert cache.uzip_rotary(_rotary(cache, **change), None, 0, None, 0) == want


APPEND = [
    (dict(dtype=4), BAD_DTYPE), (dict(backward=1), BAD_ARG), (dict(kv_heads=0), BAD_ARG), (dict(d=12, rot=12), BAD_ARG), (dict(page=0), BAD_ARG),
    (dict(v=None), BAD_ARG), (dict(slots=None), BAD_ARG), (dict(slots=FAKE + 4), BAD_ARG), (dict(k_pages=None), BAD_ARG), (dict(k_pages=FAKE + 8), BAD_ARG),
    (dict(kp_token=20), BAD_ARG), (dict(v_pages=FAKE), BAD_ARG), (dict(kp_token=8), BAD_ARG), (dict(vp_page=56), BAD_ARG), (dict(pages=-1), BAD_ARG), (dict(pages=1 << 31), BAD_ARG),
]


@pytest.mark.parametrize("change,want", APPEND)
def test_rotary_append_refuses(cache, change, want):
    assert cache.uzip_rotary_append(_append(cache, **change), None, 0, None, 0) == want


ATTENTION = [
    (dict(dtype=1), BAD_DTYPE), (dict(reserved=1), BAD_ARG), (dict(seqs=-1), BAD_ARG), (dict(seqs=65537), BAD_ARG), (dict(q_heads=3), BAD_ARG),
    (dict(q_heads=0), BAD_ARG), (dict(kv_heads=0), BAD_ARG), (dict(d=12), BAD_ARG), (dict(d=264), BAD_ARG), (dict(d=0), BAD_ARG), (dict(page=0), BAD_ARG),
    (dict(width=-1), BAD_ARG), (dict(window=-1), BAD_ARG), (dict(softcap=-1.0), BAD_ARG), (dict(softcap=math.inf), BAD_ARG), (dict(softcap=math.nan), BAD_ARG), (dict(softcap=1e-42), BAD_ARG),
    (dict(q=None), BAD_ARG), (dict(q=FAKE + 1), BAD_ARG), (dict(k_pages=FAKE + 8), BAD_ARG), (dict(kp_token=17), BAD_ARG), (dict(vp_head=-64), BAD_ARG),
    (dict(out=None), BAD_ARG), (dict(out=3 * FAKE), BAD_ARG), (dict(out_row=63), BAD_ARG), (dict(out_head=0), BAD_ARG), (dict(ldt=-5), BAD_ARG), (dict(table=None), BAD_ARG),
    (dict(table=FAKE + 2), BAD_ARG), (dict(lengths=None), BAD_ARG), (dict(lse=FAKE + 1), BAD_ARG),
]


@pytest.mark.parametrize("change,want", ATTENTION)
def test_paged_attention_refuses(cache, change, want):
    assert cache.uzip_paged_attention(_attention(cache, **change), None, 0, None, 0) == want


STATE = [dict(pages=-1), dict(page=0), dict(seqs=-1), dict(seqs=65537), dict(width=-1), dict(ldt=4), dict(refs=None), dict(refs=FAKE + 2),
         dict(table=None), dict(lengths=None)]


RESERVE = STATE + [dict(tokens=-1), dict(list=None), dict(slots=None), dict(positions=FAKE + 4), dict(pairs=None)]
FORK = STATE + [dict(n=-1), dict(list=None)]


@pytest.mark.parametrize("change", RESERVE)
def test_reserve_refuses(cache, change):
    assert cache.uzip_cache_reserve(_state(cache, **change), None, 0, None, 0) == BAD_ARG


@pytest.mark.parametrize("change", FORK)
def test_fork_and_free_refuse(cache, change):
    assert cache.uzip_cache_fork(_state(cache, **change), None, 0, None, 0) == BAD_ARG
    assert cache.uzip_cache_free(_state(cache, **change), None, 0, None, 0) == BAD_ARG


def test_fork_refuses_no_parents(cache):
    assert cache.uzip_cache_fork(_state(cache, from_=None), None, 0, None, 0) == BAD_ARG


@pytest.mark.parametrize("change", STATE + [dict(pairs=None)])
def test_compact_refuses(cache, change):
    assert cache.uzip_cache_compact(_state(cache, **change), None, 0, None, 0) == BAD_ARG


COPY = [
    (dict(dtype=1), BAD_DTYPE), (dict(reserved=1), BAD_ARG), (dict(layers=-1), BAD_ARG), (dict(heads=0), BAD_ARG), (dict(d=12), BAD_ARG),
    (dict(d=512), BAD_ARG), (dict(to_pages=1572865, from_pages=1572865), BAD_ARG), (dict(to_pages=9), BAD_ARG), (dict(k_to=FAKE + 4096), BAD_ARG),
    (dict(k=FAKE + 8, k_to=FAKE + 8), BAD_ARG), (dict(kt_page=256), BAD_ARG), (dict(k_token=8, kt_token=8), BAD_ARG), (dict(pairs=None), BAD_ARG),
    (dict(pairs=FAKE + 4), BAD_ARG), (dict(n=-1), BAD_ARG), (dict(v=FAKE, v_to=FAKE), BAD_ARG), (dict(k_to=3 * FAKE, v_to=3 * FAKE), BAD_ARG),
    (dict(k_to=3 * FAKE, v_to=FAKE), BAD_ARG), (dict(k_layer=-1024, kt_layer=-1024), BAD_ARG),
]


@pytest.mark.parametrize("change,want", COPY)
def test_copy_refuses(cache, change, want):
    assert cache.uzip_cache_copy(_copy(cache, **change), None, 0, None, 0) == want


def test_null_arguments(cache):
    lib = cache.library()
    for name in ("rotary", "rotary_append", "paged_attention", "cache_reserve", "cache_fork", "cache_free", "cache_compact", "cache_copy"):
        assert getattr(lib, f"uzip_{name}")(None, None, 0, None, None) == BAD_ARG
        assert getattr(lib, f"uzip_{name}_workspace_size")(None) == 0


def test_workspace_only_where_something_is_kept(cache):
    """Short contexts are not cut between blocks; the parts of long ones take
    two sums of every kept head for each block, whatever the sequences."""
    size = cache.uzip_paged_attention_workspace_size
    assert size(_attention(cache)) == 0
    assert size(_attention(cache, width=1 << 20, window=100)) == 0
    long = size(_attention(cache, width=1 << 20))
    assert 0 < long <= 2 * 3 * 160 * 8 * (16 + 2) * 4 + 16 * 3 * 160 + 4 * 256
    assert size(_attention(cache, width=1 << 20, seqs=1000)) <= long
    assert size(_attention(cache, width=1 << 20, d=12)) == 0
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    reserve, fork = cache.uzip_cache_reserve_workspace_size, cache.uzip_cache_fork_workspace_size
    assert reserve(_state(cache, seqs=1000, pages=5000, tokens=100)) == 0  # lists that one block keeps to itself
    assert reserve(_state(cache, seqs=3000, pages=5000, tokens=100)) == 3 * up(12000) + up(24000) + up(800)
    assert reserve(_state(cache, seqs=1000, pages=5000, tokens=100000)) == 3 * up(4000) + up(8000) + up(20000)
    assert fork(_state(cache, seqs=1000)) == 0
    assert fork(_state(cache, seqs=20000)) == up(80000) and fork(_state(cache, seqs=1000, n=1000)) == up(4000)
    assert cache.uzip_cache_compact_workspace_size(_state(cache, pages=5000)) == 2 * up(10000) + up(20000)


def test_frequencies(cache):
    f = lambda **kw: cache.rotary_frequencies(64, device="cpu", **kw)  # noqa: E731
    j = torch.arange(32, dtype=torch.float64)
    plain = 10000.0 ** (-j / 32)
    close = lambda a, b: torch.allclose(a, b, rtol=1e-13, atol=0)  # noqa: E731
    assert close(f(), plain) and close(f(base=500.0), 500.0 ** (-j / 32))
    assert close(f(scaling="linear", factor=4.0), plain / 4)
    ntk = f(scaling="ntk", factor=8.0)
    assert ntk[0] == 1 and close(ntk[-1:], plain[-1:] / 8)
    turns = 4096 * plain / (2 * math.pi)
    bands = f(scaling="bands", factor=8.0, trained=4096, fast=4.0, slow=1.0)
    assert close(bands[turns > 4], plain[turns > 4]) and close(bands[turns < 1], plain[turns < 1] / 8)
    mid = (turns > 1) & (turns < 4)
    keep = (turns - 1) / 3
    assert mid.any() and close(bands[mid], (plain * keep + plain / 8 * (1 - keep))[mid])
    yarn = f(scaling="yarn", factor=8.0, trained=4096)
    lo = math.floor(32 * math.log(4096 / (32 * 2 * math.pi)) / math.log(10000.0))
    hi = math.ceil(32 * math.log(4096 / (2 * math.pi)) / math.log(10000.0))
    ramp = ((j - lo) / (hi - lo)).clamp(0, 1)
    assert close(yarn, plain / 8 * ramp + plain * (1 - ramp))
    assert f().dtype == torch.float64 and cache.rotary_frequencies(0, device="cpu").numel() == 0


@pytest.mark.parametrize("kw", [dict(dim=63), dict(scaling="dynamic"), dict(base=0.0), dict(factor=-1.0), dict(scaling="yarn"),
                                dict(scaling="bands", trained=10, fast=1.0, slow=2.0), dict(scaling="yarn", trained=100, base=1.0), dict(dim=-2)])
def test_frequencies_refuse(cache, kw):
    from lossless_float_tensor_gb300 import UzipError

    with pytest.raises(UzipError):
        cache.rotary_frequencies(**{"dim": 64, "device": "cpu", **kw})


def test_list_cache():
    """The lists that the GPU's state is compared with, by hand."""
    from tests._cache import ListCache, Refused

    c = ListCache(6, 4, 3, 3)
    assert c.reserve([5, 0, 1], 8) == ([0, 1, 2, 3, 4, 8, -1, -1], [0, 1, 2, 3, 4, 0, 0, 0], [[-1, -1]] * 3)
    assert c.rows == [[0, 1], [], [2]] and c.refs == [1, 1, 1, 0, 0, 0]
    c.fork([0], [1])
    assert c.refs == [2, 2, 1, 0, 0, 0] and c.lengths == [5, 5, 1]
    slots, positions, copies = c.reserve([1, 1, 0], 2)
    assert copies == [[1, 3], [1, 4], [-1, -1]] and slots == [13, 17] and positions == [5, 5] and c.refs == [2, 0, 1, 1, 1, 0]
    c.free([0, -1])
    assert c.refs == [1, 0, 1, 0, 1, 0] and c.rows == [[], [0, 4], [2]]
    assert c.compact() == [[4, 1], [-1, -1], [-1, -1]] and c.rows == [[], [0, 1], [2]] and c.refs == [1, 1, 1, 0, 0, 0]
    with pytest.raises(Refused):
        c.reserve([13, 0, 0], 13)
    with pytest.raises(Refused):
        c.fork([1, 1], [0, 0])
    assert c.refs == [1, 1, 1, 0, 0, 0]
