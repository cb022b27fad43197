"""The key-value cache's operators on the GPU against their 64-bit definitions
(tests/_cache.py), and against a cache kept in lists."""
import math
import random
import threading

import pytest
import torch

from tests import _cache as ref
from tests._products import within

pytestmark = pytest.mark.gpu

DTYPES = (torch.bfloat16, torch.float16)


@pytest.fixture(scope="module")
def uz():
    import lossless_float_tensor_gb300 as uz

    return uz


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bits(t):
    return t.contiguous().view(torch.int16)


# ---- attention of one token ---------------------------------------------------

def _attend(uz, lengths, heads, group, d, page, dtype, order="heads", seed=0, q_scale=2.0, width=None, **kw):
    g = _gen(seed + d + 7 * page)
    pages = sum(-(-n // page) for n in lengths) + 3
    k, v = ref.pools(g, pages, heads, page, d, dtype, order)
    table, n = ref.tables(lengths, page, pages, seed, width)
    q = _rand(g, (len(lengths), heads * group, d), dtype, q_scale)
    out, lse = uz.paged_attention(q, k, v, table, n, with_lse=True, check=True, **kw)
    want, want_lse, off, off_lse = ref.attention64(q, k, v, table, n, **kw)
    assert within(out, want, off) <= 1.0
    empty = n == 0
    assert bool((lse[empty] == -math.inf).all()) and not bool(out[empty].any())
    assert within(lse[~empty], want_lse[~empty], off_lse[~empty]) <= 1.0
    return q, k, v, table, n, out, lse


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,heads,group,d,page", [
    ([1], 1, 1, 64, 16), ([1, 0, 2, 15, 16, 17], 2, 4, 128, 16), ([0, 0, 0], 2, 1, 64, 16), ([33, 500, 512, 513, 1], 4, 8, 128, 16),
    ([100, 7], 3, 5, 80, 24), ([257, 64, 65], 1, 7, 96, 32), ([40, 300], 2, 3, 8, 7), ([70, 129], 2, 2, 256, 64), ([70, 129], 2, 9, 256, 1),
    ([19, 77], 1, 16, 192, 16), ([300, 12], 2, 12, 128, 128), ([90], 1, 33, 64, 8), ([19, 200, 0], 2, 32, 128, 16), ([77, 300], 1, 24, 80, 16), ([33], 2, 64, 40, 16), ([31, 200], 2, 20, 104, 16), ([5, 9] * 40, 1, 4, 72, 16),
])
def test_attention(uz, lengths, heads, group, d, page, dtype):
    _attend(uz, lengths, heads, group, d, page, dtype)


# lengths over the 512 tokens up to which a head's tokens stay together, so that blocks cut them
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,heads,group,d,page", [
    ([5000], 1, 8, 128, 16), ([4096, 1, 0, 4097, 3000], 2, 4, 128, 16), ([20000, 3], 1, 1, 64, 64), ([2777, 0, 1, 900], 3, 5, 80, 24),
    ([1500, 6000], 2, 16, 128, 32), ([700, 1400], 1, 40, 96, 16), ([3333], 2, 3, 256, 5), ([1000, 2500], 1, 11, 192, 16),
    ([1300, 700], 2, 32, 128, 16), ([900, 2000, 5], 1, 17, 64, 16), ([800, 1], 2, 27, 96, 24), ([1100], 1, 71, 64, 16), ([1000, 30], 1, 48, 128, 7),
    ([1200, 3], 2, 16, 256, 16), ([1200, 3], 1, 32, 192, 16), ([600] * 150, 2, 2, 64, 16), ([513, 30] * 130, 1, 4, 128, 16), ([40000], 8, 4, 128, 16),
])
def test_attention_cut_between_blocks(uz, lengths, heads, group, d, page, dtype):
    _attend(uz, lengths, heads, group, d, page, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 1000, 5000])
def test_attention_window(uz, window, dtype):
    _attend(uz, [1, 5, 16, 99, 100, 101, 1700, 0], 2, 4, 64, 16, dtype, window=window)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("softcap,scale,q_scale", [(30.0, None, 2.0), (5.0, 0.7, 3.0), (0.0, -0.3, 1.0), (50.0, 1.0, 30.0), (0.0, 0.0, 1.0), (0.0, 2.0, 4.0)])
def test_attention_scale_and_cap(uz, softcap, scale, q_scale, dtype):
    _attend(uz, [77, 1, 900], 2, 4, 96, 16, dtype, q_scale=q_scale, softcap=softcap, scale=scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("order", ["heads", "tokens"])
@pytest.mark.parametrize("n", [1, 2, 64, 1024, 8192])
def test_attention_of_equal_scores_is_the_mean(uz, n, order, dtype):
    """Queries of zero weigh all tokens alike; sums of small whole numbers and
    divisions by powers of two are exact, so every token of every head has to be
    there once."""
    g = _gen(n)
    heads, page, d = 3, 16, 128
    pages = n // page + 5
    k, v = ref.pools(g, pages, heads, page, d, dtype, order)
    # per head and column a whole mean, and a few tokens that stand out by amounts that cancel
    v.copy_(torch.randint(-3, 4, v.shape, generator=g, device="cuda").to(dtype))
    table, lengths = ref.tables([n], page, pages)
    q = torch.zeros(1, heads * 4, d, dtype=dtype, device="cuda")
    out, lse = uz.paged_attention(q, k, v, table, lengths, with_lse=True, check=True)
    t = torch.arange(n, device="cuda")
    mean = v[table[0].long()[t // page], :, t % page].double().mean(0)
    assert torch.equal(out[0].double(), mean.repeat_interleave(4, 0).to(dtype).double())
    assert float((lse - math.log(n)).abs().max()) <= 2.0 ** -20 * (2 + math.log(n))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page,group", [(1, 1), (16, 4), (24, 9), (100, 2)])
def test_attention_finds_one_token(uz, page, group, dtype):
    """Each query head asks for one token by its key, whose value comes back as it is."""
    heads, d, n = 2, 64, 700
    g = _gen(page)
    pages = -(-n // page) + 4
    k, v = ref.pools(g, pages, heads, page, d, dtype)
    table, lengths = ref.tables([n], page, pages)
    q = torch.empty(1, heads * group, d, dtype=dtype, device="cuda")
    want = torch.empty_like(q)
    places = [0, n - 1, 1, 15, 16, 511, 512, 513, 300, 17, 255, 400, 31, 32, 63, 64, 600, 650]
    for h in range(heads * group):
        t = places[h]
        at = int(table[0, t // page]), h // group, t % page
        q[0, h] = 30 * torch.sign(k[at].float()).to(dtype)  # the token's score is that of no other: sums of |k| against random signs
        want[0, h] = v[at]
    out = uz.paged_attention(q, k, v, table, lengths, check=True)
    assert torch.equal(_bits(out), _bits(want))


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_never_uses_what_lies_behind(uz, dtype):
    """NaN and infinities in unused pages, behind the last token, before the
    window, and table entries that mean nothing."""
    g = _gen(5)
    page, heads, d, lengths = 16, 2, 64, [5, 16, 700, 0, 33]
    pages = sum(-(-n // page) for n in lengths) + 3
    k, v = ref.pools(g, pages, heads, page, d, dtype)
    table, n = ref.tables(lengths, page, pages, fill=-7, width=60)
    q = _rand(g, (5, heads * 4, d), dtype)
    for window in (0, 20):
        clean = uz.paged_attention(q, k, v, table, n, window=window, check=True)
        for bad in (math.nan, math.inf, -math.inf):
            k2, v2 = torch.full_like(k, bad), torch.full_like(v, bad)
            for i, m in enumerate(lengths):
                t = torch.arange(max(0, m - window) if window else 0, m, device="cuda")
                at = table[i].long()[t // page], slice(None), t % page
                k2[at], v2[at] = k[at], v[at]
            got = uz.paged_attention(q, k2, v2, table, n, window=window, check=True)
            assert torch.equal(_bits(got), _bits(clean))


def test_attention_not_a_number_stays_in_its_sequence(uz):
    g = _gen(6)
    for lengths in ([40, 50, 60], [1000, 900, 1100]):
        pages = 250
        k, v = ref.pools(g, pages, 2, 16, 64, torch.bfloat16)
        table, n = ref.tables(lengths, 16, pages)
        q = _rand(g, (3, 8, 64), torch.bfloat16)
        clean = uz.paged_attention(q, k, v, table, n)
        for t in (0, 17, lengths[1] - 1):
            for pool in (k, v):
                at = int(table[1, t // 16]), 1, t % 16, 9
                kept = pool[at].clone()
                pool[at] = math.nan
                out = uz.paged_attention(q, k, v, table, n, check=True)
                pool[at] = kept
                assert bool(out[1, 4:, 9].isnan().all())
                assert pool is v or bool(out[1, 4:].isnan().all())
                out[1, 4:] = clean[1, 4:]
                assert torch.equal(_bits(out), _bits(clean))
        # a value that is infinite, and weighs something, makes its column so
        at = int(table[1, 1]), 1, 3, 5
        kept = v[at].clone()
        for big in (math.inf, -math.inf):
            v[at] = big
            out = uz.paged_attention(q / 8, k, v, table, n, check=True)
            assert bool((out[1, 4:, 5] == big).all()) and int(out.isinf().sum()) == 4 and not bool(out.isnan().any())
        v[at] = kept
        # every key of a head without a finite score: the softmax of nothing but -inf is no number
        q2 = torch.zeros_like(q)
        q2[..., 3] = 1
        k2 = k.clone()
        k2[:, 0, :, 3] = -math.inf
        out = uz.paged_attention(q2, k2, v, table, n)
        assert bool(out[:, :4].isnan().all()) and bool(out[:, 4:].isfinite().all())
        # some of them: they weigh nothing
        k2 = k.clone()
        at = table[0].long()[:2]
        k2[at, 0, :, 3] = -math.inf
        out = uz.paged_attention(q2, k2, v, table, n)
        t = torch.arange(32, lengths[0], device="cuda")
        at = table[0].long()[t // 16], 0, t % 16
        want = torch.softmax(k[at].double()[:, 3] * 64 ** -0.5, 0) @ v[at].double()
        assert float((out[0, 0].double() - want).abs().max()) <= 2.0 ** -7 * float(v[at].abs().max())


@pytest.mark.parametrize("lengths", [[40, 50, 60], [1000, 900, 1100]])
def test_attention_bad_lengths_and_pages(uz, lengths):
    """What cannot be is reported, gives NaN, and leaves the other sequences alone."""
    from lossless_float_tensor_gb300 import UzipError

    g = _gen(7)
    k, v = ref.pools(g, 250, 2, 16, 128, torch.bfloat16)
    table, n = ref.tables(lengths, 16, 250)
    q = _rand(g, (3, 8, 128), torch.bfloat16)
    clean, lse = uz.paged_attention(q, k, v, table, n, with_lse=True, check=True)
    want, want_lse, off, off_lse = ref.attention64(q, k, v, table, n)
    status = torch.full((), 99, dtype=torch.int32, device="cuda")

    def bad(t, m):
        got, l2 = uz.paged_attention(q, k, v, t, m, with_lse=True, status=status)
        assert int(status) == 1 and bool(got[1].isnan().all()) and bool(l2[1].isnan().all())
        for i in (0, 2):  # where blocks cut the tokens goes by all lengths; with those the same, the bits are
            assert within(got[i], want[i], off[i]) <= 1.0 and within(l2[i], want_lse[i], off_lse[i]) <= 1.0
            assert m is not n or (torch.equal(_bits(got[i]), _bits(clean[i])) and torch.equal(l2[i], lse[i]))
        with pytest.raises(UzipError):
            uz.paged_attention(q, k, v, t, m, check=True)

    for wrong in (-1, -2 ** 31, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        m = n.clone()
        m[1] = wrong
        bad(table, m)
    for col in (0, 1, (lengths[1] - 1) // 16):
        for wrong in (-1, 250, 2 ** 31 - 1, -2 ** 31):
            t = table.clone()
            t[1, col] = wrong
            bad(t, n)
    uz.paged_attention(q, k, v, table, n, status=status)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths", [[30, 300], [900, 1500]])
def test_attention_views(uz, lengths, dtype):
    """Queries out of a fused projection, pools that are a layer of larger ones
    in another order, a wide table, an output with gaps."""
    g = _gen(8)
    d, heads, group, page, s = 80, 3, 2, 16, len(lengths)
    q, k, v, table, n, out, _ = _attend(uz, lengths, heads, group, d, page, dtype, order="heads")
    fused = _rand(g, (s, 1 + (heads * group + 5) * d), dtype)
    fused[:, 1:1 + heads * group * d] = q.flatten(1)
    q2 = fused[:, 1:1 + heads * group * d].unflatten(1, (-1, d))
    both = torch.full((k.shape[0], page, 2, heads + 1, 2 * d), 7.0, dtype=dtype, device="cuda")
    k2, v2 = both[:, :, 0, :heads, :d].transpose(1, 2), both[:, :, 1, 1:, d:].transpose(1, 2)
    k2.copy_(k)
    v2.copy_(v)
    wide = torch.full((s, table.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    room = torch.full((s, heads * group + 2, d + 3), 5.0, dtype=dtype, device="cuda")
    got = uz.paged_attention(q2, k2, v2, wide[:, :table.shape[1]], n, out=room[:, 1:-1, :d], check=True)
    assert torch.equal(_bits(got), _bits(out))
    assert bool((room[:, 0] == 5).all() and (room[:, -1] == 5).all() and (room[..., d:] == 5).all())
    # one query for all sequences, by a stride of zero
    one = q[:1].expand(s, -1, -1)
    assert torch.equal(_bits(uz.paged_attention(one, k, v, table, n)), _bits(uz.paged_attention(one.contiguous(), k, v, table, n)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,heads,group,d,page", [([30, 300, 0], 3, 2, 128, 16), ([900, 1500], 2, 5, 80, 24), ([2000, 17], 2, 20, 64, 16), ([1200], 1, 16, 256, 8)])
def test_keys_and_values_laid_out_apart(uz, lengths, heads, group, d, page, dtype):
    """Keys by head and values by token: attention, storing and copying go by each pool's own strides."""
    q, k, v, table, n, out, _ = _attend(uz, lengths, heads, group, d, page, dtype)
    by_token = v.transpose(1, 2).contiguous().transpose(1, 2)
    assert by_token.stride() != k.stride() or heads == 1 or page == 1
    assert torch.equal(_bits(uz.paged_attention(q, k, by_token, table, n, check=True)), _bits(out))
    assert torch.equal(_bits(uz.paged_attention(q, k.transpose(1, 2).contiguous().transpose(1, 2), v, table, n, check=True)), _bits(out))
    t = len(lengths)
    new = _rand(_gen(1), (t, heads, d), dtype)
    slots = torch.arange(t, device="cuda") * page
    want = v.clone()
    want[:t, :, 0] = new
    kp = k.clone()
    uz.rotary_append(q, new, new, torch.zeros(t, dtype=torch.int64, device="cuda"), uz.rotary_frequencies(d), kp, by_token, slots, check=True)
    assert torch.equal(_bits(by_token), _bits(want)) and torch.equal(_bits(kp[:t, :, 0]), _bits(new))
    last = k.shape[0] - 1
    uz.cache_copy(kp, by_token, _i32([0, last]), check=True)
    assert torch.equal(_bits(by_token[last]), _bits(want[0])) and torch.equal(_bits(kp[last]), _bits(kp[0]))


def test_attention_parts_join_by_lse(uz):
    """Attention over two halves of a context, joined by their log-sum-exps, is attention over the whole."""
    q, k, v, table, n, out, lse = _attend(uz, [960, 480], 2, 4, 128, 16, torch.float16)
    half = n // 2
    a, la = uz.paged_attention(q, k, v, table, half, with_lse=True)
    rest = torch.stack([table[i].roll(-int(half[i]) // 16) for i in range(2)])
    b, lb = uz.paged_attention(q, k, v, rest, n - half, with_lse=True)
    both = torch.logaddexp(la.double(), lb.double())
    got = a.double() * (la - both).exp()[..., None] + b.double() * (lb - both).exp()[..., None]
    assert float((both - lse).abs().max()) <= 2.0 ** -17
    _, _, off, _ = ref.attention64(q, k, v, table, n)
    assert within(got, out.double(), 3 * off) <= 1.0


def test_attention_of_pools_past_32_bits(uz):
    """Pools of over 2^32 values (8.6 GB each): the first and last pages, and pages on both sides of each border."""
    g = _gen(9)
    heads, page, d = 8, 16, 128
    pages = (1 << 32) // (heads * page * d) + 40
    k = torch.zeros(pages, heads, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    border = (1 << 31) // (heads * page * d)
    use = [0, border - 1, border, border + 1, 2 * border - 1, 2 * border, pages - 1, pages - 2, 5]
    k[use] = _rand(g, (len(use), heads, page, d), torch.bfloat16)
    v[use] = _rand(g, (len(use), heads, page, d), torch.bfloat16)
    table = _i32(use, use[::-1])
    n = _i32(len(use) * page, len(use) * page - 9)
    q = _rand(g, (2, heads * 4, d), torch.bfloat16)
    out = uz.paged_attention(q, k, v, table, n, check=True)
    want, _, off, _ = ref.attention64(q, k, v, table, n)
    assert within(out, want, off) <= 1.0
    slots = torch.tensor([(pages - 1) * page + 3, 2 * border * page, 7], device="cuda")
    new = _rand(g, (3, heads, d), torch.bfloat16)
    freqs = uz.rotary_frequencies(d)
    uz.rotary_append(q[:1].expand(3, -1, -1), new, new, torch.zeros(3, dtype=torch.int64, device="cuda"), freqs, k, v, slots, check=True)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(_bits(k[s // page, :, s % page]), _bits(new[i])) and torch.equal(_bits(v[s // page, :, s % page]), _bits(new[i]))
    uz.cache_copy(k, v, _i32([pages - 1, 3], [5, pages - 3]), check=True)
    assert torch.equal(_bits(k[3]), _bits(k[pages - 1])) and torch.equal(_bits(v[pages - 3]), _bits(v[5]))


def test_attention_of_2_to_31_tokens(uz):
    """The longest sequence, of one page of 2^20 tokens again and again (a stride
    of zero): the tokens of the page weigh as they do in one, but for the one
    that is missing at the end."""
    g = _gen(10)
    page, n = 1 << 20, 2 ** 31 - 1
    k1, v1 = ref.pools(g, 1, 1, page, 8, torch.bfloat16)
    k, v = k1.expand(2048, -1, -1, -1), v1.expand(2048, -1, -1, -1)
    table = torch.arange(2048, dtype=torch.int32, device="cuda")[None]
    q = _rand(g, (1, 2, 8), torch.bfloat16)
    out, lse = uz.paged_attention(q, k, v, table, _i32(n), with_lse=True, check=True)
    want, want_lse, off, _ = ref.attention64(q, k1, v1, _i32([0]), _i32(page))
    assert within(out, want, off + 2.0 ** -20) <= 1.0  # the missing token weighs less than 2^-31 e^20 of all
    assert float((lse.double() - want_lse - math.log(2048)).abs().max()) <= 2.0 ** -16
    short = uz.paged_attention(q, k, v, table, _i32(n), window=page - 1, check=True)
    want, _, off, _ = ref.attention64(q, k1, v1, _i32([0]), _i32(page - 1))
    assert within(short, want, off) <= 1.0


@pytest.mark.parametrize("wide", [False, True])
def test_as_many_sequences_as_there_may_be(uz, wide):
    """65536 sequences of 0 to 40 tokens (in a table for 640, where blocks cut
    rows), reserved, attended to with equal scores, half of them freed."""
    from lossless_float_tensor_gb300 import UzipError

    seqs, page, heads, d = 65536, 8, 2, 16
    width = 80 if wide else 5
    g = _gen(11)
    n = torch.randint(0, 41, (seqs,), generator=g, device="cuda").int()
    need = (n + page - 1) // page
    state = ref.state(int(need.sum()) + 5, seqs, width)
    tokens = int(n.sum()) + 9
    slots, positions, copies = uz.cache_reserve(*state, n, tokens, page, check=True)
    assert torch.equal(state[2], n) and bool((copies == -1).all()) and bool((slots[-9:] == -1).all())
    row = torch.repeat_interleave(torch.arange(seqs, device="cuda"), n.long())
    first = n.long().cumsum(0) - n
    assert torch.equal(positions[:-9], torch.arange(tokens - 9, device="cuda") - first[row])
    # pages are taken in order, so page j of sequence i is the number of pages before
    base = need.long().cumsum(0) - need
    assert torch.equal(slots[:-9], (base[row] + positions[:-9] // page) * page + positions[:-9] % page)
    k = torch.zeros(state[0].numel(), heads, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.randint(-3, 4, k.shape, generator=g, device="cuda").to(torch.bfloat16)
    q = _rand(g, (seqs, heads, d), torch.bfloat16)
    out, lse = uz.paged_attention(q, k, v, state[1], state[2], with_lse=True, check=True)
    by_token = v.transpose(1, 2).flatten(0, 1).double()[slots[:-9]]
    total = torch.zeros(seqs, heads, d, dtype=torch.float64, device="cuda").index_add_(0, row, by_token)
    want = total / n.clamp(min=1)[:, None, None]
    # sums of whole numbers are exact; the quotient is the sum times a rounded reciprocal (2 roundings of 2^-24), then
    # rounded to the type: values of 8 bits are half a step apart from the next by 2^-8 of themselves at most
    off = want.abs() * (2.0 ** -8 + 2.0 ** -20)
    assert bool(((out.double() - want).abs() <= off).all())
    assert float((lse[n > 0].double() - n[n > 0].double().log()[:, None]).abs().max()) <= 2.0 ** -17
    gone = torch.randperm(seqs, generator=g, device="cuda")[: seqs // 2].int()
    uz.cache_free(*state, gone, page, check=True)
    held = torch.ones(seqs, dtype=torch.bool, device="cuda")
    held[gone.long()] = False
    assert int(state[0].sum()) == int(need[held].sum()) and not bool(state[2][~held].any())
    moves = uz.cache_compact(*state, page, check=True)
    used = int(need[held].sum())
    assert bool((state[0][:used] == 1).all()) and not bool(state[0][used:].any())
    uz.cache_copy(k, v, moves, check=True)
    again = uz.paged_attention(q, k, v, state[1], state[2], check=True)
    assert bool(((again[held].double() - want[held]).abs() <= off[held]).all()) and not bool(again[~held].any())
    with pytest.raises(UzipError):
        uz.paged_attention(q[:1].expand(65537, -1, -1), k, v, state[1][:1].expand(65537, -1), torch.zeros(65537, dtype=torch.int32, device="cuda"))


def test_attention_repeats_its_bits(uz):
    q, k, v, table, n, out, lse = _attend(uz, [5000, 1, 2600, 800], 2, 8, 128, 16, torch.bfloat16)
    for _ in range(5):
        again, l2 = uz.paged_attention(q, k, v, table, n, with_lse=True)
        assert torch.equal(_bits(again), _bits(out)) and torch.equal(l2, lse)


def test_attention_workspace(uz):
    from lossless_float_tensor_gb300 import UzipError, cache

    q, k, v, table, n, out, _ = _attend(uz, [3000, 700], 2, 4, 128, 16, torch.bfloat16)
    a = cache.PagedAttentionArgs(dtype=0, seqs=2, q_heads=8, kv_heads=2, d=128, pages=k.shape[0], page=16, width=table.shape[1])
    need = cache.uzip_paged_attention_workspace_size(a)
    guard = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    got = uz.paged_attention(q, k, v, table, n, workspace=guard[256:256 + need])
    assert torch.equal(_bits(got), _bits(out))
    assert bool((guard[:256] == 77).all()) and bool((guard[256 + need:] == 77).all())
    with pytest.raises(UzipError):
        uz.paged_attention(q, k, v, table, n, workspace=guard[:need - 1])
    with pytest.raises(UzipError):
        uz.paged_attention(q, k, v, table, n, workspace=guard[1:])


def test_attention_refusals(uz):
    from lossless_float_tensor_gb300 import UzipError

    q, k, v, table, n, _, _ = _attend(uz, [30, 20], 2, 4, 64, 16, torch.bfloat16)
    bad = [
        (q.float(), k, v, table, n, {}), (q, k.half(), v, table, n, {}), (q[0], k, v, table, n, {}), (q, k[..., :32], v[..., :32], table, n, {}),
        (q, k, v[:-1], table, n, {}), (q, k, v, table.long(), n, {}), (q, k, v, table[:1], n, {}), (q, k, v, table, n.long(), {}),
        (q, k, v, table, n[:1], {}), (q[:, :7], k, v, table, n, {}), (q.cpu(), k, v, table, n, {}), (q, k.cpu(), v, table, n, {}),
        (q, k, v, table.cpu(), n, {}), (q, k, v, table, n.cpu(), {}), (q, k[..., ::2], v[..., ::2], table, n, {}), (q, k, v, table, n, dict(window=-1)),
        (q, k, v, table, n, dict(softcap=-2.0)), (q, k, v, table, n, dict(out=q)), (q, k, v, table, n, dict(out=q[:1])), (q, k, v, table, n, dict(out=q.float())),
        (q, k, v, table.T.contiguous().T, n, {}), (q, k, v, table, n, dict(out=q[:1].expand(2, -1, -1))),
    ]
    for i, (*args, kw) in enumerate(bad):
        with pytest.raises(UzipError):
            uz.paged_attention(*args, **kw)
            pytest.fail(f"case {i} was taken")
    with pytest.raises(UzipError):
        uz.paged_attention(q.clone().requires_grad_(), k, v, table, n)
    with torch.no_grad():
        uz.paged_attention(q.clone().requires_grad_(), k, v, table, n)
    shifted = torch.empty(k.numel() + 1, dtype=k.dtype, device="cuda")[1:].view(k.shape)
    with pytest.raises(UzipError):
        uz.paged_attention(q, shifted, v, table, n)
    none = uz.paged_attention(q[:0], k, v, table[:0], n[:0], check=True)
    assert none.shape == (0, 8, 64)
    no_pages = uz.paged_attention(q, k[:0], v[:0], table[:, :0], torch.zeros_like(n), check=True)
    assert not bool(no_pages.any())


# ---- rotary positions -----------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,hq,hk,d,rot", [
    (1, 1, 1, 64, 64), (3, 8, 2, 128, 128), (17, 5, 3, 80, 80), (100, 4, 4, 96, 48), (9, 3, 1, 64, 36), (5, 2, 2, 50, 42), (7, 3, 2, 7, 6), (2, 1, 1, 1024, 1024),
    (33, 40, 8, 128, 64), (6, 2, 1, 256, 2), (4, 3, 2, 65, 64), (3, 2, 2, 16, 0), (2000, 2, 1, 24, 16), (5, 70, 70, 8, 8), (11, 3, 1, 300, 298),
])
def test_rotary(uz, t, hq, hk, d, rot, dtype, interleaved):
    g = _gen(t + d + rot)
    q, k = _rand(g, (t, hq, d), dtype), _rand(g, (t, hk, d), dtype)
    positions = torch.randint(-5000, 200000, (t,), generator=g, device="cuda")
    freqs = uz.rotary_frequencies(rot, base=20000.0)
    kw = dict(interleaved=interleaved, scale=1.25)
    a, b = uz.rotary(q, k, positions, freqs, check=True, **kw)
    for got, x in ((a, q), (b, k)):
        want, off = ref.rotary64(x, positions, freqs, **kw)
        assert within(got, want, off) <= 1.0
        assert torch.equal(_bits(got[..., rot:]), _bits(x[..., rot:]))
    only, none = uz.rotary(q, None, positions, freqs, **kw)
    assert none is None and torch.equal(_bits(only), _bits(a))
    none, only = uz.rotary(None, k, positions, freqs, **kw)
    assert none is None and torch.equal(_bits(only), _bits(b))
    # the gradient: the transposed rotation
    a, b = uz.rotary_backward(q, k, positions, freqs, check=True, **kw)
    for got, x in ((a, q), (b, k)):
        want, off = ref.rotary64(x, positions, freqs, sign=-1.0, **kw)
        assert within(got, want, off) <= 1.0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient(uz, interleaved):
    """Against autograd of the definition in 64 bits, and against differences:
    the rotation is linear, so <dy, R(x + e) - R(x)> / |e| is <R'dy, e> / |e| at
    any step."""
    g = _gen(3)
    t, h, d = 19, 3, 96
    q, k = _rand(g, (t, h, d), torch.float16), _rand(g, (t, 1, d), torch.float16)
    dq, dk = _rand(g, (t, h, d), torch.float16), _rand(g, (t, 1, d), torch.float16)
    positions = torch.arange(t, device="cuda") * 997
    freqs = uz.rotary_frequencies(64)
    kw = dict(interleaved=interleaved, scale=0.75)
    got = uz.rotary_backward(dq, dk, positions, freqs, **kw)
    for x, dy, gx in ((q, dq, got[0]), (k, dk, got[1])):
        leaf = x.double().requires_grad_()
        rot, half = 64, 32
        a = positions.double()[:, None] * freqs
        by = torch.polar(torch.full_like(a, 0.75), a)[:, None]
        part = leaf[..., :rot]
        pair = part.unflatten(-1, (-1, 2)) if interleaved else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * by)
        flat = turned.flatten(-2) if interleaved else turned.transpose(-1, -2).flatten(-2)
        y = torch.cat([flat, leaf[..., rot:]], -1)
        (y * dy.double()).sum().backward()
        _, off = ref.rotary64(dy, positions, freqs, sign=-1.0, **kw)
        assert within(gx, leaf.grad, off) <= 1.0
        # differences of the kernel's own forward pass
        step = _rand(g, x.shape, torch.float16)
        moved = (x.double() + step.double()).half()
        e = moved.double() - x.double()
        side = dict(positions=positions, freqs=freqs, **kw)
        up, at = (uz.rotary(z, None, **side)[0].double() for z in (moved, x))
        _, off_up = ref.rotary64(moved, positions, freqs, **kw)
        _, off_at = ref.rotary64(x, positions, freqs, **kw)
        slack = (dy.double().abs() * (off_up + off_at)).sum() + (e.abs() * off).sum()
        assert abs(float((dy.double() * (up - at)).sum() - (gx.double() * e).sum())) <= float(slack)


def test_rotary_far_positions(uz):
    """Positions to 2^26, where 64-bit angles are good to 10^-8; beyond, turns by
    whole multiples: a frequency of k / 2^20 turns has the same angle 2^20
    positions on, however far."""
    g = _gen(4)
    x = _rand(g, (64, 2, 128), torch.float16)
    freqs = uz.rotary_frequencies(128)
    positions = torch.randint(2 ** 25, 2 ** 26, (64,), generator=g, device="cuda")
    got, _ = uz.rotary(x, None, positions, freqs)
    want, off = ref.rotary64(x, positions, freqs)
    assert within(got, want, off) <= 1.0
    whole = torch.arange(1, 65, dtype=torch.float64, device="cuda") * (2 * math.pi / 2 ** 20)
    near = torch.arange(64, device="cuda")
    a, _ = uz.rotary(x, None, near, whole)
    for far in (2 ** 20, 2 ** 30, -2 ** 30, 2 ** 40):
        b, _ = uz.rotary(x, None, near + far, whole)
        # the frequencies are good to 2^-53 of themselves, so far positions are off by that many turns
        want, off = ref.rotary64(x, near, whole)
        mag = x.double().abs().amax() * 2
        assert within(b, want, off + mag * 2 * math.pi * abs(far) * 64 * 2.0 ** -72) <= 1.0


@pytest.mark.parametrize("d,rot,gap", [(128, 128, 0), (128, 128, 1), (96, 48, 2), (64, 64, 8), (50, 20, 3)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_views_and_in_place(uz, d, rot, gap, interleaved):
    g = _gen(d + gap)
    t, hq, hk = 21, 6, 2
    fused = _rand(g, (t, gap + (hq + 2 * hk) * d + gap), torch.bfloat16)
    q = fused[:, gap:gap + hq * d].unflatten(1, (-1, d))
    k = fused[:, gap + hq * d:gap + (hq + hk) * d].unflatten(1, (-1, d))
    positions = torch.randint(0, 10000, (t,), generator=g, device="cuda")
    freqs = uz.rotary_frequencies(rot)
    want = uz.rotary(q.contiguous(), k.contiguous(), positions, freqs, interleaved=interleaved)
    got = uz.rotary(q, k, positions, freqs, interleaved=interleaved)
    assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(got, want))
    room = [torch.full((t, h + 1, d + 5), 3.0, dtype=q.dtype, device="cuda") for h in (hq, hk)]
    uz.rotary(q, k, positions, freqs, interleaved=interleaved, out=(room[0][:, :-1, 2:2 + d], room[1][:, 1:, :d]))
    assert torch.equal(_bits(room[0][:, :-1, 2:2 + d]), _bits(want[0])) and torch.equal(_bits(room[1][:, 1:, :d]), _bits(want[1]))
    assert bool((room[0][:, -1] == 3).all() and (room[0][..., :2] == 3).all() and (room[0][..., 2 + d:] == 3).all() and (room[1][:, 0] == 3).all())
    before = fused.clone()
    uz.rotary(q, k, positions, freqs, interleaved=interleaved, out=(q, k))
    assert torch.equal(_bits(q), _bits(want[0])) and torch.equal(_bits(k), _bits(want[1]))
    rest = gap + (hq + hk) * d
    assert torch.equal(_bits(fused[:, :gap]), _bits(before[:, :gap])) and torch.equal(_bits(fused[:, rest:]), _bits(before[:, rest:]))
    # one head's input for all heads
    one = before[:, gap:gap + d].unflatten(1, (1, d)).expand(-1, hq, -1)
    a, _ = uz.rotary(one, None, positions, freqs, interleaved=interleaved)
    b, _ = uz.rotary(one.contiguous(), None, positions, freqs, interleaved=interleaved)
    assert torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("order", ["heads", "tokens"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,hq,hk,d,rot,page", [(1, 4, 1, 128, 128, 16), (48, 32, 8, 128, 128, 16), (333, 3, 3, 80, 40, 24), (20, 5, 1, 72, 6, 1), (7, 0, 2, 256, 256, 64)])
def test_rotary_append(uz, t, hq, hk, d, rot, page, dtype, order):
    g = _gen(t + d)
    pages = -(-t // page) + 6
    kp, vp = ref.pools(g, pages, hk, page, d, dtype, order)
    k0, v0 = kp.clone(), vp.clone()
    fused = _rand(g, (t, (hq + 2 * hk) * d), dtype)
    q, k, v = (x.unflatten(1, (-1, d)) for x in fused.split((hq * d, hk * d, hk * d), 1))
    positions = torch.randint(0, 100000, (t,), generator=g, device="cuda")
    freqs = uz.rotary_frequencies(rot)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:t]
    slots[::3] = -1
    out = uz.rotary_append(q, k, v, positions, freqs, kp, vp, slots, interleaved=True, check=True)
    wq, wk = uz.rotary(q, k, positions, freqs, interleaved=True)
    assert torch.equal(_bits(out), _bits(wq))
    keep = slots >= 0
    at = slots[keep] // page, slice(None), slots[keep] % page
    k0[at], v0[at] = wk[keep], v[keep]
    assert torch.equal(_bits(kp), _bits(k0)) and torch.equal(_bits(vp), _bits(v0))


def test_rotary_append_bad_slots(uz):
    from lossless_float_tensor_gb300 import UzipError

    g = _gen(12)
    kp, vp = ref.pools(g, 5, 2, 16, 64, torch.bfloat16)
    k0, v0 = kp.clone(), vp.clone()
    x = _rand(g, (6, 2, 64), torch.bfloat16)
    positions, freqs = torch.zeros(6, dtype=torch.int64, device="cuda"), uz.rotary_frequencies(64)
    slots = torch.tensor([-2, 80, 3, 2 ** 40, -1, -2 ** 62], device="cuda")
    status = torch.zeros((), dtype=torch.int32, device="cuda")
    out = uz.rotary_append(x, x, x, positions, freqs, kp, vp, slots, status=status)
    assert int(status) == 1 and torch.equal(_bits(out), _bits(x))
    k0[0, :, 3], v0[0, :, 3] = x[2], x[2]
    assert torch.equal(_bits(kp), _bits(k0)) and torch.equal(_bits(vp), _bits(v0))
    with pytest.raises(UzipError):
        uz.rotary_append(x, x, x, positions, freqs, kp, vp, slots, check=True)


def test_rotary_refusals(uz):
    from lossless_float_tensor_gb300 import UzipError

    g = _gen(13)
    x, positions, freqs = _rand(g, (4, 2, 64), torch.bfloat16), torch.zeros(4, dtype=torch.int64, device="cuda"), uz.rotary_frequencies(64)
    kp, vp = ref.pools(g, 5, 2, 16, 64, torch.bfloat16)
    slots = torch.arange(4, device="cuda")
    bad = [(None, None, positions, freqs, {}), (x.float(), None, positions, freqs, {}), (x, x.half(), positions, freqs, {}), (x, x[:3], positions, freqs, {}),
           (x, x[..., :32], positions, freqs, {}), (x, x, positions.int(), freqs, {}), (x, x, positions[:3], freqs, {}), (x, x, positions, freqs.float(), {}),
           (x, x, positions.cpu(), freqs, {}), (x, x, positions, freqs.cpu(), {}), (x, x, positions, uz.rotary_frequencies(66), {}),
           (x[..., ::2], None, positions, freqs[:16], {}), (x, None, positions, freqs, dict(out=(x[:1].expand(4, -1, -1), None))),
           (x[0], None, positions, freqs, {}), (x, x, positions, freqs[None], {})]
    for i, (*args, kw) in enumerate(bad):
        with pytest.raises(UzipError):
            uz.rotary(*args, **kw)
            pytest.fail(f"case {i} was taken")
    with pytest.raises(UzipError):
        uz.rotary(x.clone().requires_grad_(), None, positions, freqs)
    good = [x, x, x, positions, freqs, kp, vp, slots]
    for n, wrong in ((1, None), (5, kp[:, :1]), (5, kp[..., :32]), (6, vp[:4]), (5, kp.half()), (7, slots.int()), (7, slots[:3]), (7, slots.cpu()), (2, x[:, :1]),
                     (5, kp[:1].expand(5, -1, -1, -1))):
        args = list(good)
        args[n] = wrong
        with pytest.raises(UzipError):
            uz.rotary_append(*args)
            pytest.fail(f"{n} was taken")
    a, b = uz.rotary(x[:0], x[:0], positions[:0], freqs, check=True)
    assert a.shape == (0, 2, 64) and b.shape == (0, 2, 64)


# ---- pages ------------------------------------------------------------------------

def _same(lists, state):
    ref.same_state(lists, *state)


@pytest.mark.parametrize("seed", range(6))
def test_pages_at_random(uz, seed):
    """Random operations on a small cache, some of which do not fit or cannot be, against lists after each."""
    rng = random.Random(seed)
    pages, page, seqs, width = rng.choice([(24, 4, 6, 9), (60, 16, 12, 8), (40, 1, 5, 30), (2000, 7, 40, 60)])
    lists = ref.ListCache(pages, page, seqs, width)
    state = ref.state(pages, seqs, width)
    status = torch.zeros((), dtype=torch.int32, device="cuda")
    done = {"invalid": 0, "capacity": 0, "": 0}
    for _ in range(60):
        op = rng.choice(["reserve", "reserve", "reserve", "fork", "free", "compact"])
        why = ""
        if op == "reserve":
            counts = [rng.choice([0, 0, 1, 1, 2, page, rng.randint(0, 3 * page)]) for _ in range(seqs)]
            tokens = max(0, sum(counts) + rng.choice([0, 0, 3, -1]))
            try:
                want = lists.reserve(counts, tokens)
            except ref.Refused as e:
                why = str(e)
                want = [-1] * tokens, [0] * tokens, [[-1, -1]] * seqs
            got = uz.cache_reserve(*state, _i32(*counts), tokens, page, status=status)
            assert [x.tolist() for x in got] == [list(x) for x in want]
        elif op == "fork":
            n = rng.randint(1, 3)
            empty = [i for i in range(seqs) if not lists.lengths[i]] or [0]
            parents, children = [rng.randrange(seqs) for _ in range(n)], [rng.choice(empty) for _ in range(n)]
            if rng.random() < 0.3:
                parents.append(-1)
                children.append(-1)
            if rng.random() < 0.1:
                children[0] = rng.choice([-1, seqs, -5, 2 ** 31 - 1])
            try:
                lists.fork(parents, children)
            except ref.Refused as e:
                why = str(e)
            uz.cache_fork(*state, _i32(*parents), _i32(*children), page, status=status)
        elif op == "free":
            listed = [rng.randrange(-1, seqs) for _ in range(rng.randint(1, 3))]
            if rng.random() < 0.1:
                listed[0] = rng.choice([seqs, -2])
            try:
                lists.free(listed)
            except ref.Refused as e:
                why = str(e)
            uz.cache_free(*state, _i32(*listed), page, status=status)
        else:
            assert uz.cache_compact(*state, page, status=status).tolist() == lists.compact()
        assert int(status) == {"": 0, "invalid": 1, "capacity": 3}[why], op
        done[why] += 1
        _same(lists, state)
    assert done[""] >= 20 and done["invalid"] >= 1


@pytest.mark.parametrize("pages,page,seqs,width", [(40000, 16, 300, 130), (70001, 8, 9000, 40), (9000, 64, 3, 3000), (100000, 1, 20, 5000)])
def test_pages_of_many(uz, pages, page, seqs, width):
    """Sizes at which a cluster of blocks does the work."""
    rng = random.Random(pages)
    lists = ref.ListCache(pages, page, seqs, width)
    state = ref.state(pages, seqs, width)
    budget = pages // 2
    for most in (width * page // 2, 2 * page, 1):
        counts, left = [0] * seqs, budget // 3
        for i in rng.sample(range(seqs), max(1, seqs * 2 // 3)):
            c = rng.randint(0, most)
            if c // page + 2 <= left:
                counts[i] = c
                left -= c // page + 2
        tokens = sum(counts) + 5
        want = lists.reserve(counts, tokens)
        got = uz.cache_reserve(*state, _i32(*counts), tokens, page, check=True)
        assert [x.tolist() for x in got] == [list(x) for x in want]
        _same(lists, state)
    empty = [i for i in range(seqs) if not lists.lengths[i]][:200]
    full = [i for i in range(seqs) if lists.lengths[i]]
    parents = [rng.choice(full) for _ in empty]
    if empty:
        lists.fork(parents, empty)
        uz.cache_fork(*state, _i32(*parents), _i32(*empty), page, check=True)
        _same(lists, state)
    gone = rng.sample(full, max(1, len(full) // 2))
    lists.free(gone)
    uz.cache_free(*state, _i32(*gone), page, check=True)
    _same(lists, state)
    assert uz.cache_compact(*state, page, check=True).tolist() == lists.compact()
    _same(lists, state)
    assert uz.cache_compact(*state, page, check=True).tolist() == [[-1, -1]] * (pages // 2)
    _same(lists, state)


def test_reserve_at_the_limits(uz):
    """Exactly as many pages and columns as there are, and one more."""
    page, pages, width = 4, 10, 5
    for counts, code in (([20, 20], 0), ([21, 0], 3), ([20, 17], 0), ([2 ** 31 - 1, 1], 1), ([-1, 3], 1), ([0, 0], 0)):
        state = ref.state(pages, 2, width)
        status = torch.zeros((), dtype=torch.int32, device="cuda")
        slots, positions, copies = uz.cache_reserve(*state, _i32(*counts), 40, page, status=status)
        assert int(status) == code, counts
        if code:
            assert bool((slots == -1).all()) and not bool(positions.any()) and bool((copies == -1).all())
            assert not any(bool(x.any()) for x in state)
        else:
            assert state[2].tolist() == counts and int((slots >= 0).sum()) == sum(counts)
    state = ref.state(3, 2, width)
    uz.cache_reserve(*state, _i32(4, 4), 8, page, check=True)
    before = [x.clone() for x in state]
    status = torch.zeros((), dtype=torch.int32, device="cuda")
    uz.cache_reserve(*state, _i32(4, 1), 8, page, status=status)
    assert int(status) == 3 and all(torch.equal(a, b) for a, b in zip(state, before))
    # a length near 2^31 of pages of 2^20 tokens
    state = ref.state(3000, 1, 2500)
    state[0][:2048], state[1][0, :2048] = 1, torch.arange(2048, device="cuda")
    state[2][0] = 2 ** 31 - 3
    slots, positions, _ = uz.cache_reserve(*state, _i32(2), 2, 2 ** 20, check=True)
    assert positions.tolist() == [2 ** 31 - 3, 2 ** 31 - 2] and slots.tolist() == [2047 * 2 ** 20 + 2 ** 20 - 3, 2047 * 2 ** 20 + 2 ** 20 - 2]
    uz.cache_reserve(*state, _i32(2), 2, 2 ** 20, status=status)
    assert int(status) == 3 and int(state[2]) == 2 ** 31 - 1


def test_state_that_cannot_be(uz):
    """Lengths, pages and reference counts that contradict one another change nothing."""
    page = 4
    good = ref.state(12, 3, 4)
    uz.cache_reserve(*good, _i32(9, 5, 0), 14, page, check=True)

    def broken(refs=None, table=None, length=None):
        s = [x.clone() for x in good]
        if refs:
            s[0][refs[0]] = refs[1]
        if table:
            s[1][table[0], table[1]] = table[2]
        if length:
            s[2][length[0]] = length[1]
        return s

    status = torch.zeros((), dtype=torch.int32, device="cuda")
    page_of = good[1].tolist()
    for s in (broken(length=(0, -1)), broken(length=(0, 17)), broken(table=(0, 2, -1)), broken(table=(0, 2, 12)), broken(table=(0, 2, 2 ** 31 - 1)),
              broken(refs=(page_of[0][2], 0))):
        before = [x.clone() for x in s]
        for call in (lambda: uz.cache_reserve(*s, _i32(1, 0, 0), 4, page, status=status), lambda: uz.cache_fork(*s, _i32(0), _i32(2), page, status=status),
                     lambda: uz.cache_free(*s, _i32(0), page, status=status), lambda: uz.cache_compact(*s, page, status=status)):
            call()
            assert int(status) == 1 and all(torch.equal(a, b) for a, b in zip(s, before))


def test_smallest_caches(uz):
    """No sequences, no columns, no pages, one page, no tokens."""
    status = torch.zeros((), dtype=torch.int32, device="cuda")
    none = _i32()
    for pages, seqs, width, counts, tokens, code in ((5, 0, 4, [], 3, 0), (5, 0, 4, [], 0, 0), (5, 2, 0, [0, 0], 2, 0), (5, 2, 0, [0, 1], 2, 3),
                                                     (0, 2, 3, [0, 0], 0, 0), (0, 2, 3, [1, 0], 1, 3), (1, 1, 1, [1], 1, 0), (1, 1, 1, [5], 5, 3), (1, 3, 2, [0, 4, 0], 4, 0)):
        state = ref.state(pages, seqs, width)
        slots, positions, copies = uz.cache_reserve(*state, _i32(*counts), tokens, 4, status=status)
        assert int(status) == code, (pages, seqs, width, counts)
        real = 0 if code else sum(counts)
        assert slots.tolist() == list(range(real)) + [-1] * (tokens - real) and copies.shape == (seqs, 2)
        assert positions.tolist() == list(range(real)) + [0] * (tokens - real)
        moves = uz.cache_compact(*state, 4, check=True)
        assert moves.shape == (pages // 2, 2) and bool((moves == -1).all())
        uz.cache_fork(*state, none, none, 4, check=True)
        uz.cache_free(*state, none, 4, check=True)
        uz.cache_fork(*state, _i32(-1, -1), _i32(-1, -1), 4, check=True)
        uz.cache_free(*state, _i32(-1), 4, check=True)
        uz.cache_free(*state, _i32(0), 4, status=status)
        assert int(status) == (0 if seqs else 1)
        assert not bool(state[0].any()) or seqs > 1
    k = torch.zeros(0, 1, 4, 8, dtype=torch.bfloat16, device="cuda")
    uz.cache_copy(k, k.clone(), none.view(0, 2), check=True)
    uz.cache_copy(k, k.clone(), _i32([-1, -1]), check=True)


def test_pages_in_a_graph(uz):
    """Fork, free and compact captured once and replayed on states that change in between."""
    page, pages, seqs, width = 4, 60, 8, 10
    lists = [ref.ListCache(pages, page, seqs, width) for _ in range(2)]
    state, want = ref.state(pages, seqs, width), None
    parents, children, gone = _i32(0, 1), _i32(6, 7), _i32(1, 2, -1)

    def work():
        uz.cache_fork(*state, parents, children, page)
        uz.cache_free(*state, gone, page)
        return uz.cache_compact(*state, page)

    eager = work()
    assert bool((eager == -1).all())
    for x in state:
        x.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moves = work()
    for n, counts in enumerate(([9, 5, 7, 1, 0, 4, 0, 0], [1, 30, 2, 0, 0, 0, 0, 0])):
        for x in state:
            x.zero_()
        lists[n].reserve(counts, sum(counts))
        uz.cache_reserve(*state, _i32(*counts), sum(counts), page, check=True)
        graph.replay()
        lists[n].fork([0, 1], [6, 7])
        lists[n].free([1, 2])
        want = lists[n].compact()
        assert moves.tolist() == want
        _same(lists[n], state)


def test_pages_refusals(uz):
    from lossless_float_tensor_gb300 import UzipError

    refs, table, n = ref.state(8, 3, 4)
    c = _i32(1, 1, 1)
    for args in ((refs.long(), table, n), (refs, table.long(), n), (refs, table, n.long()), (refs, table, n[:2]), (refs.cpu(), table, n), (refs, table[0], n),
                 (refs, table.T.contiguous().T, n), (refs[::2], table, n), (refs, table.cpu(), n)):
        for call in (lambda: uz.cache_reserve(*args, c, 3, 4), lambda: uz.cache_fork(*args, c[:1], c[:1], 4), lambda: uz.cache_free(*args, c[:1], 4),
                     lambda: uz.cache_compact(*args, 4)):
            with pytest.raises(UzipError):
                call()
                pytest.fail("taken")
    for call in (lambda: uz.cache_reserve(refs, table, n, c[:2], 3, 4), lambda: uz.cache_reserve(refs, table, n, c.long(), 3, 4),
                 lambda: uz.cache_fork(refs, table, n, c, c[:2], 4), lambda: uz.cache_free(refs, table, n, c[:, None], 4),
                 lambda: uz.cache_reserve(refs, table, n, c, 3, 0), lambda: uz.cache_compact(refs, table, n, 4, out=c)):
        with pytest.raises(UzipError):
            call()
            pytest.fail("taken")
    # a table that is a part of a wider one
    wide = torch.full((3, 9), 5, dtype=torch.int32, device="cuda")
    slots, _, _ = uz.cache_reserve(refs, wide[:, 2:6], n, _i32(5, 0, 4), 9, 4, check=True)
    assert wide[0].tolist() == [5, 5, 0, 1, 5, 5, 5, 5, 5] and wide[2, 2] == 2 and slots.tolist() == list(range(5)) + [8, 9, 10, 11]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layers,heads,page,d", [(1, 1, 1, 8), (2, 3, 16, 64), (3, 2, 24, 80), (1, 8, 64, 128), (2, 1, 5, 256)])
@pytest.mark.parametrize("order,to_order", [("heads", "heads"), ("tokens", "tokens"), ("heads", "tokens"), ("gaps", "tokens")])
def test_copy_pages(uz, layers, heads, page, d, order, to_order, dtype):
    g = _gen(d + page)

    def cache(pages, order):
        if order == "gaps":
            return [_rand(g, (layers, pages, heads + 1, page + 2, 2 * d), dtype)[:, :, 1:, 1:-1, :d] for _ in range(2)]
        shape = (layers, pages, heads, page, d) if order == "heads" else (layers, pages, page, heads, d)
        both = [_rand(g, shape, dtype) for _ in range(2)]
        return both if order == "heads" else [x.transpose(2, 3) for x in both]

    k, v = cache(20, order)
    pairs = _i32([3, 9], [-1, 4], [0, 0], [19, 1], [2, -1], [3, 11], [-1, -1])
    kt, vt = cache(12, to_order)
    want = kt.clone(), vt.clone()
    for a, b in ((3, 9), (0, 0), (19, 1), (3, 11)):
        want[0][:, b], want[1][:, b] = k[:, a], v[:, a]
    uz.cache_copy(k, v, pairs, to=(kt, vt), check=True)
    assert torch.equal(_bits(kt), _bits(want[0])) and torch.equal(_bits(vt), _bits(want[1]))
    want = k.clone(), v.clone()
    pairs = _i32([3, 9], [-1, -1], [19, 1], [3, 11], [12, 0])
    for a, b in ((3, 9), (19, 1), (3, 11), (12, 0)):
        want[0][:, b], want[1][:, b] = want[0][:, a], want[1][:, a]
    uz.cache_copy(k, v, pairs, check=True)
    assert torch.equal(_bits(k), _bits(want[0])) and torch.equal(_bits(v), _bits(want[1]))
    uz.cache_copy(k[0], v[0], _i32([5, 6]), check=True)
    assert torch.equal(_bits(k[0, 6]), _bits(k[0, 5])) and torch.equal(_bits(k[1:]), _bits(want[0][1:]))


def test_copy_of_many_pages(uz):
    g = _gen(20)
    k, v = _rand(g, (2, 9000, 2, 16, 64), torch.bfloat16), _rand(g, (2, 9000, 2, 16, 64), torch.bfloat16)
    order = torch.randperm(9000, generator=g, device="cuda").int()
    pairs = torch.stack([order[:4000], order[4000:8000]], 1).contiguous()
    pairs[::7] = -1
    want = k.clone(), v.clone()
    keep = pairs[:, 0] >= 0
    a, b = pairs[keep, 0].long(), pairs[keep, 1].long()
    want[0][:, b], want[1][:, b] = want[0][:, a], want[1][:, a]
    uz.cache_copy(k, v, pairs, check=True)
    assert torch.equal(_bits(k), _bits(want[0])) and torch.equal(_bits(v), _bits(want[1]))


def test_copy_refuses_pairs_that_collide(uz):
    from lossless_float_tensor_gb300 import UzipError

    g = _gen(21)
    k, v = _rand(g, (8, 2, 16, 64), torch.float16), _rand(g, (8, 2, 16, 64), torch.float16)
    kt, vt = _rand(g, (4, 2, 16, 64), torch.float16), _rand(g, (4, 2, 16, 64), torch.float16)
    status = torch.zeros((), dtype=torch.int32, device="cuda")
    kept = [x.clone() for x in (k, v, kt, vt)]
    for pairs in ([[0, 1], [2, 1]], [[0, 1], [1, 2]], [[3, 3]], [[0, 8]], [[8, 0]], [[-2, 0]], [[0, -2]], [[2 ** 31 - 1, 1]]):
        uz.cache_copy(k, v, _i32(*pairs), status=status)
        assert int(status) == 1, pairs
    for pairs in ([[0, 1], [2, 1]], [[0, 4]], [[8, 0]], [[5, -9]]):
        uz.cache_copy(k, v, _i32(*pairs), to=(kt, vt), status=status)
        assert int(status) == 1, pairs
    assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip((k, v, kt, vt), kept))
    uz.cache_copy(k, v, _i32([3, 3], [2, 0], [3, 1]), to=(kt, vt), check=True)
    for bad in (dict(to=(kt.bfloat16(), vt)), dict(to=(kt[..., :32], vt[..., :32])), dict(to=(k, vt)), dict(to=(kt[:3], vt))):
        with pytest.raises(UzipError):
            uz.cache_copy(k, v, _i32([0, 1]), **bad)
    for args in ((k, v, _i32(0, 1)), (k, v, _i32([0, 1]).long()), (k, v[:4], _i32([0, 1])), (k[0], v[0], _i32([0, 1])), (k, v, _i32([0, 1]).cpu())):
        with pytest.raises(UzipError):
            uz.cache_copy(*args)
    uz.cache_copy(k, v, torch.empty(0, 2, dtype=torch.int32, device="cuda"), check=True)


def test_c_entry_points_refuse_one_wrong_thing(uz):
    """Arguments that are taken as they are, and refused with any one of the
    changes that the tests without a GPU list."""
    from lossless_float_tensor_gb300 import cache
    from tests import test_cache_host as host

    room = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    # each pointer its own 16 KB, zeros: lengths of 0, pages and slots of 0, frequencies of 0; status behind
    status = torch.zeros((), dtype=torch.int32, device="cuda")

    def real(a):
        for n, (name, kind) in enumerate(a._fields_):
            if kind is cache._vp and getattr(a, name):
                setattr(a, name, room.data_ptr() + n * 16384)
        if isinstance(a, cache.CacheCopyArgs):  # within one pool
            a.k_to, a.v_to = a.k, a.v
        return a

    def check(entry, build, changes):
        size = getattr(cache, entry.__name__ + "_workspace_size")
        a = real(build(cache))
        assert size(a) <= 1 << 18
        call = lambda a: entry(a, room.data_ptr() + (3 << 18), 1 << 18, status.data_ptr(), stream)  # noqa: E731
        assert call(a) == 0, entry.__name__
        torch.cuda.synchronize()
        for change in changes:
            change, want = change if isinstance(change, tuple) else (change, host.BAD_ARG)
            a = real(build(cache))
            for name, v in change.items():
                if isinstance(v, int) and v >= host.FAKE:  # the same place off its boundary, or another pointer's
                    v = (getattr(a, name) or room.data_ptr()) + v % host.FAKE if v % host.FAKE else None
                if v is None and change[name] is not None:
                    break
                setattr(a, name, v)
            else:
                assert call(a) == want, (entry.__name__, change)
                torch.cuda.synchronize()

    check(cache.uzip_rotary, host._rotary, [c for c in host.ROTARY if "slots" not in c[0]])
    check(cache.uzip_rotary_append, host._append, host.APPEND)
    check(cache.uzip_paged_attention, host._attention, host.ATTENTION)
    check(cache.uzip_cache_reserve, host._state, host.RESERVE)
    check(cache.uzip_cache_fork, host._state, host.FORK + [dict(from_=None)])
    check(cache.uzip_cache_free, host._state, host.FORK)
    check(cache.uzip_cache_compact, host._state, host.STATE + [dict(pairs=None)])
    check(cache.uzip_cache_copy, host._copy, [c for c in host.COPY if "k_to" not in c[0]])
    # pointers that have to differ, or to agree
    for build, entry, same in ((host._append, cache.uzip_rotary_append, ("v_pages", "k_pages")), (host._attention, cache.uzip_paged_attention, ("out", "q")),
                               (host._copy, cache.uzip_cache_copy, ("v_to", "k_to"))):
        a = real(build(cache))
        setattr(a, same[0], getattr(a, same[1]))
        assert entry(a, None, 0, status.data_ptr(), stream) == host.BAD_ARG
    a = real(host._rotary(cache))
    a.slots = room.data_ptr()
    assert cache.uzip_rotary(a, None, 0, status.data_ptr(), stream) == host.BAD_ARG
    # memory that is not the device's, or ends too early
    for name in ("q", "k_pages", "table", "lengths", "out"):
        a = real(host._attention(cache))
        setattr(a, name, host.FAKE)
        assert cache.uzip_paged_attention(a, None, 0, None, stream) == host.BAD_ARG, name


# ---- together ---------------------------------------------------------------------

class _Server:
    """A layer's cache as a server keeps it, beside the keys and values of each
    sequence in plain tensors."""

    def __init__(self, uz, pages=300, page=16, seqs=8, width=80, hq=8, hk=2, d=64, layers=2, dtype=torch.bfloat16):
        self.uz, self.page, self.hq, self.hk, self.d, self.layers, self.dtype = uz, page, hq, hk, d, layers, dtype
        self.k = torch.full((layers, pages, hk, page, d), math.nan, dtype=dtype, device="cuda")
        self.v = torch.full_like(self.k, math.inf)
        self.state = ref.state(pages, seqs, width)
        self.freqs = uz.rotary_frequencies(d, scaling="linear", factor=2.0)
        self.plain = [[(torch.empty(0, hk, d, dtype=dtype, device="cuda"),) * 2 for _ in range(layers)] for _ in range(seqs)]
        self.g = _gen(31)

    def step(self, counts):
        uz = self.uz
        tokens = sum(counts) + 3
        slots, positions, copies = uz.cache_reserve(*self.state, _i32(*counts), tokens, self.page, check=True)
        uz.cache_copy(self.k, self.v, copies, check=True)
        for layer in range(self.layers):
            fused = _rand(self.g, (tokens, (self.hq + 2 * self.hk) * self.d), self.dtype)
            q, k, v = (x.unflatten(1, (-1, self.d)) for x in fused.split((self.hq * self.d, self.hk * self.d, self.hk * self.d), 1))
            q2 = uz.rotary_append(q, k, v, positions, self.freqs, self.k[layer], self.v[layer], slots, check=True)
            turned = uz.rotary(q, k, positions, self.freqs)
            assert torch.equal(_bits(q2), _bits(turned[0]))
            at = 0
            for i, c in enumerate(counts):
                pk, pv = self.plain[i][layer]
                self.plain[i][layer] = torch.cat([pk, turned[1][at:at + c]]), torch.cat([pv, v[at:at + c]])
                at += c

    def attend(self, window=0):
        out = []
        for layer in range(self.layers):
            q = _rand(_gen(77 + layer), (self.state[1].shape[0], self.hq, self.d), self.dtype)
            got, lse = self.uz.paged_attention(q, self.k[layer], self.v[layer], self.state[1], self.state[2], window=window, with_lse=True, check=True)
            for i, rows in enumerate(self.plain):
                pk, pv = rows[layer]
                assert pk.shape[0] == int(self.state[2][i])
                one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
                n = _i32(pk.shape[0])
                want, _, off, _ = ref.attention64(q[i:i + 1], pk.transpose(0, 1)[None] if n else pk.new_zeros(1, self.hk, 1, self.d),
                                                  pv.transpose(0, 1)[None] if n else pv.new_zeros(1, self.hk, 1, self.d), one, n, window=window)
                assert within(got[i:i + 1], want, off) <= 1.0
            out.append(got)
        return out


def test_a_server_at_work(uz):
    """Prompts, single tokens, forks with copies on write, freed sequences,
    compaction, and the cache sent to another one through the codec: attention
    agrees with plain keys and values throughout, and to the bit after moves."""
    s = _Server(uz)
    s.step([100, 33, 0, 640, 1, 0, 0, 0])
    s.attend()
    s.step([1, 1, 0, 1, 1, 0, 0, 0])
    uz.cache_fork(*s.state, _i32(3, 0, 3, -1), _i32(5, 6, 7, -1), s.page, check=True)
    s.plain[5], s.plain[6], s.plain[7] = list(s.plain[3]), list(s.plain[0]), list(s.plain[3])
    s.attend()
    for _ in range(3):
        s.step([1, 1, 0, 1, 0, 1, 1, 1])
    s.attend(window=50)
    uz.cache_free(*s.state, _i32(3, 1, -1), s.page, check=True)
    for i in (1, 3):
        s.plain[i] = [(x[:0], y[:0]) for x, y in s.plain[i]]
    before = s.attend()
    s.step([0, 7, 0, 0, 0, 0, 0, 0])
    before = s.attend()
    moves = uz.cache_compact(*s.state, s.page, check=True)
    uz.cache_copy(s.k, s.v, moves, check=True)
    used = int((s.state[0] > 0).sum())
    assert int((moves[:, 0] >= 0).sum()) > 0 and not bool(s.state[0][used:].any())
    assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(s.attend(), before))
    # the used pages, in one buffer, compressed, sent, and put into another server's cache
    n = used
    box = torch.empty(2, s.layers, n, s.hk, s.page, s.d, dtype=s.dtype, device="cuda")
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    uz.cache_copy(s.k, s.v, torch.stack([ids, ids], 1).contiguous(), to=(box[0], box[1]), check=True)
    buf, size = uz.compress(box)
    arrived = uz.decompress(uz.compressed_bytes(buf, size).clone(), s.dtype, box.numel()).view(box.shape)
    other_k, other_v = torch.zeros_like(s.k), torch.zeros_like(s.v)
    place = torch.randperm(s.k.shape[1], generator=_gen(3), device="cuda")[:n].int()
    uz.cache_copy(arrived[0], arrived[1], torch.stack([ids, place], 1).contiguous(), to=(other_k, other_v), check=True)
    at = place[s.state[1].clamp(0, n - 1).long()]
    for layer in range(s.layers):
        q = _rand(_gen(77 + layer), (8, s.hq, s.d), s.dtype)
        got = uz.paged_attention(q, other_k[layer], other_v[layer], at, s.state[2], check=True)
        assert torch.equal(_bits(got), _bits(before[layer]))


def test_a_decoding_step_in_a_graph(uz):
    """A whole step captured once and replayed as the sequences grow, over page
    borders and from whole rows to rows that blocks cut."""
    page, seqs, hq, hk, d = 16, 3, 8, 2, 64
    g = _gen(40)
    k, v = ref.pools(g, 400, hk, page, d, torch.bfloat16)
    state = ref.state(400, seqs, 100)
    freqs = uz.rotary_frequencies(d)
    fused = _rand(g, (seqs, (hq + 2 * hk) * d), torch.bfloat16)
    uz.cache_reserve(*state, _i32(15, 1, 600), 616, page, check=True)
    kept = [x.clone() for x in (*state, k, v)]
    counts = _i32(1, 1, 1)

    def step():
        slots, positions, copies = uz.cache_reserve(*state, counts, seqs, page)
        uz.cache_copy(k, v, copies)
        q, kk, vv = (x.unflatten(1, (-1, d)) for x in fused.split((hq * d, hk * d, hk * d), 1))
        q = uz.rotary_append(q, kk, vv, positions, freqs, k, v, slots)
        return uz.paged_attention(q, k, v, state[1], state[2], with_lse=True)

    def inputs(i):
        fused.copy_(_rand(_gen(1000 + i), fused.shape, fused.dtype))

    eager = []
    for i in range(20):
        inputs(i)
        eager.append([x.clone() for x in step()])
    end = [x.clone() for x in (*state, k, v)]
    for a, b in zip((*state, k, v), kept):
        a.copy_(b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for a, b in zip((*state, k, v), kept):
        a.copy_(b)
    for i in range(20):
        inputs(i)
        graph.replay()
        assert torch.equal(_bits(got[0]), _bits(eager[i][0])) and torch.equal(got[1], eager[i][1])
    assert all(torch.equal(a, b) for a, b in zip(state, end))
    assert torch.equal(_bits(k), _bits(end[3])) and torch.equal(_bits(v), _bits(end[4]))


def test_streams_and_threads(uz):
    """Calls on streams of their own, from several threads, give what one call gives."""
    cases = []
    for n in range(4):
        g = _gen(50 + n)
        k, v = ref.pools(g, 400, 2, 16, 128, torch.bfloat16)
        table, lengths = ref.tables([3000 - n, 40, 700], 16, 400, seed=n)
        q = _rand(g, (3, 8, 128), torch.bfloat16)
        pos = torch.tensor([3000, 40, 700], device="cuda")
        cases.append((q, k, v, table, lengths, pos))
    freqs = uz.rotary_frequencies(128)
    want = [(uz.paged_attention(*c[:5]), uz.rotary(c[0], None, c[5], freqs)[0]) for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(n):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                got[n] = uz.paged_attention(*cases[n][:5], stream=stream), uz.rotary(cases[n][0], None, cases[n][5], freqs, stream=stream)[0]
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for (a, b), (c, e) in zip(got, want):
        assert torch.equal(_bits(a), _bits(c)) and torch.equal(_bits(b), _bits(e))
