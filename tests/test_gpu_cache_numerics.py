"""Attention of one token where its arithmetic could lose digits: capped scores
of any cap, weights far below the largest.  Bounds here go by the scores and the weights themselves, so that
none of them grows with what it is to bound."""
import math

import pytest
import torch

from tests import _cache as ref
from tests._products import ROUND, TINY, within

pytestmark = pytest.mark.gpu

DTYPES = (torch.bfloat16, torch.float16)


@pytest.fixture(scope="module")
def uz():
    import lossless_float_tensor_gb300 as uz

    return uz


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _f32(x):
    """What a float argument is in 32 bits."""
    return float(torch.tensor(x, dtype=torch.float32))


# ---- capped scores ------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cap", [1e-3, 1.0, 30.0, 50.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e20, 1e37, 3e38])
def test_a_capped_score_keeps_its_digits(uz, cap, dtype):
    """The log-sum-exp of one token is its score.  Keys with a single 1 give
    products without rounding, so all that is off is the cap: the factors in 32
    bits (scale, cap, scale over cap, log2 e, ln 2: together some 8 roundings of
    2^-24), 2^-21 for the exponential, its reciprocal and their difference from
    half the cap on, 2^-23 for the polynomial below.  2^-19 of the score bounds
    them all."""
    d, heads = 64, 8
    u = 10.0 ** torch.linspace(-7, 1.5, 400, dtype=torch.float64)
    u = torch.cat([u, torch.linspace(0.4, 0.6, 200, dtype=torch.float64), 10.0 ** torch.linspace(-38, -7, 200, dtype=torch.float64)])
    x = (cap * torch.cat([u, -u])).to(dtype)
    x = x[x.double().abs().ge(2.0 ** -24 if dtype == torch.float16 else 1e-30) & x.double().abs().le(6e4 if dtype == torch.float16 else 5e37)]
    # scores of ordinary size, whatever the cap
    x = torch.cat([x, torch.linspace(-40, 40, 333, dtype=torch.float64).to(dtype)])
    x = torch.cat([x, x[: -x.numel() % heads]]).view(-1, heads).cuda()
    q = torch.zeros(x.shape[0], heads, d, dtype=dtype, device="cuda")
    q[..., 5] = x
    k = torch.zeros(1, 1, 1, d, dtype=dtype, device="cuda")
    k[..., 5] = 1
    v = torch.randn(k.shape, generator=_gen(1), device="cuda").to(dtype)
    table = torch.zeros(x.shape[0], 1, dtype=torch.int32, device="cuda")
    for scale in (1.0, -0.25):
        out, lse = uz.paged_attention(q, k, v, table, table[:, 0] + 1, scale=scale, softcap=cap, with_lse=True, check=True)
        s = x.double() * scale
        want = _f32(cap) * torch.tanh(s / _f32(cap))
        assert within(lse, want, 2.0 ** -19 * want.abs() + 2.0 ** -126) <= 1.0
        assert torch.equal(out, v[0, 0, 0].expand_as(out))


def attention64(q, k, v, table, lengths, scale=None, softcap=0.0):
    """(out, lse, bound of |out - computed|, bound of |lse - computed|).

    A score is off by the 32-bit sum of d products (each addition by at most
    2^-23 of the magnitudes so far) and by 2^-19 of itself for what is done to
    it, capped or not.  A weight is off by that in numerator and sum, 2^-20 for
    the exponential, and its rounding to the type: by half a step of itself, in
    fp16 (where the largest is 2^15 and steps are no less than 2^-24) by no less
    than 2^-40 of the largest.  Sums over tokens run in 32 bits, and the result
    is rounded once."""
    u, tiny = ROUND[q.dtype], TINY[q.dtype]
    least = 2.0 ** -40 if q.dtype == torch.float16 else 0.0
    s, hq, d = q.shape
    heads, page = k.shape[1], k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, lse = torch.zeros(s, hq, d, dtype=torch.float64, device=q.device), torch.zeros(s, hq, dtype=torch.float64, device=q.device)
    off, off_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for i, n in enumerate(lengths.tolist()):
        t = torch.arange(n, device=q.device)
        at = table[i].long()[t // page]
        kk, vv = k[at, :, t % page].double(), v[at, :, t % page].double()  # [n, heads, d]
        qq = q[i].double().view(heads, hq // heads, d)
        z = torch.einsum("hgd,nhd->hgn", qq, kk) * scale
        slip = (d + 4) * 2.0 ** -23 * abs(scale) * torch.einsum("hgd,nhd->hgn", qq.abs(), kk.abs())
        if softcap:
            z = softcap * torch.tanh(z / softcap)
        slip = slip + 2.0 ** -19 * z.abs()
        # the sum weighs each token's slip as the result does; one token is off by its own
        w = torch.softmax(z, -1)
        worst = (w * slip).sum(-1, keepdim=True)
        each = u + 1.1 * (slip + worst) + 2.0 ** -19 + (n + 8) * 2.0 ** -23
        err = torch.einsum("hgn,nhd->hgd", w * each, vv.abs()) + n * least * vv.abs().amax(0)[:, None]
        o, total = torch.einsum("hgn,nhd->hgd", w, vv), torch.logsumexp(z, -1)
        out[i], lse[i] = o.reshape(hq, d), total.reshape(hq)
        off[i] = (u * (o.abs() + err) + err + tiny).reshape(hq, d)
        off_lse[i] = (1.1 * worst[..., 0] + 2.0 ** -20 * (2 + total.abs()) + (n + 8) * 2.0 ** -23).reshape(hq)
    return out, lse, off, off_lse


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cap", [30.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e20, 3.4e38])
@pytest.mark.parametrize("lengths,heads,group,d", [([77, 1, 300], 2, 4, 96), ([900, 2000], 1, 8, 128), ([700, 40], 1, 17, 64), ([650], 1, 12, 256)])
def test_attention_of_large_caps(uz, lengths, heads, group, d, cap, dtype):
    """A cap far above the scores is hardly any: no digits of them are lost."""
    g = _gen(d)
    pages = sum(-(-n // 16) for n in lengths) + 3
    k, v = ref.pools(g, pages, heads, 16, d, dtype)
    table, n = ref.tables(lengths, 16, pages)
    q = (torch.randn(len(lengths), heads * group, d, generator=g, device="cuda") * 2).to(dtype)
    got = uz.paged_attention(q, k, v, table, n, softcap=cap, with_lse=True, check=True)
    want, want_lse, off, off_lse = attention64(q, k, v, table, n, softcap=_f32(cap))
    assert within(got[0], want, off) <= 1.0 and within(got[1], want_lse, off_lse) <= 1.0
    if cap >= 1e8:  # (x / cap)^2 is below half a step of 32 bits: nothing is left of the cap
        plain = uz.paged_attention(q, k, v, table, n, with_lse=True)
        assert torch.equal(got[0].view(torch.int16), plain[0].view(torch.int16)) and torch.equal(got[1], plain[1])


def test_infinite_scores_meet_the_cap(uz):
    """A product past 32 bits, or an infinite key, is a score of plus or minus the cap; what is no number stays none."""
    d = 64
    q = torch.zeros(4, 1, d, dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = torch.tensor([1.0, -1.0, 3e38, math.nan], device="cuda")
    k = torch.zeros(1, 1, 1, d, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    table = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    for key, signs in ((math.inf, (1, -1, 1)), (-3e38, (-1, 1, -1))):
        k[..., 0] = key
        for cap in (5.0, 1e6, 1e30):
            _, lse = uz.paged_attention(q, k, v, table, table[:, 0] + 1, scale=1.0, softcap=cap, with_lse=True)
            want = cap * torch.tensor(signs, dtype=torch.float64, device="cuda")
            assert float(((lse[:3, 0].double() - want) / want).abs().max()) <= 2.0 ** -20 and bool(lse[3].isnan().all())


# ---- weights far below the largest ----------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("below", [(0, 0), (13, 15), (20.3, 20.3), (16, 24), (24.7, 24.7), (25, 30), (30, 34), (5, 39)])
@pytest.mark.parametrize("group,d", [(1, 64), (8, 128), (16, 256), (32, 96)])
def test_small_weights_keep_their_digits(uz, group, d, below, dtype):
    """One token has a score some powers of two over all others, and a value of
    0: the result is what the others add up to."""
    g = _gen(d)
    lengths = [2, 17, 40, 300, 2000, 2000, 2000]
    sinks = [0, 16, 5, 299, 0, 1000, 1999]
    pages = sum(-(-n // 16) for n in lengths) + 3
    k, v = ref.pools(g, pages, 2, 16, d, dtype, scale=1024.0)  # results in the type's normal range
    k[..., 3] = -(below[0] + (below[1] - below[0]) * torch.rand(k.shape[:-1], generator=g, device="cuda")).to(dtype)
    table, n = ref.tables(lengths, 16, pages)
    for i, t in enumerate(sinks):
        at = int(table[i, t // 16]), slice(None), t % 16
        k[at] = 0
        v[at] = 0
    q = torch.zeros(len(lengths), 2 * group, d, dtype=dtype, device="cuda")
    q[..., 3] = 1
    scale = _f32(math.log(2))
    out, lse = uz.paged_attention(q, k, v, table, n, scale=scale, with_lse=True, check=True)
    want, want_lse, off, off_lse = attention64(q, k, v, table, n, scale=scale)
    assert within(out, want, off) <= 1.0 and within(lse, want_lse, off_lse) <= 1.0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,heads,group,d,page", [
    ([1, 0, 2, 15, 16, 17], 2, 4, 128, 16), ([33, 500, 512, 513, 1], 4, 8, 128, 16), ([100, 7], 3, 5, 80, 24), ([70, 129], 2, 9, 256, 1),
    ([19, 200, 0], 2, 32, 128, 16), ([20000, 3], 1, 1, 64, 64), ([1500, 6000], 2, 16, 128, 32), ([900, 2000, 5], 1, 17, 64, 16), ([1000, 2500], 1, 11, 192, 16),
])
def test_attention_within_the_bounds_of_its_weights(uz, lengths, heads, group, d, page, dtype):
    g = _gen(d + page)
    pages = sum(-(-n // page) for n in lengths) + 3
    k, v = ref.pools(g, pages, heads, page, d, dtype)
    table, n = ref.tables(lengths, page, pages)
    q = (torch.randn(len(lengths), heads * group, d, generator=g, device="cuda") * 6).to(dtype)
    out, lse = uz.paged_attention(q, k, v, table, n, with_lse=True, check=True)
    some = n > 0
    want, want_lse, off, off_lse = attention64(q[some], k, v, table[some], n[some])
    assert within(out[some], want, off) <= 1.0 and within(lse[some], want_lse, off_lse) <= 1.0


def test_large_scores_and_values_in_fp16(uz):
    """Scores up to where 32 bits step by more than one, and the largest values: the factor of the weights makes nothing infinite."""
    d, n = 64, 1000
    g = _gen(3)
    k, v = ref.pools(g, 80, 1, 16, d, torch.float16)
    v.copy_(torch.where(torch.rand(v.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0) * 65504)
    k.fill_(60000.0)
    table, lengths = ref.tables([n], 16, 80)
    q = torch.full((1, 4, d), 60000.0, dtype=torch.float16, device="cuda")
    for scale in (1.0, 1e-3, -1e4):  # equal scores of 2.3e11, 2.3e8, -2.3e15
        out, lse = uz.paged_attention(q, k, v, table, lengths, scale=scale, with_lse=True, check=True)
        t = torch.arange(n, device="cuda")
        want = v[table[0].long()[t // 16], 0, t % 16].double().mean(0)
        # sums of at most 1000 terms of 65504 in 32 bits, one rounding of the result
        assert within(out, want.expand(1, 4, d), 2.0 ** -11 * want.abs() + 65504 * 1008 * 2.0 ** -23) <= 1.0
        score = 3.6e9 * d * scale
        assert float((lse.double() - score).abs().max()) <= 2.0 ** -20 * abs(score)


# ---- sums over long contexts ----------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,group,d", [([131072], 8, 128), ([100003], 3, 64), ([40000, 7, 65536], 4, 80), ([20001], 32, 96), ([9999], 16, 256)])
def test_long_sums_keep_32_bits(uz, lengths, group, d, dtype):
    """Weights of 1, 1/2, 1/4 and 1/8 and values that are small whole numbers
    of both signs: every product and every partial sum is a multiple of 1/8 (in
    fp16 times 2^15) of at most 2^20, which 32 bits hold exactly, while the
    result is what is left of them.  So it is off by its one rounding and by
    what the weights are in sum: 2^-18, for the exponentials' 2^-22, the sum's
    and the reciprocal's roundings."""
    g = _gen(d)
    page = 16
    pages = sum(-(-n // page) for n in lengths) + 3
    k, v = ref.pools(g, pages, 1, page, d, dtype)
    table, n = ref.tables(lengths, page, pages)
    v.copy_(torch.randint(-3, 4, v.shape, generator=g, device="cuda").to(dtype))
    # each tile of 16 tokens has a token of the largest score: the maximum never moves, and no sum is scaled
    k[:, 0, :, 3] = -torch.tensor([0, 1, 2, 3, 1, 0, 3, 2] * 2, device="cuda").to(dtype)
    q = torch.zeros(len(lengths), group, d, dtype=dtype, device="cuda")
    q[..., 3] = 1
    out, lse = uz.paged_attention(q, k, v, table, n, scale=_f32(math.log(2)), with_lse=True, check=True)
    for i, m in enumerate(lengths):
        t = torch.arange(m, device="cuda")
        at = table[i].long()[t // page]
        w = 2.0 ** k[at, 0, t % page, 3].double()
        want = (w[:, None] * v[at, 0, t % page].double()).sum(0) / w.sum()
        assert within(out[i], want.expand(group, d), (ROUND[dtype] + 2.0 ** -18) * want.abs() + TINY[dtype]) <= 1.0
        assert float((lse[i].double() - w.sum().log()).abs().max()) <= 2.0 ** -19 * (2 + math.log(m))


def _rounds(lengths, page, pages):
    """A table whose rows go round and round through the pool, each from another
    page on, and how often each sequence has each of the pool's tokens."""
    width = -(-max(lengths) // page)
    starts = torch.arange(len(lengths)) * 5 % pages
    table = ((starts[:, None] + torch.arange(width)) % pages).int().cuda()
    n, all_ = torch.tensor(lengths)[:, None], pages * page
    place = (torch.arange(all_)[None] - starts[:, None] * page) % all_  # of the pool's token in a round
    return table, n[:, 0].int().cuda(), ((n - place + all_ - 1) // all_).clamp(min=0).double().cuda()


# a warp's sum of 512 tiles by instructions that cut toward zero, each by less than 2^-23 of the sum so far, and as many
# additions of two weights in 32 bits, then a few roundings: less than 2 * 2^-14 + 2^-16
SUMS = 2.0 ** -12.5


def _of_rounds(uz, lengths, group, d, dtype, page=16, pages=64, q_scale=2.0, positive=False):
    g = _gen(d + group)
    k, v = ref.pools(g, pages, 1, page, d, dtype)
    if positive:
        v.copy_((1 + torch.rand(v.shape, generator=g, device="cuda")).to(dtype))
    table, n, often = _rounds(lengths, page, pages)
    q = (torch.randn(len(lengths), group, d, generator=g, device="cuda") * q_scale).to(dtype)
    out, lse = uz.paged_attention(q, k, v, table, n, with_lse=True, check=True)
    kk, vv, qq = k.flatten(0, 2).double(), v.flatten(0, 2).double(), q.double()
    z = qq @ kk.T * d ** -0.5
    slip = (d + 4) * 2.0 ** -23 * d ** -0.5 * (qq.abs() @ kk.abs().T) + 2.0 ** -19 * z.abs()
    z = z + often.log()[:, None]  # tokens that a sequence does not have: -inf
    w, total = torch.softmax(z, -1), torch.logsumexp(z, -1)
    worst = (w * slip).sum(-1, keepdim=True)
    u, least = ROUND[dtype], 2.0 ** -40 if dtype == torch.float16 else 0.0
    want = w @ vv
    err = (w * (u + 1.1 * (slip + worst) + 2.0 ** -19 + SUMS)) @ vv.abs() + least * n[:, None, None] * vv.abs().max()
    assert within(out, want, u * (want.abs() + err) + err + TINY[dtype]) <= 1.0
    assert within(lse, total, 1.1 * worst[..., 0] + 2.0 ** -20 * (2 + total.abs()) + SUMS) <= 1.0
    return q, k, v, table, n, out, lse, want


# rows that a block takes more than 32768 tokens of: a row for each block, and rows that many blocks share
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group,d", [(1, 64), (8, 128), (12, 128), (32, 128), (32, 64), (32, 96), (3, 192), (16, 256)])
@pytest.mark.parametrize("lengths", [[32767, 32768, 32769, 32784, 65536, 65537, 98304, 99999, 5, 1] * 61, [30 * 10 ** 6], [10 ** 7, 3, 40 * 10 ** 5, 10 ** 7]])
def test_rows_of_many_chunks(uz, lengths, group, d, dtype):
    _of_rounds(uz, lengths, group, d, dtype)


@pytest.mark.parametrize("group,d", [(1, 64), (8, 128), (32, 96)])
def test_long_sums_of_one_sign_do_not_fall_short(uz, group, d):
    """A row of 524288 tokens for each block, values between 1 and 2: the
    results agree with 64 bits by the sums' bound and one rounding (the weights'
    own roundings are at random here: 2^-11 over the root of some thousand)."""
    *_, out, _, want = _of_rounds(uz, [524288] * 500, group, d, torch.float16, page=256, pages=64, q_scale=0.5, positive=True)
    assert within(out, want, (ROUND[torch.float16] + SUMS) * want) <= 1.0


def test_a_bad_page_of_an_early_chunk(uz):
    q, k, v, table, n, out, lse, _ = _of_rounds(uz, [100000] * 500, 4, 64, torch.bfloat16)
    status = torch.zeros((), dtype=torch.int32, device="cuda")
    for col in (0, 2047, 2048, 6249):
        t = table.clone()
        t[250, col] = 64
        got, got_lse = uz.paged_attention(q, k, v, t, n, with_lse=True, status=status)
        assert int(status) == 1 and bool(got[250].isnan().all()) and bool(got_lse[250].isnan().all())
        got[250], got_lse[250] = out[250], lse[250]
        assert torch.equal(got, out) and torch.equal(got_lse, lse)
