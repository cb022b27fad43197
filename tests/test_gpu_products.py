"""The matrix-product operators on the GPU against their 64-bit definitions.

Random inputs are held to the error bounds of tests/_products.py, element by
element.  Small whole numbers, whose products and sums every type here holds
exactly, have to come out equal, so that a wrong index anywhere shows.
"""
import pytest
import torch

from tests import _products as ref

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


def _whole(g, shape, dtype, most=2, share=1.0):
    v = torch.randint(-most, most + 1, shape, generator=g, device="cuda")
    if share < 1.0:
        v = v * (torch.rand(shape, generator=g, device="cuda") < share)
    return v.to(dtype)


def _ok(got, pair):
    want, bound = pair
    assert ref.within(got, want, bound) <= 1.0


def _same(got, want, dtype):
    assert torch.equal(got.double(), want.to(dtype).double())


SIZES = [(1, 1, 1), (1, 64, 64), (1, 4096, 130), (3, 100, 7), (7, 9, 257), (16, 512, 1000), (33, 65, 129), (64, 1024, 96),
         (100, 72, 300), (127, 130, 515), (128, 128, 256), (129, 520, 255), (200, 1001, 64), (255, 63, 1024),
         (257, 264, 513), (300, 2048, 384), (1000, 192, 777), (2049, 136, 128)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", SIZES)
def test_linear_whole_numbers(uz, m, k, n, dtype):
    g = _gen(m + 3 * k + 7 * n)
    share = min(1.0, 24.0 / k)  # sums of few terms stay within the 8 bits of bf16
    x, w = _whole(g, (m, k), dtype, 2, share), _whole(g, (n, k), dtype, 1)
    b, r = _whole(g, (n,), dtype, 3), _whole(g, (m, n), dtype, 3)
    z = x.double() @ w.double().T + b.double()
    y, pre = uz.linear(x, w, b, activation="relu", residual=r, save_preact=True, check=True)
    _same(pre, z, dtype)
    _same(y, z.clamp(min=0) + r.double(), dtype)
    _same(uz.linear(x, w), x.double() @ w.double().T, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", SIZES)
def test_linear_backward_whole_numbers(uz, m, k, n, dtype):
    g = _gen(m + 5 * k + 11 * n)
    dy, x, w = _whole(g, (m, n), dtype, 2, min(1.0, 24.0 / max(m, n))), _whole(g, (m, k), dtype, 1), _whole(g, (n, k), dtype, 1)
    z = _whole(g, (m, n), dtype, 1)
    for act in ("none", "relu"):
        dz = dy.double() * ref.slope64(z.double(), act)
        dx, dw, db = uz.linear_backward(dy, x, w, z, activation=act, check=True)
        _same(dx, dz @ w.double(), dtype)
        _same(dw, dz.T @ x.double(), dtype)
        _same(db, dz.sum(0), dtype)
    only = uz.linear_backward(dy, x, w, need_dx=False, need_db=False)
    assert only[0] is None and only[2] is None
    _same(only[1], dy.double().T @ x.double(), dtype)


# sizes at which one tile is split over its depth (long depths, few tiles), by
# single blocks and by pairs, and at which pairs take tiles of every width
WIDE = [(20, 9000, 130), (300, 12000, 260), (640, 16400, 513), (1100, 300, 4200), (2300, 520, 2112), (1030, 4100, 1033)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", WIDE)
def test_linear_whole_numbers_split_and_paired(uz, m, k, n, dtype):
    g = _gen(m + k + 13 * n)
    x, w = _whole(g, (m, k), dtype, 2, 24.0 / k), _whole(g, (n, k), dtype, 1)
    b, r = _whole(g, (n,), dtype, 3), _whole(g, (m, n), dtype, 3)
    dy = _whole(g, (m, n), dtype, 2, 24.0 / max(m, n))
    y, z = uz.linear(x, w, b, activation="relu", residual=r, save_preact=True, check=True)
    want = x.double() @ w.double().T + b.double()
    _same(z, want, dtype)
    _same(y, want.clamp(min=0) + r.double(), dtype)
    dx, dw, db = uz.linear_backward(dy, x, w, check=True)
    _same(dx, dy.double() @ w.double(), dtype)
    _same(dw, dy.double().T @ x.double(), dtype)
    _same(db, dy.double().sum(0), dtype)
    # and the transposed shapes, whose gradients sum over k and n
    dy2, x2 = _whole(g, (k, m), dtype, 2, 24.0 / max(k, m)), _whole(g, (k, n), dtype, 1)
    _, dw, db = uz.linear_backward(dy2, x2, torch.zeros(m, n, dtype=dtype, device="cuda"), need_dx=False, check=True)
    _same(dw, dy2.double().T @ x2.double(), dtype)
    _same(db, dy2.double().sum(0), dtype)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", [(1, 1024, 512), (5, 333, 70), (40, 4096, 384), (130, 257, 264), (513, 640, 1030)])
def test_linear_bounds(uz, m, k, n, dtype, act):
    g = _gen(m + k + n)
    x, w = _rand(g, (m, k), dtype), _rand(g, (n, k), dtype, k ** -0.5)
    b, r, dy = _rand(g, (n,), dtype, 0.5), _rand(g, (m, n), dtype), _rand(g, (m, n), dtype)
    y, z = uz.linear(x, w, b, activation=act, residual=r, save_preact=True)
    y64, z64, y_off, z_off = ref.linear64(x, w, b, r, act)
    _ok(y, (y64, y_off))
    _ok(z, (z64, z_off))
    for got, pair in zip(uz.linear_backward(dy, x, w, z, activation=act), ref.linear_grad64(dy, x, w, z, act)):
        _ok(got, pair)


def test_signs_kept_for_relu(uz):
    """relu's slope is a step, so a value kept for its gradient has to have its
    sign: tensor-core sums of 4096 products get about 15 of 16 million signs
    wrong (of values below 1e-5), 32-bit sums about 4.  Over three draws at
    most as many as twice the latter may be, by the dense and by the grouped
    product."""
    wrong = [0, 0]
    for seed in range(3):
        g = _gen(40 + seed)
        x, w, b = _rand(g, (4096, 4096), torch.float16), _rand(g, (4096, 4096), torch.float16, 1 / 64), _rand(g, (4096,), torch.float16, 0.5)
        sign = x.double() @ w.double().T + b.double() > 0
        off = torch.tensor([0, 1000, 4096], device="cuda")
        wrong[0] += int(((uz.linear(x, w, b, activation="relu", save_preact=True)[1] > 0) != sign).sum())
        z = uz.grouped_linear(x, torch.stack([w, w]), off, torch.stack([b, b]), activation="relu", save_preact=True)[1]
        wrong[1] += int(((z > 0) != sign).sum())
    assert max(wrong) <= 24


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_strided_views_and_odd_addresses(uz, dtype):
    g = _gen(5)
    m, k, n = 70, 200, 150
    for lead, pad in ((0, 8), (1, 3), (8, 56), (4, 4)):
        x = _whole(g, (m, lead + k + pad), dtype, 2, 0.1)[:, lead:lead + k]
        w = _whole(g, (n, lead + k + pad), dtype, 1)[:, lead:lead + k]
        r = _whole(g, (m, lead + n + pad), dtype)[:, lead:lead + n]
        dy = _whole(g, (m, lead + n + pad), dtype, 1, 0.1)[:, lead:lead + n]
        out = torch.full((m, lead + n + pad), 77.0, dtype=dtype, device="cuda")
        got = uz.linear(x, w, residual=r, out=out[:, lead:lead + n])
        _same(got, x.double() @ w.double().T + r.double(), dtype)
        assert bool((out[:, :lead] == 77).all()) and bool((out[:, lead + n:] == 77).all())
        dx, dw, db = uz.linear_backward(dy, x, w)
        _same(dx, dy.double() @ w.double(), dtype)
        _same(dw, dy.double().T @ x.double(), dtype)
        _same(db, dy.double().sum(0), dtype)


def test_rows_of_every_other_matrix_row(uz):
    g = _gen(6)
    x, w = _whole(g, (80, 128), torch.float16)[::2], _whole(g, (96, 128), torch.float16, 1)[::3]
    _same(uz.linear(x, w), x.double() @ w.double().T, torch.float16)


@pytest.mark.parametrize("m,k,n", [(0, 8, 8), (8, 0, 8), (8, 8, 0), (0, 0, 0), (1, 0, 1), (300, 0, 600)])
def test_linear_lengths_of_zero(uz, m, k, n):
    x, w = torch.ones(m, k, device="cuda", dtype=torch.bfloat16), torch.ones(n, k, device="cuda", dtype=torch.bfloat16)
    b, dy = torch.full((n,), 2.0, device="cuda", dtype=torch.bfloat16), torch.ones(m, n, device="cuda", dtype=torch.bfloat16)
    y = uz.linear(x, w, b, check=True)
    assert y.shape == (m, n) and bool((y == 2 + k).all())
    dx, dw, db = uz.linear_backward(dy, x, w, check=True)
    assert dx.shape == (m, k) and bool((dx == n).all())
    assert dw.shape == (n, k) and bool((dw == m).all())
    assert db.shape == (n,) and bool((db == m).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", [(40, 136, 300), (300, 72, 520)])
def test_not_a_number_and_infinity_stay_in_their_rows(uz, m, k, n, dtype):
    g = _gen(7)
    x, w = _rand(g, (m, k), dtype), _rand(g, (n, k), dtype, 0.1)
    clean = uz.linear(x, w)
    x[3, k - 1] = float("nan")
    x[m - 1, 0] = float("inf")
    got = uz.linear(x, w)
    keep = [i for i in range(m) if i not in (3, m - 1)]
    assert torch.equal(got[keep], clean[keep])
    assert bool(torch.isnan(got[3]).all())
    assert not bool(torch.isfinite(got[m - 1]).any())


def test_activations_far_out(uz):
    z = torch.tensor([-3e38, -1e4, -200.0, -89.0, -30.0, 0.0, 30.0, 89.0, 200.0, 1e4, 3e38], device="cuda").to(torch.bfloat16)
    one = torch.ones(1, 1, device="cuda", dtype=torch.bfloat16)
    for act in ("relu", "gelu", "silu"):
        y = uz.linear(one, z[:, None], activation=act)[0].double()
        want = torch.where(z.double() > 0, z.double(), 0.0)
        assert torch.allclose(y, want, rtol=2.0 ** -8, atol=1e-11), act
        dx, _, db = uz.linear_backward(torch.ones(1, 11, device="cuda", dtype=torch.bfloat16), one, z[:, None], z[None, :],
                                       activation=act)
        want = (z > 0).double()
        want[5] = 0.0 if act == "relu" else 0.5
        assert torch.allclose(db.double(), want, rtol=0, atol=1e-10), act


# ---- grouped ---------------------------------------------------------------------

COUNTS = [[5], [0, 0, 3], [1, 0, 2, 1], [64, 64], [63, 65, 1, 0, 200], [0, 130, 0, 129, 17, 0], [300, 1, 1, 1, 40],
          [16] * 12, [0, 0], [1] * 40, [700, 0, 513, 256, 1, 900], [257] * 9]


def _offsets(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k,n", [(64, 64), (72, 300), (201, 130), (512, 257)])
@pytest.mark.parametrize("counts", COUNTS)
def test_grouped_whole_numbers(uz, counts, k, n, dtype):
    g = _gen(sum(counts) + k + n)
    e, m = len(counts), sum(counts)
    off = _offsets(counts)
    x, w, b = _whole(g, (m, k), dtype, 2, min(1.0, 24.0 / k)), _whole(g, (e, n, k), dtype, 1), _whole(g, (e, n), dtype, 3)
    dy, z = _whole(g, (m, n), dtype, 2, 24.0 / 512), _whole(g, (m, n), dtype, 1)
    y, pre = uz.grouped_linear(x, w, off, b, activation="relu", save_preact=True, check=True)
    dx, dw, db = uz.grouped_linear_backward(dy, x, w, off, z, activation="relu", check=True)
    dz = dy.double() * (z > 0)
    at = 0
    for i, c in enumerate(counts):
        rows = slice(at, at + c)
        at += c
        pz = x[rows].double() @ w[i].double().T + b[i].double()
        _same(pre[rows], pz, dtype)
        _same(y[rows], pz.clamp(min=0), dtype)
        _same(dx[rows], dz[rows] @ w[i].double(), dtype)
        _same(dw[i], dz[rows].T @ x[rows].double(), dtype)
        _same(db[i], dz[rows].sum(0), dtype)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_grouped_bounds(uz, dtype, act):
    counts, k, n = [37, 0, 1, 150, 12], 264, 200
    g = _gen(8)
    off, m = _offsets(counts), sum(counts)
    x, w, b = _rand(g, (m, k), dtype), _rand(g, (5, n, k), dtype, k ** -0.5), _rand(g, (5, n), dtype, 0.5)
    dy = _rand(g, (m, n), dtype)
    y, z = uz.grouped_linear(x, w, off, b, activation=act, save_preact=True)
    dx, dw, db = uz.grouped_linear_backward(dy, x, w, off, z, activation=act)
    at = 0
    for i, c in enumerate(counts):
        rows = slice(at, at + c)
        at += c
        y64, z64, y_off, z_off = ref.linear64(x[rows], w[i], b[i], None, act)
        _ok(y[rows], (y64, y_off))
        _ok(z[rows], (z64, z_off))
        for got, pair in zip((dx[rows], dw[i], db[i]), ref.linear_grad64(dy[rows], x[rows], w[i], z[rows], act)):
            _ok(got, pair)


def test_grouped_neighbours_do_not_leak(uz):
    """Rows that are not finite reach only their own expert's gradients."""
    counts = [20, 45, 0, 31]
    g = _gen(9)
    off, m, k, n = _offsets(counts), 96, 128, 136
    x, w, dy = (_rand(g, s, torch.bfloat16) for s in ((m, k), (4, n, k), (m, n)))
    y0 = uz.grouped_linear(x, w, off)
    _, dw0, db0 = uz.grouped_linear_backward(dy, x, w, off)
    x[20:65] = float("nan")
    dy[20:65] = float("inf")
    y1 = uz.grouped_linear(x, w, off)
    dx1, dw1, db1 = uz.grouped_linear_backward(dy, x, w, off)
    for i in (0, 2, 3):
        assert torch.equal(dw0[i], dw1[i]) and torch.equal(db0[i], db1[i])
    assert torch.equal(y0[:20], y1[:20]) and torch.equal(y0[65:], y1[65:])
    assert bool(torch.isnan(dw1[1]).all()) and bool(torch.isfinite(dx1[:20]).all()) and bool(torch.isfinite(dx1[65:]).all())


@pytest.mark.parametrize("offsets", [[1, 5, 10], [0, 5, 9], [0, 11, 10], [0, 5, 11], [0, -1, 10], [0, 7, 3]])
def test_grouped_bad_offsets(uz, offsets):
    off = torch.tensor(offsets, dtype=torch.int64, device="cuda")
    x, w = torch.ones(10, 64, device="cuda", dtype=torch.float16), torch.ones(2, 72, 64, device="cuda", dtype=torch.float16)
    status = torch.full((), -1, dtype=torch.int32, device="cuda")
    y, z = uz.grouped_linear(x, w, off, save_preact=True, status=status)
    assert int(status.item()) == uz.UZIP_ERR_INVALID_ARG
    assert bool(torch.isnan(y).all()) and bool(torch.isnan(z).all())
    for part in uz.grouped_linear_backward(y, x, w, off, status=status):
        assert bool(torch.isnan(part).all())
    assert int(status.item()) == uz.UZIP_ERR_INVALID_ARG
    with pytest.raises(uz.UzipError, match="invalid argument"):
        uz.grouped_linear(x, w, off, check=True)


# ---- cross entropy -----------------------------------------------------------------

LOSS_SIZES = [(1, 1, 1), (1, 1000, 64), (5, 33, 40), (64, 512, 128), (65, 257, 129), (130, 1030, 200), (300, 5000, 72),
              (513, 700, 513)]


def _loss_inputs(t, v, d, dtype, seed, drop=0.2):
    g = _gen(seed)
    h, w = _rand(g, (t, d), dtype), _rand(g, (v, d), dtype, 2 * d ** -0.5)
    targets = torch.randint(0, v, (t,), generator=g, device="cuda")
    targets[torch.rand(t, generator=g, device="cuda") < drop] = -100
    return h, w, targets, 0.5 + torch.rand(t, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,v,d", LOSS_SIZES)
def test_cross_entropy_bounds(uz, t, v, d, dtype):
    h, w, targets, dloss = _loss_inputs(t, v, d, dtype, t + v + d)
    loss, lse = uz.cross_entropy(h, w, targets, check=True)
    want, want_lse, off = ref.loss64(h, w, targets)
    _ok(loss, (want, off))
    _ok(lse, (want_lse, off))
    assert bool((loss[targets == -100] == 0).all())
    for piece in (0, 256, 40):
        got = uz.cross_entropy_backward(dloss, h, w, targets, lse, piece=piece, check=True)
        for a, pair in zip(got, ref.loss_grad64(h, w, targets, dloss)):
            _ok(a, pair)


@pytest.mark.parametrize("scale", [1e-30, 3e-6, 1.0, 4096.0])
def test_cross_entropy_gradient_at_any_scale(uz, scale):
    """The softmax gradient keeps its precision for small and large weights."""
    h, w, targets, dloss = _loss_inputs(90, 3000, 104, torch.bfloat16, 21)
    _, lse = uz.cross_entropy(h, w, targets)
    got = uz.cross_entropy_backward(dloss * scale, h, w, targets, lse)
    for a, pair in zip(got, ref.loss_grad64(h, w, targets, dloss * scale)):
        _ok(a, pair)


@pytest.mark.parametrize("dtype", DTYPES)
def test_cross_entropy_gradient_of_a_mean(uz, dtype):
    """Equal weights that are no power of two: a target's gradient is nearly the
    weight itself, so its rounding is the same for all tokens and does not
    average out.  The results' own rounding is u / sqrt(3) of their size or
    less; the whole error has to stay below twice that."""
    g = _gen(28)
    h, w = _rand(g, (600, 256), dtype), _rand(g, (20000, 256), dtype, 1 / 16)
    targets = torch.randint(0, 20000, (600,), generator=g, device="cuda")
    for weight in (1 / 600, 0.7, 1.3):
        dloss = torch.full((600,), weight * (512 if dtype == torch.float16 else 1), device="cuda")
        _, lse = uz.cross_entropy(h, w, targets)
        for a, (want, _) in zip(uz.cross_entropy_backward(dloss, h, w, targets, lse), ref.loss_grad64(h, w, targets, dloss)):
            assert float((a.double() - want).norm() / want.norm()) <= 2 * ref.ROUND[dtype] / 3 ** 0.5


def test_cross_entropy_ignored_rows_may_hold_anything(uz):
    h, w, targets, dloss = _loss_inputs(200, 900, 136, torch.bfloat16, 22)
    drop = targets == -100
    loss0, lse0 = uz.cross_entropy(h, w, targets)
    dh0, dw0 = uz.cross_entropy_backward(dloss, h, w, targets, lse0)
    at = torch.nonzero(drop).flatten()
    h[at[0]] = float("nan")
    h[at[1], 5] = float("inf")
    dloss[at[2]] = float("nan")
    loss1, lse1 = uz.cross_entropy(h, w, targets)
    dh1, dw1 = uz.cross_entropy_backward(dloss, h, w, targets, lse1)
    assert torch.equal(loss0, loss1) and torch.equal(lse0, lse1)
    assert torch.equal(dh0, dh1) and torch.equal(dw0, dw1)
    assert bool((dh1[drop] == 0).all())


def test_cross_entropy_all_ignored_and_no_tokens(uz):
    h, w, targets, dloss = _loss_inputs(70, 300, 64, torch.float16, 23)
    targets[:] = -100
    loss, lse = uz.cross_entropy(h, w, targets, check=True)
    dh, dw = uz.cross_entropy_backward(dloss, h, w, targets, lse, check=True)
    assert not loss.any() and not dh.any() and not dw.any()
    loss, lse = uz.cross_entropy(h[:0], w, targets[:0], check=True)
    dh, dw = uz.cross_entropy_backward(dloss[:0], h[:0], w, targets[:0], lse, check=True)
    assert loss.shape == (0,) and dh.shape == (0, 64) and not dw.any()


def test_cross_entropy_other_ignore_index(uz):
    h, w, targets, dloss = _loss_inputs(50, 300, 64, torch.float16, 24, drop=0.0)
    targets[::4] = 7
    loss, lse = uz.cross_entropy(h, w, targets, ignore_index=7)
    want, _, off = ref.loss64(h, w, targets, ignore=7)
    _ok(loss, (want, off))
    for a, pair in zip(uz.cross_entropy_backward(dloss, h, w, targets, lse, ignore_index=7),
                       ref.loss_grad64(h, w, targets, dloss, ignore=7)):
        _ok(a, pair)


def test_cross_entropy_large_logits(uz):
    """Logits of several hundred, where exp alone overflows."""
    h, w, targets, _ = _loss_inputs(40, 500, 64, torch.bfloat16, 25)
    h = h * 100
    loss, _ = uz.cross_entropy(h, w, targets)
    want, _, off = ref.loss64(h, w, targets)
    _ok(loss, (want, off))


@pytest.mark.parametrize("bad", [300, -1, 1 << 40])
def test_cross_entropy_bad_target(uz, bad):
    h, w, targets, dloss = _loss_inputs(40, 300, 64, torch.bfloat16, 26, drop=0.0)
    good, _ = uz.cross_entropy(h, w, targets)
    targets[9] = bad
    status = torch.zeros((), dtype=torch.int32, device="cuda")
    loss, lse = uz.cross_entropy(h, w, targets, status=status)
    assert int(status.item()) == uz.UZIP_ERR_INVALID_ARG
    assert bool(torch.isnan(loss[9])) and torch.equal(loss[:9], good[:9]) and torch.equal(loss[10:], good[10:])
    dh, dw = uz.cross_entropy_backward(dloss, h, w, targets, lse, status=status)
    assert int(status.item()) == uz.UZIP_ERR_INVALID_ARG
    assert bool(torch.isnan(dh[9]).all()) and bool(torch.isnan(dw).all())


def test_cross_entropy_strided(uz):
    h, w, targets, dloss = _loss_inputs(60, 400, 208, torch.float16, 27)
    for lead in (0, 8, 3):
        hv, wv = h[:, lead:lead + 150], w[::2, lead:lead + 150]
        tv = torch.where(targets >= 0, targets // 2, targets)
        loss, lse = uz.cross_entropy(hv, wv, tv)
        want, _, off = ref.loss64(hv, wv, tv)
        _ok(loss, (want, off))
        for a, pair in zip(uz.cross_entropy_backward(dloss, hv, wv, tv, lse), ref.loss_grad64(hv, wv, tv, dloss)):
            _ok(a, pair)


# ---- how the calls behave ------------------------------------------------------------

def test_same_inputs_give_the_same_bits(uz):
    g = _gen(30)
    x, w, dy = (_rand(g, s, torch.bfloat16) for s in ((40, 4096), (512, 4096), (40, 512)))
    h, wv, targets, dloss = _loss_inputs(150, 2000, 256, torch.bfloat16, 31)
    _, lse = uz.cross_entropy(h, wv, targets)
    first = None
    for _ in range(4):
        out = [uz.linear(x, w), *uz.linear_backward(dy, x, w), *uz.cross_entropy(h, wv, targets),
               *uz.cross_entropy_backward(dloss, h, wv, targets, lse, piece=512)]
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


@pytest.mark.parametrize("m,k,n", [(354, 1072, 1616), (586, 4280, 273), (90, 512, 1003), (21, 3600, 3176)])
def test_same_bits_where_a_tile_ends_inside_a_patch(uz, m, k, n):
    """Values kept for relu's gradient are compared with their neighbours' size:
    only with neighbours that exist.  Other calls in between leave other values
    behind in the columns past the end."""
    g = _gen(34)
    x, w, b = _rand(g, (m, k), torch.float16), _rand(g, (2, n, k), torch.float16, k ** -0.5), _rand(g, (2, n), torch.float16)
    off = torch.tensor([0, m // 3, m], device="cuda")
    other = _rand(g, (m, k), torch.float16, 1000.0), _rand(g, (2048, k), torch.float16), _rand(g, (2048,), torch.float16, 30000.0)
    first = None
    for i in range(6):
        if i % 2:
            uz.linear(other[0], other[1], other[2], activation="relu", save_preact=True)
        out = [*uz.linear(x, w[0], b[0], activation="relu", save_preact=True),
               *uz.grouped_linear(x, w, off, b, activation="relu", save_preact=True)]
        first = first or out
        assert all(torch.equal(p, q) for p, q in zip(first, out))


def test_streams_of_their_own(uz):
    g = _gen(32)
    x, w, dy = _whole(g, (130, 201), torch.bfloat16, 1, 0.1), _whole(g, (260, 201), torch.bfloat16, 1), \
        _whole(g, (130, 260), torch.bfloat16, 1, 0.05)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for s in streams * 4:
        got.append((uz.linear(x, w, stream=s), *uz.linear_backward(dy, x, w, stream=s)))
    torch.cuda.synchronize()
    for y, dx, dw, db in got:
        _same(y, x.double() @ w.double().T, torch.bfloat16)
        _same(dx, dy.double() @ w.double(), torch.bfloat16)
        _same(dw, dy.double().T @ x.double(), torch.bfloat16)


def test_graph_capture(uz):
    g = _gen(33)
    x, w = _whole(g, (24, 512), torch.bfloat16, 2, 0.05), _whole(g, (700, 512), torch.bfloat16, 1)
    y = torch.empty(24, 700, dtype=torch.bfloat16, device="cuda")
    uz.linear(x, w, out=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uz.linear(x, w, out=y)
    x.copy_(_whole(g, (24, 512), torch.bfloat16, 2, 0.05))
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    _same(y, x.double() @ w.double().T, torch.bfloat16)


def test_a_workspace_given_and_too_small(uz):
    from lossless_float_tensor_gb300 import ops

    x, w = torch.ones(9, 33, device="cuda", dtype=torch.float16), torch.ones(50, 33, device="cuda", dtype=torch.float16)
    y = torch.empty(9, 50, device="cuda", dtype=torch.float16)
    a = ops.LinearArgs(dtype=2, m=9, n=50, k=33, x=x.data_ptr(), ldx=33, w=w.data_ptr(), ldw=33, y=y.data_ptr(), ldy=50)
    need = ops.uzip_linear_workspace_size(a)
    assert need > 0  # rows of 33 values are copied to 16-byte boundaries
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert ops.uzip_linear(a, ws.data_ptr(), need - 1, None, stream) == uz.UZIP_ERR_CAPACITY
    assert ops.uzip_linear(a, None, 0, None, stream) == uz.UZIP_ERR_INVALID_ARG
    assert ops.uzip_linear(a, ws.data_ptr(), need, None, stream) == uz.UZIP_OK
    assert bool((y == 33).all())
    a.y = y.data_ptr() + 2 * 9 * 50  # the last row would end past the allocation's end unless the allocator rounds up
    a.ldy = 1 << 30
    assert ops.uzip_linear(a, ws.data_ptr(), need, None, stream) == uz.UZIP_ERR_INVALID_ARG


def test_refusals(uz):
    half = lambda *s: torch.ones(*s, device="cuda", dtype=torch.float16)  # noqa: E731
    x, w = half(4, 8), half(6, 8)
    off = torch.tensor([0, 4], device="cuda")
    bad = [
        lambda: uz.linear(x, half(6, 9)),
        lambda: uz.linear(x, w.bfloat16()),
        lambda: uz.linear(x, w, half(7)),
        lambda: uz.linear(x, w, residual=half(4, 7)),
        lambda: uz.linear(x, w, activation="tanh"),
        lambda: uz.linear(x.float(), w.float()),
        lambda: uz.linear(x.t(), half(6, 4)),
        lambda: uz.linear(x.cpu(), w),
        lambda: uz.linear(x[0], w),
        lambda: uz.linear(half(1, 8).expand(4, 8), w),
        lambda: uz.linear(x, w, out=half(4, 7)),
        lambda: uz.linear_backward(half(4, 6), x, w, activation="gelu"),
        lambda: uz.linear_backward(half(4, 7), x, w),
        lambda: uz.grouped_linear(x, w, off),
        lambda: uz.grouped_linear(x, half(1, 6, 8), off.int()),
        lambda: uz.grouped_linear(x, half(2, 6, 8), off),
        lambda: uz.grouped_linear(x, half(0, 6, 8), off[:1]),
        lambda: uz.cross_entropy(x, w, torch.zeros(4, dtype=torch.int32, device="cuda")),
        lambda: uz.cross_entropy(x, w, torch.zeros(5, dtype=torch.int64, device="cuda")),
        lambda: uz.cross_entropy(x, half(0, 8), torch.zeros(4, dtype=torch.int64, device="cuda")),
        lambda: uz.cross_entropy_backward(half(4), x, w, torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")),
        lambda: uz.cross_entropy_backward(torch.ones(4, device="cuda"), x, w, torch.zeros(4, dtype=torch.int64, device="cuda"),
                                          torch.zeros(4, device="cuda"), piece=-1),
    ]
    for f in bad:
        with pytest.raises(uz.UzipError):
            f()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("grouped", (False, True))
def test_relu_keeps_the_sign_of_sums_that_cancel(uz, dtype, grouped):
    # Every fourth row against every 64th column: 64 products, then the same ones negated, sixteen times, and +-2^-26 at
    # last.  Sums of 32 bits are off by more, and fp16 has no value that small.
    m, n, k = 300, 512, 2048
    g = _gen(5)
    x = _rand(g, (m, k), dtype)
    w = _rand(g, (3, n, k) if grouped else (n, k), dtype)
    sign = torch.randint(0, 2, (m,), generator=g, device="cuda") * 2 - 1
    rows, cols = slice(0, m, 4), slice(7, n, 64)
    xs, ws = x.view(m, k // 128, 2, 64), w.view(-1, n, k // 128, 2, 64)
    xs[rows, :, 1] = xs[rows, :, 0]
    ws[:, cols, :, 1] = -ws[:, cols, :, 0]
    x[rows, k - 65] = 0
    x[rows, k - 1] = (sign[rows] * 2.0**-13).to(dtype)
    w[..., cols, k - 1] = 2.0**-13
    if grouped:
        offsets = torch.tensor([0, 130, 130, m], device="cuda")
        z = uz.grouped_linear(x, w, offsets, activation="relu", save_preact=True)[1]
    else:
        z = uz.linear(x, w, activation="relu", save_preact=True)[1]
    small = z[rows, cols]
    assert torch.equal(small > 0, (sign[rows, None] > 0).expand_as(small))
    assert float(small.abs().max()) <= 2.0**-24
