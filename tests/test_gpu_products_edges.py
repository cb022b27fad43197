"""The matrix-product operators where rounding, range, size or the order of calls
could show: signs kept for relu, confident tokens, long sums, tails of the
activations, tokens by the thousand, graphs and threads."""
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


# ---- signs kept for relu's gradient ------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", [(4096, 4096, 4096), (2048, 14336, 4096), (1024, 32768, 2048)])
def test_no_kept_sign_is_wrong(uz, m, k, n, dtype):
    """A value near zero is summed again as good as exactly, and one that is not
    is further from zero than its sum's error: every sign of six draws is that
    of the 64-bit sum."""
    g = _gen(7)
    for _ in range(6):
        x, w, b = _rand(g, (m, k), dtype), _rand(g, (n, k), dtype, k ** -0.5), _rand(g, (n,), dtype, 0.5)
        sign = x.double() @ w.double().T + b.double() > 0
        z = uz.linear(x, w, b, activation="relu", save_preact=True)[1]
        assert int(((z > 0) != sign).sum()) == 0


def test_no_kept_sign_is_wrong_by_expert(uz):
    """37 experts with ragged and odd rows: 50 draws, 77 million values."""
    e, m, k, n = 37, 1531, 520, 1003
    for seed in range(50):
        g = _gen(seed)
        x, w, b = _rand(g, (m, k), torch.float16), _rand(g, (e, n, k), torch.float16, k ** -0.5), _rand(g, (e, n), torch.float16, 0.5)
        cuts = torch.randint(0, m + 1, (e - 1,), generator=g, device="cuda").sort().values
        off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), m)])
        z = uz.grouped_linear(x, w, off, b, activation="relu", save_preact=True)[1]
        ends = off.tolist()
        for i in range(e):
            rows = slice(ends[i], ends[i + 1])
            assert torch.equal(z[rows] > 0, x[rows].double() @ w[i].double().T + b[i].double() > 0)


# ---- grouped products with a residual (C entry point) ------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k,n", [(72, 300), (512, 512), (201, 130)])
@pytest.mark.parametrize("counts", [[3, 0, 2, 1], [16] * 12, [63, 65, 1, 0, 200], [700, 0, 513, 256], [257] * 9])
def test_grouped_residual(uz, counts, k, n, dtype):
    """The residual is added whichever way the product is taken: few rows for
    each expert, or many."""
    from lossless_float_tensor_gb300 import ops

    g = _gen(sum(counts) + k)
    e, m = len(counts), sum(counts)
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int64, device="cuda")
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, w, b, r = whole(m, k), whole(e, n, k), whole(e, n), whole(m, n)
    x *= torch.rand(m, k, generator=g, device="cuda") < 16.0 / k
    y, z = torch.empty_like(r), torch.empty_like(r)
    a = ops.LinearArgs(dtype=uz.UZIP_BF16 if dtype == torch.bfloat16 else uz.UZIP_FP16, act=ops.UZIP_ACT_RELU, m=m, n=n, k=k,
                       groups=e, offsets=off.data_ptr(), x=x.data_ptr(), ldx=k, w=w.data_ptr(), ldw=k, w_group=n * k,
                       bias=b.data_ptr(), residual=r.data_ptr(), ldr=n, y=y.data_ptr(), ldy=n, z=z.data_ptr(), ldz=n)
    ws = torch.empty(ops.uzip_grouped_linear_workspace_size(a), dtype=torch.uint8, device="cuda")
    status = torch.full((), -1, dtype=torch.int32, device="cuda")
    st = ops.uzip_grouped_linear(a, ws.data_ptr() if ws.numel() else None, ws.numel(), status.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream)
    assert st == uz.UZIP_OK and int(status.item()) == uz.UZIP_OK
    at = 0
    for i, c in enumerate(counts):
        rows = slice(at, at + c)
        at += c
        pz = x[rows].double() @ w[i].double().T + b[i].double()
        assert torch.equal(z[rows].double(), pz.to(dtype).double())
        assert torch.equal(y[rows].double(), (pz.clamp(min=0) + r[rows].double()).to(dtype).double())


# ---- tokens that the model is sure of ----------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_confident_tokens(uz, dtype):
    """A target with p between 0.999 and 0.99999: p - 1 is the difference of two
    near numbers, and the whole row of dh hangs on it.  Off by: the rounding of
    lse (half a unit of a value below 32, 2^-20) and of the exponential (2^-21)
    against 1 - p; logits whose sums of 1024 depths are cut 256 times by 2^-23 of
    at most 8 (four of them: 2^-10); two roundings to the type."""
    g = _gen(35)
    d, v, t = 4096, 8192, 512
    w = _rand(g, (v, d), dtype, d ** -0.5)
    targets = torch.randint(0, v, (t,), generator=g, device="cuda")
    sure = torch.linspace(14, 24, t, device="cuda")[:, None]
    h = (w[targets].float() * sure + 0.1 * torch.randn(t, d, generator=g, device="cuda")).to(dtype)
    s = h.double() @ w.double().T
    p = torch.softmax(s, 1)
    rest = p.scatter(1, targets[:, None], 0.0).sum(1)
    want = 16384 * (p.scatter(1, targets[:, None], -rest[:, None]) @ w.double())
    _, lse = uz.cross_entropy(h, w, targets)
    dh, dw = uz.cross_entropy_backward(torch.full((t,), 16384.0, device="cuda"), h, w, targets, lse, check=True)
    off = (dh.double() - want).norm(dim=1) / want.norm(dim=1)
    bound = 2 * ref.ROUND[dtype] + 2.0 ** -10 + (2.0 ** -20 + 2.0 ** -21) / rest
    judged = (rest < 1e-3) & (rest > 1e-5)
    assert int(judged.sum()) > 64 and float(lse.max()) < 32
    assert float((off / bound)[judged].max()) <= 1.0
    # and the classes' rows, of which only confident tokens have a part
    only = torch.where(judged, 16384.0, 0.0)
    _, dw = uz.cross_entropy_backward(only.float(), h, w, targets, lse, need_dh=False, check=True)
    dl = p.scatter(1, targets[:, None], -rest[:, None]) * only.double()[:, None]
    at = torch.unique(targets[judged])
    want, most = (dl.T @ h.double())[at], (dl.abs() * bound[:, None]).T @ h.double().abs()
    assert float(((dw[at].double() - want).abs() / (most[at] + ref.ROUND[dtype] * want.abs() + 2.0 ** -24)).max()) <= 1.0


# ---- depths of many thousands ------------------------------------------------------

def _whole(g, shape, dtype, most=2, share=None):
    """Whole numbers, of which a share may be kept and the others be zero."""
    v = torch.randint(-most, most + 1, shape, generator=g, device="cuda")
    if share is not None:
        v = v * (torch.rand(shape, generator=g, device="cuda") < share)
    return v.to(dtype)


def _same(got, want, dtype):
    assert torch.equal(got.double(), want.to(dtype).double())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", [(1, 300000, 40), (20, 200001, 130), (300, 150000, 260), (1100, 70000, 1201), (2300, 17000, 4200)])
def test_long_depths_whole_numbers(uz, m, k, n, dtype):
    """Depths over 16384 are added up from chunks: every sum is exact here, as a
    product of x and w, and with the same lengths as one of dy and w or x."""
    g = _gen(m + k + n)
    x, w = _whole(g, (m, k), dtype, 2, 24.0 / k), _whole(g, (n, k), dtype, 1)
    b, r = _whole(g, (n,), dtype, 3), _whole(g, (m, n), dtype, 3)
    z = x.double() @ w.double().T + b.double()
    for act in ("relu", "none"):
        y, pre = uz.linear(x, w, b, activation=act, residual=r, save_preact=True, check=True)
        _same(pre, z, dtype)
        _same(y, ref.act64(z, act) + r.double(), dtype)
    wt, xt = _whole(g, (k, n), dtype, 1), _whole(g, (m, n), dtype, 1)  # depth k in dx
    dx, _, _ = uz.linear_backward(x, xt, wt, need_dw=False, need_db=False, check=True)
    _same(dx, x.double() @ wt.double(), dtype)
    dy, xl = x.T.contiguous(), _whole(g, (k, n), dtype, 1)  # depth k in dw
    _, dw, _ = uz.linear_backward(dy, xl, torch.zeros(m, n, dtype=dtype, device="cuda"), need_dx=False, need_db=False, check=True)
    _same(dw, dy.double().T @ xl.double(), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,k,n", [([20000, 0, 17000, 300], 136, 200), ([16, 3, 0, 40], 17001, 264), ([300, 5, 700], 17000, 520),
                                        ([16, 3, 0, 40], 264, 17001), ([300, 5, 700], 520, 17000), ([40000, 1], 72, 64)])
def test_long_depths_by_expert(uz, counts, k, n, dtype):
    g = _gen(sum(counts) + k)
    e, m = len(counts), sum(counts)
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int64, device="cuda")
    x, w = _whole(g, (m, k), dtype, 2, 24.0 / k), _whole(g, (e, n, k), dtype, 1)
    dy = _whole(g, (m, n), dtype, 2, 24.0 / max(n, max(counts)))
    y = uz.grouped_linear(x, w, off, check=True)
    dx, dw, _ = uz.grouped_linear_backward(dy, x, w, off, need_db=False, check=True)
    at = 0
    for i, c in enumerate(counts):
        rows = slice(at, at + c)
        at += c
        _same(y[rows], x[rows].double() @ w[i].double().T, dtype)
        _same(dx[rows], dy[rows].double() @ w[i].double(), dtype)
        _same(dw[i], dy[rows].double().T @ x[rows].double(), dtype)


@pytest.mark.parametrize("rows", [1 << 17, 1 << 18, 1 << 20])
def test_long_sums_are_not_short(uz, rows):
    """Sums of one sign.  A chunk of 16384 depths is 1024 steps of at most four
    additions, each cut by less than 2^-23 of the sum so far, which grows evenly:
    2^-12 at worst, and 2^-18 for up to 64 chunks added with rounding.  Beyond
    that only the result's own rounding is left, which has no direction: its
    mean over some thousand values is within 2^-15."""
    g = _gen(36)
    x = (torch.rand(rows, 64, generator=g, device="cuda") + 0.5).half()
    dy = ((torch.rand(rows, 96, generator=g, device="cuda") + 0.5) * (2.0 ** 14 / rows)).half()
    want = dy.double().T @ x.double()
    worst, mean = 2.0 ** -12 + 2.0 ** -18, 2.0 ** -15
    w = torch.zeros(1, 96, 64, device="cuda", dtype=torch.half)
    off = torch.tensor([0, rows], device="cuda")
    for got in (uz.linear_backward(dy, x, w[0], need_dx=False, need_db=False, check=True)[1],
                uz.grouped_linear_backward(dy, x, w, off, need_dx=False, need_db=False, check=True)[1][0],
                uz.linear(dy.T.contiguous(), x.T.contiguous(), check=True),
                uz.linear_backward(dy.T.contiguous(), torch.zeros(96, 64, device="cuda", dtype=torch.half), x, need_dw=False,
                                   need_db=False, check=True)[0]):
        short = (got.double() - want) / want
        assert float(short.abs().max()) <= ref.ROUND[torch.float16] + worst
        assert abs(float(short.mean())) <= worst + mean


def test_long_sum_over_tokens_is_not_short(uz):
    """The same for the gradient of a loss over 2^17 tokens that all have class
    0: every other class's row is a sum of one sign.  The softmax gradient's
    rounding to fp16 has no direction either."""
    t, v, d = 1 << 17, 64, 64
    g = _gen(37)
    h = (torch.rand(t, d, generator=g, device="cuda") + 0.5).half()
    w = _rand(g, (v, d), torch.float16, 0.05)
    targets = torch.zeros(t, dtype=torch.int64, device="cuda")
    _, lse = uz.cross_entropy(h, w, targets)
    dw = uz.cross_entropy_backward(torch.full((t,), 1.0 / 1024, device="cuda"), h, w, targets, lse, need_dh=False, check=True)[1]
    p = torch.softmax(h.double() @ w.double().T, 1)
    want = (p.T @ h.double() / 1024)[1:]
    short = (dw[1:].double() - want) / want
    assert float(short.abs().max()) <= 2 * ref.ROUND[torch.float16] + 2.0 ** -12 + 2.0 ** -18
    assert abs(float(short.mean())) <= 2.0 ** -12 + 2.0 ** -18 + 2.0 ** -15


# ---- tokens by the thousand --------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t", [1023, 1024, 1025, 2049, 5000])
def test_cross_entropy_of_thousands_of_tokens(uz, t, dtype):
    """Tokens are counted 1024 at a time: some thousands with runs of ignored
    ones longer than that, at the start, in the middle or at the end."""
    v, d = 300, 72
    g = _gen(t)
    h, w = _rand(g, (t, d), dtype), _rand(g, (v, d), dtype, 2 * d ** -0.5)
    dloss = 0.5 + torch.rand(t, generator=g, device="cuda")
    base = torch.randint(0, v, (t,), generator=g, device="cuda")
    base[torch.rand(t, generator=g, device="cuda") < 0.3] = -100
    for gone in (slice(0, 0), slice(0, t // 2), slice(t // 4, t // 4 + 1100), slice(t // 2, t)):
        targets = base.clone()
        targets[gone] = -100
        loss, lse = uz.cross_entropy(h, w, targets, check=True)
        want, want_lse, off = ref.loss64(h, w, targets)
        assert ref.within(loss, want, off) <= 1.0 and ref.within(lse, want_lse, off) <= 1.0
        assert bool((loss[targets == -100] == 0).all())
        got = uz.cross_entropy_backward(dloss, h, w, targets, lse, check=True)
        for a, (r, bound) in zip(got, ref.loss_grad64(h, w, targets, dloss)):
            assert ref.within(a, r, bound) <= 1.0
        assert bool((got[0][targets == -100] == 0).all())


@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_cross_entropy_of_half_a_million_tokens(uz, drop):
    """More tokens than a block lists at once before it copies their rows: each
    token's loss and dh, and dw, against 64 bits."""
    t, v, d = 700_001, 24, 16
    g = _gen(38)
    h, w = _rand(g, (t, d), torch.float16), _rand(g, (v, d), torch.float16, 2 * d ** -0.5)
    dloss = 0.5 + torch.rand(t, generator=g, device="cuda")
    targets = torch.randint(0, v, (t,), generator=g, device="cuda")
    targets[torch.rand(t, generator=g, device="cuda") < drop] = -100
    loss, lse = uz.cross_entropy(h, w, targets, check=True)
    want, want_lse, off = ref.loss64(h, w, targets)
    assert ref.within(loss, want, off) <= 1.0 and ref.within(lse, want_lse, off) <= 1.0
    for a, (r, bound) in zip(uz.cross_entropy_backward(dloss, h, w, targets, lse, check=True), ref.loss_grad64(h, w, targets, dloss)):
        assert ref.within(a, r, bound) <= 1.0


# ---- graphs and threads ------------------------------------------------------------

def test_calls_of_many_launches_in_a_graph(uz):
    """Calls that pack, multiply several times and join, captured and replayed on
    other values: the same bits as the calls themselves."""
    g = _gen(39)
    m, k, n, e, v = 300, 201, 261, 5, 1003
    off = torch.tensor([0, 40, 40, 170, 171, m], device="cuda")
    x, w, we, b, be = (_rand(g, s, torch.bfloat16, 0.2) for s in ((m, k), (n, k), (e, n, k), (n,), (e, n)))
    dy, head = _rand(g, (m, n), torch.bfloat16), _rand(g, (v, k), torch.bfloat16, 0.2)
    targets = torch.randint(0, v, (m,), generator=g, device="cuda")
    targets[::5] = -100
    dloss = torch.rand(m, generator=g, device="cuda")

    def step():
        y, z = uz.linear(x, w, b, activation="gelu", residual=dy, save_preact=True)
        ye, ze = uz.grouped_linear(x, we, off, be, activation="relu", save_preact=True)
        loss, lse = uz.cross_entropy(x, head, targets)
        return [y, z, ye, ze, loss, lse, *uz.linear_backward(dy, x, w, z, activation="gelu"),
                *uz.grouped_linear_backward(dy, x, we, off, ze, activation="relu"),
                *uz.cross_entropy_backward(dloss, x, head, targets, lse, piece=256)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (40, 41, 42):
        for a in (x, w, we, b, be, dy, head):
            a.copy_(_rand(_gen(seed), a.shape, a.dtype, 0.2))
        targets.copy_(targets.roll(7))
        for o in out:
            o.fill_(7)
        graph.replay()
        graph.replay()  # each replay starts from the other's leavings
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(p, q) for p, q in zip(got, step()))


def test_calls_from_several_threads(uz):
    """Threads with streams of their own and sizes in different orders get what
    one thread gets."""
    import threading

    g = _gen(43)
    sizes = [(1, 256, 96), (40, 201, 130), (300, 520, 264), (130, 72, 1003)]
    data = []
    for m, k, n in sizes:
        x, w, dy = (_rand(g, s, torch.float16, 0.2) for s in ((m, k), (n, k), (m, n)))
        off = torch.tensor([0, m // 3, m], device="cuda")
        data.append((x, w, dy, torch.stack([w, -w]), off))

    def calls(i):
        x, w, dy, we, off = data[i]
        y, z = uz.linear(x, w, activation="silu", save_preact=True)
        return [y, *uz.linear_backward(dy, x, w, z, activation="silu"), uz.grouped_linear(x, we, off),
                *uz.grouped_linear_backward(dy, x, we, off)]

    want = [calls(i) for i in range(len(sizes))]
    torch.cuda.synchronize()
    faults = []

    def work(first):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for turn in range(12):
                    i = (first + turn) % len(sizes)
                    got = calls(i)
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        faults.append((first, turn))
        except Exception as err:  # a thread's error would be lost
            faults.append(err)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join(120)
    assert not faults and not any(th.is_alive() for th in threads)


# ---- the ends of the types' ranges -------------------------------------------------

@pytest.mark.parametrize("grouped", [False, True])
def test_relu_keeps_signs_below_the_types_range(uz, grouped):
    """Values that fp16 rounds to zero still have their sign in what is kept, and
    so their gradient; the result itself is rounded as ever (half of 2^-24)."""
    g = _gen(44)
    m, k, n = 200, 96, 264
    x, w, dy = _rand(g, (m, k), torch.float16, 2.0 ** -14), _rand(g, (2, n, k), torch.float16, 2.0 ** -18), _rand(g, (m, n), torch.float16)
    if grouped:
        off = torch.tensor([0, 30, m], device="cuda")
        y, z = uz.grouped_linear(x, w, off, activation="relu", save_preact=True)
        dx, _, db = uz.grouped_linear_backward(dy, x, w, off, z, activation="relu")
        rows = [(slice(0, 30), 0), (slice(30, m), 1)]
    else:
        y, z = uz.linear(x, w[0], activation="relu", save_preact=True)
        dx, _, db = uz.linear_backward(dy, x, w[0], z, activation="relu")
        rows, db = [(slice(0, m), 0)], db[None]
    for r, i in rows:
        z64 = x[r].double() @ w[i].double().T
        assert float(z64.abs().max()) < 2.0 ** -25 and bool((z64 != 0).all())
        assert torch.equal(z[r] > 0, z64 > 0)
        assert float((y[r].double() - z64.clamp(min=0)).abs().max()) <= 2.0 ** -25
        dz = dy[r].double() * (z64 > 0)
        want, mag = dz.sum(0), dz.abs().sum(0)
        assert ref.within(db[i], want, ref.ROUND[torch.float16] * want.abs() + (m + 4) * 2.0 ** -22 * mag + 2.0 ** -24) <= 1.0


@pytest.mark.parametrize("act", ("relu", "gelu", "silu"))
@pytest.mark.parametrize("dtype", DTYPES)
def test_gradients_where_the_kept_value_is_infinite(uz, dtype, act):
    """A value past the type's range is kept as infinity: the slope there is 1
    or 0, as it is next to it.  One that is not a number stays one."""
    inf = float("inf")
    z = torch.tensor([[-inf, inf, 1.0, float("nan"), -inf, 0.5, inf, -2.0]], device="cuda").to(dtype)
    for n in (8, 5):  # 16-byte rows, and others
        dy, x, w = (torch.ones(s, device="cuda", dtype=dtype) for s in ((1, n), (1, 3), (n, 3)))
        _, dw, db = uz.linear_backward(dy, x, w, z[:, :n].contiguous(), activation=act)
        for got in (db, dw[:, 0]):
            assert got[0] == 0 and got[1] == 1 and got[4] == 0 and bool(torch.isnan(got[3]))
            assert bool(torch.isfinite(got[[2, 0, 1, 4]]).all())


def test_silu_gradient_of_a_value_that_overflows_fp16(uz):
    x, w = torch.full((2, 1), 300.0, device="cuda").half(), torch.tensor([[-300.0], [0.01]], device="cuda").half()
    y, z = uz.linear(x, w, activation="silu", save_preact=True)
    assert bool((y[:, 0] == 0).all()) and bool(torch.isinf(z[:, 0]).all())
    dx, dw, db = uz.linear_backward(torch.ones_like(y), x, w, z, activation="silu")
    assert float(db[0]) == 0 and float(dw[0]) == 0 and bool(torch.isfinite(dx).all())


# ---- the tails of the activations --------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
def test_gelu_keeps_its_precision_in_the_tail(uz, dtype):
    """gelu and its slope for z from -12 to -2, relative to themselves: one
    rounding, the exponential's argument (up to 104, rounded twice: 104 2^-23
    ln 2 = 9e-6) and the fitted tail (1e-6), below 2^-16 together.  In the slope
    Phi(z) - |z| phi(z) the errors are up to 1.6 times the difference's own."""
    z = torch.linspace(-12, -2, 4001, device="cuda").to(dtype).unique()
    one = torch.ones(1, 1, device="cuda", dtype=dtype)
    y = uz.linear(one, z[:, None], activation="gelu")[0].double()
    want = ref.act64(z.double(), "gelu")
    u, tiny = ref.ROUND[dtype], ref.TINY[dtype]
    assert float(((y - want).abs() / ((u + 2.0 ** -16) * want.abs() + tiny)).max()) <= 1.0
    dx, _, db = uz.linear_backward(torch.ones(1, z.numel(), device="cuda", dtype=dtype), one, z[:, None], z[None], activation="gelu")
    want = ref.slope64(z.double(), "gelu")
    assert float(((db.double() - want).abs() / ((u + 2.0 ** -15) * want.abs() + tiny)).max()) <= 1.0


@pytest.mark.parametrize("dtype", DTYPES)
def test_silu_keeps_its_precision_in_the_tail(uz, dtype):
    """The same for silu from -80 to -2: exp(-z)'s argument is up to 116, rounded
    twice (1e-5), below 2^-16 with the reciprocal."""
    z = torch.linspace(-80, -2, 4001, device="cuda").to(dtype).unique()
    one = torch.ones(1, 1, device="cuda", dtype=dtype)
    y = uz.linear(one, z[:, None], activation="silu")[0].double()
    want = ref.act64(z.double(), "silu")
    assert float(((y - want).abs() / ((ref.ROUND[dtype] + 2.0 ** -16) * want.abs() + ref.TINY[dtype])).max()) <= 1.0


# ---- waits that run out ------------------------------------------------------------

STARVED = [(1, 4096, 1024), (20, 9000, 130), (300, 520, 264), (1100, 300, 4200), (640, 16400, 513)]


def _starved(uz, call):
    """What call() gives while no product gets its first operand, its waits 50
    ms long, and the status that it reports."""
    import ctypes

    hook = uz.library().uzip_debug_starve_products
    hook.argtypes, hook.restype = [ctypes.c_int64], None
    status = torch.full((), -1, dtype=torch.int32, device="cuda")
    hook(100_000_000)
    try:
        out = call(status)
    finally:
        hook(0)
    torch.cuda.synchronize()
    return out, int(status.item())


@pytest.mark.parametrize("m,k,n", STARVED)
def test_waits_that_run_out_are_reported(uz, m, k, n):
    """Single blocks, pairs and clusters of both give up, and the next call is
    as good as ever."""
    g = _gen(45)
    x, w = _whole(g, (m, k), torch.bfloat16, 1, 8.0 / k), _whole(g, (n, k), torch.bfloat16, 1)
    assert _starved(uz, lambda s: uz.linear(x, w, status=s))[1] == uz.UZIP_ERR_TIMEOUT
    with pytest.raises(uz.UzipError, match="time"):
        _starved(uz, lambda s: uz.linear(x, w, check=True))
    _same(uz.linear(x, w, check=True), x.double() @ w.double().T, torch.bfloat16)


@pytest.mark.parametrize("m,k,n", STARVED)
def test_waits_that_run_out_leave_nan(uz, m, k, n):
    """What could not be computed is NaN also for a caller who asks for no
    status, in every output and schedule."""
    g = _gen(46)
    x, w, dy = (_rand(g, s, torch.float16, 0.2) for s in ((m, k), (n, k), (m, n)))
    off = torch.tensor([0, m // 3, m // 3, m], device="cuda")
    we = torch.stack([w, w, w])
    calls = [lambda s: uz.linear(x, w, activation="relu", save_preact=True), lambda s: [uz.linear(x, w)],
             lambda s: uz.linear_backward(dy, x, w, need_db=False)[:2],
             lambda s: uz.grouped_linear(x, we, off, activation="gelu", save_preact=True),
             lambda s: [uz.grouped_linear_backward(dy, x, we, off, need_dw=False, need_db=False)[0]],
             # (the expert in the middle has no rows: nothing of its is waited for)
             lambda s: list(uz.grouped_linear_backward(dy, x, we, off, need_dx=False, need_db=False)[1][(2 if m < 3 else 0)::2])]
    for call in calls:
        for t in _starved(uz, call)[0]:
            assert bool(torch.isnan(t).all())


def test_waits_that_run_out_leave_nan_losses(uz):
    g = _gen(47)
    for t in (20, 300):
        h, w = _rand(g, (t, 200), torch.bfloat16), _rand(g, (1003, 200), torch.bfloat16, 0.2)
        targets = torch.randint(0, 1003, (t,), generator=g, device="cuda")
        targets[3] = -100
        _, lse = uz.cross_entropy(h, w, targets)
        (loss, bad), _ = _starved(uz, lambda s: uz.cross_entropy(h, w, targets, status=s))
        used = targets != -100
        assert bool(torch.isnan(loss[used]).all() & torch.isnan(bad[used]).all() & (loss[~used] == 0).all())
        (dh, dw), _ = _starved(uz, lambda s: uz.cross_entropy_backward(torch.ones(t, device="cuda"), h, w, targets, lse, piece=256))
        assert bool(torch.isnan(dh[used]).all() & torch.isnan(dw).all() & (dh[~used] == 0).all())
        assert bool(torch.isfinite(uz.cross_entropy(h, w, targets, check=True)[0]).all())


# ---- what the torch functions refuse -----------------------------------------------

def test_tensors_that_require_gradients_are_refused(uz):
    """Autograd does not know these calls: a result without a gradient would be
    a silent hole in a training step."""
    half = lambda *s: torch.ones(*s, device="cuda", dtype=torch.float16)  # noqa: E731
    x, w, b, y = half(4, 8), half(6, 8), half(6), half(4, 6)
    targets, off = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.tensor([0, 4], device="cuda")
    ones = torch.ones(4, device="cuda")
    leaf = lambda t: t.clone().requires_grad_()  # noqa: E731
    calls = [lambda f: uz.linear(f(x), w), lambda f: uz.linear(x, f(w)), lambda f: uz.linear(x, w, f(b)),
             lambda f: uz.linear(x, w, residual=f(y)), lambda f: uz.linear_backward(f(y), x, w),
             lambda f: uz.linear_backward(y, f(x), f(w)), lambda f: uz.grouped_linear(x, f(w)[None], off),
             lambda f: uz.grouped_linear(f(x), w[None], off), lambda f: uz.cross_entropy(f(x), w, targets),
             lambda f: uz.cross_entropy(x, f(w), targets), lambda f: uz.cross_entropy_backward(f(ones), x, w, targets, ones)]
    for call in calls:
        with pytest.raises(uz.UzipError, match="requires gradients"):
            call(leaf)
        with torch.no_grad():
            got = call(leaf)
        want = call(lambda t: t)
        for p, q in zip(got if isinstance(got, tuple) else [got], want if isinstance(want, tuple) else [want]):
            assert torch.equal(p, q)


def test_a_workspace_or_status_that_is_not_one(uz):
    """A strided workspace would be written between its values, a status word of
    another type beyond its end; a workspace of wider values has all its bytes."""
    x, w = torch.ones(9, 33, device="cuda", dtype=torch.float16), torch.ones(50, 33, device="cuda", dtype=torch.float16)
    wide = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(uz.UzipError, match="workspace"):
        uz.linear(x, w, workspace=wide[::2])
    assert not wide.any()
    words = torch.zeros(8, dtype=torch.uint8, device="cuda")
    for bad in (words[0], words.view(torch.int64)[0], torch.zeros(4, device="cuda")[0], torch.zeros(0, dtype=torch.int32, device="cuda")):
        with pytest.raises(uz.UzipError, match="status"):
            uz.linear(x, w, status=bad)
    assert not words.any()
    need = -(-(9 + 50) * 40 * 2 // 256) * 256 + 256
    y = uz.linear(x, w, workspace=torch.empty(need // 4, dtype=torch.float32, device="cuda"), check=True)
    assert bool((y == 33).all())


# ---- token weights of many sizes ---------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
def test_cross_entropy_weights_of_many_sizes(uz, dtype):
    """Weights from 1 to 2^-20 of the largest: each row of dh to its own size,
    with what fp16 cannot hold beside the largest (2^-35 of it a class)."""
    t, v, d = 210, 4000, 136
    g = _gen(48)
    h, w = _rand(g, (t, d), dtype), _rand(g, (v, d), dtype, 2 * d ** -0.5)
    targets = torch.randint(0, v, (t,), generator=g, device="cuda")
    dloss = 2.0 ** (13 - torch.arange(t, device="cuda") % 21).float()
    _, lse = uz.cross_entropy(h, w, targets)
    dh, _ = uz.cross_entropy_backward(dloss, h, w, targets, lse, need_dw=False, check=True)
    s = h.double() @ w.double().T
    dl = dloss.double()[:, None] * (torch.softmax(s, 1) - torch.nn.functional.one_hot(targets, v))
    want, u = dl @ w.double(), ref.ROUND[dtype]
    lost = 2.0 ** -35 * 2.0 ** 13 if dtype == torch.float16 else 0.0
    slip = 4 * (d + 4) * 2.0 ** -23 * (h.double().abs() @ w.double().abs().T).amax(1, keepdim=True) + 2.0 ** -18 * (2 + s.abs())
    off = (dl.abs() * (u + slip) + lost) @ w.double().abs()
    off = off * (1 + 2.0 ** -10) + (v + 4) * 2.0 ** -23 * (dl.abs() @ w.double().abs())
    assert float(((dh.double() - want).abs() / (off + u * want.abs() + ref.TINY[dtype])).max()) <= 1.0
