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
