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
