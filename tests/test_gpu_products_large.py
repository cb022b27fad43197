"""Products over matrices of more than 2^31 values, whose offsets pass 32 bits."""
import pytest
import torch

from tests import _products as ref

pytestmark = pytest.mark.gpu

ROWS, COLS = 140_003, 16_384  # 2.29e9 values


@pytest.fixture(scope="module")
def uz():
    import lossless_float_tensor_gb300 as uz

    return uz


@pytest.fixture(scope="module")
def big():
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(ROWS, COLS, dtype=torch.bfloat16, device="cuda")
    for part in w.split(20_000):
        part.copy_(torch.randint(-8, 9, part.shape, generator=g, device="cuda"))
    yield w
    del w
    torch.cuda.empty_cache()


def test_weight_rows_and_columns(uz, big):
    at = torch.tensor([0, 5, COLS - 1], device="cuda")
    x = torch.zeros(3, COLS, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(3), at] = 1
    assert torch.equal(uz.linear(x, big, check=True), big[:, at].T)
    rows = torch.tensor([1, ROWS // 2, ROWS - 1], device="cuda")
    dy = torch.zeros(3, ROWS, dtype=torch.bfloat16, device="cuda")
    dy[torch.arange(3), rows] = 1
    dx, dw, db = uz.linear_backward(dy, x, big, check=True)
    assert torch.equal(dx, big[rows])
    assert int(dw.count_nonzero()) == 3 and bool((dw[rows, at] == 1).all())
    assert int(db.count_nonzero()) == 3 and bool((db[rows] == 1).all())


def test_experts_far_apart(uz, big):
    experts, n = 100, 1400
    w = big[: experts * n].view(experts, n, COLS)
    counts = torch.zeros(experts, dtype=torch.int64)
    counts[0], counts[57], counts[99] = 2, 1, 3
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).cuda()
    owner = torch.repeat_interleave(torch.arange(experts), counts).cuda()
    at = torch.tensor([3, COLS - 1, 64, 1, COLS - 2, 8000], device="cuda")
    x = torch.zeros(6, COLS, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(6), at] = 1
    assert torch.equal(uz.grouped_linear(x, w, off, check=True), w[owner, :, at])
    dy = torch.zeros(6, n, dtype=torch.bfloat16, device="cuda")
    dy[:, n - 1] = 1
    dx, dw, _ = uz.grouped_linear_backward(dy, x, w, off, need_db=False, check=True)
    assert torch.equal(dx, w[owner, n - 1])
    assert int(dw.count_nonzero()) == 6 and bool((dw[owner, n - 1, at] == 1).all())


def test_result_of_many_values(uz, big):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randint(-3, 4, (ROWS, 16), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-3, 4, (COLS, 16), generator=g, device="cuda").to(torch.bfloat16)
    out = big  # its values have served
    uz.linear(x, w, out=out, check=True)
    for rows in (slice(0, 300), slice(ROWS // 2, ROWS // 2 + 300), slice(ROWS - 300, ROWS)):
        assert torch.equal(out[rows].double(), x[rows].double() @ w.double().T)


def test_vocabulary_of_many_values(uz):
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty(ROWS, COLS, dtype=torch.float16, device="cuda")
    for part in w.split(20_000):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * (2 * COLS ** -0.5))
    h = torch.randn(3, COLS, generator=g, device="cuda").half()
    targets = torch.tensor([0, ROWS - 1, 77_777], device="cuda")
    loss, lse = uz.cross_entropy(h, w, targets, check=True)
    s = torch.cat([h.double() @ part.double().T for part in w.split(10_000)], 1)
    want = torch.logsumexp(s, 1) - s[torch.arange(3), targets]
    mag = torch.cat([h.double().abs() @ part.double().abs().T for part in w.split(10_000)], 1).amax(1)
    off = 2 * (COLS + 4) * 2.0 ** -23 * mag + 2.0 ** -20 * (1 + want.abs() + want.abs())
    assert ref.within(loss, want, off) <= 1.0
    dh, dw = uz.cross_entropy_backward(torch.full((3,), 64.0, device="cuda"), h, w, targets, lse, check=True)
    p = torch.exp(s - torch.logsumexp(s, 1, keepdim=True))
    p[torch.arange(3), targets] -= 1
    for rows in (slice(0, 100), slice(ROWS - 100, ROWS)):
        want = (64 * p[:, rows]).T @ h.double()
        bound = 2.0 ** -9 * (64 * p[:, rows].abs()).T @ h.double().abs() + 2.0 ** -24
        assert ref.within(dw[rows], want, bound) <= 1.0
