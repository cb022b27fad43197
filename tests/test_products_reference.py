"""The 64-bit definitions that the product operators are tested against, held
to central differences, and the constants of their error bounds to a grid."""
import pytest
import torch

from tests import _products as ref


def _difference(f, at, step=1e-5):
    g = torch.zeros_like(at)
    flat, out = at.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + step
        hi = f()
        flat[i] = keep - step
        lo = f()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * step)
    return g


@pytest.mark.parametrize("act", ref.ACTS)
def test_linear_gradient_against_differences(act):
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 4), (6, 4)))
    b, dy = torch.randn(6, generator=g, dtype=torch.float64), torch.randn(5, 6, generator=g, dtype=torch.float64)
    f = lambda: float((ref.act64(x @ w.T + b, act) * dy).sum())  # noqa: E731
    dz = dy * ref.slope64(x @ w.T + b, act)
    # a central difference is off by step^2 times the third derivative plus 2^-52 / step of the value
    for at, want in ((x, dz @ w), (w, dz.T @ x), (b, dz.sum(0))):
        assert torch.allclose(_difference(f, at), want, rtol=0, atol=1e-8)


def test_loss_gradient_against_differences():
    g = torch.Generator().manual_seed(4)
    h, w = torch.randn(4, 3, generator=g, dtype=torch.float64), torch.randn(7, 3, generator=g, dtype=torch.float64)
    t, dl = torch.tensor([2, -100, 6, 0]), torch.randn(4, generator=g, dtype=torch.float64)

    def f():
        s = h @ w.T
        loss = torch.logsumexp(s, 1) - s[torch.arange(4), t.clamp(min=0)]
        return float((loss * dl)[t != -100].sum())

    ref.ROUND[torch.float64], ref.TINY[torch.float64] = 0.0, 0.0
    (dh, _), (dw, _) = ref.loss_grad64(h, w, t, dl)
    del ref.ROUND[torch.float64], ref.TINY[torch.float64]
    assert torch.allclose(_difference(f, h), dh, rtol=0, atol=1e-8)
    assert torch.allclose(_difference(f, w), dw, rtol=0, atol=1e-8)


@pytest.mark.parametrize("act", ref.ACTS)
def test_bound_constants(act):
    z = torch.linspace(-30, 30, 600001, dtype=torch.float64)
    s = ref.slope64(z, act)
    assert float(s.abs().max()) <= ref.SLOPE_MAX[act]
    if act != "relu":  # its slope is a step
        curve = (s[2:] - s[:-2]) / (z[2:] - z[:-2])
        assert float((z[1:-1] * curve).abs().max()) <= ref.CURVE_MAX[act] + 1e-9
