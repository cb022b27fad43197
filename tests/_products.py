"""64-bit definitions of the matrix-product operators and the error bounds that
their tests use (torch, any device)."""
import math

import torch

ACTS = ("none", "relu", "gelu", "silu")
# largest relative error of one rounding to the type: half a unit in the last place
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# what a rounding below the normal range may lose
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z.clone()


def slope64(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        q = torch.sigmoid(z)
        return q * (1 + z * (1 - q))
    return torch.ones_like(z)


# max over z of |act'(z)| and of |z act''(z)| (how far rounding z moves act'),
# each rounded up: gelu'' = phi(z)(2 - z^2), silu'' = q(1-q)(2 + z(1-2q))
SLOPE_MAX = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "silu": 1.1}
CURVE_MAX = {"none": 0.0, "relu": 0.0, "gelu": 0.6, "silu": 0.45}


def linear64(x, w, b=None, r=None, act="none"):
    """(y, z, bound of |y - computed|, bound of |z - computed|): one rounding
    of the result, a 32-bit sum of k products (each addition off by at most
    2^-23 of the sum of magnitudes so far), and 2^-20 for the activation's
    exponential or error function."""
    dt = x.dtype
    xd, wd = x.double(), w.double()
    z = xd @ wd.T
    mag = xd.abs() @ wd.abs().T
    if b is not None:
        z = z + b.double()
        mag = mag + b.double().abs()
    acc = (x.shape[1] + 4) * 2.0 ** -23 * mag
    y = act64(z, act)
    off = acc * SLOPE_MAX[act] + (0 if act in ("none", "relu") else 2.0 ** -20 * (z.abs() + 1))
    if r is not None:
        y = y + r.double()
        off = off + 2.0 ** -23 * y.abs()
    u, tiny = ROUND[dt], TINY[dt]
    return y, z, u * (y.abs() + off) + off + tiny, u * (z.abs() + acc) + acc + tiny


def linear_grad64(dy, x, w, z, act):
    """dx, dw, db and the bounds of their errors, given the saved z (which the
    operator reads as it was rounded): dz is rounded once more for the
    products, the results once, sums run in 32 bits."""
    dt = x.dtype
    u, tiny = ROUND[dt], TINY[dt]
    xd, wd, dyd = x.double(), w.double(), dy.double()
    dz = dyd * slope64(z.double(), act)
    off = dyd.abs() * (0 if act in ("none", "relu") else 2.0 ** -19)
    dzr = off + (0 if act == "none" else u) * (dz.abs() + off) + (0 if act == "none" else tiny)
    m, n = dz.shape
    out = []
    for ref, mag, err, terms in (
            (dz @ wd, dz.abs() @ wd.abs(), dzr @ wd.abs(), n),
            (dz.T @ xd, dz.abs().T @ xd.abs(), dzr.T @ xd.abs(), m),
            (dz.sum(0), dz.abs().sum(0), off.sum(0), m)):
        acc = err + (terms + 4) * 2.0 ** -23 * (mag + err)
        out.append((ref, u * (ref.abs() + acc) + acc + tiny))
    return out


def loss64(h, w, targets, ignore=-100):
    """loss, lse, bound of their errors: a logit is off by the 32-bit sum of d
    products, the log-sum-exp by no more than the worst logit plus 2^-20 for
    the exponentials, the logarithm and the sum of v terms' partial sums."""
    hd, wd = h.double(), w.double()
    s = hd @ wd.T
    mag = (hd.abs() @ wd.abs().T).amax(1)
    used = targets != ignore
    at = targets.clamp(0, w.shape[0] - 1)
    lse = torch.logsumexp(s, 1)
    loss = lse - s[torch.arange(s.shape[0], device=s.device), at]
    off = 2 * (h.shape[1] + 4) * 2.0 ** -23 * mag + 2.0 ** -20 * (1 + lse.abs() + loss.abs())
    zero = torch.zeros_like(loss)
    return torch.where(used, loss, zero), torch.where(used, lse, zero), off


def loss_grad64(h, w, targets, dloss, ignore=-100):
    """dh, dw and the bounds of their errors: the softmax gradient is rounded
    once (relative to its own size, and never below the type's smallest step
    after scaling the largest weight to 2^10), its exponent is off by the
    logits' error; the results are rounded once."""
    dt = h.dtype
    u, tiny = ROUND[dt], TINY[dt]
    used = targets != ignore
    hd, wd = torch.where(used[:, None], h.double(), 0.0), w.double()
    s = hd @ wd.T
    lse = torch.logsumexp(s, 1, keepdim=True)
    g = torch.where(used, dloss.double(), 0.0)[:, None]
    p = torch.exp(s - lse)
    hit = torch.nn.functional.one_hot(targets.clamp(0, w.shape[0] - 1), w.shape[0]).double()
    dl = g * (p - hit)
    top = float(g.abs().max()) if g.numel() else 0.0
    slip = 4 * (h.shape[1] + 4) * 2.0 ** -23 * (hd.abs() @ wd.abs().T).amax(1, keepdim=True) \
        + 2.0 ** -19 * (2 + s.abs() + lse.abs())
    first = g.abs() * (p * slip + 2.0 ** -22 * hit)
    err = first + u * (dl.abs() + first) + tiny * top * 2.0 ** -9
    out = []
    for ref, mag, e, terms in ((dl @ wd, dl.abs() @ wd.abs(), err @ wd.abs(), w.shape[0]),
                               (dl.T @ hd, dl.abs().T @ hd.abs(), err.T @ hd.abs(), h.shape[0])):
        acc = e + (terms + 4) * 2.0 ** -23 * (mag + e)
        out.append((ref, u * (ref.abs() + acc) + acc + tiny))
    return out


def within(got, ref, bound):
    """Largest error as a share of its bound (at most 1 passes)."""
    if not ref.numel():
        return 0.0
    d = (got.double() - ref).abs()
    if not torch.isfinite(got).all():
        return math.inf
    return float((d / bound).max())
