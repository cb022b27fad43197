"""The framework's matrix-product operators as their users call them, for measurement.

Three operators over the weights that the library stores and moves: a linear
layer with bias, activation and residual (`linear`), the same product grouped
by expert with ragged row counts (`grouped`), and softmax cross entropy over a
vocabulary whose logits are never kept (`ce`).  Each case is a serving call
(the forward result) or a training step (forward and gradients).

With `own` false, run() computes the plain form in 32 bits from elementary
torch operations; with `own` true it calls the library.
"""
import math

import torch

own = False

if torch.cuda.is_available():  # the plain form's products stay in 32 bits
    torch.backends.cuda.matmul.allow_tf32 = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}

# The costliest listed case bounds the drawn ones (useful operations of a pass).
_MOST_FLOPS = 1.3e13


def _linear(name, dtype, m, k, n, act="none", bias=False, residual=False, train=False):
    c = {"op": "linear", "dtype": dtype, "m": m, "k": k, "n": n, "act": act, "bias": bias, "residual": residual, "train": train}
    return dict(c, name=name) if name else c


def _grouped(name, dtype, t, e, k, n, act="none", bias=False, train=False, skew=1.0):
    c = {"op": "grouped", "dtype": dtype, "t": t, "e": e, "k": k, "n": n, "act": act, "bias": bias, "train": train, "skew": skew}
    return dict(c, name=name) if name else c


def _ce(name, dtype, t, v, d, ignored=0.0, train=False):
    c = {"op": "ce", "dtype": dtype, "t": t, "v": v, "d": d, "ignored": ignored, "train": train}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through the key projection of a decoder layer: latency
        _linear("linear_token_kv", "bf16", 1, 4096, 1024),
        # a batch of single tokens through the gate projection: the weights' bandwidth
        _linear("linear_tokens_gate", "bf16", 16, 4096, 14336, act="silu"),
        # a prompt through the down projection, added to the residual stream
        _linear("linear_prompt_down", "fp16", 2048, 14336, 4096, bias=True, residual=True),
        # a training step on sizes that fill no tile and no 16-byte row
        _linear("linear_odd_train", "fp16", 777, 1001, 1237, act="gelu", bias=True, residual=True, train=True),
        # a training step of the gate projection on a large batch
        _linear("linear_gate_train", "bf16", 8192, 4096, 14336, act="silu", bias=True, train=True),
        # single tokens spread over many small experts: most experts have none or one
        _grouped("grouped_tokens", "bf16", 24, 64, 2048, 1408, act="silu", skew=1.0),
        # a prompt over many small experts, uneven, biased
        _grouped("grouped_prompt", "fp16", 8192, 64, 2048, 1408, act="gelu", bias=True, skew=1.0),
        # a training step of eight large experts
        _grouped("grouped_train", "bf16", 8192, 8, 4096, 14336, act="silu", train=True, skew=0.5),
        # a training step with empty experts, ragged sizes and odd rows
        _grouped("grouped_odd_train", "fp16", 1531, 37, 520, 1003, act="relu", bias=True, train=True, skew=2.0),
        # scoring a few tokens against a vocabulary of an 8-billion-value model: the weights' bandwidth
        _ce("ce_score", "bf16", 48, 128256, 4096),
        # a training step of that vocabulary with a part of the tokens ignored
        _ce("ce_train", "bf16", 4096, 128256, 4096, ignored=0.1, train=True),
        # a training step on an odd vocabulary and batch
        _ce("ce_odd_train", "fp16", 1001, 32003, 1000, ignored=0.3, train=True),
    ]


def _log(rng, lo, hi, round_to=True):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = max(lo, min(hi, v))
    if round_to and v > 64:  # widths: half are multiples of 64, a quarter of 8, a quarter as they fall
        step = rng.choice((64, 64, 8, 1))
        v = v // step * step
    return v + 64 if v == 3072 else v


def draw(rng):
    while True:
        op = rng.choice(("linear", "grouped", "ce"))
        dtype = rng.choice(("bf16", "fp16"))
        train = rng.random() < 0.5
        act = rng.choice(("none", "relu", "gelu", "silu"))
        if op == "linear":
            c = _linear(None, dtype, _log(rng, 1, 8192, False), _log(rng, 64, 14336), _log(rng, 64, 14336), act,
                        rng.random() < 0.5, rng.random() < 0.5, train)
        elif op == "grouped":
            c = _grouped(None, dtype, _log(rng, 1, 16384, False), _log(rng, 2, 96, False), _log(rng, 64, 4096), _log(rng, 64, 8192), act,
                         rng.random() < 0.5, train, rng.choice((0.0, 0.5, 1.0, 2.0)))
            # the experts' weights, and the plain form's padded rows, stay within the largest listed case's
            if c["e"] * c["k"] * c["n"] > 8 * 4096 * 14336 or c["t"] * c["k"] > 8192 * 4096 * 2:
                continue
        else:
            c = _ce(None, dtype, _log(rng, 1, 4096, False), _log(rng, 1000, 128256, False), _log(rng, 64, 4096),
                    rng.choice((0.0, 0.1, 0.5)), train)
        if work(c)["flops"] <= _MOST_FLOPS:
            return c


def _counts(case, seed):
    """Rows of each expert: weights (rank + 1)^-skew/2 in a shuffled order, so that some experts have none."""
    g = torch.Generator().manual_seed(seed * 7919 + 11)
    e, t = case["e"], case["t"]
    p = torch.arange(1, e + 1, dtype=torch.float64) ** (-0.5 * case["skew"])
    p = p[torch.randperm(e, generator=g)]
    hit = torch.multinomial(p / p.sum(), t, replacement=True, generator=g)
    return torch.bincount(hit, minlength=e)


def _normal(g, shape, scale, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DT[case["dtype"]]
    s = dict(case)
    if case["op"] == "ce":
        t, v, d = case["t"], case["v"], case["d"]
        s["h"] = _normal(g, (t, d), 1.0, dt)
        s["w"] = _normal(g, (v, d), 2.0 / math.sqrt(d), dt)
        s["targets"] = torch.randint(0, v, (t,), generator=g, device="cuda")
        drop = torch.rand(t, generator=g, device="cuda") < case["ignored"]
        s["targets"][drop] = -100
        if case["train"]:  # a weight for each token; fp16 steps scale their loss
            scale = 512.0 if case["dtype"] == "fp16" else 1.0
            s["dloss"] = (0.5 + torch.rand(t, generator=g, device="cuda")) * (scale / t)
        return s
    k, n = case["k"], case["n"]
    if case["op"] == "linear":
        rows, lead = case["m"], ()
    else:
        rows, lead = case["t"], (case["e"],)
        counts = _counts(case, int(seed))
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).cuda()
        s["most"] = int(counts.max())
    s["x"] = _normal(g, (rows, k), 1.0, dt)
    s["w"] = torch.empty(lead + (n, k), dtype=dt, device="cuda")
    for part in s["w"].view(-1, n, k):  # an expert at a time: no 32-bit copy of them all
        part.copy_(torch.randn((n, k), generator=g, device="cuda") * (1.0 / math.sqrt(k)))
    s["b"] = _normal(g, lead + (n,), 0.5, dt) if case["bias"] else None
    s["r"] = _normal(g, (rows, n), 1.0, dt) if case.get("residual") else None
    s["dy"] = _normal(g, (rows, n), 1.0, dt) if case["train"] else None
    return s


# ---- plain forms (32 bits, rounded once at the end) ------------------------

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    return torch.ones_like(z)


def _plain_linear(s):
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.T
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    if not s["train"]:
        return [y.to(dt)]
    dz = s["dy"].float() * _act_grad(z, s["act"])
    out = [y.to(dt), (dz @ w).to(dt), (dz.T @ x).to(dt)]
    if s["b"] is not None:
        out.append(dz.sum(0).to(dt))
    return out


def _plain_grouped(s):
    # every expert's rows padded to the longest, one batched product
    dt = s["x"].dtype
    x, w, off = s["x"].float(), s["w"].float(), s["offsets"]
    at = off[:-1, None] + torch.arange(s["most"], device=x.device)
    there = at < off[1:, None]
    at = at.clamp(max=x.shape[0] - 1)
    xp = x[at] * there[..., None]
    z = torch.bmm(xp, w.transpose(1, 2))
    if s["b"] is not None:
        z = z + s["b"].float()[:, None, :]
    y = _act(z, s["act"])[there]
    if not s["train"]:
        return [y.to(dt)]
    dz = s["dy"].float()[at] * there[..., None] * _act_grad(z, s["act"])
    out = [y.to(dt), torch.bmm(dz, w)[there].to(dt), torch.bmm(dz.transpose(1, 2), xp).to(dt)]
    if s["b"] is not None:
        out.append(dz.sum(1).to(dt))
    return out


def _plain_ce(s):
    dt = s["h"].dtype
    h, w, t = s["h"].float(), s["w"].float(), s["targets"]
    used = t >= 0
    rows, at = torch.arange(t.numel(), device=t.device), t.clamp(min=0)
    logits = h @ w.T
    top = logits.max(1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse = torch.log(total) + top
    loss = torch.where(used, lse[:, 0] - logits[rows, at], 0.0)
    if not s["train"]:
        return [loss]
    e /= total
    e[rows, at] -= 1
    e *= torch.where(used, s["dloss"], 0.0)[:, None]
    return [loss, (e @ w).to(dt), (e.T @ h).to(dt)]


# ---- the library's operators -------------------------------------------------

def _own_linear(s):
    import lossless_float_tensor_gb300 as uz

    if not s["train"]:
        return [uz.linear(s["x"], s["w"], s["b"], activation=s["act"], residual=s["r"])]
    y, z = uz.linear(s["x"], s["w"], s["b"], activation=s["act"], residual=s["r"], save_preact=True)
    dx, dw, db = uz.linear_backward(s["dy"], s["x"], s["w"], z, activation=s["act"], need_db=s["b"] is not None)
    return [y, dx, dw] + ([db] if db is not None else [])


def _own_grouped(s):
    import lossless_float_tensor_gb300 as uz

    if not s["train"]:
        return [uz.grouped_linear(s["x"], s["w"], s["offsets"], s["b"], activation=s["act"])]
    y, z = uz.grouped_linear(s["x"], s["w"], s["offsets"], s["b"], activation=s["act"], save_preact=True)
    dx, dw, db = uz.grouped_linear_backward(s["dy"], s["x"], s["w"], s["offsets"], z, activation=s["act"],
                                            need_db=s["b"] is not None)
    return [y, dx, dw] + ([db] if db is not None else [])


def _own_ce(s):
    import lossless_float_tensor_gb300 as uz

    loss, lse = uz.cross_entropy(s["h"], s["w"], s["targets"])
    if not s["train"]:
        return [loss]
    dh, dw = uz.cross_entropy_backward(s["dloss"], s["h"], s["w"], s["targets"], lse)
    return [loss, dh, dw]


def run(state):
    if own:
        return {"linear": _own_linear, "grouped": _own_grouped, "ce": _own_ce}[state["op"]](state)
    return {"linear": _plain_linear, "grouped": _plain_grouped, "ce": _plain_ce}[state["op"]](state)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    if case["op"] == "ce":
        t, v, d = case["t"], case["v"], case["d"]
        read = 2 * (t * d + v * d) + 8 * t
        if not case["train"]:
            return {"bytes": read + 4 * t, "flops": 2 * t * v * d}
        return {"bytes": read + 4 * t + 4 * t + 2 * (t * d + v * d), "flops": 6 * t * v * d}
    k, n = case["k"], case["n"]
    if case["op"] == "linear":
        rows, experts, live = case["m"], 1, 1
    else:
        rows, experts = case["t"], case["e"]
        # experts with rows, expected over the seeds
        p = [(i + 1) ** (-0.5 * case["skew"]) for i in range(experts)]
        live = sum(1 - (1 - q / sum(p)) ** rows for q in p)
    bias = n if case["bias"] else 0
    res = rows * n if case.get("residual") else 0
    bytes_ = 2 * (rows * k + live * (n * k + bias) + res + rows * n)
    if case["op"] == "grouped":
        bytes_ += 8 * (experts + 1)
    if not case["train"]:
        return {"bytes": bytes_, "flops": 2 * rows * n * k}
    bytes_ += 2 * (rows * n + rows * k + experts * (n * k + bias))
    return {"bytes": bytes_, "flops": 6 * rows * n * k}


# ---- the definitions in 64 bits ------------------------------------------------

_PHI = 1 / math.sqrt(2 * math.pi)


def _exact_block(x, w, b, r, dy, act):
    """One dense block: [y] or [y, dx, dw, db], all in 64 bits."""
    z = torch.einsum("mk,nk->mn", x, w) + (0 if b is None else b)
    if act == "relu":
        y, slope = z.clamp(min=0), torch.heaviside(z, torch.zeros_like(z))
    elif act == "gelu":
        cdf = torch.special.ndtr(z)
        y, slope = z * cdf, cdf + z * _PHI * torch.exp(-z.square() / 2)
    elif act == "silu":
        sg = torch.special.expit(z)
        y, slope = z * sg, sg + z * sg * torch.special.expit(-z)
    else:
        y, slope = z, torch.ones_like(z)
    y = y if r is None else y + r
    if dy is None:
        return [y]
    dz = dy * slope
    return [y, torch.einsum("mn,nk->mk", dz, w), torch.einsum("mn,mk->nk", dz, x), dz.sum(0)]


def exact(case, seed):
    work_flops = work(case)["flops"]
    if work_flops > 3e12:  # 64-bit products run at about 1 TFLOP/s
        return None
    s = prepare(case, seed)
    f64 = lambda v: None if v is None else v.to(torch.float64)  # noqa: E731
    if case["op"] == "linear":
        out = _exact_block(f64(s["x"]), f64(s["w"]), f64(s["b"]), f64(s["r"]), f64(s["dy"]), case["act"])
        return out if case["bias"] else out[:3]
    if case["op"] == "grouped":
        ends = s["offsets"].tolist()
        parts = []
        for e in range(case["e"]):
            cut = slice(ends[e], ends[e + 1])
            parts.append(_exact_block(f64(s["x"][cut]), f64(s["w"][e]), None if s["b"] is None else f64(s["b"][e]), None,
                                      None if s["dy"] is None else f64(s["dy"][cut]), case["act"]))
        out = [torch.cat([p[0] for p in parts])]
        if case["train"]:
            out += [torch.cat([p[1] for p in parts]), torch.stack([p[2] for p in parts])]
            if case["bias"]:
                out.append(torch.stack([p[3] for p in parts]))
        return out
    h, w, t = f64(s["h"]), f64(s["w"]), s["targets"]
    keep = torch.nonzero(t != -100).flatten()
    loss = torch.zeros(t.numel(), dtype=torch.float64, device=h.device)
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for part in keep.split(512):
        logp = torch.log_softmax(torch.einsum("td,vd->tv", h[part], w), 1)
        hit = torch.nn.functional.one_hot(t[part], case["v"])
        loss[part] = -(logp * hit).sum(1)
        if case["train"]:
            dl = (logp.exp() - hit) * s["dloss"][part].to(torch.float64)[:, None]
            dh[part] = torch.einsum("tv,vd->td", dl, w)
            dw += torch.einsum("tv,td->vd", dl, h[part])
    return [loss, dh, dw] if case["train"] else [loss]
