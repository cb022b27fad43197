"""The operators around a paged key-value cache as their users call them, for measurement.

Three groups.  `attn`: attention of one new token for each sequence over the
cache's pages.  `rope`: rotary positions, for serving fused with the store of
keys and values into the pages, for training with the gradient.  `pages`:
reserving, forking, freeing, compacting and copying pages.

A cache is k and v, each [layers, pages, kv heads, page size, head size], with
int32 reference counts for the pages, a table of pages for each sequence and
the sequences' lengths.

With `own` false, run() computes the plain form in 32 bits (angles in 64) from
elementary torch operations; with `own` true it calls the library.
"""
import math

import torch

own = False

if torch.cuda.is_available():  # the plain form's products stay in 32 bits
    torch.backends.cuda.matmul.allow_tf32 = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_BASE = 500000.0  # of the rotary frequencies

# The costliest listed case bounds the drawn ones (bytes of a pass).
_MOST_BYTES = 4.2e9


def _attn(name, dtype, seqs, heads, group, d, page, least, most, cap=0.0, window=0, order="heads"):
    c = {"op": "attn", "dtype": dtype, "seqs": seqs, "heads": heads, "group": group, "d": d, "page": page, "least": least, "most": most,
         "cap": cap, "window": window, "order": order}
    return dict(c, name=name) if name else c


def _rope(name, dtype, t, hq, hkv, d, rot, kind, interleaved=False, scale=1.0, page=16, far=8192):
    c = {"op": "rope", "dtype": dtype, "t": t, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "kind": kind, "interleaved": interleaved,
         "scale": scale, "page": page, "far": far}
    return dict(c, name=name) if name else c


def _pages(name, kind, dtype, layers, pages, heads, page, d, seqs, least, most, new=1):
    c = {"op": "pages", "kind": kind, "dtype": dtype, "layers": layers, "pages": pages, "heads": heads, "page": page, "d": d, "seqs": seqs,
         "least": least, "most": most, "new": new}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short conversation: latency
        _attn("attn_token", "bf16", 1, 8, 4, 128, 16, 400, 400),
        # a batch of conversations of uneven lengths
        _attn("attn_batch", "bf16", 64, 8, 4, 128, 16, 16, 4096),
        # one long document: the length is all there is to split
        _attn("attn_long", "bf16", 1, 8, 8, 128, 64, 131072, 131072),
        # a head of keys for each query head, capped scores, a window, pages by token; lengths of zero and one
        _attn("attn_window", "fp16", 24, 16, 1, 64, 32, 0, 6000, cap=30.0, window=1024, order="tokens"),
        # sizes that fill no tile, pages that end inside one
        _attn("attn_odd", "fp16", 37, 3, 5, 80, 24, 0, 2777),
        # a full server
        _attn("attn_large", "bf16", 128, 8, 4, 128, 16, 1024, 12288),
        # a decoding step's tokens into the cache
        _rope("rope_step", "bf16", 48, 32, 8, 128, 128, "step", far=131072),
        # a prompt into the cache
        _rope("rope_prompt", "bf16", 8192, 32, 8, 128, 128, "prompt"),
        # a training step, a part of each head, neighbouring values paired, amplitude of a stretched context
        _rope("rope_train", "fp16", 8191, 24, 8, 96, 48, "train", interleaved=True, scale=1.1386),
        # a decoding step's pages: some sequences still share their last page
        _pages("pages_step", "reserve", "bf16", 4, 8192, 8, 16, 128, 96, 64, 1024),
        # many answers from one prompt: fork, a token each, page copies, free
        _pages("pages_fork", "fork", "fp16", 4, 2048, 8, 16, 128, 33, 2001, 2001),
        # a pool's used pages moved together, for all layers
        _pages("pages_compact", "compact", "bf16", 4, 16384, 8, 16, 128, 128, 64, 1984),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("attn", "attn", "rope", "pages"))
        dtype = rng.choice(("bf16", "fp16"))
        d = rng.choice((64, 64, 128, 128, 128, 256, 8 * rng.randint(2, 32)))
        if op == "attn":
            most = _log(rng, 1, 131072)
            least = rng.choice((most, 0, rng.randint(0, most)))
            c = _attn(None, dtype, _log(rng, 1, 256), rng.choice((1, 2, 3, 4, 5, 8, 8, 16, 32)), rng.choice((1, 2, 4, 4, 5, 7, 8, 16, 32)), d,
                      rng.choice((1, 8, 16, 16, 24, 32, 64, 128)), least, most, rng.choice((0.0, 0.0, 30.0, 50.0)),
                      rng.choice((0, 0, 0, _log(rng, 16, 8192))), rng.choice(("heads", "heads", "tokens")))
            # the plain form pads every sequence to the longest
            if c["heads"] * c["group"] > 128 or c["seqs"] * most * c["heads"] * d > 2.2e9 or c["seqs"] * most * c["heads"] * c["group"] > 3e8:
                continue
        elif op == "rope":
            hkv = rng.choice((1, 2, 4, 8, 8, 16))
            rot = rng.choice((d, d, d, d // 2 // 2 * 2, 2 * rng.randint(1, d // 2)))
            c = _rope(None, dtype, _log(rng, 1, 16384), hkv * rng.choice((1, 2, 4, 8)), hkv, d, rot, rng.choice(("step", "prompt", "train")),
                      rng.random() < 0.4, rng.choice((1.0, 1.0, 1.25)), rng.choice((8, 16, 24, 64)), _log(rng, 1024, 2000000))
            if c["t"] * c["hq"] * d > 2 ** 28 or (c["kind"] == "step" and c["t"] > 512):
                continue
        else:
            seqs, page = _log(rng, 2, 512), rng.choice((8, 16, 16, 24, 32, 64))
            most = _log(rng, 1, 16384)
            new = rng.choice((1, 1, _log(rng, 1, 2048)))
            need = seqs * (-(-(most + new) // page) + 1) + 8
            layers, heads = rng.choice((1, 2, 4, 8, 16)), rng.choice((1, 2, 4, 8))
            c = _pages(None, rng.choice(("reserve", "fork", "compact", "send")), dtype, layers, int(need * rng.choice((1.0, 1.3, 2.0))) + 1, heads, page, d,
                       seqs, rng.randint(1, most), most, new)
            if c["pages"] > 300000 or c["pages"] * layers * heads * page * d > 1.6e9:
                continue
        if work(c)["bytes"] <= _MOST_BYTES:
            return c


# ---- inputs ------------------------------------------------------------------

def _normal(g, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for part in flat.split(1 << 28):  # no 32-bit copy of a whole pool
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda") * scale)
    return out


def _spread(case):
    """Lengths of the sequences, evenly from the least to the most; zero and one occur where they may."""
    n, lo, hi = case["seqs"], case["least"], case["most"]
    out = [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]
    if lo == 0 and n > 3:
        out[-2] = min(1, hi)
    return out


def _lengths(case, seed):
    g = torch.Generator().manual_seed(seed * 7919 + 5)
    return torch.tensor(_spread(case))[torch.randperm(case["seqs"], generator=g)]


def _counts(case):
    """New tokens of the sequences: one each, or evenly up to the most."""
    n, new = case["seqs"], case["new"]
    return [1] * n if new == 1 else [new * i // (n - 1) for i in range(n)]


def _table(counts, width, pages, seed):
    """Page tables of sequences with `counts` pages each: pages in a shuffled order, page 0 the first; -1 behind."""
    g = torch.Generator().manual_seed(seed * 104729 + 3)
    order = torch.randperm(pages, generator=g)
    order[order == 0] = order[0].clone()
    order[0] = 0
    at = torch.arange(width)
    there = at < counts[:, None]
    table = torch.full((counts.numel(), width), -1, dtype=torch.int64)
    table[there] = order[: int(counts.sum())]
    return table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DT[case["dtype"]]
    s = dict(case)
    return {"attn": _prepare_attn, "rope": _prepare_rope, "pages": _prepare_pages}[case["op"]](case, int(seed), g, dt, s)


def _prepare_attn(case, seed, g, dt, s):
    n, page = _lengths(case, seed), case["page"]
    counts = -(-n // page)
    pages = int(counts.sum()) + 8
    if case["order"] == "heads":  # a head's tokens of a page lie together
        shape = (pages, case["heads"], page, case["d"])
        s["k"], s["v"] = _normal(g, shape, dt), _normal(g, shape, dt)
    else:  # a token's heads lie together
        shape = (pages, page, case["heads"], case["d"])
        s["k"], s["v"] = _normal(g, shape, dt).transpose(1, 2), _normal(g, shape, dt).transpose(1, 2)
    s["table"] = _table(counts, max(1, -(-case["most"] // page)), pages, seed).int().cuda()
    s["lengths"] = n.int().cuda()
    # scores with a deviation of 2: some tokens carry much of the weight
    s["q"] = _normal(g, (case["seqs"], case["heads"] * case["group"], case["d"]), dt, 2.0)
    return s


def _frequencies(rot):
    return _BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


def _prepare_rope(case, seed, g, dt, s):
    t, hq, hkv, d, page = case["t"], case["hq"], case["hkv"], case["d"], case["page"]
    s["freqs"] = _frequencies(case["rot"])
    if case["kind"] == "train":  # positions start again with each packed document
        s["q"], s["k"] = _normal(g, (t, hq, d), dt), _normal(g, (t, hkv, d), dt)
        s["dq"], s["dk"] = _normal(g, (t, hq, d), dt), _normal(g, (t, hkv, d), dt)
        s["positions"] = torch.arange(t, device="cuda") % (1000 + seed % 97)
        return s
    qkv = _normal(g, (t, (hq + 2 * hkv) * d), dt)  # as one projection gives them
    s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in qkv.split((hq * d, hkv * d, hkv * d), 1))
    if case["kind"] == "step":  # a token of each sequence, each in a page of its own
        pages = t + 8
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda")
        s["slots"] = torch.randperm(pages, generator=g, device="cuda")[:t] * page + s["positions"] % page
    else:  # one prompt, in shuffled pages, the first page entered before
        pages = -(-(t + page) // page) + 8
        s["positions"] = torch.arange(t, device="cuda") + seed % page
        s["slots"] = torch.randperm(pages, generator=g, device="cuda")[s["positions"] // page] * page + s["positions"] % page
    s["kp"], s["vp"] = _normal(g, (pages, hkv, page, d), dt), _normal(g, (pages, hkv, page, d), dt)
    return s


def _prepare_pages(case, seed, g, dt, s):
    seqs, page, pages, kind = case["seqs"], case["page"], case["pages"], case["kind"]
    n = _lengths(case, seed)
    counts = -(-n // page)
    width = -(-(case["most"] + case["new"]) // page) + 1
    if kind == "fork":  # one prompt, the other sequences unused
        n[:], counts[:] = 0, 0
        n[0], counts[0] = case["most"], -(-case["most"] // page)
    table = _table(counts, width, pages, seed)
    if kind == "reserve":  # every fourth sequence was forked from the one before it and has not gone on
        for i in range(3, seqs, 4):
            table[i], n[i] = table[i - 1], n[i - 1]
    refs = torch.bincount(table[table >= 0], minlength=pages)
    s["saved"] = torch.cat([refs, table.flatten(), n]).int().cuda()
    s["live"] = s["saved"].clone()
    s["refs"], s["lengths"] = s["live"][:pages], s["live"][pages + seqs * width:]
    s["table"] = s["live"][pages: pages + seqs * width].view(seqs, width)
    shape = (case["layers"], pages, case["heads"], page, case["d"])
    s["k"], s["v"] = _normal(g, shape, dt), _normal(g, shape, dt)
    if kind == "reserve":
        c = torch.tensor(_counts(case), dtype=torch.int32)
        s["counts"] = c[torch.randperm(seqs, generator=torch.Generator().manual_seed(seed))].cuda()
        s["tokens"] = -(-int(c.sum()) // 8) * 8  # a step's batch is padded
    elif kind == "fork":
        s["parents"] = torch.zeros(seqs - 1, dtype=torch.int32, device="cuda")
        s["children"] = torch.arange(1, seqs, dtype=torch.int32, device="cuda")
        s["counts"], s["tokens"] = torch.ones(seqs, dtype=torch.int32, device="cuda"), seqs - 1
        s["counts"][0] = 0
    elif kind == "send":  # the pages of every sequence, one after another, into a buffer to be sent
        a = table[table >= 0]
        s["pairs"] = torch.stack([a, torch.arange(a.numel())], 1).int().cuda()
        out = (case["layers"], a.numel(), case["heads"], page, case["d"])
        s["ko"], s["vo"] = torch.zeros(out, dtype=dt, device="cuda"), torch.zeros(out, dtype=dt, device="cuda")
    return s


# ---- plain forms (32 bits, rounded once at the end) ------------------------

def _plain_attn(s):
    n, at, page = s["lengths"], s["table"].long().clamp(min=0), s["page"]
    rows, width = at.shape
    take = lambda x: x[at].transpose(1, 2).reshape(rows, s["heads"], width * page, s["d"]).float()  # noqa: E731
    q = s["q"].float().view(rows, s["heads"], s["group"], s["d"])
    z = q @ take(s["k"]).transpose(2, 3) * (1 / math.sqrt(s["d"]))
    if s["cap"]:
        z = s["cap"] * torch.tanh(z / s["cap"])
    pos = torch.arange(width * page, device=n.device)
    live = pos < n[:, None]
    if s["window"]:
        live &= pos >= n[:, None] - s["window"]
    live = live[:, None, None, :]
    z = torch.where(live, z, -math.inf)
    top = z.max(3, keepdim=True).values
    p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    o = p @ take(s["v"]) / torch.where(total == 0, 1.0, total)
    return [o.view(s["q"].shape).to(s["q"].dtype)]


def _plain_rotate(x, positions, s, sign=1.0):
    rot, half = s["rot"], s["rot"] // 2
    a = positions.double()[:, None] * s["freqs"]
    c, sn = (torch.cos(a) * s["scale"]).float()[:, None, :], (torch.sin(a) * (sign * s["scale"])).float()[:, None, :]
    y = x.float()
    if s["interleaved"]:
        u, w = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([u * c - w * sn, u * sn + w * c], -1).flatten(-2)
    else:
        u, w = y[..., :half], y[..., half:rot]
        turned = torch.cat([u * c - w * sn, u * sn + w * c], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_rope(s):
    pos = s["positions"]
    if s["kind"] == "train":
        return [_plain_rotate(s["q"], pos, s), _plain_rotate(s["k"], pos, s), _plain_rotate(s["dq"], pos, s, -1.0), _plain_rotate(s["dk"], pos, s, -1.0)]
    q, k = _plain_rotate(s["q"], pos, s), _plain_rotate(s["k"], pos, s)
    page, off = s["slots"] // s["page"], s["slots"] % s["page"]
    s["kp"][page, :, off] = k
    s["vp"][page, :, off] = s["v"]
    return [q, s["kp"], s["vp"]]


def _plain_copy(k, v, pairs):
    # a pair of -1 stands for none: page 0, which nothing is copied to, onto itself
    src, to = pairs[:, 0].long().clamp(min=0), pairs[:, 1].long().clamp(min=0)
    k[:, to] = k[:, src]
    v[:, to] = v[:, src]


def _place(values, where, at, size):
    """A list of `size` whose entry at[i] is values[i] wherever where[i]; -1 elsewhere."""
    out = torch.full((size + 1,), -1, dtype=torch.int64, device=values.device)
    out[torch.where(where, at, size)] = values
    return out[:size]


def _plain_reserve(s):
    refs, table, n, page, count = s["refs"], s["table"], s["lengths"].long(), s["page"], s["counts"].long()
    pages, width = refs.numel(), table.shape[1]
    have, want = (n + page - 1) // page, (n + count + page - 1) // page
    last = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long()
    cow = (count > 0) & (n % page != 0) & (refs[last.clamp(min=0)] > 1)
    need = want - have + cow
    first = need.cumsum(0) - need
    free = refs == 0
    ids = torch.arange(pages, device=refs.device)
    lowest = _place(ids, free, free.cumsum(0) - 1, pages)
    col = torch.arange(width, device=refs.device)
    moved = cow[:, None] & (col == have[:, None] - 1)
    grown = (col >= have[:, None]) & (col < want[:, None])
    at = torch.where(moved, first[:, None], (first + cow - have)[:, None] + col)
    got = lowest[at.clamp(0, pages - 1)].int()
    copies = torch.where(cow[:, None], torch.stack([last, lowest[first.clamp(max=pages - 1)]], 1), -1).int()
    table.copy_(torch.where(moved | grown, got, table))
    refs.copy_(torch.where(free & (free.cumsum(0) <= need.sum()), 1, refs))
    refs.index_add_(0, last.clamp(min=0), -cow.int())
    ends = count.cumsum(0)
    i = torch.arange(s["tokens"], device=refs.device)
    real = i < ends[-1]
    row = torch.searchsorted(ends, i, right=True).clamp(max=count.numel() - 1)
    positions = torch.where(real, n[row] + i - (ends - count)[row], 0)
    slots = torch.where(real, table[row, positions // page] * page + positions % page, -1)
    s["lengths"] += s["counts"]
    return slots, positions, copies


def _plain_fork(s, parents, children):
    rows, n = s["table"][parents.long()], s["lengths"][parents.long()]
    there = torch.arange(rows.shape[1], device=rows.device) < ((n + s["page"] - 1) // s["page"])[:, None]
    s["refs"].index_add_(0, rows.clamp(min=0).flatten(), there.flatten().int())
    s["table"][children.long()] = torch.where(there, rows, -1)
    s["lengths"][children.long()] = n


def _plain_free(s, rows):
    rows = rows.long()
    held, n = s["table"][rows], s["lengths"][rows]
    there = torch.arange(held.shape[1], device=held.device) < ((n + s["page"] - 1) // s["page"])[:, None]
    s["refs"].index_add_(0, held.clamp(min=0).flatten(), -there.flatten().int())
    s["table"][rows] = -1
    s["lengths"][rows] = 0


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    pages = refs.numel()
    used, ids = refs > 0, torch.arange(pages, device=refs.device)
    low = ids < used.sum()
    hole, move = ~used & low, used & ~low
    holes = _place(ids, hole, hole.cumsum(0) - 1, pages)
    rank = move.cumsum(0) - 1
    goes = torch.where(move, holes[rank.clamp(min=0)], ids)
    moves = torch.stack([_place(ids, move, rank, pages // 2), _place(goes, move, rank, pages // 2)], 1).int()
    table.copy_(torch.where(table >= 0, goes[table.long().clamp(min=0)].int(), table))
    refs.copy_(torch.zeros_like(refs).index_add_(0, goes, refs))
    return moves


def _plain_pages(s):
    kind = s["kind"]
    if kind == "send":
        src, to = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
        s["ko"][:, to] = s["k"][:, src]
        s["vo"][:, to] = s["v"][:, src]
        return [s["ko"], s["vo"]]
    if kind == "fork":
        _plain_fork(s, s["parents"], s["children"])
        slots, positions, copies = _plain_reserve(s)
        _plain_copy(s["k"], s["v"], copies)
        _plain_free(s, s["children"])
        out = [slots, positions, copies]
    elif kind == "reserve":
        s["live"].copy_(s["saved"])
        out = list(_plain_reserve(s))
        _plain_copy(s["k"], s["v"], out[2])
    else:
        s["live"].copy_(s["saved"])
        out = [_plain_compact(s)]
        _plain_copy(s["k"], s["v"], out[0])
    return out + [s["refs"], s["table"], s["lengths"], s["k"], s["v"]]


# ---- the library's operators -------------------------------------------------

def _own_attn(s):
    import lossless_float_tensor_gb300 as uz

    return [uz.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lengths"], softcap=s["cap"], window=s["window"])]


def _own_rope(s):
    import lossless_float_tensor_gb300 as uz

    if s["kind"] == "train":
        return [*uz.rotary(s["q"], s["k"], s["positions"], s["freqs"], interleaved=s["interleaved"], scale=s["scale"]),
                *uz.rotary_backward(s["dq"], s["dk"], s["positions"], s["freqs"], interleaved=s["interleaved"], scale=s["scale"])]
    q = uz.rotary_append(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["kp"], s["vp"], s["slots"], interleaved=s["interleaved"],
                         scale=s["scale"])
    return [q, s["kp"], s["vp"]]


def _own_pages(s):
    import lossless_float_tensor_gb300 as uz

    state, kind = (s["refs"], s["table"], s["lengths"]), s["kind"]
    if kind == "send":
        uz.cache_copy(s["k"], s["v"], s["pairs"], to=(s["ko"], s["vo"]))
        return [s["ko"], s["vo"]]
    if kind == "fork":
        uz.cache_fork(*state, s["parents"], s["children"], s["page"])
        out = list(uz.cache_reserve(*state, s["counts"], s["tokens"], s["page"]))
        uz.cache_copy(s["k"], s["v"], out[2])
        uz.cache_free(*state, s["children"], s["page"])
    elif kind == "reserve":
        s["live"].copy_(s["saved"])
        out = list(uz.cache_reserve(*state, s["counts"], s["tokens"], s["page"]))
        uz.cache_copy(s["k"], s["v"], out[2])
    else:
        s["live"].copy_(s["saved"])
        out = [uz.cache_compact(*state, s["page"])]
        uz.cache_copy(s["k"], s["v"], out[0])
    return out + [s["refs"], s["table"], s["lengths"], s["k"], s["v"]]


def run(state):
    if own:
        return {"attn": _own_attn, "rope": _own_rope, "pages": _own_pages}[state["op"]](state)
    return {"attn": _plain_attn, "rope": _plain_rope, "pages": _plain_pages}[state["op"]](state)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    d = case["d"]
    if case["op"] == "attn":
        tokens = sum(min(n, case["window"] or n) for n in _spread(case))
        hq = case["heads"] * case["group"]
        return {"bytes": 4 * tokens * case["heads"] * d + 4 * case["seqs"] * hq * d + 4 * tokens / case["page"] + 4 * case["seqs"],
                "flops": 4 * tokens * hq * d}
    if case["op"] == "rope":
        t, hq, hkv = case["t"], case["hq"], case["hkv"]
        if case["kind"] == "train":
            return {"bytes": 8 * t * (hq + hkv) * d + 8 * t, "flops": 6 * t * (hq + hkv) * case["rot"]}
        return {"bytes": 4 * t * (hq + 2 * hkv) * d + 16 * t, "flops": 3 * t * (hq + hkv) * case["rot"]}
    seqs, page, pages, kind = case["seqs"], case["page"], case["pages"], case["kind"]
    whole = 4 * case["layers"] * case["heads"] * page * d  # keys and values of a page, over all layers
    held = sum(-(-n // page) for n in _spread(case))
    if kind == "send":
        return {"bytes": 2 * whole * held + 8 * held, "flops": 0}
    if kind == "fork":  # the children's rows are written and cleared, their pages counted twice, one page copied for each
        return {"bytes": (seqs - 1) * (2 * whole + 16 * -(-case["most"] // page) + 48) + 4 * pages, "flops": 0}
    if kind == "reserve":  # a quarter of the sequences, and those that they share with, copy their last page
        tokens = sum(_counts(case))
        return {"bytes": seqs // 2 * 2 * whole * (1 - 1 / page) + 16 * tokens + 32 * seqs + 4 * pages, "flops": 0}
    moved = held * (1 - held / pages)  # used pages above as many lowest ones as are used
    return {"bytes": 2 * whole * moved + 8 * moved + 8 * pages + 8 * held, "flops": 0}


# ---- the definitions in 64 bits ------------------------------------------------

def _exact_attn(case, s):
    outs = []
    for i, n in enumerate(s["lengths"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        spot = torch.arange(lo, n, device="cuda")
        page, off = s["table"][i].long()[spot // case["page"]], spot % case["page"]
        k, v = (x[page, :, off].to(torch.float64) for x in (s["k"], s["v"]))  # [tokens, heads, d]
        q = s["q"][i].to(torch.float64).reshape(case["heads"], case["group"], case["d"])
        z = torch.einsum("hgd,nhd->hgn", q, k) / case["d"] ** 0.5
        if case["cap"]:
            z = torch.tanh(z / case["cap"]) * case["cap"]
        w = torch.softmax(z, -1) if n else z
        outs.append(torch.einsum("hgn,nhd->hgd", w, v).reshape(-1, case["d"]))
    return [torch.stack(outs)]


def _exact_turned(case, s, x, back=False):
    """The rotation as a product of complex numbers."""
    angle = torch.outer(s["positions"].to(torch.float64), s["freqs"]) * (-1 if back else 1)
    by = torch.polar(torch.full_like(angle, case["scale"]), angle)[:, None]
    out = x.to(torch.float64).clone()
    part = out[..., : case["rot"]]
    pair = part.unflatten(-1, (-1, 2)) if case["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * by)
    out[..., : case["rot"]] = turned.flatten(-2) if case["interleaved"] else turned.transpose(-1, -2).flatten(-2)
    return out


def _exact_rope(case, s):
    q, k = _exact_turned(case, s, s["q"]), _exact_turned(case, s, s["k"])
    if case["kind"] == "train":
        return [q, k, _exact_turned(case, s, s["dq"], True), _exact_turned(case, s, s["dk"], True)]
    pools = []
    for pool, rows in ((s["kp"], k), (s["vp"], s["v"].to(torch.float64))):
        by_token = pool.to(torch.float64).transpose(1, 2).flatten(0, 1)  # [slots, heads, d]
        by_token[s["slots"]] = rows
        pools.append(by_token.unflatten(0, (-1, case["page"])).transpose(1, 2))
    return [q] + pools


def _exact_pages(case, s):
    """The pools after the calls, from lists of pages kept on the host."""
    if case["pages"] * case["layers"] * case["heads"] * case["page"] * case["d"] > 4e9:
        return None
    page, f64 = case["page"], torch.float64
    k, v = s["k"].to(f64), s["v"].to(f64)
    if case["kind"] == "send":
        src = s["pairs"][:, 0].long()
        return [k[:, src], v[:, src]]
    refs, table, n = s["refs"].tolist(), s["table"].tolist(), s["lengths"].tolist()
    copies = []
    if case["kind"] == "compact":
        used = [p for p in range(case["pages"]) if refs[p]]
        holes = [p for p in range(len(used)) if not refs[p]]
        copies = list(zip([p for p in used if p >= len(used)], holes))
    else:
        if case["kind"] == "fork":
            for c in range(1, case["seqs"]):
                table[c], n[c] = list(table[0]), n[0]
            for p in table[0][: -(-n[0] // page)]:
                refs[p] += case["seqs"] - 1
        spare = iter([p for p in range(case["pages"]) if not refs[p]])
        for i, c in enumerate(s["counts"].tolist()):
            have = -(-n[i] // page)
            if c and n[i] % page and refs[table[i][have - 1]] > 1:
                copies.append((table[i][have - 1], next(spare)))
            for _ in range(-(-(n[i] + c) // page) - have):
                next(spare)
    if copies:
        src, to = (list(x) for x in zip(*copies))
        k[:, to], v[:, to] = k[:, src], v[:, src]
    whole = [None] if case["kind"] == "compact" else [None] * 3
    return whole + [None] * 3 + [k, v]


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "rope": _exact_rope, "pages": _exact_pages}[case["op"]](case, s)
