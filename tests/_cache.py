"""64-bit definitions of the cache operators, the error bounds that their tests
use, and a cache kept in lists on the host (torch, any device)."""
import math

import torch

from tests._products import ROUND, TINY


def pools(g, pages, heads, page, d, dtype, order="heads", scale=1.0):
    """k and v pools [pages, heads, page, d]; order "tokens": a token's heads lie together."""
    shape = (pages, heads, page, d) if order == "heads" else (pages, page, heads, d)
    out = [(torch.randn(shape, generator=g, device="cuda") * scale).to(dtype) for _ in range(2)]
    return out if order == "heads" else [x.transpose(1, 2) for x in out]


def tables(lengths, page, pages, seed=0, width=None, fill=-1):
    """int32 table with shuffled pages for each sequence, and int32 lengths, on the GPU."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // page) for n in lengths]
    order = torch.randperm(pages, generator=g).tolist()
    width = width or max(1, max(counts, default=1))
    table = torch.full((len(lengths), width), fill, dtype=torch.int32)
    for i, c in enumerate(counts):
        table[i, :c] = torch.tensor([order.pop() for _ in range(c)], dtype=torch.int32)
    return table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda()


def attention64(q, k, v, table, lengths, scale=None, softcap=0.0, window=0):
    """(out, lse, bound of |out - computed|, bound of |lse - computed|).

    A score is off by the 32-bit sum of d products (each addition by at most
    2^-23 of the magnitudes so far) and 2^-21 of itself for the scaling, of the
    cap for its exponential.  A weight is off by twice that and 2^-20 for the
    exponential, and rounded to the type, relative to the largest (fp16: by no
    less than 2^-25); sums over tokens run in 32 bits; the result is rounded
    once."""
    dt = q.dtype
    u, tiny = ROUND[dt], TINY[dt]
    s, hq, d = q.shape
    heads, page = k.shape[1], k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, lse = torch.zeros(s, hq, d, dtype=torch.float64, device=q.device), torch.full((s, hq), -math.inf, dtype=torch.float64, device=q.device)
    off, off_lse = torch.full_like(out, tiny), torch.full_like(lse, tiny)
    for i, n in enumerate(lengths.tolist()):
        lo = max(0, n - window) if window else 0
        if n == 0:
            continue
        t = torch.arange(lo, n, device=q.device)
        at = table[i].long()[t // page]
        kk, vv = k[at, :, t % page].double(), v[at, :, t % page].double()  # [n, heads, d]
        qq = q[i].double().view(heads, hq // heads, d)
        z = torch.einsum("hgd,nhd->hgn", qq, kk) * scale
        slip = (d + 4) * 2.0 ** -23 * abs(scale) * torch.einsum("hgd,nhd->hgn", qq.abs(), kk.abs()) + 2.0 ** -21 * z.abs()
        if softcap:
            z = softcap * torch.tanh(z / softcap)
            slip = slip + 2.0 ** -20 * softcap
        w = torch.softmax(z, -1)
        o = torch.einsum("hgn,nhd->hgd", w, vv)
        mag = torch.einsum("hgn,nhd->hgd", w, vv.abs())
        worst = slip.amax(-1, keepdim=True)
        each = u + 4 * worst + 2.0 ** -19 + (n - lo + 8) * 2.0 ** -23
        low = (n - lo) * 2.0 ** -25 * vv.abs().amax(0)[:, None] if dt == torch.float16 else 0.0
        err = mag * each + low
        out[i], lse[i] = o.reshape(hq, d), torch.logsumexp(z, -1).reshape(hq)
        off[i] = (u * (o.abs() + err) + err + tiny).reshape(hq, d)
        off_lse[i] = (2 * worst[..., 0] + 2.0 ** -20 * (2 + torch.logsumexp(z, -1).abs()) + (n - lo + 8) * 2.0 ** -23).reshape(hq)
    return out, lse, off, off_lse


def rotary64(x, positions, freqs, interleaved=False, scale=1.0, sign=1.0):
    """(y, bound of |y - computed|): cosines and sines off by 2^-20 (the angle in
    turns to 32 bits, the functions to a few units), two products and a sum in 32
    bits, rounded once; copied values exact."""
    rot, half = 2 * freqs.numel(), freqs.numel()
    a = positions.double()[:, None] * freqs
    c, s = torch.cos(a)[:, None] * scale, torch.sin(a)[:, None] * (scale * sign)
    y, mag = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    cut = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    u, w = x.double()[..., cut[0]], x.double()[..., cut[1]]
    y[..., cut[0]], y[..., cut[1]] = u * c - w * s, u * s + w * c
    mag[..., cut[0]] = mag[..., cut[1]] = (u.abs() + w.abs()) * abs(scale)
    off = mag * 2.0 ** -20
    rounding, tiny = ROUND[x.dtype], TINY[x.dtype]
    return y, rounding * (y.abs() * (mag > 0) + off) + off + tiny


class Refused(Exception):
    pass


class ListCache:
    """The state of a cache in lists, by the definition of each operation."""

    def __init__(self, pages, page, seqs, width):
        self.page, self.width = page, width
        self.refs, self.rows, self.lengths = [0] * pages, [[] for _ in range(seqs)], [0] * seqs

    def reserve(self, counts, tokens):
        if sum(counts) > tokens or min(counts, default=0) < 0:
            raise Refused("invalid")
        free = [p for p, r in enumerate(self.refs) if r == 0]
        refs, rows, lengths = list(self.refs), [list(r) for r in self.rows], list(self.lengths)
        slots, positions, copies = [], [], [[-1, -1] for _ in counts]
        for i, c in enumerate(counts):
            n = lengths[i]
            if n + c > self.width * self.page:
                raise Refused("capacity")
            if c and n % self.page and self.refs[rows[i][-1]] > 1:
                if not free:
                    raise Refused("capacity")
                copies[i] = [rows[i][-1], free[0]]
                refs[rows[i][-1]] -= 1
                rows[i][-1] = free.pop(0)
                refs[rows[i][-1]] = 1
            for t in range(n, n + c):
                if t // self.page == len(rows[i]):
                    if not free:
                        raise Refused("capacity")
                    rows[i].append(free.pop(0))
                    refs[rows[i][-1]] = 1
                slots.append(rows[i][t // self.page] * self.page + t % self.page)
                positions.append(t)
            lengths[i] = n + c
        self.refs, self.rows, self.lengths = refs, rows, lengths
        pad = tokens - len(slots)
        return slots + [-1] * pad, positions + [0] * pad, copies

    def fork(self, parents, children):
        pairs = [(p, c) for p, c in zip(parents, children) if (p, c) != (-1, -1)]
        kids = [c for _, c in pairs]
        if any(not 0 <= x < len(self.rows) for pc in pairs for x in pc) or len(set(kids)) < len(kids):
            raise Refused("invalid")
        if any(self.lengths[c] for c in kids) or any(p in kids for p, _ in pairs):
            raise Refused("invalid")
        for p, c in pairs:
            self.rows[c], self.lengths[c] = list(self.rows[p]), self.lengths[p]
            for x in self.rows[p]:
                self.refs[x] += 1

    def free(self, sequences):
        listed = [s for s in sequences if s != -1]
        if any(not 0 <= s < len(self.rows) for s in listed) or len(set(listed)) < len(listed):
            raise Refused("invalid")
        for s in listed:
            for x in self.rows[s]:
                self.refs[x] -= 1
            self.rows[s], self.lengths[s] = [], 0

    def compact(self):
        used = [p for p, r in enumerate(self.refs) if r]
        moves = list(zip([p for p in used if p >= len(used)], [p for p in range(len(used)) if not self.refs[p]]))
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        return [list(m) for m in moves] + [[-1, -1]] * (len(self.refs) // 2 - len(moves))


def state(pages, seqs, width):
    """refs, table and lengths of a new cache."""
    return (torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.zeros(seqs, width, dtype=torch.int32, device="cuda"),
            torch.zeros(seqs, dtype=torch.int32, device="cuda"))


def same_state(lists, refs, table, lengths):
    assert refs.tolist() == lists.refs
    assert lengths.tolist() == lists.lengths
    for row, want in zip(table.tolist(), lists.rows):
        assert row[:len(want)] == want
