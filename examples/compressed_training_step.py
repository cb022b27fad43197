"""One training step of a small mixture-of-experts block whose weights live
compressed, then single-token serving from the same containers.

The weights of a gate projection, of eight experts and of a vocabulary are kept
as containers (about two thirds of their size).  The step decompresses each
weight into a workspace on a side stream while the products before it run,
multiplies, takes the loss over the vocabulary without keeping its logits, runs
the gradients, and compresses each gradient as it would be sent.

    python examples/compressed_training_step.py [--tokens 2048] [--width 1024] [--vocab 32000]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_float_tensor_gb300 as uz  # noqa: E402

EXPERTS = 8


class Kept:
    """A weight held as a container; open() decompresses it on `stream`."""

    def __init__(self, w):
        self.shape, self.dtype = w.shape, w.dtype
        buf, size = uz.compress(w)
        self.box = uz.compressed_bytes(buf, size).clone()

    def open(self, stream):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            w = uz.decompress(self.box, self.dtype, self.shape.numel(), check=False).view(self.shape)
            ready = torch.cuda.Event()
            ready.record(stream)
        w.record_stream(torch.cuda.current_stream())
        return w, ready


def use(opened):
    w, ready = opened
    torch.cuda.current_stream().wait_event(ready)
    return w


def make_model(width, hidden, vocab, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5).to(dtype)  # noqa: E731
    weights = {"gate": rand(hidden, width), "up": rand(EXPERTS, width, hidden), "head": rand(vocab, width)}
    bias = torch.zeros(hidden, dtype=dtype, device="cuda")
    return weights, {name: Kept(w) for name, w in weights.items()}, bias


def sort_by_expert(t):
    """Tokens in the order of their experts, and where each expert's begin (a
    fixed assignment stands in for a router)."""
    owner = torch.arange(t, device="cuda") * 2654435761 % 4294967296 % EXPERTS
    order = torch.argsort(owner, stable=True)
    counts = torch.bincount(owner, minlength=EXPERTS)
    return order, torch.cat([counts.new_zeros(1), counts.cumsum(0)])


def forward(kept, bias, x, offsets, side, save=False):
    """Gate projection with silu, the tokens' experts, added to the input."""
    gate, up = kept["gate"].open(side), kept["up"].open(side)
    a = uz.linear(x, use(gate), bias, activation="silu", save_preact=save)
    a, z = a if save else (a, None)
    y = uz.grouped_linear(a, use(up), offsets)
    return y + x, (gate[0], up[0], a, z)


def train_step(kept, bias, x, offsets, targets, side):
    head = kept["head"].open(side)
    h, (gate, up, a, z) = forward(kept, bias, x, offsets, side, save=True)
    w = use(head)
    loss, lse = uz.cross_entropy(h, w, targets)
    used = targets != -100
    dloss = used.float() / used.sum()
    dh, dhead = uz.cross_entropy_backward(dloss, h, w, targets, lse)
    da, dup, _ = uz.grouped_linear_backward(dh, a, up, offsets, need_db=False)
    dx, dgate, dbias = uz.linear_backward(da, x, gate, z, activation="silu")
    grads = {"gate": dgate, "up": dup, "head": dhead}
    sent = {name: uz.compress(g) for name, g in grads.items()}
    return loss, dx + dh, {**grads, "bias": dbias}, sent


def serve_token(kept, bias, x, offsets, side):
    """The next token's loss against every class is not needed: the greedy
    choice is the class of the largest logit."""
    h, _ = forward(kept, bias, x, offsets, side)
    return uz.linear(h, use(kept["head"].open(side))).argmax(1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args(argv)
    dtype = torch.bfloat16
    weights, kept, bias = make_model(a.width, a.hidden, a.vocab, dtype)
    raw = sum(2 * w.numel() for w in weights.values())
    boxes = sum(k.box.numel() for k in kept.values())
    print(f"weights: {raw / 1e6:.1f} MB, kept in {boxes / 1e6:.1f} MB ({boxes / raw:.3f})")
    g = torch.Generator(device="cuda").manual_seed(1)
    order, offsets = sort_by_expert(a.tokens)
    x = torch.randn(a.tokens, a.width, generator=g, device="cuda").to(dtype)[order]
    targets = torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda")[order]
    targets[::10] = -100  # a prompt's tokens, say
    side = torch.cuda.Stream()
    loss, dx, grads, sent = train_step(kept, bias, x, offsets, targets, side)
    torch.cuda.synchronize()
    mean = float(loss.sum() / (targets != -100).sum())
    size = sum(int(s.item()) for _, s in sent.values())
    print(f"training step: mean loss {mean:.4f}, gradients of {raw / 1e6:.1f} MB sent in {size / 1e6:.1f} MB ({size / raw:.3f})")
    one = torch.tensor([0, 1] + [1] * (EXPERTS - 1), device="cuda")
    token = serve_token(kept, bias, x[:1], one, side)
    print(f"next class for one token: {int(token.item())}")
    return weights, kept, bias, x, offsets, targets, loss, dx, grads, sent, token


if __name__ == "__main__":
    main()
