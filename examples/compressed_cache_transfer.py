"""A prompt's key-value cache, sent compressed from the server that read the
prompt to one that decodes several answers from it.

The prompt server projects the prompt, stores rotated keys and values into the
pages of its cache, gathers the prompt's pages into one buffer and compresses
it.  The token server decompresses the buffer into pages of its own, forks the
prompt into as many sequences as answers are wanted (they share its pages, and
copy the last one when they write to it), and decodes a token of each at a time.

    python examples/compressed_cache_transfer.py [--prompt 3001] [--answers 4] [--tokens 8] [--layers 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_float_tensor_gb300 as uz  # noqa: E402

PAGE, HEADS, GROUP, D = 16, 4, 4, 128  # tokens of a page, key heads, query heads of each, values of a head


class Cache:
    """Pools for all layers, and the state: reference counts, page tables, lengths."""

    def __init__(self, layers, pages, sequences, width, dtype):
        self.k = torch.zeros(layers, pages, HEADS, PAGE, D, dtype=dtype, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.state = (torch.zeros(pages, dtype=torch.int32, device="cuda"),
                      torch.zeros(sequences, width, dtype=torch.int32, device="cuda"),
                      torch.zeros(sequences, dtype=torch.int32, device="cuda"))

    def reserve(self, counts, tokens):
        """Room for new tokens; pages that are shared and written to are copied, for all layers."""
        slots, positions, copies = uz.cache_reserve(*self.state, counts, tokens, PAGE, check=True)
        uz.cache_copy(self.k, self.v, copies, check=True)
        return slots, positions


def layer_inputs(x, w):
    """Queries, keys and values of one projection."""
    qkv = uz.linear(x, w)
    return (p.unflatten(1, (-1, D)) for p in qkv.split((HEADS * GROUP * D, HEADS * D, HEADS * D), 1))


def read_prompt(cache, x, weights, freqs):
    n = x.shape[0]
    slots, positions = cache.reserve(torch.tensor([n] + [0] * (cache.state[2].numel() - 1), dtype=torch.int32, device="cuda"), n)
    for layer, (w_in, _) in enumerate(weights):
        q, k, v = layer_inputs(x, w_in)
        uz.rotary_append(q, k, v, positions, freqs, cache.k[layer], cache.v[layer], slots, check=True)


def send(cache, pages, n):
    """The first sequence's pages, in order, as a container."""
    held = cache.state[1][0, :pages]
    box = torch.empty((2,) + cache.k.shape[:1] + (pages,) + cache.k.shape[2:], dtype=cache.k.dtype, device="cuda")
    places = torch.arange(pages, dtype=torch.int32, device="cuda")
    uz.cache_copy(cache.k, cache.v, torch.stack([held, places], 1), to=(box[0], box[1]), check=True)
    if n % PAGE:  # whatever lies behind the last token is not sent
        box[:, :, -1, :, n % PAGE:].zero_()
    buf, size = uz.compress(box)
    return uz.compressed_bytes(buf, size).clone(), box


def receive(cache, container, pages, n):
    shape = (2,) + cache.k.shape[:1] + (pages,) + cache.k.shape[2:]
    box = uz.decompress(container, cache.k.dtype, torch.Size(shape).numel()).view(shape)
    cache.reserve(torch.tensor([n] + [0] * (cache.state[2].numel() - 1), dtype=torch.int32, device="cuda"), n)
    places = torch.arange(pages, dtype=torch.int32, device="cuda")
    uz.cache_copy(box[0], box[1], torch.stack([places, cache.state[1][0, :pages]], 1), to=(cache.k, cache.v), check=True)


def decode_token(cache, x, weights, freqs, counts):
    """One token of each answer through all layers; the last layer's attention beside the new hidden states."""
    answers = x.shape[0]
    slots, positions = cache.reserve(counts, answers)
    for layer, (w_in, w_out) in enumerate(weights):
        q, k, v = layer_inputs(x, w_in)
        q = uz.rotary_append(q, k, v, positions, freqs, cache.k[layer], cache.v[layer], slots)
        seen = uz.paged_attention(q, cache.k[layer], cache.v[layer], cache.state[1][1:], cache.state[2][1:])
        x = uz.linear(seen.flatten(1), w_out, residual=x)
    return x, q, seen


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompt", type=int, default=3001)
    ap.add_argument("--answers", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args(argv)
    dtype, width = torch.bfloat16, HEADS * GROUP * D
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s, scale=1.0: (torch.randn(s, generator=g, device="cuda") * scale).to(dtype)  # noqa: E731
    weights = [(rand((HEADS * GROUP + 2 * HEADS) * D, width, scale=width ** -0.5), rand(width, width, scale=width ** -0.5)) for _ in range(a.layers)]
    freqs = uz.rotary_frequencies(D)
    pages = -(-a.prompt // PAGE)

    prompt_server = Cache(a.layers, pages + 5, 1, pages + 1, dtype)
    read_prompt(prompt_server, rand(a.prompt, width), weights, freqs)
    container, box = send(prompt_server, pages, a.prompt)
    print(f"{a.prompt} tokens: {box.nbytes / 1e6:.1f} MB of cache sent as {container.numel() / 1e6:.1f} MB")

    tokens_each = -(-a.tokens // PAGE) + 1
    server = Cache(a.layers, pages + a.answers * tokens_each, 1 + a.answers, pages + tokens_each, dtype)
    receive(server, container, pages, a.prompt)
    one = torch.tensor([0] + [1] * a.answers, dtype=torch.int32, device="cuda")
    uz.cache_fork(*server.state, torch.zeros(a.answers, dtype=torch.int32, device="cuda"),
                  torch.arange(1, a.answers + 1, dtype=torch.int32, device="cuda"), PAGE, check=True)
    x = rand(a.answers, width)
    for _ in range(a.tokens):
        x, q, seen = decode_token(server, x, weights, freqs, one)
    table, lengths = server.state[1].clone(), server.state[2].clone()
    used, alone = int((server.state[0] > 0).sum()), int((-(-lengths // PAGE)).sum())
    print(f"{a.answers} answers of {a.tokens} tokens beside the prompt in {used} pages; unshared they would be {alone}")
    uz.cache_free(*server.state, torch.arange(a.answers + 1, dtype=torch.int32, device="cuda"), PAGE, check=True)
    return prompt_server, server, box, table, lengths, q, seen


if __name__ == "__main__":
    main()
