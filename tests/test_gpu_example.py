"""The example training step runs and agrees with the same step in 64 bits."""
import importlib.util
import os

import pytest
import torch

from tests import _products as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_compressed_training_step():
    import lossless_float_tensor_gb300 as uz

    spec = importlib.util.spec_from_file_location("_example", os.path.join(ROOT, "examples", "compressed_training_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    weights, kept, bias, x, offsets, targets, loss, dx, grads, sent, token = ex.main(
        ["--tokens", "300", "--width", "256", "--hidden", "512", "--vocab", "3001"])
    # the same step in 64 bits by autograd, from the weights as they were before compression
    leaf = {k: v.double().requires_grad_() for k, v in {**weights, "bias": bias, "x": x}.items()}
    a = torch.nn.functional.silu(leaf["x"] @ leaf["gate"].T + leaf["bias"])
    ends = offsets.tolist()
    y = torch.cat([a[ends[e]:ends[e + 1]] @ leaf["up"][e].T for e in range(ex.EXPERTS)])
    logits = (y + leaf["x"]) @ leaf["head"].T
    want = torch.nn.functional.cross_entropy(logits, targets, reduction="none")
    want[targets != -100].mean().backward()
    # relative 2-norms: activations are rounded to 8 bits at three places before the loss, gradients at six
    def off(got, ref64):
        return float((got.double() - ref64).norm() / ref64.norm())

    u = ref.ROUND[torch.bfloat16]
    assert off(loss, want.detach()) <= 3 * u
    assert off(dx, leaf["x"].grad) <= 6 * u
    for name, g in grads.items():
        assert off(g, leaf[name].grad) <= 6 * u, name
    for name, (buf, _) in sent.items():
        g = grads[name]
        assert torch.equal(uz.decompress(buf, g.dtype, g.numel()).view(torch.int16), g.reshape(-1).view(torch.int16))
    best = ((y + leaf["x"]) @ leaf["head"].T)[0].detach()
    one = ex.forward(kept, bias, x[:1], torch.tensor([0, 1] + [1] * 7, device="cuda"), torch.cuda.Stream())[0]
    assert off(one, (y + leaf["x"])[:1].detach()) <= 3 * u
    assert float(best.max() - best[int(token.item())]) <= 6 * u * float(best.abs().max())
