"""Tensors with a tangent of forward-mode differentiation are refused, by
whichever argument they come in; the results had none and said nothing."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def uz():
    import lossless_float_tensor_gb300 as uz

    return uz


def _calls(uz):
    """name -> (function, keyword arguments, names of those that may have a tangent)"""
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, w, wg, dy = rand(4, 64), rand(32, 64), rand(2, 32, 64), rand(4, 32)
    offsets, targets = torch.tensor([0, 1, 4], device="cuda"), torch.tensor([0, 5, 31, 2], device="cuda")
    q, k, pools = rand(4, 4, 64), rand(4, 2, 64), [rand(8, 2, 16, 64) for _ in range(4)]
    positions, freqs = torch.arange(4, device="cuda"), uz.rotary_frequencies(64)
    table, lengths = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2), torch.full((4,), 20, dtype=torch.int32, device="cuda")
    lse, dloss = torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
    pages = dict(k_pages=pools[0], v_pages=pools[1])
    return {
        "linear": (uz.linear, dict(x=x, w=w, bias=rand(32), residual=rand(4, 32), out=rand(4, 32)), "x w bias residual out"),
        "linear_backward": (uz.linear_backward, dict(dy=dy, x=x, w=w, preact=rand(4, 32), activation="silu"), "dy x w preact"),
        "grouped_linear": (uz.grouped_linear, dict(x=x, w=wg, offsets=offsets, bias=rand(2, 32)), "x w bias"),
        "grouped_linear_backward": (uz.grouped_linear_backward, dict(dy=dy, x=x, w=wg, offsets=offsets), "dy x w"),
        "cross_entropy": (uz.cross_entropy, dict(h=x, w=w, targets=targets), "h w"),
        "cross_entropy_backward": (uz.cross_entropy_backward, dict(dloss=dloss, h=x, w=w, targets=targets, lse=lse), "dloss h w lse"),
        "rotary": (uz.rotary, dict(q=q, k=k, positions=positions, freqs=freqs), "q k freqs"),
        "rotary_backward": (uz.rotary_backward, dict(dq=q, dk=k, positions=positions, freqs=freqs), "dq dk freqs"),
        "rotary_append": (uz.rotary_append, dict(q=q, k=k, v=k + 1, positions=positions, freqs=freqs, slots=positions, out=rand(4, 4, 64), **pages),
                          "q k v freqs k_pages v_pages out"),
        "paged_attention": (uz.paged_attention, dict(q=q, table=table, lengths=lengths, out=rand(4, 4, 64), **pages), "q k_pages v_pages out"),
        "cache_copy": (uz.cache_copy, dict(pairs=table[:2] + 4, **pages), "k_pages v_pages"),
    }


@pytest.mark.parametrize("name", ["linear", "linear_backward", "grouped_linear", "grouped_linear_backward", "cross_entropy", "cross_entropy_backward", "rotary",
                                  "rotary_backward", "rotary_append", "paged_attention", "cache_copy"])
def test_tangents_are_refused(uz, name):
    f, args, dual = _calls(uz)[name]
    f(**args)
    with forward_ad.dual_level():
        f(**args)  # tensors without one are taken there as elsewhere
        for n in dual.split():
            with_tangent = forward_ad.make_dual(args[n], torch.ones_like(args[n]))
            assert not with_tangent.requires_grad
            with pytest.raises(uz.UzipError, match="has a tangent"):
                f(**(args | {n: with_tangent}))
            f(**(args | {n: forward_ad.unpack_dual(with_tangent).primal}))


def test_tangents_of_pairs_are_refused(uz):
    """Outputs and destinations that come in twos."""
    _, args, _ = _calls(uz)["rotary"]
    _, copy, _ = _calls(uz)["cache_copy"]
    with forward_ad.dual_level():
        for n in (0, 1):
            outs = [torch.empty_like(args["q"]), torch.empty_like(args["k"])]
            uz.rotary(**args, out=outs)
            outs[n] = forward_ad.make_dual(outs[n], torch.ones_like(outs[n]))
            with pytest.raises(uz.UzipError, match="has a tangent"):
                uz.rotary(**args, out=outs)
            to = [torch.empty_like(copy["k_pages"]), torch.empty_like(copy["v_pages"])]
            uz.cache_copy(**copy, to=to)
            to[n] = forward_ad.make_dual(to[n], torch.ones_like(to[n]))
            with pytest.raises(uz.UzipError, match="has a tangent"):
                uz.cache_copy(**copy, to=to)


def test_function_transforms_are_refused(uz):
    """What torch.func hands in has no memory of its own."""
    _, args, _ = _calls(uz)["rotary"]
    q = args["q"]
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda x: uz.rotary(x, None, args["positions"], args["freqs"])[0], (q,), (q,))
