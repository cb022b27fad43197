"""The example that sends a cache runs; what the answers attend to agrees with
64 bits over the prompt server's own cache."""
import importlib.util
import os

import pytest
import torch

from tests import _cache as ref
from tests._products import within

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("prompt", [48, 1001])
def test_compressed_cache_transfer(prompt):
    spec = importlib.util.spec_from_file_location("_example", os.path.join(ROOT, "examples", "compressed_cache_transfer.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    sender, server, box, table, lengths, q, seen = ex.main(["--prompt", str(prompt), "--answers", "3", "--tokens", "5"])
    assert lengths.tolist() == [prompt] + [prompt + 5] * 3 and not any(bool(x.any()) for x in (server.state[0], server.state[2]))
    # the prompt arrived to the bit
    t = torch.arange(prompt, device="cuda")
    for mine, theirs in ((sender.k, server.k), (sender.v, server.v)):
        a = mine[:, sender.state[1][0].long()[t // ex.PAGE], :, t % ex.PAGE]
        b = theirs[:, table[0].long()[t // ex.PAGE], :, t % ex.PAGE]
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # answers share the prompt's whole pages and have their last ones to themselves
    whole = prompt // ex.PAGE
    assert all(torch.equal(table[i, :whole], table[0, :whole]) for i in (1, 2, 3))
    assert len({int(table[i, whole]) for i in (1, 2, 3)}) == 3
    want, _, off, _ = ref.attention64(q, server.k[-1], server.v[-1], table[1:], lengths[1:])
    assert within(seen, want, off) <= 1.0
