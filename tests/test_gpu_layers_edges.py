"""The layer operators where they are easily wrong: waits that give up, outputs
over their inputs, mixed saved forms, odd pitches of codes, empty sums. The
definitions and bounds are those of test_gpu_layers.py."""
import time

import pytest
import torch

import tile_level_collective_gb300 as P
from test_gpu_layers import gen, rnd

pytestmark = pytest.mark.gpu


# ---- waits that give up ------------------------------------------------------------

@pytest.mark.parametrize("tokens, hidden, inter, experts, local, top_k", [
    (1, 7168, 512, 16, 16, 8),           # tiles of many parts
    (7, 512, 2048, 8, 8, 2),             # whole tiles in phase 1
    (16, 4096, 1536, 64, 64, 8),         # hundreds of stages per block: the ring turns many times
    (40, 1024, 72, 32, 8, 4),
    (64, 640, 640, 16, 16, 4),
])
def test_moe_waits_that_give_up_end_the_call(monkeypatch, tokens, hidden, inter, experts, local, top_k):
    """With a bound of 1 ns waits give up at any stage of either phase (the
    copies are valid and land soon after): every call returns without the full
    bound of a wait for a copy that was never started, and the next call with
    the default bound has the bits of the first."""
    g, t = gen(tokens + hidden), torch.bfloat16
    x = rnd(g, (tokens, hidden), t)
    layer = P.MoeLayer(rnd(g, (experts, hidden), t, 0.1), rnd(g, (local, 2 * inter, hidden), t, hidden ** -0.5),
                       rnd(g, (local, hidden, inter), t, inter ** -0.5), top_k)
    want, got, ws = torch.empty_like(x), torch.empty_like(x), layer.workspace(tokens)
    torch.cuda.synchronize()
    P.ptoc_wait_faults()
    layer(x, want, workspace=ws)
    torch.cuda.synchronize()
    assert P.ptoc_wait_faults() == 0
    for _ in range(20):
        monkeypatch.setenv("PTOC_WAIT_NS", "1")
        start = time.monotonic()
        layer(x, got, workspace=ws)
        torch.cuda.synchronize()
        took = time.monotonic() - start
        faults = P.ptoc_wait_faults()
        monkeypatch.delenv("PTOC_WAIT_NS")
        assert faults > 0 or torch.equal(got, want)
        assert took < 1.5
        layer(x, got, workspace=ws)
        torch.cuda.synchronize()
        assert P.ptoc_wait_faults() == 0 and torch.equal(got, want)
