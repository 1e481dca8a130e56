"""The example that runs the layer operators together, against the same steps
in 64 bits (loosely: bf16 roundings pass from layer to layer), and its command."""
import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


def test_decode_matches_plain_steps():
    import layer_step
    tokens, hidden, inter, experts, top_k, ranks, steps = 5, 1024, 512, 32, 4, 4, 1
    stream, normed = layer_step.decode(tokens, hidden, inter, experts, top_k, ranks, steps)
    g = torch.Generator(device="cuda").manual_seed(0)

    def weights(*shape, std):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)

    router = weights(experts, hidden, std=hidden ** -0.5).double()
    w_in = weights(experts, 2 * inter, hidden, std=hidden ** -0.5).double()
    w_out = weights(experts, hidden, inter, std=inter ** -0.5).double()
    post, pre = (1 + weights(hidden, std=0.1)).double(), (1 + weights(hidden, std=0.1)).double()
    gate = (weights(hidden, std=0.1) + 0.5).double()
    s = weights(tokens, hidden, std=1.0).double()

    def norm(v, w):
        return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w

    x = norm(s, pre).to(torch.bfloat16).double()
    score = torch.softmax(x @ router.t(), 1)
    ids = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :top_k]
    w = score.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    y = torch.zeros_like(s)
    for t in range(tokens):
        for k in range(top_k):
            gu = w_in[ids[t, k]] @ x[t]
            y[t] += w[t, k] * (w_out[ids[t, k]] @ (torch.nn.functional.silu(gu[:inter]) * gu[inter:]))
    s = s + gate * norm(y, post)
    # the windows' and h's roundings: a few bf16 units of the row's rms
    assert float((stream.double() - s).abs().max()) <= 4 * 2.0 ** -8 * float(s.abs().max())
    assert float((normed.double() - norm(s, pre)).abs().max()) <= 8 * 2.0 ** -8 * float(norm(s, pre).abs().max())


def test_training_lowers_the_loss():
    import layer_step
    losses = layer_step.train()
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_command():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "layer_step.py")], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "decode: stream (5, 1024)" in r.stdout and "train: loss" in r.stdout
