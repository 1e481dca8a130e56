"""The layer operators together, as a model split over ranks uses them.

decode(): one decoding step of a mixture-of-experts layer whose experts are
spread over N ranks (all on this GPU, as everywhere in this library). Each rank
computes its experts' part of the layer's output into its window; block_norm
sums the windows, norms the sum, gates it into the residual stream and norms
the next layer's input, in one launch.

train(): one training step of the same norms for a block whose output is spread
over N windows: the forward pass keeps the block output and the stream in 8
bits, and the backward pass reads them back. The weight and gate gradients are
applied; the parts' and the residual's gradients are what a model would pass on.

    python examples/layer_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tile_level_collective_gb300 as ptoc  # noqa: E402


def decode(tokens=5, hidden=1024, inter=512, experts=32, top_k=4, ranks=4, steps=3, seed=0):
    """The residual stream after `steps` layers and the next layer's input."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16

    def weights(*shape, std):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(0, std, generator=g)

    router = weights(experts, hidden, std=hidden ** -0.5)
    w_in = weights(experts, 2 * inter, hidden, std=hidden ** -0.5)
    w_out = weights(experts, hidden, inter, std=inter ** -0.5)
    post, pre = 1 + weights(hidden, std=0.1), 1 + weights(hidden, std=0.1)
    gate = weights(hidden, std=0.1) + 0.5
    per = experts // ranks
    layers = [ptoc.MoeLayer(router, w_in[r * per:(r + 1) * per], w_out[r * per:(r + 1) * per], top_k,
                            first_expert=r * per) for r in range(ranks)]
    workspaces = [layer.workspace(tokens) for layer in layers]
    windows = [torch.empty(tokens, hidden, dtype=dt, device="cuda") for _ in range(ranks)]
    stream = weights(tokens, hidden, std=1.0)
    normed = torch.empty_like(stream)
    # the first layer's input: the stream normed, with nothing to add to it
    ptoc.block_norm([torch.zeros_like(stream)], stream, stream, normed, post_norm=False, pre_weight=pre)
    for _ in range(steps):
        for layer, window, workspace in zip(layers, windows, workspaces):
            layer(normed, window, workspace=workspace)
        ptoc.block_norm(windows, stream, stream, normed, post_weight=post, pre_weight=pre, gate=gate)
    return stream, normed


def train(rows=512, cols=2048, ranks=2, steps=4, lr=0.02, seed=0):
    """The loss of each step of fitting the norms' weights and the gate."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16

    def rand():
        return torch.empty(rows, cols, dtype=dt, device="cuda").normal_(0, 1, generator=g)

    parts, x, target = [rand() for _ in range(ranks)], rand(), rand()
    post, pre, gate = (torch.ones(cols, device="cuda") for _ in range(3))
    out, normed, d_x, d_part = (torch.empty_like(x) for _ in range(4))
    block8, stream8 = ptoc.Checkpoint8(rows, cols), ptoc.Checkpoint8(rows, cols)
    rstd = torch.empty(2, rows, device="cuda")
    d_post, d_pre, d_gate = (torch.empty(cols, device="cuda") for _ in range(3))
    workspace = ptoc.block_norm_backward_workspace(rows, cols)
    losses = []
    for _ in range(steps):
        ptoc.block_norm(parts, x, out, normed, post_weight=post, pre_weight=pre, gate=gate, rstd=rstd,
                        block_ckpt=block8, stream_ckpt=stream8)
        error = normed.float() - target.float()
        losses.append(float(error.square().mean()))
        d_normed = error.to(dt)
        ptoc.block_norm_backward(block8, stream8, rstd, d_normed, d_x, d_part, d_pre, d_post_weight=d_post,
                                 d_gate=d_gate, post_weight=post, pre_weight=pre, gate=gate, workspace=workspace)
        for w, d in ((post, d_post), (pre, d_pre), (gate, d_gate)):
            w -= lr / rows * d
    return losses


if __name__ == "__main__":
    stream, normed = decode()
    rms = [float(t.float().square().mean().sqrt()) for t in (stream, normed)]
    print("decode: stream %s, rms %.4f; next input rms %.4f" % (tuple(stream.shape), *rms))
    print("train: loss " + ", ".join("%.4f" % v for v in train()))
