"""The layer operators where they are easily wrong: waits that give up, bits
of activations, empty sums. The definitions and bounds are those of
test_gpu_layers.py."""
import time

import pytest
import torch

import tile_level_collective_gb300 as P
from test_gpu_layers import DT, E, FILL, TINY, U, close, gate_shape, gen, rnd


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


# ---- the experts' activations keep more bits than their type ----------------------------

def check_moe_parts(tokens, hidden, inter, experts, top_k, dtype, scale=1.0, renorm=True, w_lead=0, spread=1.0):
    """y against 64 bits, given the kernel's own choice and weights. A sum of n
    products in binary32 is off by n * 2^-24 of their magnitudes, silu's slope
    is at most 1.1, and an activation is kept to 2^-17 (bf16) or 2^-22 (f16) of
    itself, in steps of 2^-35 in f16: without a rounding to the type."""
    g, t = gen(tokens * 31 + hidden), DT[dtype]
    x = rnd(g, (tokens, hidden), t)
    router = rnd(g, (experts, hidden), t, spread * hidden ** -0.5)

    def packed(shape, std):
        n = shape[0] * shape[1] * shape[2]
        return rnd(g, (n + w_lead,), t, std)[w_lead:].view(shape)

    w_in, w_out = packed((experts, 2 * inter, hidden), hidden ** -0.5), packed((experts, hidden, inter), inter ** -0.5)
    layer = P.MoeLayer(router, w_in, w_out, top_k, renormalize=renorm, scale=scale)
    y = torch.empty_like(x)
    ids = torch.empty(tokens, top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(tokens, top_k, device="cuda")
    layer(x, y, ids=ids, weights=w, workspace=layer.workspace(tokens))
    keep, step = (2.0 ** -17, 0.0) if dtype == "bf16" else (2.0 ** -22, 2.0 ** -36)
    want, bound = (torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda") for _ in range(2))
    for tok in range(tokens):
        for k in range(top_k):
            e, we, v = int(ids[tok, k]), float(w[tok, k]), x[tok].double()
            wi, wo = w_in[e].double(), w_out[e].double()
            gu, mag = wi @ v, wi.abs() @ v.abs()
            gate, up = gu[:inter], gu[inter:]
            act = gate / (1 + torch.exp(-gate))
            h = we * act * up
            dh = we * hidden * E * (1.1 * mag[:inter] * up.abs() + act.abs() * mag[inter:]) + \
                h.abs() * (8 * E + keep) + step
            want[tok] += wo @ h
            bound[tok] += wo.abs() @ dh + (top_k * inter + 8) * E * (wo.abs() @ h.abs())
    close(y, want, bound * 1.01 + U[t] * want.abs() + (TINY if dtype == "f16" else 0.0), "y")
    return w


@pytest.mark.parametrize("tokens", [1, 8, 9, 33, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_moe_activations_are_not_rounded_to_the_type(tokens, dtype):
    check_moe_parts(tokens, 512, 200, 12, 3, dtype)
    check_moe_parts(tokens, 200, 72, 6, 2, dtype, w_lead=1)              # weights at odd places


@pytest.mark.parametrize("tokens", [2, 40])
@pytest.mark.parametrize("w_lead", [0, 1])
def test_moe_small_f16_weights(tokens, w_lead):
    """Routing weights that push activations below the smallest normal f16
    (2^-14): softmax scores over 256 experts, not renormalised, times 2^-6."""
    w = check_moe_parts(tokens, 256, 104, 256, 4, "f16", scale=2.0 ** -6, renorm=False, w_lead=w_lead, spread=0.25)
    assert float(w.max()) < 2.0 ** -12


@pytest.mark.parametrize("w_lead", [0, 1])
def test_moe_f16_activations_beyond_the_range_are_infinite(w_lead):
    """One huge activation of one token: its row has infinities or NaN where
    the output weights are not zero, the other tokens' rows are those of a call
    without it."""
    g, t = gen(77), torch.float16
    tokens, hidden, inter, experts = 5, 256, 64, 4
    x = rnd(g, (tokens, hidden), t)
    router = rnd(g, (experts, hidden), t, 0.1)

    def packed(shape, std):
        n = shape[0] * shape[1] * shape[2]
        return rnd(g, (n + w_lead,), t, std)[w_lead:].view(shape)

    w_in, w_out = packed((experts, 2 * inter, hidden), 0.06), packed((experts, hidden, inter), 0.1)
    layer = P.MoeLayer(router, w_in, w_out, 2)
    clean, y = torch.empty_like(x), torch.empty_like(x)
    ids = torch.empty(tokens, 2, dtype=torch.int32, device="cuda")
    layer(x, clean, ids=ids, workspace=layer.workspace(tokens))
    x[3] *= 30
    x[3].clamp_(-100, 100)
    w_in[:, 5] = torch.sign(x[3].float()).to(t) * 4                       # gate and up of activation 5
    w_in[:, inter + 5] = w_in[:, 5]
    layer(x, clean, ids=ids, workspace=layer.workspace(tokens))
    assert float((w_in[0, 5].double() @ x[3].double())) > 2000            # so activation 5 is beyond 65504
    x2 = x.clone()
    x2[3] = 0
    layer(x2, y, workspace=layer.workspace(tokens))
    others = [0, 1, 2, 4]
    assert torch.equal(clean[others], y[others]) and bool(torch.isfinite(y[others]).all())
    assert not bool(torch.isfinite(clean[3]).any())


def exact_inputs(tokens, hidden, inter, experts, dtype, g):
    """Tokens with two elements other than 0, so that the first product has no
    rounding to speak of."""
    x = torch.zeros(tokens, hidden, dtype=DT[dtype], device="cuda")
    x[:, 3] = rnd(g, (tokens,), DT[dtype], 0.5, 2.0)
    x[:, 10] = rnd(g, (tokens,), DT[dtype])
    return x, rnd(g, (experts, 2 * inter, hidden), DT[dtype]), rnd(g, (experts, hidden, inter), DT[dtype], 4.0)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -9], ids=["ordinary", "small"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens", [1, 8, 20, 64])
@pytest.mark.parametrize("hidden", [256, 252])
def test_moe_second_product_of_nearly_exact_activations(tokens, hidden, dtype, scale):
    """With a first product of two terms and a second one of 32, the bound is
    that of y's rounding and little else; `small`: activations around 2^-14,
    where f16 has steps of 2^-24. 252 columns take the plain kernels."""
    inter, experts, top_k = 16, 8, 2
    g, t = gen(tokens + hidden), DT[dtype]
    x, w_in, w_out = exact_inputs(tokens, hidden, inter, experts, dtype, g)
    layer = P.MoeLayer(rnd(g, (experts, hidden), t, 0.1), w_in, w_out, top_k, scale=scale)
    y = torch.empty_like(x)
    ids = torch.empty(tokens, top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(tokens, top_k, device="cuda")
    layer(x, y, ids=ids, weights=w, workspace=layer.workspace(tokens))
    keep, step = (2.0 ** -17, 0.0) if dtype == "bf16" else (2.0 ** -22, 2.0 ** -36)
    want, bound = (torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda") for _ in range(2))
    for k in range(top_k):
        e, v = ids[:, k].long(), x.double()
        gu, mag = (torch.einsum("tih,th->ti", f(w_in[e].double()), f(v)) for f in (lambda z: z, torch.abs))
        gate, up = gu[:, :inter], gu[:, inter:]
        act = gate / (1 + torch.exp(-gate))
        h = w[:, k:k + 1].double() * act * up
        dh = w[:, k:k + 1].double() * 2 * E * (1.1 * mag[:, :inter] * up.abs() + act.abs() * mag[:, inter:]) + \
            h.abs() * (8 * E + keep) + step
        wo = w_out[e].double()
        want += torch.einsum("thi,ti->th", wo, h)
        bound += torch.einsum("thi,ti->th", wo.abs(), dh + (top_k * inter + 8) * E * h.abs())
    close(y, want, bound * 1.01 + U[t] * want.abs() + (TINY if dtype == "f16" else 0.0), "y")


# ---- values that are not finite cost no more than others ---------------------------------

def elapsed_ms(f):
    times = []
    for _ in range(4):
        torch.cuda.synchronize()
        start = time.monotonic()
        f()
        torch.cuda.synchronize()
        times.append((time.monotonic() - start) * 1e3)
    return min(times)


@pytest.mark.parametrize("tokens, hidden, inter, experts", [(1, 2048, 1024, 8), (64, 2048, 1024, 8), (64, 40960, 128, 4)])
def test_moe_activations_beyond_the_range_take_no_longer(tokens, hidden, inter, experts):
    """One f16 activation of every token beyond 65504, with finite weights: the
    sums over experts need no second look. (Ten times the time of a call with
    ordinary values, and a millisecond, are far above the noise.)"""
    g, t = gen(hidden + tokens), torch.float16
    x = rnd(g, (tokens, hidden), t)
    x[:, 0] = 60.0
    router, w_in = rnd(g, (experts, hidden), t, 0.02), rnd(g, (experts, 2 * inter, hidden), t, hidden ** -0.5)
    layer = P.MoeLayer(router, w_in, rnd(g, (experts, hidden, inter), t, 0.05), 4)
    y, ws = torch.empty_like(x), layer.workspace(tokens)
    ordinary = elapsed_ms(lambda: layer(x, y, workspace=ws))
    assert bool(torch.isfinite(y).all())
    w_in[:, 7, 0] = 60.0
    w_in[:, inter + 7, 0] = 60.0
    took = elapsed_ms(lambda: layer(x, y, workspace=ws))
    assert not bool(torch.isfinite(y).any()) and bool(torch.isinf(y).any())
    assert took <= 10 * ordinary + 1, (took, ordinary)


# ---- empty sums ----------------------------------------------------------------------

@pytest.mark.parametrize("rows, cols", [(5, 0), (0, 40), (0, 0)])
@pytest.mark.parametrize("gate", ["scalar", "one", "channel", "token"])
def test_gradients_of_an_empty_matrix_are_zero(rows, cols, gate):
    """What is summed over no element is zero, also where the rows have no columns."""
    z = lambda: torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    given = torch.ones(gate_shape(gate, rows, cols), dtype=torch.bfloat16, device="cuda")
    dpre, dpost, dgate = (torch.full(s, FILL, device="cuda") for s in ((cols,), (cols,), given.shape))
    P.block_norm_backward(z(), z(), torch.empty(2, rows, device="cuda"), z(), z(), z(), dpre, d_post_weight=dpost,
                          d_gate=dgate, gate=given, workspace=P.block_norm_backward_workspace(rows, cols))
    assert all(bool((v == 0).all()) for v in (dpre, dpost, dgate))
