"""The layer operators where they are easily wrong: waits that give up, bits
of activations, empty sums, outputs over their inputs, mixed saved forms, odd
pitches of codes. The definitions and bounds are those of test_gpu_layers.py."""
import time

import pytest
import torch

import tile_level_collective_gb300 as P
from test_gpu_layers import (CHAIN, DT, E, FILL, TINY, U, Box, back64, close, decode64, encode64, gate_shape, gen,
                             norm_inputs, reduce_gate, rnd, rows_at, same_values)

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


# ---- outputs over their inputs, and what the forward pass saved -------------------------

# the forms of both passes: aligned rows, odd pitches, odd bases, a gate for each element, wide rows
FORMS = [
    ("bf16", 333, 1024, 2, "channel", True, 0, 0),
    ("f16", 500, 1003, 1, "token", True, 2, 0),
    ("f32", 320, 2051, 2, "scalar", True, 0, 0),
    ("bf16", 60, 515, 1, "token", True, 4, 3),
    ("f16", 40, 1000, 2, "element", True, 8, 0),
    ("f32", 21, 8200, 1, "channel", True, 0, 0),
    ("bf16", 9, 9001, 2, "one", False, 0, 0),
    ("bf16", 350, 4097, 1, "none", False, 0, 0),
]
IDS = lambda c: "-".join(str(v) for v in c)


def backward_inputs(case, seed=0):
    dtype, rows, cols, _, gate, post, pad, lead = case
    t, d = DT[dtype], norm_inputs(*case)
    g = gen(99 + cols + seed)
    a, s = d["parts"][0], d["x"]
    rstd = torch.stack([1 / (v.float().square().mean(1) + 1e-5).sqrt() for v in (a, s)])
    boxes = [Box(rows, cols, t, pad, lead) for _ in range(4)]
    for b in boxes[:2]:
        b.view.copy_(rnd(g, (rows, cols), torch.float32))
    return d, a, s, rstd, boxes


def backward(case, d, a, s, rstd, dy, du, dx, da):
    """One call; the gradients of the weights and the gate."""
    _, rows, cols, _, _, post, _, _ = case
    sums = dict(d_post_weight=torch.full((cols,), FILL, device="cuda") if post else None,
                d_gate=None if d["gate"] is None else torch.full(d["gate"].shape, FILL, device="cuda"))
    dpre = torch.full((cols,), FILL, device="cuda")
    P.block_norm_backward(a, s, rstd, dy, dx, da, dpre, d_stream=du, post_norm=post, post_weight=d["wpost"],
                          pre_weight=d["wpre"], gate=d["gate"], residual_scale=0.75, branch_scale=-1.5,
                          workspace=P.block_norm_backward_workspace(rows, cols), **sums)
    return dict(sums, dpre=dpre)


def check_gradients(case, d, a, s, rstd, dy, du, dx, da, sums):
    """Against 64 bits, with the bounds of test_gpu_layers.check_back."""
    dtype, rows, _, _, _, post, _, _ = case
    f = back64(a, s, rstd[0], rstd[1], dy, du, d["wpost"], d["wpre"], d["gate"], 0.75, -1.5, post)
    u, c = U[DT[dtype]], 2 * CHAIN * E
    close(dx, f["dx"], u * f["dx"].abs() + c * f["mdx"] + TINY, "d_residual")
    close(da, f["da"], u * f["da"].abs() + c * f["mda"] + TINY, "d_block")
    per = c + (rows + 8) * E
    close(sums["dpre"], f["dpre"], per * f["mpre"], "d_pre_weight")
    if post:
        close(sums["d_post_weight"], f["dpost"], per * f["mpost"], "d_post_weight")
    if d["gate"] is not None:
        shape = d["gate"].shape
        close(sums["d_gate"], reduce_gate(f["dg"], shape), (per + CHAIN * E) * reduce_gate(f["mdg"], shape), "d_gate")


@pytest.mark.parametrize("case", FORMS, ids=IDS)
def test_block_norm_over_its_residual(case):
    dtype, rows, cols, _, _, post, pad, lead = case
    d = norm_inputs(*case)
    call = lambda x, out, normed: P.block_norm(d["parts"], x, out, normed, post_norm=post, post_weight=d["wpost"],
                                               pre_weight=d["wpre"], gate=d["gate"], residual_scale=0.75)
    apart, normed, over, normed2 = (Box(rows, cols, DT[dtype], pad, lead) for _ in range(4))
    call(d["x"], apart.view, normed.view)
    over.view.copy_(d["x"])
    call(over.view, over.view, normed2.view)
    assert torch.equal(over.view, apart.view) and torch.equal(normed2.view, normed.view)
    assert over.outside_intact()


@pytest.mark.parametrize("ckpt", [False, True], ids=["saved", "ckpt"])
@pytest.mark.parametrize("case", FORMS, ids=IDS)
def test_block_norm_backward_over_its_inputs(case, ckpt):
    """d_residual over du, and d_block over the saved block output: the bits of
    a call with outputs of their own, which is compared with 64 bits."""
    d, a, s, rstd, (dy, du, dx, da) = backward_inputs(case)
    rows, cols = a.shape
    saved = a, s
    if ckpt:
        saved = P.Checkpoint8(rows, cols), P.Checkpoint8(rows, cols)
        P.checkpoint8(a, saved[0])
        P.checkpoint8(s, saved[1])
        a, s = (decode64(k.codes, k.exps) for k in saved)
    sums = backward(case, d, *saved, rstd, dy.view, du.view, dx.view, da.view)
    check_gradients(case, d, a, s, rstd, dy.view, du.view, dx.view, da.view, sums)
    block = Box(rows, cols, DT[case[0]], case[6], case[7]).view if ckpt else saved[0]
    again = backward(case, d, *saved, rstd, dy.view, du.view, du.view, block)
    assert torch.equal(du.view, dx.view) and torch.equal(block, da.view)
    assert all(v is None or torch.equal(v, sums[k]) for k, v in again.items())
    assert du.outside_intact()


@pytest.mark.parametrize("kept", ["block", "stream"])
@pytest.mark.parametrize("case", FORMS, ids=IDS)
def test_block_norm_backward_from_one_matrix_and_one_checkpoint(case, kept):
    d, a, s, rstd, (dy, du, dx, da) = backward_inputs(case)
    k = P.Checkpoint8(*a.shape)
    P.checkpoint8(s if kept == "block" else a, k)
    small = decode64(k.codes, k.exps)
    saved, exact = ((a, k), (a, small)) if kept == "block" else ((k, s), (small, s))
    sums = backward(case, d, *saved, rstd, dy.view, du.view, dx.view, da.view)
    check_gradients(case, d, *exact, rstd, dy.view, du.view, dx.view, da.view, sums)
    assert dx.outside_intact() and da.outside_intact()


# ---- codes and exponents at any pitch ---------------------------------------------------

class CodeBox:
    """A Checkpoint8 whose rows lie `pad` bytes apart, from byte `lead` on, in
    filled memory."""

    def __init__(self, rows, cols, pad, lead, exps_pad=0, exps_lead=0):
        nb = (cols + 31) // 32
        self.parts = []
        for width, more, first, dtype in ((cols, pad, lead, torch.int8), (nb, exps_pad, exps_lead, torch.uint8)):
            raw = torch.full((first + (rows + 1) * (width + more) + 32,), 7, dtype=dtype, device="cuda")
            self.parts.append((raw, raw.as_strided((rows, width), (width + more, 1), first)))
        self.k = P.Checkpoint8.of(self.parts[0][1], self.parts[1][1], cols)

    def outside_intact(self):
        ok = True
        for raw, view in self.parts:
            keep = raw.clone()
            keep.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(7)
            ok = ok and bool((keep == 7).all())
        return ok


CODES = [(1, 0, 0, 0), (5, 0, 1, 0), (0, 0, 3, 0), (8, 0, 0, 0), (3, 5, 0, 0), (0, 8, 0, 4), (0, 0, 0, 1), (11, 1, 2, 3)]


@pytest.mark.parametrize("codes", CODES, ids=IDS)
@pytest.mark.parametrize("dtype, rows, cols, pad", [("bf16", 37, 1003, 0), ("f16", 330, 520, 8), ("f32", 41, 2047, 1),
                                                    ("f32", 19, 96, 0), ("bf16", 11, 9001, 0), ("bf16", 40, 4096, 0)])
def test_codes_at_any_pitch(dtype, rows, cols, pad, codes):
    """Kept, restored, written by the forward pass and read by the backward
    pass, with rows of codes that begin anywhere in their 16 bytes."""
    case = (dtype, rows, cols, 1, "channel", True, pad, 0)
    d, a, s, rstd, (dy, du, dx, da) = backward_inputs(case)
    bk, sk, again = (CodeBox(rows, cols, *codes) for _ in range(3))
    for k, x in ((bk, a), (sk, s)):
        P.checkpoint8(x, k.k)
        want = encode64(x)
        assert torch.equal(k.k.codes, want[0]) and torch.equal(k.k.exps, want[1]) and k.outside_intact()
        back = Box(rows, cols, DT[dtype], pad)
        P.restore8(k.k, back.view)
        assert same_values(back.view, decode64(*want).to(DT[dtype])) and back.outside_intact()
    sums = backward(case, d, bk.k, sk.k, rstd, dy.view, du.view, dx.view, da.view)
    a8, s8 = (decode64(k.k.codes, k.k.exps) for k in (bk, sk))
    check_gradients(case, d, a8, s8, rstd, dy.view, du.view, dx.view, da.view, sums)
    assert dx.outside_intact() and da.outside_intact()
    # the forward pass's checkpoints of the sum of one part, and of the stream
    out = Box(rows, cols, DT[dtype], pad)
    P.block_norm([a], s, out.view, post_weight=d["wpost"], gate=d["gate"], block_ckpt=again.k, stream_ckpt=sk.k)
    for k, x in ((again, a), (sk, out.view)):
        want = encode64(x)
        assert torch.equal(k.k.codes, want[0]) and torch.equal(k.k.exps, want[1]) and k.outside_intact()


@pytest.mark.parametrize("pitch", [2 ** 30 + 8, 2 ** 30 + 1])
def test_rows_past_32_bits_against_the_definition(pitch):
    """What test_rows_past_32_bits_have_the_same_bits compares between pitches,
    against 64 bits at the far one."""
    cols = 1000
    case = ("bf16", 3, cols, 1, "channel", True, 0, 0)
    d, a, s, rstd, (dy, du, _, _) = backward_inputs(case)
    part, x, y, v = (rows_at(pitch).copy_(m) for m in (a, s, dy.view, du.view))
    dx, da, restored = (rows_at(pitch) for _ in range(3))
    bk, sk = (P.Checkpoint8.of(rows_at(pitch, torch.int8), rows_at(pitch, torch.uint8, 32)) for _ in range(2))
    for k, m in ((bk, part), (sk, x)):
        P.checkpoint8(m, k)
        want = encode64(m)
        assert torch.equal(k.codes, want[0]) and torch.equal(k.exps, want[1])
        P.restore8(k, restored)
        assert same_values(restored, decode64(*want).to(torch.bfloat16))
    sums = backward(case, d, bk, sk, rstd, y, v, dx, da)
    a8, s8 = (decode64(k.codes, k.exps) for k in (bk, sk))
    check_gradients(case, d, a8, s8, rstd, y, v, dx, da, sums)


# ---- alignments that no kernel needs cost nothing ---------------------------------------

def device_us(f):
    """The shortest of several stretches of calls, per call."""
    times = []
    for _ in range(6):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(10):
            f()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 100)
    return min(times)


@pytest.mark.parametrize("odd", ["gate", "exponents", "codes"])
def test_alignments_that_no_kernel_needs_cost_nothing(odd):
    """A gate of one number at an odd element, exponents from an odd byte on,
    codes from a multiple of 8 on: the time is that of the same call with all
    of them aligned (with the element-wide kernels 115 us where these take 62)."""
    rows, cols, t = 4096, 4096, torch.bfloat16
    g = gen(4)
    a, s, dy, out, normed, dx, da = (rnd(g, (rows, cols), t) for _ in range(7))
    rstd, gates = torch.ones(2, rows, device="cuda"), torch.ones(16, dtype=t, device="cuda")
    ws = P.block_norm_backward_workspace(rows, cols)
    times = []
    for shifted in (False, True):
        at = dict(gate=(1, 0, 0), exponents=(0, 0, 3), codes=(0, 8, 0))[odd] if shifted else (0, 0, 0)
        gate = gates[at[0]:at[0] + 1]
        bk, sk = (CodeBox(rows, cols, 0, at[1], 0, at[2]) for _ in range(2))

        def step():
            P.block_norm([a], s, out, normed, gate=gate, rstd=rstd, block_ckpt=bk.k, stream_ckpt=sk.k)
            P.block_norm_backward(bk.k, sk.k, rstd, dy, dx, da, gate=gate, workspace=ws)

        times.append(device_us(step))
    assert times[1] <= 1.4 * times[0], times


# ---- factors that are not finite ----------------------------------------------------------

@pytest.mark.parametrize("cols, lead", [(96, 0), (1000, 0), (1003, 0), (515, 1), (9000, 0), (9001, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_norm_infinite_gates_reach_only_their_rows(dtype, cols, lead):
    """An infinite gate makes its row infinite, whose statistic is then 0 at
    every width: nothing past the row's end takes part."""
    rows, t = 5, DT[dtype]
    g = gen(cols)
    boxes = [Box(rows, cols, t, 0, lead) for _ in range(4)]
    part, x, out, normed = (b.view for b in boxes)
    for v in (part, x):
        v.copy_(rnd(g, (rows, cols), torch.float32).abs() + 1)
    gate = torch.ones(rows, 1, dtype=t, device="cuda")
    gate[2] = float("inf")
    rstd = torch.empty(2, rows, device="cuda")
    P.block_norm([part], x, out, normed, gate=gate, rstd=rstd)
    assert bool(torch.isinf(out[2]).all()) and float(rstd[1, 2]) == 0
    others = [0, 1, 3, 4]
    assert bool(torch.isfinite(out[others]).all()) and bool((rstd[:, others] > 0).all())
    P.block_norm([part], x, out, normed, post_norm=False, rstd=rstd, residual_scale=float("inf"))
    assert bool(torch.isinf(out).all()) and bool((rstd[1] == 0).all())
