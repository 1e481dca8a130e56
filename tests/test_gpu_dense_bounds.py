"""The dense block's operators where a bound on the whole result hides an error.
Tolerances are derived as in test_gpu_dense.py."""
import pytest
import torch

import tile_level_collective_gb300 as P
from test_gpu_dense import F64, act64, box, check_clip, ffn_back_want, ffn_inputs, ffn_want, product, rounded
from test_gpu_layers import DT, E, TINY, U, Box, close, rnd

pytestmark = pytest.mark.gpu


# ---- the gradients' norm -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("place", ["in", "out"])
def test_clip_norm_beyond_binary32(dtype, place):
    """A finite set whose norm binary32 cannot hold: the caller reads an infinite norm, and finds scale 1
    and its gradients as they were."""
    t = torch.full((2,), 3e38, dtype=DT[dtype], device="cuda")
    before, out, result = t.clone(), torch.zeros_like(t), torch.zeros(2, device="cuda")
    s = P.Gradients([t], None if place == "in" else [out])
    s.clip(1.0, result, workspace=s.workspace())
    assert result.tolist() == [float("inf"), 1.0]
    assert torch.equal(t, before) and (place == "in" or torch.equal(out, before))


def test_clip_largest_norm():
    """The largest norms that binary32 holds are finite, and limited."""
    check_clip([torch.full((2,), 2.4e38, device="cuda")], None, 1e30)
    check_clip([torch.full((3,), 1.9e38, device="cuda")], [torch.empty(3, device="cuda")], 1e30)


# ---- the activations --------------------------------------------------------------------------

# An activation is off by at most this part of its value (see the header).
ACT_REL = 2.0 ** -19


def picked(gates, dt, hidden):
    """[n, hidden] rows whose first product with a unit vector is the gate."""
    w = torch.zeros(gates.numel(), hidden, dtype=dt, device="cuda")
    w[:, 0] = gates
    return w


GATES = {torch.float16: (-5.5, 2.0 ** 13), torch.bfloat16: (-12.0, 1.0)}       # the lowest gate, and u, which keeps h normal


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,odd", [(5, 0), (5, 1), (100, 0), (100, 1), (150, 0)])
def test_activation_tail(dtype, act, tokens, odd):
    """h one by one, at gates down to where it is nearly zero: relative to itself."""
    dt = DT[dtype]
    low, up = GATES[dt]
    width = 512 + odd
    g = torch.linspace(low, -0.5, width, device="cuda").to(dt)
    w_in = torch.cat([picked(g, dt, width), picked(torch.full_like(g, up), dt, width)])
    w_out = torch.eye(width, dtype=dt, device="cuda")
    x = torch.zeros(tokens, width, dtype=dt, device="cuda")
    x[:, 0] = 1
    y = torch.empty_like(x)
    f = P.GatedFfn(w_in, w_out, act)
    f(x, y, workspace=f.workspace(tokens))
    want = (act64(g.to(F64), act)[0] * up).expand(tokens, width)
    # one rounding (two where h enters as one number: the second one is exact), and the activation's arithmetic
    close(y, want, (U[dt] + 2 * ACT_REL) * want.abs(), act)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,odd", [(5, 0), (5, 1), (100, 0), (150, 0)])
def test_slope_tail(dtype, act, tokens, odd):
    """dg and du one by one, as dx and as a weight's gradient shows them."""
    dt = DT[dtype]
    low, up = GATES[dt]
    width = 512 + odd
    g = torch.linspace(low, -3.0, width, device="cuda").to(dt)
    pre = torch.cat([g, torch.full_like(g, up)]).expand(tokens, -1).contiguous()
    dy = torch.full((tokens, width), 1.0, dtype=dt, device="cuda")
    eye, none = torch.eye(width, dtype=dt, device="cuda"), torch.zeros(width, width, dtype=dt, device="cuda")
    x = torch.zeros(tokens, width, dtype=dt, device="cuda")
    x[0, 0] = 1                                           # d_w_in's first column is the first token's dg and du
    a, slope = act64(g.to(F64), act)
    for gate in (True, False):
        f = P.GatedFfn(torch.cat([eye, none] if gate else [none, eye]), eye, act)
        dx, dw = torch.empty_like(x), torch.empty_like(f.w_in)
        f.backward(x, pre, dy, d_x=dx, d_w_in=dw, workspace=f.backward_workspace(tokens))
        # act' is a sum of two terms of opposite signs, which below -3 add to 2.1 times it at most
        d = slope * up if gate else a
        bound = (U[dt] + 4 * ACT_REL) * d.abs() + (TINY if dt == torch.float16 else 0)
        close(dx, d.expand(tokens, width), bound, "dg" if gate else "du")
        both = torch.cat([slope * up, a])
        close(dw[:, 0], both, (U[dt] + 4 * ACT_REL) * both.abs() + (TINY if dt == torch.float16 else 0), "d_w_in")


# ---- rows at the end of binary32 -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [1024, 1001, 8192, 16384])
def test_layer_norm_warps_far_apart(dtype, cols):
    """Rows whose warps' means are far apart, up to deviations whose squares binary32 cannot add: those
    have a standard deviation of infinity, so that rstd is 0 and y the bias."""
    dt = DT[dtype]
    x = torch.zeros(3, cols, dtype=dt, device="cuda")
    # a sum of squared deviations of 2.56e38 (cols / 4 times the square), and larger ones
    x[0, :cols // 2], x[1, :cols // 2], x[2, cols // 2:] = 2.5e17 * (16384 / cols) ** 0.5, 1e19, -1e19
    y, stats, bias = torch.empty_like(x), torch.empty(2, 3, device="cuda"), torch.full((cols,), 0.5, dtype=dt, device="cuda")
    for rows in (x, x[:1]):
        P.layer_norm([rows], y[:len(rows)], bias=bias, stats=stats[:, :len(rows)].contiguous())
        s = x[:1].to(F64)
        d = s - s.mean()
        want = d / d.square().mean().sqrt()
        # sums of a warp's equal values, and of the warps: as in norm_want
        close(y[:1], want + 0.5, 256 * E * want.abs() + U[dt] * (want + 0.5).abs())
        assert bool((y[1:len(rows)] == 0.5).all())


# ---- numbers that a second product takes in two parts ------------------------------------------------

# A number of the type and what it leaves, rounded again: relative to the number.
PARTS = {torch.float16: 2.0 ** -22, torch.bfloat16: 2.0 ** -16}


def own_rounding(got, want, dt, what):
    """The error of a result that is rounded once, against that of rounding the 64-bit one: a second
    rounding of every operand would make it 1.4 times as much."""
    once = float((want.to(dt).to(F64) - want).norm())
    off = float((got.to(F64) - want).norm())
    assert off <= 1.1 * once, "%s: %.3g times a rounding" % (what, off / once)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,hidden,inter,pad", [(1, 4096, 1000, 0), (8, 512, 520, 0), (9, 512, 520, 8), (37, 264, 1000, 0),
                                                     (64, 256, 512, 0), (1, 2049, 333, 0), (8, 512, 520, 1), (40, 255, 401, 0),
                                                     (64, 256, 512, 3)])
def test_few_tokens_are_rounded_once(dtype, act, tokens, hidden, inter, pad):
    """Up to 64 tokens h, dg and du reach y and dx in more bits than the type has, at any width and pitch."""
    dt = DT[dtype]
    x, w_in, w_out, g = ffn_inputs(tokens, hidden, inter, dt, tokens + hidden)
    x, w_in, w_out = box(x, pad), box(w_in, pad), box(w_out, pad)
    f = P.GatedFfn(w_in.view, w_out.view, act)
    y = Box(tokens, hidden, dt, pad)
    f(x.view, y.view, workspace=f.workspace(tokens))
    pre, dy = box(rnd(g, (tokens, 2 * inter), dt), pad), box(rnd(g, (tokens, hidden), dt), pad)
    dx = Box(tokens, hidden, dt, pad)
    f.backward(x.view, pre.view, dy.view, d_x=dx.view, workspace=f.backward_workspace(tokens))

    x, w_in, w_out, pre, dy = (b.view.to(F64) for b in (x, w_in, w_out, pre, dy))
    gu, err = product(x, w_in.t())
    a, slope = act64(gu[:, :inter], act)
    u = gu[:, inter:]
    h = a * u
    err_h = (slope.abs() * err[:, :inter] + err[:, :inter] ** 2) * u.abs() + a.abs() * err[:, inter:] \
        + 2 * ACT_REL * h.abs() + 1.2 * err[:, :inter] * err[:, inter:]
    want, bound = product(h, w_out.t(), err_h + PARTS[dt] * h.abs() + 2.0 ** -36)
    close(y.view, want, rounded(want, bound, dt), "y")
    own_rounding(y.view, want, dt, "y")

    dh, err = product(dy, w_out)
    a, slope = act64(pre[:, :inter], act)
    u = pre[:, inter:]
    # act' is a sum of two terms of at most 1.2 together
    d = torch.cat([dh * u * slope, dh * a], 1)
    err_d = torch.cat([err * (u * slope).abs() + 4 * ACT_REL * (dh.abs() + err) * u.abs() * 1.2,
                       err * a.abs() + 2 * ACT_REL * (dh.abs() + err) * a.abs()], 1)
    want, bound = product(d, w_in, err_d + PARTS[dt] * d.abs() + 2.0 ** -36)
    close(dx.view, want, rounded(want, bound, dt), "dx")
    own_rounding(dx.view, want, dt, "dx")


# ---- gradients along the gradient --------------------------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,hidden,inter", [(40, 64, 96), (100, 64, 96), (200, 136, 96), (40, 65, 97)])
def test_gated_ffn_gradient_along_itself(act, tokens, hidden, inter):
    """The library's forward pass in f16 along each of its own gradients: the loss sum(y dy) changes by
    the gradient times the way, and by nothing near a gradient that is zero, negated or doubled."""
    dt, part = torch.float16, 2.0 ** -4
    x, w_in, w_out, g = ffn_inputs(tokens, hidden, inter, dt, 9)
    dy = rnd(g, (tokens, hidden), dt)
    f = P.GatedFfn(w_in, w_out, act)
    ws = f.workspace(tokens)
    pre, y = torch.empty(tokens, 2 * inter, dtype=dt, device="cuda"), torch.empty_like(x)
    f(x, y, pre=pre, workspace=ws)
    got = dict(d_x=torch.empty_like(x), d_w_in=torch.empty_like(w_in), d_w_out=torch.empty_like(w_out))
    f.backward(x, pre, dy, **got, workspace=f.backward_workspace(tokens))
    bounds = ffn_back_want(x, pre, dy, w_in, w_out, act, dt)
    y_bound = float((ffn_want(x, w_in, w_out, act, dt)["y"][1] * dy.to(F64).abs()).sum())
    for t, name in ((x, "d_x"), (w_in, "d_w_in"), (w_out, "d_w_out")):
        d = got[name].to(F64)
        v = d * (float(t.to(F64).norm()) / float(d.norm()))
        base, change, way = t.clone(), [], []
        for h in (part, 2 * part):
            ends = []
            for sign in (h, -h):
                t.copy_((base.to(F64) + sign * v).to(dt))
                f(x, y, workspace=ws)
                ends.append((t.to(F64), float((y.to(F64) * dy.to(F64)).sum())))
            change.append(ends[0][1] - ends[1][1])
            way.append(ends[0][0] - ends[1][0])
        t.copy_(base)
        want = [float((d * m).sum()) for m in way]
        # the cube's part of a difference, which a way twice as long has eight times
        cubic = (change[1] - 2 * change[0] - (want[1] - 2 * want[0])) / 6
        off = abs(change[0] - want[0] - cubic)
        # roundings of y at the four ends (the far two count a third) and of the gradient; the kept g and u are
        # rounded too, which moves the gradient by what three roundings of dg and du do at most; the way is
        # 1/16 of the tensor's norm, so that the fifth power's part (4/16^4) and that of the square, which the ends'
        # own roundings leave (U a 1/16), stay below a hundredth
        bound = 4 * y_bound + 4 * float((bounds[name][1] * way[0].abs()).sum()) + 0.1 * abs(cubic) + 0.01 * abs(want[0])
        assert bound < abs(want[0]) / 4, name
        assert off <= bound, name
        for wrong in (0.0, -1.0, 2.0):
            far = (change[1] - 2 * change[0] - wrong * (want[1] - 2 * want[0])) / 6
            assert abs(change[0] - wrong * want[0] - far) > bound, name


# ---- two parts where the caller asks for them --------------------------------------------------------------

TWO_SHAPES = [  # tokens, hidden, inter, pad: streamed and not, both widths of tiles, any pitch and width
    (1, 520, 512, 0), (37, 264, 1000, 0), (64, 256, 512, 8), (65, 256, 512, 0), (128, 520, 264, 0), (130, 264, 200, 0),
    (300, 1000, 600, 8), (1300, 2056, 136, 0), (140, 136, 8200, 0), (8, 512, 520, 1), (70, 255, 401, 0), (150, 64, 64, 3)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,hidden,inter,pad", TWO_SHAPES)
def test_two_parts(dtype, act, tokens, hidden, inter, pad):
    """At any number of tokens, y and all three gradients have the error of their own rounding."""
    dt = DT[dtype]
    x, w_in, w_out, g = ffn_inputs(tokens, hidden, inter, dt, tokens + hidden)
    x, w_in, w_out = box(x, pad), box(w_in, pad), box(w_out, pad)
    f = P.GatedFfn(w_in.view, w_out.view, act, parts=2)
    pre, dy = box(rnd(g, (tokens, 2 * inter), dt), pad), box(rnd(g, (tokens, hidden), dt), pad)
    got = dict(y=Box(tokens, hidden, dt, pad), d_x=Box(tokens, hidden, dt, pad), d_w_in=Box(2 * inter, hidden, dt, pad),
               d_w_out=Box(hidden, inter, dt, pad))
    kept = Box(tokens, 2 * inter, dt, pad)
    ws, bws = f.workspace(tokens), f.backward_workspace(tokens)
    grads = {k: got[k].view for k in ("d_x", "d_w_in", "d_w_out")}
    for k in range(2):                                     # what a workspace held does not matter
        ws.fill_(255), bws.fill_(255)
        f(x.view, got["y"].view, pre=kept.view if k else None, workspace=ws)
        f.backward(x.view, pre.view, dy.view, **grads, workspace=bws)
        again = [b.view.clone() for b in got.values()]
        if k:
            assert all(torch.equal(a, b) for a, b in zip(again, first))
        first = again
    for name, v in grads.items():                          # asked for alone: the same bits
        one = torch.empty_like(v)
        f.backward(x.view, pre.view, dy.view, **{name: one}, workspace=bws)
        assert torch.equal(one, v), name
    assert all(b.outside_intact() for b in (kept, *got.values())) and P.ptoc_wait_faults() == 0

    low = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -130       # half a step of the second number
    x, w_in, w_out, pre, dy = (b.view.to(F64) for b in (x, w_in, w_out, pre, dy))
    gu, err = product(x, w_in.t())
    close(kept.view, gu, rounded(gu, err, dt), "pre")
    a, slope = act64(gu[:, :inter], act)
    u, eg, eu = gu[:, inter:], err[:, :inter], err[:, inter:]
    h = a * u
    err_h = (slope.abs() * eg + eg * eg) * u.abs() + a.abs() * eu + 2 * ACT_REL * h.abs() + 1.2 * eg * eu
    want = dict(y=product(h, w_out.t(), err_h + PARTS[dt] * h.abs() + low))
    dh, err = product(dy, w_out)
    a, slope = act64(pre[:, :inter], act)
    u = pre[:, inter:]
    d, h = torch.cat([dh * u * slope, dh * a], 1), a * u
    err_d = torch.cat([err * (u * slope).abs() + 4 * ACT_REL * (dh.abs() + err) * u.abs() * 1.2,
                       err * a.abs() + 2 * ACT_REL * (dh.abs() + err) * a.abs()], 1) + PARTS[dt] * d.abs() + low
    want["d_x"], want["d_w_in"] = product(d, w_in, err_d), product(d.t(), x, err_d.t())
    v, e = product(h.t(), dy, ((2 * ACT_REL + PARTS[dt]) * h.abs() + low).t())
    want["d_w_out"] = v.t(), e.t()
    for name, (v, e) in want.items():
        close(got[name].view, v, rounded(v, e, dt), name)
        if v.numel() >= 2000:
            own_rounding(got[name].view, v, dt, name)


@pytest.mark.parametrize("tokens", [3, 70, 300])
def test_two_parts_rows_stay_apart(tokens):
    """An infinity or a NaN in a token's row changes no other row, and an h beyond f16 is infinite."""
    for dt in (torch.bfloat16, torch.float16):
        x, w_in, w_out, _ = ffn_inputs(tokens, 136, 200, dt, 5)
        f = P.GatedFfn(w_in, w_out, parts=2)
        ws = f.workspace(tokens)
        clean, y = torch.empty_like(x), torch.empty_like(x)
        f(x, clean, workspace=ws)
        x[1, 3], x[2, 100] = float("inf"), float("nan")
        if dt == torch.float16:
            x[0] *= 300
        f(x, y, workspace=ws)
        assert not bool(torch.isfinite(y[1:3]).any()) and (dt == torch.bfloat16 or not bool(torch.isfinite(y[0]).all()))
        assert torch.equal(y[3:], clean[3:])


@pytest.mark.parametrize("tokens", [40, 200])
def test_two_parts_captured_and_on_streams(tokens):
    """Overlapping calls with a workspace each, eager and replayed, give the bits of one call; so does a call
    after one whose waits gave up."""
    dt, jobs = torch.bfloat16, []
    for k in range(3):
        x, w_in, w_out, g = ffn_inputs(tokens, 512, 776, dt, k)
        f = P.GatedFfn(w_in, w_out, parts=2)
        pre, dy = torch.empty(tokens, 1552, dtype=dt, device="cuda"), rnd(g, (tokens, 512), dt)
        out = [torch.empty_like(v) for v in (x, x, w_in, w_out)]
        spaces = f.workspace(tokens), f.backward_workspace(tokens)

        def run(f=f, x=x, pre=pre, dy=dy, out=out, spaces=spaces):
            f(x, out[0], pre=pre, workspace=spaces[0])
            f.backward(x, pre, dy, d_x=out[1], d_w_in=out[2], d_w_out=out[3], workspace=spaces[1])
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        jobs.append((run, graph, out, [v.clone() for v in out], torch.cuda.Stream()))
    for i in range(6):
        for run, graph, out, _, stream in jobs:
            with torch.cuda.stream(stream):
                for v in out:
                    v.zero_()
                graph.replay() if i & 1 else run()
    torch.cuda.synchronize()
    for _, _, out, want, _ in jobs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert P.ptoc_wait_faults() == 0


@pytest.mark.parametrize("parts,tokens,hidden,inter", [(2, 150, 2048, 1000), (1, 40000, 264, 264), (1, 130, 264, 33000)])
def test_two_parts_and_long_sums_waits_that_give_up(parts, tokens, hidden, inter, monkeypatch):
    """With a bound of 1 ns waits on valid copies run out: the calls end, and the next ones are whole."""
    dt = torch.bfloat16
    x, w_in, w_out, g = ffn_inputs(tokens, hidden, inter, dt, 3)
    f = P.GatedFfn(w_in, w_out, parts=parts)
    ws, bws = f.workspace(tokens), f.backward_workspace(tokens)
    y, pre, dy = torch.empty_like(x), torch.empty(tokens, 2 * inter, dtype=dt, device="cuda"), rnd(g, (tokens, hidden), dt)
    out = [y, *(torch.empty_like(v) for v in (x, w_in, w_out))]

    def run():
        f(x, y, pre=pre, workspace=ws)
        f.backward(x, pre, dy, d_x=out[1], d_w_in=out[2], d_w_out=out[3], workspace=bws)
        torch.cuda.synchronize()

    run()
    want = [v.clone() for v in out]
    monkeypatch.setenv("PTOC_WAIT_NS", "1")
    for _ in range(3):
        run()
    assert P.ptoc_wait_faults() > 0
    monkeypatch.delenv("PTOC_WAIT_NS")
    run()
    assert P.ptoc_wait_faults() == 0 and all(torch.equal(a, b) for a, b in zip(out, want))


# ---- calls at the limits, and several threads' ------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("tokens,hidden,inter", [
    (3, P.FFN_MAX_WIDTH, 8), (3, 8, P.FFN_MAX_WIDTH), (200, P.FFN_MAX_WIDTH, 8), (200, 8, P.FFN_MAX_WIDTH),
    (P.FFN_MAX_TOKENS, 8, 8), (100001, 64, 72), (300000, 40, 24), (130, 264, 33000), (500, 33000, 264), (33000, 264, 520),
    (33000, 1024, 2048)])
def test_gated_ffn_long_sums(dtype, tokens, hidden, inter, parts):
    """The widest blocks and the longest batches keep the error of their roundings. (In one chain 2^22
    tokens lose 4e-3 of the weights' gradients: the tensor cores cut sums off.)"""
    dt = DT[dtype]
    x, w_in, w_out, g = ffn_inputs(tokens, hidden, inter, dt, 11)
    f = P.GatedFfn(w_in, w_out, parts=parts)
    y, pre, dy = torch.empty_like(x), torch.empty(tokens, 2 * inter, dtype=dt, device="cuda"), rnd(g, (tokens, hidden), dt)
    f(x, y, pre=pre, workspace=f.workspace(tokens))
    got = dict(d_x=torch.empty_like(x), d_w_in=torch.empty_like(w_in), d_w_out=torch.empty_like(w_out))
    f.backward(x, pre, dy, **got, workspace=f.backward_workspace(tokens))
    assert P.ptoc_wait_faults() == 0
    x, w_in, w_out, dy = (t.to(F64) for t in (x, w_in, w_out, dy))
    gu = x @ w_in.t()
    want = dict(pre=gu, y=(act64(gu[:, :inter], "silu")[0] * gu[:, inter:]) @ w_out.t())
    p = pre.to(F64)
    a, slope = act64(p[:, :inter], "silu")
    dh = dy @ w_out
    d = torch.cat([dh * p[:, inter:] * slope, dh * a], 1)
    want.update(d_x=d @ w_in, d_w_in=d.t() @ x, d_w_out=dy.t() @ (a * p[:, inter:]))
    for name, v in dict(got, y=y, pre=pre).items():
        once = float((want[name].to(dt).to(F64) - want[name]).norm() / want[name].norm())
        off = float((v.to(F64) - want[name]).norm() / want[name].norm())
        # one rounding, and of what enters the product another one (of the same size: independent of it), a tenth
        # for the few values that a result may have; a chain of 32768 elements (of the two parts 65536) cut off at every
        # 16th is off by at most 2^-24 for each of its sums on the average, which lie between 0 and the last one
        roundings = 1.1 * once * (2 ** 0.5 if parts == 1 else 1)
        assert off <= roundings + 2048 * 2.0 ** -25, "%s: %.3g, %.3g times a rounding" % (name, off, off / once)


@pytest.mark.parametrize("shared", [True, False])
def test_threads_at_once(shared):
    """Threads that call on one stream, launch between launch, or on a stream each, with tensors and
    workspaces of their own: the bits of calls one after another."""
    import threading
    dt, jobs = torch.bfloat16, []
    for k, tokens in enumerate((1, 33, 100, 200)):
        x, w_in, w_out, g = ffn_inputs(tokens, 512, 776, dt, k)
        f = P.GatedFfn(w_in, w_out, parts=1 + k % 2)
        pre, dy = torch.empty(tokens, 1552, dtype=dt, device="cuda"), rnd(g, (tokens, 512), dt)
        out = [torch.empty_like(v) for v in (x, x, w_in, w_out)]
        spaces = f.workspace(tokens), f.backward_workspace(tokens)
        result, normed = torch.empty(2, device="cuda"), torch.empty_like(x)
        grads = P.Gradients(out[2:], [torch.empty_like(v) for v in out[2:]])
        cs = grads.workspace()

        def run(stream, f=f, x=x, pre=pre, dy=dy, out=out, spaces=spaces, grads=grads, cs=cs, result=result, normed=normed):
            P.layer_norm([x], normed, stream=stream)
            f(normed, out[0], pre=pre, workspace=spaces[0], stream=stream)
            f.backward(normed, pre, dy, d_x=out[1], d_w_in=out[2], d_w_out=out[3], workspace=spaces[1], stream=stream)
            grads.clip(1.0, result, workspace=cs, stream=stream)
        jobs.append((run, out + grads.outs + [result, normed, pre]))
    one = torch.cuda.Stream()
    for run, _ in jobs:
        run(one)
    torch.cuda.synchronize()
    want = [[v.clone() for v in out] for _, out in jobs]
    for _, out in jobs:
        for v in out:
            v.zero_()
    torch.cuda.synchronize()
    failed = []

    def work(run, stream):
        try:
            for _ in range(30):
                run(stream)
        except Exception as e:                             # shown by the test's thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(run, one if shared else torch.cuda.Stream())) for run, _ in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and P.ptoc_wait_faults() == 0
    for (_, out), ref in zip(jobs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
