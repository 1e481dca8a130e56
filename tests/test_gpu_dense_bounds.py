"""The dense block's operators where a bound on the whole result hides an error.
Tolerances are derived as in test_gpu_dense.py."""
import pytest
import torch

import tile_level_collective_gb300 as P
from test_gpu_dense import F64, act64, check_clip
from test_gpu_layers import DT, E, TINY, U, close

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
