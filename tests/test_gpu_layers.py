"""The layer operators on the GPU against plain 64-bit implementations.

Tolerances are the a-priori rounding bounds of the documented arithmetic: one
rounding to the stored type (u * |value|, u = 2^-24, 2^-11, 2^-8 for f32, f16,
bf16), plus binary32 arithmetic over the terms of each formula (a multiple of
2^-24 of the sum of their magnitudes; the multiple counts the operations on
the longest path), plus half the smallest f16 step where results may be
subnormal. A checkpoint's codes, routing choices and copies are compared
exactly."""
import math

import pytest
import torch

import tile_level_collective_gb300 as P

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E = 2.0 ** -24
TINY = 2.0 ** -25          # half the smallest f16 step
FILL = 7.0                 # what surrounds an output and must survive


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, shape, dtype, std=1.0, mean=0.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(mean, std, generator=g)


class Box:
    """A [rows, cols] view inside a filled buffer: `pad` extra columns, `lead`
    elements before it (so that the base can be odd), a row after it."""

    def __init__(self, rows, cols, dtype, pad=0, lead=0, fill=FILL):
        self.ld = cols + pad
        self.raw = torch.full((lead + (rows + 1) * self.ld + 8,), fill, device="cuda").to(dtype)
        self.view = torch.as_strided(self.raw, (rows, cols), (self.ld, 1), lead)

    def outside_intact(self):
        keep = self.raw.clone()
        torch.as_strided(keep, self.view.shape, self.view.stride(), self.view.storage_offset()).fill_(FILL)
        return bool((keep.float() == FILL).all())


def close(got, want, bound, what=""):
    """|got - want| <= bound elementwise; equal NaNs and infinities agree."""
    got = got.double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~(same | ((got - want).abs() <= bound))
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g times its bound" % (
        what, int(bad.sum()), bad.numel(), float(((got - want).abs() / bound)[bad].max()))


# ---- checkpoints ---------------------------------------------------------------

def encode64(x):
    """Codes and exponent bytes of the definition, in 64 bits."""
    rows, cols = x.shape
    x = x.double()
    nb = (cols + 31) // 32
    v = torch.zeros(rows, nb * 32, dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, nb, 32)
    top = v.abs().amax(2)
    finite = torch.isfinite(v).all(2)
    e = torch.full_like(top, -127.0)
    for k in range(-127, 123):                                # the smallest e with top <= 127 * 2^e
        e = torch.where(top > 127.0 * 2.0 ** k, torch.full_like(e, k + 1.0), e)
    codes = torch.where(finite[..., None], torch.round(v * torch.exp2(-e)[..., None]), torch.zeros_like(v))
    byte = torch.where(finite, e + 127, torch.full_like(e, 255.0))
    return codes.view(rows, nb * 32)[:, :cols].to(torch.int8), byte.to(torch.uint8)


def decode64(codes, exps):
    scale = torch.exp2(exps.double() - 127)
    scale = torch.where(exps == 255, torch.full_like(scale, float("nan")), scale)
    return codes.double() * scale.repeat_interleave(32, 1)[:, :codes.shape[1]]


def same_values(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,lead", [(1, 1, 0, 0), (1, 32, 0, 0), (3, 31, 0, 0), (5, 33, 1, 1),
                                                (7, 255, 1, 0), (4, 256, 0, 0), (9, 1003, 5, 3), (2, 8192, 8, 8),
                                                (300, 520, 8, 0)])
def test_checkpoint_codes_and_values(dtype, rows, cols, pad, lead):
    g = gen(rows * 1000 + cols)
    src = Box(rows, cols, DT[dtype], pad, lead)
    src.view.copy_(rnd(g, (rows, cols), torch.float32) * torch.exp2(rnd(g, (rows, cols), torch.float32, 4.0).round()))
    k = P.Checkpoint8(rows, cols)
    P.checkpoint8(src.view, k)
    codes, exps = encode64(src.view)
    assert torch.equal(k.codes, codes) and torch.equal(k.exps, exps)
    for out_dtype in ("f32", "bf16", "f16"):
        dst = Box(rows, cols, DT[out_dtype], pad, lead)
        P.restore8(k, dst.view)
        assert same_values(dst.view, decode64(codes, exps).to(DT[out_dtype]))
        assert dst.outside_intact()


def test_checkpoint_of_special_values():
    """Zeros, subnormals, the largest floats, exact ties and 127-multiples,
    infinities and NaN, each filling a block of its own."""
    inf, nan, big = float("inf"), float("nan"), torch.finfo(torch.float32).max
    blocks = [[0.0], [-0.0, 0.0], [1e-45, -3e-45], [2.0 ** -126, 1.5 * 2.0 ** -140], [big, -big, 1.0],
              [127.0, 0.5, 1.5, 2.5, -0.5], [127.0000076, 1.0], [254.0, 1.0, 3.0], [inf, 1.0], [-inf], [nan, 2.0],
              [64.0, 63.5], [2.0 ** -120 * 127]]
    x = torch.zeros(2, 32 * len(blocks) + 3, device="cuda")
    for i, b in enumerate(blocks):
        for r in range(2):                    # the second row: the same values at the block's end
            at = 32 * i + (0 if r == 0 else 32 - len(b))
            x[r, at:at + len(b)] = torch.tensor(b, device="cuda")
    codes, exps = encode64(x)
    for view in (x, torch.cat([x, x], 1)[:, 1:x.shape[1] + 1]):       # aligned, and at an odd base
        src = x if view is x else torch.as_strided(view.contiguous(), x.shape, x.stride())
        k = P.Checkpoint8(*x.shape)
        P.checkpoint8(src, k)
        c, e = (codes, exps) if view is x else encode64(src)
        assert torch.equal(k.codes, c) and torch.equal(k.exps, e)
        out = torch.empty_like(x)
        P.restore8(k, out)
        assert same_values(out, decode64(c, e).float())            # the largest floats round up to 2^128


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [5, 37, 263, 1001, 1030])
def test_checkpoint_of_special_values_at_odd_rows(dtype, cols):
    """Infinities and NaN in the run that the end of a row cuts, in the first
    run and between, at every place of a row in its 16 bytes."""
    g, t = gen(cols), DT[dtype]
    src, dst = Box(17, cols, t, 1, 1), Box(17, cols, t, 1, 1)
    src.view.copy_(rnd(g, (17, cols), torch.float32))
    for r, c in ((1, cols - 1), (4, 0), (6, cols // 2), (9, cols - 2)):
        src.view[r, c] = float("nan") if r % 3 else float("inf")
    src.view[12] = 0
    k = P.Checkpoint8(17, cols)
    P.checkpoint8(src.view, k)
    codes, exps = encode64(src.view)
    assert torch.equal(k.codes, codes) and torch.equal(k.exps, exps)
    P.restore8(k, dst.view)
    assert same_values(dst.view, decode64(codes, exps).to(t))
    assert dst.outside_intact()


# ---- block_norm ------------------------------------------------------------------

def gate_shape(kind, rows, cols):
    return {"none": None, "scalar": (), "one": (1,), "channel": (cols,), "token": (rows, 1),
            "element": (rows, cols)}[kind]


def norm64(parts, x, wpost, wpre, gate, rs, bs, eps, post):
    """The forward pass, with the magnitudes that its rounding bounds need."""
    a, mag = torch.zeros_like(x.double()), torch.zeros_like(x.double())
    for p in parts:
        a, mag = a + p.double(), mag + p.double().abs()
    ra = 1 / torch.sqrt(a.square().mean(1, keepdim=True) + eps) if post else torch.ones_like(a[:, :1])
    w = wpost.double() if wpost is not None else 1.0
    g = gate.double() if gate is not None else torch.ones((), dtype=torch.float64, device=x.device)
    n = a * ra * w if post else a
    s = rs * x.double() + bs * g * n
    r = 1 / torch.sqrt(s.square().mean(1, keepdim=True) + eps)
    v = wpre.double() if wpre is not None else 1.0
    size = abs(rs) * x.double().abs() + abs(bs) * g.abs() * mag * ra * (w.abs() if wpost is not None and post else 1.0)
    # a's own error reaches s through ra too: relative to the row's rms
    row = size.square().mean(1, keepdim=True).sqrt()
    return dict(a=a, ra=ra, n=n, s=s, r=r, y=s * r * v, mag=mag, size=size,
                ysize=(size + s.abs() * r * row) * r * (v.abs() if wpre is not None else 1.0))


# the longest chain of binary32 operations on a row: 8 columns of up to 4 chunks
# in one thread, 5 + 5 exchange steps, and the handful of the formula; each
# of the parts adds one
CHAIN = 64

CASES = [
    # dtype, rows, cols, parts, gate, post, pad, lead
    ("bf16", 1, 7168, 8, "channel", True, 0, 0),
    ("bf16", 5, 1, 1, "scalar", True, 0, 0),
    ("f32", 3, 7, 2, "none", True, 0, 0),
    ("f16", 4, 64, 3, "element", True, 0, 0),
    ("bf16", 9, 257, 1, "token", False, 7, 0),
    ("f32", 33, 1003, 4, "token", True, 2, 1),
    ("f16", 17, 1000, 5, "channel", False, 8, 8),
    ("bf16", 6, 4096, 16, "element", True, 64, 0),
    ("bf16", 3, 8200, 2, "channel", True, 0, 0),
    ("f32", 2, 12000, 9, "one", True, 4, 4),
    ("f16", 2, 20001, 1, "none", True, 1, 1),
    ("bf16", 2, 32768, 2, "channel", True, 0, 0),
    ("f32", 700, 96, 64, "none", False, 0, 0),
    ("bf16", 400, 4097, 3, "channel", True, 0, 0),         # odd pitch, more rows than blocks
    ("f16", 701, 1031, 1, "scalar", True, 0, 0),
    ("f32", 350, 2051, 2, "token", True, 1, 0),
    ("bf16", 40, 8191, 2, "channel", True, 2, 0),
    ("f16", 33, 515, 13, "token", True, 0, 1),             # odd base
    ("f32", 17, 8190, 1, "channel", False, 0, 3),
    ("bf16", 5, 9001, 2, "token", True, 0, 0),
]


def norm_inputs(dtype, rows, cols, parts, gate, post, pad, lead, params_f32=False, seed=0):
    g = gen(seed + rows + 7 * cols)
    t, q = DT[dtype], torch.float32 if params_f32 else DT[dtype]
    box = [Box(rows, cols, t, pad, lead) for _ in range(parts)]
    for b in box:
        b.view.copy_(rnd(g, (rows, cols), torch.float32))
    x = Box(rows, cols, t, pad, lead)
    x.view.copy_(rnd(g, (rows, cols), torch.float32, 3.0))
    shape = gate_shape(gate, rows, cols)
    return dict(parts=[b.view for b in box], x=x.view, wpost=rnd(g, (cols,), q, 0.2, 1.0) if post else None,
                wpre=rnd(g, (cols,), q, 0.2, 1.0), gate=None if shape is None else rnd(g, shape, q, 0.4, 0.6))


def check_norm(case, params_f32=False, **given):
    dtype, rows, cols, parts, gate, post, pad, lead = case
    d = dict(norm_inputs(*case, params_f32=params_f32), **given)
    t, rs, bs, eps = DT[dtype], 0.75, -1.5, 1e-5
    out, normed, blk = (Box(rows, cols, t, pad, lead) for _ in range(3))
    rstd = torch.empty(2, rows, device="cuda")
    bk, sk = P.Checkpoint8(rows, cols), P.Checkpoint8(rows, cols)
    P.block_norm(d["parts"], d["x"], out.view, normed.view, post_norm=post, post_weight=d["wpost"],
                 pre_weight=d["wpre"], gate=d["gate"], residual_scale=rs, branch_scale=bs, eps=eps,
                 block_out=blk.view, block_ckpt=bk, stream_ckpt=sk, rstd=rstd)
    f = norm64(d["parts"], d["x"], d["wpost"], d["wpre"], d["gate"], rs, bs, eps, post)
    c = (CHAIN + parts) * E
    close(out.view, f["s"], U[t] * f["s"].abs() + c * f["size"] + TINY, "stream")
    close(normed.view, f["y"], U[t] * f["y"].abs() + c * f["ysize"] + TINY, "normed")
    close(blk.view, f["a"], U[t] * f["a"].abs() + c * f["mag"] + TINY, "block_out")
    # a statistic's relative error: that of its positive sum, and twice that of a
    rel = c * (1 + 2 * (f["mag"].square().mean(1) / f["a"].square().mean(1).clamp_min(1e-300)).sqrt())
    close(rstd[0], f["ra"][:, 0], f["ra"][:, 0] * (rel if post else 0 * rel), "ra")
    rel = c * (1 + 2 * (f["size"].square().mean(1) / f["s"].square().mean(1).clamp_min(1e-300)).sqrt())
    close(rstd[1], f["r"][:, 0], f["r"][:, 0] * rel, "r")
    # a checkpoint of what is stored: the stream's codes are those of the stored
    # stream, the block's those of the binary32 sum in rank order
    sum32 = d["parts"][0].float()
    for p in d["parts"][1:]:
        sum32 = sum32 + p.float()
    for k, src in ((bk, sum32), (sk, out.view)):
        codes, exps = encode64(src)
        assert torch.equal(k.codes, codes) and torch.equal(k.exps, exps)
    assert torch.equal(blk.view, sum32.to(t))
    for b in (out, normed, blk):
        assert b.outside_intact()
    return d, out, normed, rstd


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_block_norm(case):
    check_norm(case)


def test_block_norm_with_f32_parameters():
    for case in (CASES[0], CASES[3], CASES[4], CASES[6]):
        check_norm(case, params_f32=True)


def test_block_norm_sum_is_the_collective_sum():
    """block_out has the bits that treduce leaves for the same windows."""
    d = norm_inputs("bf16", 13, 520, 7, "none", True, 0, 0)
    out, blk, dst = (torch.empty(13, 520, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    P.block_norm(d["parts"], d["x"], out, block_out=blk)
    P.treduce(d["parts"], dst)
    assert torch.equal(blk, dst)


def test_block_norm_in_place_and_defaults():
    d = norm_inputs("f16", 21, 776, 3, "none", True, 0, 0)
    out, normed = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    P.block_norm(d["parts"], d["x"], out, normed)
    f = norm64(d["parts"], d["x"], None, None, None, 1.0, 1.0, 1e-6, True)
    close(out, f["s"], U[torch.float16] * f["s"].abs() + (CHAIN + 3) * E * f["size"] + TINY)
    x = d["x"].clone()
    n2 = torch.empty_like(normed)
    P.block_norm(d["parts"], x, x, n2)
    assert torch.equal(x, out) and torch.equal(n2, normed)
    x = d["x"].clone()
    P.block_norm(d["parts"], x, x)                                # no norm before a next block
    assert torch.equal(x, out)


@pytest.mark.parametrize("cols", [72, 1003, 9000])
def test_block_norm_rows_of_zeros_and_specials(cols):
    """A row of zeros stays zero (eps bounds the statistic); infinities and NaN
    stay in their rows."""
    d = norm_inputs("f32", 6, cols, 2, "none", True, 0, 0)
    for p in d["parts"]:
        p[1] = 0
    d["x"][1] = 0
    d["parts"][0][2, cols // 2] = float("nan")
    d["x"][3, 5] = float("inf")
    d["parts"][1][4, cols - 1] = float("-inf")
    out, normed = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    P.block_norm(d["parts"], d["x"], out, normed, post_weight=d["wpost"], pre_weight=d["wpre"])
    assert bool((out[1] == 0).all()) and bool((normed[1] == 0).all())
    assert bool(torch.isfinite(out[[0, 5]]).all()) and bool(torch.isfinite(normed[[0, 5]]).all())
    f = norm64(d["parts"], d["x"], d["wpost"], d["wpre"], None, 1.0, 1.0, 1e-6, True)
    for r in (2, 3, 4):
        assert torch.equal(torch.isnan(out[r]), torch.isnan(f["s"][r])), r
        assert torch.equal(torch.isnan(normed[r]), torch.isnan(f["y"][r])), r


def back64(a, s, ra, r, dy, du, wpost, wpre, gate, rs, bs, post):
    a, s, dy, ra, r = a.double(), s.double(), dy.double(), ra.double()[:, None], r.double()[:, None]
    wpre = wpre.double() if wpre is not None else torch.ones_like(s[0])
    wpost = wpost.double() if wpost is not None else torch.ones_like(s[0])
    g = gate.double() if gate is not None else torch.ones((), dtype=torch.float64, device=s.device)
    sh, up = s * r, wpre * dy
    ds = r * (up - sh * (up * sh).mean(1, keepdim=True))
    mds = r * (up.abs() + sh.abs() * (up * sh).abs().mean(1, keepdim=True))
    if du is not None:
        ds, mds = ds + du.double(), mds + du.double().abs()
    dn, mdn = bs * g * ds, abs(bs) * g.abs() * mds
    ah = a * ra if post else a
    n = ah * wpost if post else a
    if post:
        da = ra * (wpost * dn - ah * (wpost * dn * ah).mean(1, keepdim=True))
        mda = ra * (wpost.abs() * mdn + ah.abs() * (wpost.abs() * mdn * ah.abs()).mean(1, keepdim=True))
    else:
        da, mda = dn, mdn
    dg, mdg = bs * ds * n, abs(bs) * mds * n.abs()
    return dict(dx=rs * ds, mdx=abs(rs) * mds, da=da, mda=mda, dpre=(dy * sh).sum(0), mpre=(dy * sh).abs().sum(0),
                dpost=(dn * ah).sum(0), mpost=(mdn * ah.abs()).sum(0), dg=dg, mdg=mdg)


def reduce_gate(t, shape):
    """Sum a [rows, cols] tensor to the gate's shape."""
    full = (1,) * (2 - len(shape)) + tuple(shape)
    for axis in (0, 1):
        if full[axis] == 1:
            t = t.sum(axis, keepdim=True)
    return t.reshape(shape)


def check_back(case, ckpt, with_du=True, params_f32=False):
    dtype, rows, cols, _, gate, post, pad, lead = case
    t, rs, bs = DT[dtype], 0.75, -1.5
    d = norm_inputs(dtype, rows, cols, 1, gate, post, pad, lead, params_f32=params_f32)
    g = gen(99 + cols)
    a, s = d["parts"][0], d["x"]
    rstd = torch.stack([1 / (a.float().square().mean(1) + 1e-5).sqrt(), 1 / (s.float().square().mean(1) + 1e-5).sqrt()])
    dy, du = Box(rows, cols, t, pad, lead), Box(rows, cols, t, pad, lead)
    dy.view.copy_(rnd(g, (rows, cols), torch.float32))
    du.view.copy_(rnd(g, (rows, cols), torch.float32))
    a_in, s_in = a, s
    if ckpt:
        a_in, s_in = P.Checkpoint8(rows, cols), P.Checkpoint8(rows, cols)
        P.checkpoint8(a, a_in)
        P.checkpoint8(s, s_in)
        a, s = decode64(a_in.codes, a_in.exps), decode64(s_in.codes, s_in.exps)
    dx, da = Box(rows, cols, t, pad, lead), Box(rows, cols, t, pad, lead)
    dpre = torch.full((cols,), FILL, device="cuda")
    dpost = torch.full((cols,), FILL, device="cuda") if post else None
    dg = None if d["gate"] is None else torch.full(d["gate"].shape, FILL, device="cuda")
    P.block_norm_backward(a_in, s_in, rstd, dy.view, dx.view, da.view, dpre, d_post_weight=dpost, d_gate=dg,
                          d_stream=du.view if with_du else None, post_norm=post, post_weight=d["wpost"],
                          pre_weight=d["wpre"], gate=d["gate"], residual_scale=rs, branch_scale=bs,
                          workspace=P.block_norm_backward_workspace(rows, cols))
    f = back64(a, s, rstd[0], rstd[1], dy.view, du.view if with_du else None, d["wpost"], d["wpre"], d["gate"], rs, bs,
               post)
    c = 2 * CHAIN * E                              # two statistics, one after the other
    close(dx.view, f["dx"], U[t] * f["dx"].abs() + c * f["mdx"] + TINY, "d_residual")
    close(da.view, f["da"], U[t] * f["da"].abs() + c * f["mda"] + TINY, "d_block")
    sums = c + (rows + 8) * E                      # a chain over the rows in the worst case
    close(dpre, f["dpre"], sums * f["mpre"], "d_pre_weight")
    if post:
        close(dpost, f["dpost"], sums * f["mpost"], "d_post_weight")
    if dg is not None:
        close(dg, reduce_gate(f["dg"], dg.shape), (sums + CHAIN * E) * reduce_gate(f["mdg"], dg.shape), "d_gate")
    assert dx.outside_intact() and da.outside_intact()


@pytest.mark.parametrize("ckpt", [False, True], ids=["saved", "ckpt"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_block_norm_backward(case, ckpt):
    check_back(case, ckpt)


def test_block_norm_backward_variants():
    check_back(("bf16", 40, 2056, 1, "channel", True, 0, 0), True, with_du=False)
    check_back(("f16", 11, 515, 1, "scalar", True, 0, 0), False, params_f32=True)
    check_back(("bf16", 2000, 264, 1, "channel", True, 0, 0), True)           # more rows than blocks
    check_back(("bf16", 1500, 4096, 1, "scalar", True, 0, 0), True)
    check_back(("f32", 900, 135, 1, "token", False, 0, 0), False)


def test_block_norm_gradients_against_differences():
    """Central differences of <y, dy> + <s, du> in 64 bits along random
    directions of every input, against the kernel's gradients in binary32.
    The difference quotient's own error (h^2 times third derivatives of order
    one, and cancellation at 2^-53 / h) is below 1e-6 of the magnitudes."""
    rows, cols, eps, rs, bs = 6, 41, 1e-3, 0.75, -1.5
    g = gen(5)
    f64 = torch.float64
    v = {k: rnd(g, sh, torch.float32).to(f64) for k, sh in
         dict(p0=(rows, cols), p1=(rows, cols), x=(rows, cols), wpost=(cols,), wpre=(cols,), gate=(cols,),
              dy=(rows, cols), du=(rows, cols)).items()}

    def loss(q):
        f = norm64([q["p0"], q["p1"]], q["x"], q["wpost"], q["wpre"], q["gate"], rs, bs, eps, True)
        return (f["y"] * v["dy"]).sum() + (f["s"] * v["du"]).sum()

    q32 = {k: t.float() for k, t in v.items()}
    out, normed, blk = (torch.empty(rows, cols, device="cuda") for _ in range(3))
    rstd = torch.empty(2, rows, device="cuda")
    P.block_norm([q32["p0"], q32["p1"]], q32["x"], out, normed, post_weight=q32["wpost"], pre_weight=q32["wpre"],
                 gate=q32["gate"], residual_scale=rs, branch_scale=bs, eps=eps, block_out=blk, rstd=rstd)
    dx, da = torch.empty_like(out), torch.empty_like(out)
    dpre, dpost, dgate = (torch.empty(cols, device="cuda") for _ in range(3))
    P.block_norm_backward(blk, out, rstd, q32["dy"], dx, da, dpre, d_post_weight=dpost, d_gate=dgate,
                          d_stream=q32["du"], post_weight=q32["wpost"], pre_weight=q32["wpre"], gate=q32["gate"],
                          residual_scale=rs, branch_scale=bs, eps=eps,
                          workspace=P.block_norm_backward_workspace(rows, cols))
    grads = dict(p0=da, p1=da, x=dx, wpost=dpost, wpre=dpre, gate=dgate)
    h = 1e-5
    for k, grad in grads.items():
        for trial in range(3):
            u = rnd(g, tuple(v[k].shape), torch.float32).to(f64)
            plus, minus = (loss(dict(v, **{k: v[k] + sign * h * u})) for sign in (1, -1))
            want = float((plus - minus) / (2 * h))
            got = float((grad.double() * u).sum())
            size = float((grad.double() * u).abs().sum())
            assert abs(got - want) <= 1e-5 * size + 1e-6, (k, got, want)


def test_block_norm_backward_empty_rows_clear_the_sums():
    z = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    dpre, dpost, dgate = (torch.full((64,), FILL, device="cuda") for _ in range(3))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    P.block_norm_backward(z, z, torch.empty(2, 0, device="cuda"), z, z.clone(), z.clone(), dpre, d_post_weight=dpost,
                          d_gate=dgate, post_weight=w, gate=w, workspace=P.block_norm_backward_workspace(0, 64))
    assert all(bool((t == 0).all()) for t in (dpre, dpost, dgate))
    P.block_norm([z], z, z)


# ---- the mixture of experts --------------------------------------------------------

def route64(logits, bias, top_k, score, renorm, scale):
    sc = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    key = logits if score == "softmax" and bias is None else sc + (bias.double() if bias is not None else 0)
    key = torch.where(torch.isnan(key), torch.full_like(key, -math.inf), key)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top_k]
    w = sc.gather(1, ids)
    return ids, (w / w.sum(1, keepdim=True) if renorm else w) * scale


def moe_case(tokens, hidden, inter, experts, first, local, top_k, dtype, score="softmax", bias=False, renorm=True,
             router_f32=False, pad=0, lead=0, seed=0, w_lead=0):
    g = gen(seed + tokens + hidden)
    t = DT[dtype]
    x = Box(tokens, hidden, t, pad, lead)
    x.view.copy_(rnd(g, (tokens, hidden), torch.float32))
    def packed(shape, std):
        n = math.prod(shape)
        return rnd(g, (n + w_lead,), t, std)[w_lead:].view(shape)
    router = rnd(g, (experts, hidden), torch.float32 if router_f32 else t, 2 / math.sqrt(hidden))
    b = rnd(g, (experts,), torch.float32, 0.1) if bias else None
    w_in = packed((local, 2 * inter, hidden), 1 / math.sqrt(hidden))
    w_out = packed((local, hidden, inter), 1 / math.sqrt(inter))
    scale = 1.75
    y = Box(tokens, hidden, t, pad, lead)
    ids = torch.full((tokens, top_k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((tokens, top_k), FILL, device="cuda")
    layer = P.MoeLayer(router, w_in, w_out, top_k, bias=b, first_expert=first, score=score, renormalize=renorm,
                       scale=scale)
    layer(x.view, y.view, ids=ids, weights=w, workspace=layer.workspace(tokens))
    assert y.outside_intact()

    xd, rd = x.view.double(), router.double()
    logits = xd @ rd.t()
    err = hidden * E * (xd.abs() @ rd.abs().t())                   # of a logit
    # every choice is the exact one, or its key is as large to within the keys'
    # error (a score's slope is at most 1); ties are tested on exact logits below
    want_ids = route64(logits, b, top_k, score, renorm, scale)[0]
    key = logits if score == "softmax" and b is None else \
        (torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)) + (0 if b is None else b.double())
    chosen = ids.long()
    assert bool(((chosen >= 0) & (chosen < experts)).all())
    assert all(len(set(row)) == top_k for row in chosen.tolist())
    off = (key.gather(1, chosen) - key.gather(1, want_ids)).abs()
    assert bool((off <= 2 * err.amax(1, keepdim=True) + 16 * E).all())
    want_ids = chosen
    w_all = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    want_w = w_all.gather(1, chosen)
    want_w = (want_w / want_w.sum(1, keepdim=True) if renorm else want_w) * scale
    # exp(d) - 1 for a logit error d, on the score and on the sum
    rel = 4 * err.amax(1, keepdim=True) + 32 * E
    close(w, want_w, rel * want_w.abs() + E * 1e-6, "weights")

    want, bound = torch.zeros_like(xd), torch.zeros_like(xd)
    c1, c2 = hidden * E, inter * E
    for e in range(local):
        hit = want_ids == first + e
        for tok in torch.nonzero(hit.any(1))[:, 0].tolist():
            we = (want_w[tok] * hit[tok]).sum()
            wi, wo = w_in[e].double(), w_out[e].double()
            gu, mag = wi @ xd[tok], wi.abs() @ xd[tok].abs()
            gt, up = gu[:inter], gu[inter:]
            act = gt / (1 + torch.exp(-gt))
            h = we * act * up
            # silu's slope is at most 1.1; one rounding of h to the type
            dh = we * (1.1 * c1 * mag[:inter] * up.abs() + act.abs() * c1 * mag[inter:]) + \
                h.abs() * (rel[tok] + 8 * E + U[t]) + (TINY if t == torch.float16 else 0.0)
            want[tok] += wo @ h
            bound[tok] += wo.abs() @ dh + c2 * (wo.abs() @ h.abs())
    close(y.view, want, bound * 1.01 + U[t] * want.abs() + TINY, "y")
    return ids, y.view


MOE = [
    # tokens, hidden, inter, experts, first, local, top_k, dtype
    (1, 64, 64, 4, 0, 4, 2, "bf16"),
    (1, 7168, 256, 16, 0, 16, 8, "bf16"),
    (2, 72, 40, 8, 2, 3, 3, "f16"),
    (5, 520, 136, 60, 0, 60, 4, "bf16"),
    (13, 1000, 200, 16, 8, 8, 6, "f16"),
    (16, 256, 512, 8, 0, 8, 8, "bf16"),
    (17, 384, 64, 128, 32, 64, 8, "bf16"),
    (31, 136, 1000, 5, 0, 5, 1, "f16"),
    (33, 2048, 96, 32, 0, 32, 4, "bf16"),
    (48, 512, 128, 16, 4, 1, 2, "bf16"),
    (64, 1024, 320, 40, 0, 40, 5, "bf16"),
    (64, 128, 64, 1, 0, 1, 1, "f16"),
    (7, 640, 192, 1024, 0, 64, 16, "bf16"),
    # not multiples of 8
    (3, 33, 17, 4, 0, 4, 2, "bf16"),
    (9, 1001, 65, 12, 3, 9, 4, "f16"),
    (64, 100, 30, 6, 0, 6, 3, "bf16"),
]


@pytest.mark.parametrize("case", MOE, ids=lambda c: "-".join(str(v) for v in c))
def test_moe(case):
    moe_case(*case)


def test_moe_scores_and_layouts():
    moe_case(11, 264, 72, 24, 0, 24, 5, "bf16", score="sigmoid", bias=True)
    moe_case(11, 264, 72, 24, 6, 12, 5, "f16", score="softmax", bias=True, renorm=False)
    moe_case(20, 264, 72, 24, 0, 24, 5, "bf16", score="sigmoid", renorm=False, router_f32=True)
    moe_case(6, 256, 64, 16, 0, 16, 4, "bf16", pad=8)                # a pitch above the width, aligned
    moe_case(6, 256, 64, 16, 0, 16, 4, "bf16", pad=3, lead=1)        # x and y at odd places
    moe_case(6, 256, 64, 16, 0, 16, 4, "bf16", w_lead=1)             # weights at odd places


def test_moe_many_tokens_choose_one_expert():
    """Every token's first choice is one expert: 64 rows for it, few for others."""
    tokens, hidden, inter, experts = 64, 256, 96, 12
    g = gen(3)
    x = rnd(g, (tokens, hidden), torch.bfloat16)
    x[:, 0] = 8.0
    router = rnd(g, (experts, hidden), torch.bfloat16, 0.05)
    router[:, 0] = 0
    router[7, 0] = 4.0
    w_in = rnd(g, (experts, 2 * inter, hidden), torch.bfloat16, 1 / 16)
    w_out = rnd(g, (experts, hidden, inter), torch.bfloat16, 0.1)
    layer = P.MoeLayer(router, w_in, w_out, 1)
    y = torch.empty_like(x)
    ids = torch.empty(tokens, 1, dtype=torch.int32, device="cuda")
    layer(x, y, ids=ids, workspace=layer.workspace(tokens))
    assert bool((ids == 7).all())
    gu = x.double() @ w_in[7].double().t()
    h = torch.nn.functional.silu(gu[:, :inter]) * gu[:, inter:]
    want = h @ w_out[7].double().t()
    size = h.abs() @ w_out[7].double().abs().t()
    close(y, want, 2 * U[torch.bfloat16] * size + U[torch.bfloat16] * want.abs(), "y")


def test_moe_ties_and_absent_experts():
    """Equal logits go to the lowest index (exact in every summation order:
    small integers), and a token without a local expert gets a row of zeros."""
    tokens, hidden, experts, k = 9, 64, 32, 5
    g = gen(8)
    x = torch.randint(-2, 3, (tokens, hidden), generator=g, device="cuda").to(torch.bfloat16)
    router = torch.randint(-1, 2, (experts, hidden), generator=g, device="cuda").to(torch.bfloat16)
    router[9] = router[4]
    router[20:28] = 0
    x[0] = 0                                                        # every logit is zero
    w_in = rnd(g, (2, 128, hidden), torch.bfloat16)
    w_out = rnd(g, (2, hidden, 64), torch.bfloat16)
    layer = P.MoeLayer(router, w_in, w_out, k, first_expert=30)
    y = torch.full((tokens, hidden), FILL, device="cuda").to(torch.bfloat16)
    ids = torch.empty(tokens, k, dtype=torch.int32, device="cuda")
    layer(x, y, ids=ids, workspace=layer.workspace(tokens))
    want = torch.sort(x.double() @ router.double().t(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    assert ids[0].tolist() == [0, 1, 2, 3, 4]
    none = ~(want >= 30).any(1)
    assert bool(none.any()) and bool((y[none] == 0).all())


def test_moe_nan_and_infinite_logits_choose_valid_experts():
    hidden, experts, k = 64, 8, 3
    g = gen(2)
    x = rnd(g, (4, hidden), torch.bfloat16)
    x[1, 3] = float("nan")                       # every logit of token 1 is NaN
    router = rnd(g, (experts, hidden), torch.bfloat16)
    router[2, 0] = float("nan")                  # expert 2 is the last choice of every token
    router[5, 1] = float("inf")
    layer = P.MoeLayer(router, rnd(g, (8, 64, hidden), torch.bfloat16), rnd(g, (8, hidden, 32), torch.bfloat16), k)
    y = torch.empty_like(x)
    ids = torch.empty(4, k, dtype=torch.int32, device="cuda")
    layer(x, y, ids=ids, workspace=layer.workspace(4))
    assert ids[1].tolist() == [0, 1, 2]
    for t in (0, 2, 3):
        row = ids[t].tolist()
        assert len(set(row)) == k and 2 not in row and all(0 <= e < experts for e in row)
        logits = (x[t].double() @ router.double().t()).nan_to_num(nan=-math.inf)
        assert row == torch.sort(logits, descending=True, stable=True).indices[:k].tolist()
    assert bool(torch.isnan(y[1]).all())


@pytest.mark.parametrize("tokens, hidden, inter, first, local", [
    (1, 64, 64, 0, 4), (5, 512, 320, 0, 8), (40, 4096, 128, 2, 4), (20, 40960, 64, 0, 8), (9, 100, 36, 0, 8)])
def test_moe_infinite_and_nan_weights_stay_with_their_expert(tokens, hidden, inter, first, local):
    """Only tokens that chose the expert see what its w_out holds; the products
    of all tokens are taken together, in tiles that one block sums or several."""
    g, t, experts, k = gen(hidden + tokens), torch.bfloat16, 8, 2
    x, router = rnd(g, (tokens, hidden), t), rnd(g, (experts, hidden), t, 0.1)
    w_in = rnd(g, (local, 2 * inter, hidden), t, 1 / math.sqrt(hidden))
    w_out = rnd(g, (local, hidden, inter), t, 1 / math.sqrt(inter))
    layer = P.MoeLayer(router, w_in, w_out, k, first_expert=first)
    ids = torch.empty(tokens, k, dtype=torch.int32, device="cuda")
    w = torch.empty(tokens, k, device="cuda")
    clean, y = torch.empty_like(x), torch.empty_like(x)
    layer(x, clean, ids=ids, weights=w, workspace=layer.workspace(tokens))
    w_out[1, 3::5, inter // 2] = float("nan")
    w_out[2, 4::5, inter - 1] = float("inf")
    layer(x, y, workspace=layer.workspace(tokens))
    # sizes of the sums, for the binary32 roundings of a sum in another order
    size = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    hit = torch.zeros(tokens, local, dtype=torch.bool, device="cuda")
    for e in range(local):
        of = torch.where(ids == first + e, w, torch.zeros_like(w)).sum(1).double()
        hit[:, e] = (ids == first + e).any(1)
        a = x.double() @ w_in[e].double().t()
        h = (of[:, None] * torch.nn.functional.silu(a[:, :inter]) * a[:, inter:]).abs()
        size += 1.02 * h @ w_out[e].nan_to_num(nan=1.0, posinf=1.0).double().abs().t()
    nan_cols = torch.zeros(hidden, dtype=torch.bool, device="cuda")
    inf_cols = nan_cols.clone()
    nan_cols[3::5], inf_cols[4::5] = True, True
    gone = hit[:, 1:2] & nan_cols | hit[:, 2:3] & inf_cols
    assert torch.equal(~torch.isfinite(y), gone)
    assert torch.equal(torch.isnan(y) & nan_cols, hit[:, 1:2] & nan_cols)
    keep = lambda v: torch.where(gone, torch.zeros_like(v), v)
    close(keep(y), keep(clean).double(), 2 * (k * inter + 8) * E * size + 2 * U[t] * clean.double().abs(), "y")


def test_moe_parts_of_expert_parallel_ranks_add_up():
    """Each rank's y is its part: block_norm over the ranks' parts equals
    block_norm over the whole layer's output, to the parts' rounding."""
    tokens, hidden, inter, experts, k = 12, 512, 128, 16, 4
    g = gen(31)
    t = torch.bfloat16
    x = rnd(g, (tokens, hidden), t)
    router = rnd(g, (experts, hidden), t, 0.1)
    w_in, w_out = rnd(g, (experts, 2 * inter, hidden), t, 0.05), rnd(g, (experts, hidden, inter), t, 0.1)
    ranks, per = 4, 4
    parts = [torch.empty_like(x) for _ in range(ranks)]
    for r in range(ranks):
        layer = P.MoeLayer(router, w_in[r * per:(r + 1) * per], w_out[r * per:(r + 1) * per], k, first_expert=r * per)
        layer(x, parts[r], workspace=layer.workspace(tokens))
    layer, whole = P.MoeLayer(router, w_in, w_out, k), torch.empty_like(x)
    layer(x, whole, workspace=layer.workspace(tokens))
    sizes = sum(p.double().abs() for p in parts)
    close(whole, sum(p.double() for p in parts), 2 * U[t] * sizes + U[t] * whole.double().abs(), "sum of parts")


def test_moe_recovers_from_waits_that_gave_up(monkeypatch):
    """With a bound of 1 ns a wait may give up (valid copies that are merely
    not there yet): the call returns, the count says so, and the next call with
    the default bound is right."""
    g = gen(12)
    x = rnd(g, (9, 512), torch.bfloat16)
    layer = P.MoeLayer(rnd(g, (16, 512), torch.bfloat16, 0.1), rnd(g, (16, 256, 512), torch.bfloat16, 0.05),
                       rnd(g, (16, 512, 128), torch.bfloat16, 0.1), 4)
    want, got, ws = torch.empty_like(x), torch.empty_like(x), layer.workspace(9)
    torch.cuda.synchronize()
    P.ptoc_wait_faults()
    layer(x, want, workspace=ws)
    torch.cuda.synchronize()
    assert P.ptoc_wait_faults() == 0
    monkeypatch.setenv("PTOC_WAIT_NS", "1")
    layer(x, got, workspace=ws)
    torch.cuda.synchronize()
    faults = P.ptoc_wait_faults()
    monkeypatch.delenv("PTOC_WAIT_NS")
    assert faults > 0 or torch.equal(got, want)
    layer(x, got, workspace=ws)
    torch.cuda.synchronize()
    assert P.ptoc_wait_faults() == 0 and torch.equal(got, want)


# ---- offsets past 32 bits -----------------------------------------------------------------

def rows_at(pitch, dtype=torch.bfloat16, cols=1000):
    """Three rows at any pitch, whose memory between them stays untouched."""
    raw = torch.empty(2 * pitch + cols, dtype=dtype, device="cuda")
    return torch.as_strided(raw, (3, cols), (pitch, 1))


@pytest.mark.parametrize("near, far", [(1008, 2 ** 30 + 8), (1001, 2 ** 30 + 1)])
def test_rows_past_32_bits_have_the_same_bits(near, far):
    g, cols = gen(5), 1000
    given = [rnd(g, (3, cols), torch.bfloat16) for _ in range(4)]
    w = rnd(g, (cols,), torch.bfloat16, 0.2, 1.0)
    results = []
    for pitch in (near, far):
        part, x, dy, du = (rows_at(pitch).copy_(v) for v in given)
        out, normed, restored, dx, da = (rows_at(pitch) for _ in range(5))
        bk, sk, nk = (P.Checkpoint8.of(rows_at(pitch, torch.int8), rows_at(pitch, torch.uint8, 32)) for _ in range(3))
        rstd, dw = torch.empty(2, 3, device="cuda"), torch.empty(cols, device="cuda")
        P.block_norm([part], x, out, normed, post_weight=w, pre_weight=w, gate=w, block_ckpt=bk, stream_ckpt=sk,
                     rstd=rstd)
        P.checkpoint8(normed, nk)
        P.restore8(nk, restored)
        P.block_norm_backward(bk, sk, rstd, dy, dx, da, dw, d_stream=du, post_weight=w, pre_weight=w, gate=w,
                              workspace=P.block_norm_backward_workspace(3, cols))
        results.append([v.clone() for v in (out, normed, restored, dx, da, rstd, dw, bk.codes, bk.exps, sk.codes,
                                            sk.exps, nk.codes, nk.exps)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    f = norm64([given[0]], given[1], w, w, w, 1.0, 1.0, 1e-6, True)
    close(results[1][0], f["s"], U[torch.bfloat16] * f["s"].abs() + (CHAIN + 1) * E * f["size"])


def test_many_rows():
    """More than 2^31 elements; the rows at the end are compared."""
    rows, cols, t = 2 ** 21 + 3, 1032, torch.bfloat16
    g = gen(6)
    part, x = rnd(g, (rows, cols), t), rnd(g, (rows, cols), t)
    out, normed, k = torch.empty_like(x), torch.empty_like(x), P.Checkpoint8(rows, cols)
    rstd = torch.empty(2, rows, device="cuda")
    P.block_norm([part], x, out, normed, rstd=rstd)
    f = norm64([part[-50:]], x[-50:], None, None, None, 1.0, 1.0, 1e-6, True)
    close(out[-50:], f["s"], U[t] * f["s"].abs() + (CHAIN + 1) * E * f["size"])
    close(normed[-50:], f["y"], U[t] * f["y"].abs() + (CHAIN + 1) * E * f["ysize"])
    P.checkpoint8(out, k)
    codes, exps = encode64(out[-50:])
    assert torch.equal(k.codes[-50:], codes) and torch.equal(k.exps[-50:], exps)
    dx, da = x, torch.empty_like(x)
    P.block_norm_backward(part, out, rstd, normed, dx, da, workspace=P.block_norm_backward_workspace(rows, cols))
    b = back64(part[-50:], out[-50:], rstd[0, -50:], rstd[1, -50:], normed[-50:], None, None, None, None, 1.0, 1.0, True)
    close(dx[-50:], b["dx"], U[t] * b["dx"].abs() + 2 * CHAIN * E * b["mdx"])
    close(da[-50:], b["da"], U[t] * b["da"].abs() + 2 * CHAIN * E * b["mda"])
    P.restore8(k, dx)
    assert same_values(dx[-50:], decode64(codes, exps).to(t))


def test_moe_weights_past_32_bits():
    ids, _ = moe_case(8, 8192, 2048, 72, 0, 72, 16, "bf16")
    assert int(ids.max()) >= 64                                        # past 2^31 elements of w_in


# ---- streams, graphs, repeats ---------------------------------------------------------

def test_repeats_have_the_same_bits_and_streams_and_graphs_work():
    rows, cols = 333, 1024
    d = norm_inputs("bf16", rows, cols, 2, "channel", True, 0, 0)
    g = gen(1)
    layer = P.MoeLayer(rnd(g, (16, cols), torch.bfloat16, 0.1), rnd(g, (16, 256, cols), torch.bfloat16, 0.03),
                       rnd(g, (16, cols, 128), torch.bfloat16, 0.1), 4)
    ws, bws = layer.workspace(24), P.block_norm_backward_workspace(rows, cols)

    def buffers():
        o = {k: torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda") for k in ("s", "y", "dx", "da")}
        o.update(rstd=torch.zeros(2, rows, device="cuda"), dpre=torch.zeros(cols, device="cuda"),
                 dgate=torch.zeros(cols, device="cuda"), moe=torch.zeros(24, cols, dtype=torch.bfloat16, device="cuda"),
                 bk=P.Checkpoint8(rows, cols), sk=P.Checkpoint8(rows, cols))
        return o

    def step(o):
        P.block_norm(d["parts"], d["x"], o["s"], o["y"], post_weight=d["wpost"], pre_weight=d["wpre"], gate=d["gate"],
                     block_ckpt=o["bk"], stream_ckpt=o["sk"], rstd=o["rstd"])
        layer(o["y"][:24], o["moe"], workspace=ws)
        P.block_norm_backward(o["bk"], o["sk"], o["rstd"], o["y"], o["dx"], o["da"], o["dpre"], d_gate=o["dgate"],
                              post_weight=d["wpost"], pre_weight=d["wpre"], gate=d["gate"], workspace=bws)

    def tensors(o):
        return [t for t in o.values() if torch.is_tensor(t)] + [o["bk"].codes, o["sk"].exps]

    first, second, third = buffers(), buffers(), buffers()
    step(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(second)
    torch.cuda.synchronize()
    for a, b in zip(tensors(first), tensors(second)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(third)
    for t in tensors(third):
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(tensors(first), tensors(third)):
        assert torch.equal(a, b)
