"""The layer operators as they are measured: block_norm, its backward pass,
8-bit activation checkpoints and the mixture-of-experts layer for a few tokens.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end), or, where ``own`` is true, through the
library's calls. ``exact`` restates the definitions in 64 bits.

Formulas (one row of H columns; all sums over the row unless said otherwise)

    block_norm   a = sum_r part_r in rank order
                 n = a * ra * post_weight,  ra = rsqrt(mean(a^2) + eps)   (n = a and ra = 1 without the norm after)
                 s = residual_scale * x + branch_scale * gate * n
                 y = s * r * pre_weight,    r = rsqrt(mean(s^2) + eps)
    backward     ds = du + r * (wpre * dy) - s * r^3 / H * sum(wpre * dy * s)
                 dx = residual_scale * ds;  dn = branch_scale * gate * ds
                 da = ra * (wpost * dn) - a * ra^3 / H * sum(wpost * dn * a)
                 dwpre = sum_rows dy * s * r;  dwpost = sum_rows dn * a * ra
                 dgate = branch_scale * ds * n, summed over the axes along which the gate is broadcast
    checkpoint8  blocks of 32 columns: the smallest e with max|x| <= 127 * 2^e, codes rint(x / 2^e)
    moe          logits = router x; the top_k experts by score (+ bias); w = their scores, renormalised, * scale
                 y = sum over the chosen experts that are held here of w * down(silu(gate x) * (up x))
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
BLOCK = 32


def _size(dtype):
    return 4 if dtype == "f32" else 2


# ---- cases ------------------------------------------------------------------

def _norm(rows, cols, dtype, parts, gate, post=True, ckpt=False, pad=0, name=None):
    c = dict(op="norm", rows=rows, cols=cols, dtype=dtype, parts=parts, gate=gate, post=post, ckpt=ckpt, pad=pad)
    return dict(c, name=name) if name else c


def _back(rows, cols, dtype, gate, post=True, ckpt=True, pad=0, name=None):
    c = dict(op="norm_backward", rows=rows, cols=cols, dtype=dtype, gate=gate, post=post, ckpt=ckpt, pad=pad)
    return dict(c, name=name) if name else c


def _ckpt(rows, cols, dtype, pad=0, name=None):
    c = dict(op="checkpoint", rows=rows, cols=cols, dtype=dtype, pad=pad)
    return dict(c, name=name) if name else c


def _moe(tokens, hidden, inter, experts, local, first, top_k, dtype, score, name=None):
    c = dict(op="moe", tokens=tokens, hidden=hidden, inter=inter, experts=experts, local=local, first=first,
             top_k=top_k, dtype=dtype, score=score)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token, 8 ranks' partial outputs: the latency of the call
        _norm(1, 7168, "bf16", 8, "channel", name="norm_token"),
        # a small batch of odd width in 32 bits, rows at an odd pitch, a gate for each token
        _norm(257, 1003, "f32", 4, "token", pad=2, name="norm_ragged"),
        # a training step's forward pass: one partial output, both 8-bit checkpoints written
        _norm(8192, 4096, "bf16", 1, "channel", ckpt=True, name="norm_train"),
        # prefill of 16384 tokens after a block split over 8 ranks
        _norm(16384, 8192, "bf16", 8, "none", name="norm_prefill"),
        # a short, odd batch in f16 from activations saved in 16 bits, without the norm after the block
        _back(77, 1000, "f16", "scalar", post=False, ckpt=False, pad=8, name="back_small"),
        # the backward pass of norm_train, from its 8-bit checkpoints
        _back(8192, 4096, "bf16", "channel", name="back_train"),
        # a long batch of wide rows with a gate for each token
        _back(16384, 8192, "bf16", "token", name="back_wide"),
        # one small activation of odd width kept and restored
        _ckpt(33, 1003, "f32", name="ckpt_small"),
        # one block's activations of a long batch
        _ckpt(16384, 8192, "bf16", name="ckpt_wide"),
        # one decoded token through a layer of 64 wide experts
        _moe(1, 7168, 2048, 64, 64, 0, 8, "bf16", "softmax", name="moe_token"),
        # a batch of 13 in f16 on the rank that holds experts 32 to 95 of 128, scored by sigmoids with a selection bias
        _moe(13, 4096, 1536, 128, 64, 32, 8, "f16", "sigmoid", name="moe_slice"),
        # the largest batch, which touches nearly every expert
        _moe(64, 4096, 1536, 128, 128, 0, 8, "bf16", "softmax", name="moe_batch"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, of=1):
    """A multiple of `of` between lo * of and hi * of, spread over the logarithm; 3072 gives way to its neighbour."""
    w = of * _log_int(rng, lo, hi)
    return w + of if w == 3072 else w


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "checkpoint", "moe"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "moe":
        dtype = rng.choice(["f16", "bf16"])
        experts = rng.choice([8, 16, 60, 64, 128])
        local = rng.choice([experts, max(1, experts // 2), max(1, experts // 4)])
        first = rng.randint(0, experts - local)
        hidden = _width(rng, 64, 896, 8)
        # the weights of every expert held stay below the largest listed layer's
        most = 128 * 1536 * 4096 // (local * hidden)
        inter = _width(rng, 16, max(17, min(2048, most) // 8), 8)
        return _moe(_log_int(rng, 1, 64), hidden, inter, experts, local, first, rng.randint(1, min(8, experts)),
                    dtype, rng.choice(["softmax", "sigmoid"]))
    cols = _width(rng, 4, 127, 64) if rng.random() < 0.5 else _width(rng, 256, 8191)
    pad = rng.choice([0, 0, 1, 8, 64])
    rows = _width(rng, 1, 16384)
    if dtype == "f32":
        rows = max(1, rows // 2)
    gate = rng.choice(["none", "scalar", "channel", "token"])
    if op == "norm":
        parts = rng.choice([1, 1, 2, 4, 8])
        return _norm(rows, cols, dtype, parts, gate, post=rng.random() < 0.7, ckpt=rng.random() < 0.3, pad=pad)
    if op == "norm_backward":
        return _back(rows, cols, dtype, gate, post=rng.random() < 0.7, ckpt=rng.random() < 0.6, pad=pad)
    return _ckpt(rows, cols, dtype, pad=pad)


# ---- inputs -----------------------------------------------------------------

class _Random:
    """Seeded values on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, shape, dtype, std=1.0, mean=0.0):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t.normal_(mean, std, generator=self.g)

    def rows(self, rows, cols, pad, dtype, std=1.0):
        """A [rows, cols] view at pitch cols + pad."""
        return self.normal((rows, cols + pad), dtype, std)[:, :cols]


def _empty_rows(rows, cols, pad, dtype):
    return torch.empty(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _gate(case, rnd, dtype):
    shape = {"none": None, "scalar": (1,), "channel": (case["cols"],), "token": (case["rows"], 1)}[case["gate"]]
    return None if shape is None else rnd.normal(shape, dtype, 0.3, 0.7)


def _power_of_two(biased):
    """2^(biased - 127) in 32 bits, from the exponent field (0 stands for the subnormal 2^-127)."""
    return torch.where(biased > 0, biased << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _encode8(x):
    """Codes and exponent bytes of a [rows, cols] tensor, in torch."""
    rows, cols = x.shape
    nb = (cols + BLOCK - 1) // BLOCK
    v = torch.zeros(rows, nb * BLOCK, dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, nb, BLOCK)
    bits = v.abs().amax(2).view(torch.int32)
    # the exponent of max|x| / 127 rounded up to a power of two, biased by 127
    e = (((bits + 0x1FFFF) >> 23) - 6).clamp(0, 254)                # finite values only
    codes = torch.round(v * _power_of_two(254 - e)[..., None]).to(torch.int8)
    return codes.view(rows, nb * BLOCK)[:, :cols], e.to(torch.uint8)


def _decode8(codes, exps, dtype=torch.float32):
    scale = _power_of_two(exps.to(torch.int32)).to(dtype)
    scale = scale.repeat_interleave(BLOCK, dim=1)[:, :codes.shape[1]]
    return codes.to(dtype) * scale


def prepare(case, seed):
    rnd = _Random(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    st = dict(case=case)
    if op == "moe":
        t, h, i, e = case["tokens"], case["hidden"], case["inter"], case["local"]
        st["x"] = rnd.normal((t, h), dtype)
        st["router"] = rnd.normal((case["experts"], h), dtype, 1.5 / math.sqrt(h))
        st["bias"] = rnd.normal((case["experts"],), torch.float32, 0.05) if case["score"] == "sigmoid" else None
        st["w_in"] = rnd.normal((e, 2 * i, h), dtype, 1.0 / math.sqrt(h))
        st["w_out"] = rnd.normal((e, h, i), dtype, 1.0 / math.sqrt(i))
        st["y"] = torch.empty(t, h, dtype=dtype, device="cuda")
        st["ids"] = torch.empty(t, case["top_k"], dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty(t, case["top_k"], dtype=torch.float32, device="cuda")
        if own:
            import tile_level_collective_gb300 as ptoc
            st["layer"] = ptoc.MoeLayer(st["router"], st["w_in"], st["w_out"], case["top_k"], bias=st["bias"],
                                        first_expert=case["first"], score=case["score"], scale=2.5)
            st["workspace"] = st["layer"].workspace(t)
        return st

    rows, cols, pad = case["rows"], case["cols"], case["pad"]
    if op == "checkpoint":
        # activations: a few channels are much larger than the rest
        x = rnd.rows(rows, cols, pad, dtype)
        x[:, ::97] *= 20
        st["x"], st["out"] = x, _empty_rows(rows, cols, pad, dtype)
        if own:
            import tile_level_collective_gb300 as ptoc
            st["ckpt"] = ptoc.Checkpoint8(rows, cols)
        return st

    st["gate"] = _gate(case, rnd, dtype)
    st["post_weight"] = rnd.normal((cols,), dtype, 0.1, 1.0) if case["post"] else None
    st["pre_weight"] = rnd.normal((cols,), dtype, 0.1, 1.0)
    if op == "norm":
        n = case["parts"]
        st["parts"] = [rnd.rows(rows, cols, pad, dtype, 1.0 / math.sqrt(n)) for _ in range(n)]
        st["x"] = rnd.rows(rows, cols, pad, dtype, 3.0)
        st["out"], st["normed"] = _empty_rows(rows, cols, pad, dtype), _empty_rows(rows, cols, pad, dtype)
        st["rstd"] = torch.empty(2, rows, dtype=torch.float32, device="cuda")
        if own and case["ckpt"]:
            import tile_level_collective_gb300 as ptoc
            st["block_ckpt"], st["stream_ckpt"] = ptoc.Checkpoint8(rows, cols), ptoc.Checkpoint8(rows, cols)
        return st

    # backward: what the forward pass saved, and the gradients that arrive
    block = rnd.rows(rows, cols, pad, dtype)
    stream = rnd.rows(rows, cols, pad, dtype, 3.0)
    bf, sf = block.float(), stream.float()
    st["rstd"] = torch.stack([torch.rsqrt((bf * bf).mean(1) + EPS), torch.rsqrt((sf * sf).mean(1) + EPS)])
    if case["ckpt"]:
        st["block8"], st["stream8"] = _encode8(bf), _encode8(sf)
        if own:
            import tile_level_collective_gb300 as ptoc
            st["block"] = ptoc.Checkpoint8.of(*st["block8"], cols)
            st["stream"] = ptoc.Checkpoint8.of(*st["stream8"], cols)
    else:
        st["block"], st["stream"] = block, stream
    st["d_normed"] = rnd.rows(rows, cols, pad, dtype)
    st["d_stream"] = rnd.rows(rows, cols, pad, dtype)
    st["d_residual"], st["d_block"] = _empty_rows(rows, cols, pad, dtype), _empty_rows(rows, cols, pad, dtype)
    f32 = dict(dtype=torch.float32, device="cuda")
    st["d_pre_weight"] = torch.empty(cols, **f32)
    st["d_post_weight"] = torch.empty(cols, **f32) if case["post"] else None
    st["d_gate"] = None if st["gate"] is None else torch.empty(st["gate"].shape, **f32)
    if own:
        import tile_level_collective_gb300 as ptoc
        st["workspace"] = ptoc.block_norm_backward_workspace(rows, cols)
    return st


RESIDUAL_SCALE, BRANCH_SCALE = 0.9, 1.25


# ---- one pass ---------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return {"norm": _run_norm, "norm_backward": _run_back, "checkpoint": _run_ckpt, "moe": _run_moe}[op](state)


def _given(**tensors):
    """The gradients that the case has."""
    return {k: v for k, v in tensors.items() if v is not None}


def _run_norm(st):
    case = st["case"]
    if own:
        import tile_level_collective_gb300 as ptoc
        ptoc.block_norm(st["parts"], st["x"], st["out"], st["normed"], post_norm=case["post"],
                        post_weight=st["post_weight"], pre_weight=st["pre_weight"], gate=st["gate"],
                        residual_scale=RESIDUAL_SCALE, branch_scale=BRANCH_SCALE, eps=EPS, rstd=st["rstd"],
                        block_ckpt=st.get("block_ckpt"), stream_ckpt=st.get("stream_ckpt"))
        out = dict(stream=st["out"], normed=st["normed"], rstd=st["rstd"])
        if case["ckpt"]:
            for k in ("block_ckpt", "stream_ckpt"):
                v = torch.empty_like(st["x"])
                ptoc.restore8(st[k], v)
                out[k] = v
        return out
    dtype = st["x"].dtype
    a = st["parts"][0].float()
    for p in st["parts"][1:]:
        a = a + p.float()
    ra, n = torch.ones_like(a[:, :1]), a
    if case["post"]:
        ra = torch.rsqrt((a * a).mean(1, keepdim=True) + EPS)
        n = a * ra * st["post_weight"].float()
    if st["gate"] is not None:
        n = n * st["gate"].float()
    s = RESIDUAL_SCALE * st["x"].float() + BRANCH_SCALE * n
    r = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)
    y = s * r * st["pre_weight"].float()
    out = dict(stream=s.to(dtype), normed=y.to(dtype), rstd=torch.cat([ra, r], 1).t().contiguous())
    if case["ckpt"]:
        out["block_ckpt"] = _decode8(*_encode8(a)).to(dtype)
        out["stream_ckpt"] = _decode8(*_encode8(out["stream"])).to(dtype)
    return out


def _run_back(st):
    case = st["case"]
    if own:
        import tile_level_collective_gb300 as ptoc
        ptoc.block_norm_backward(st["block"], st["stream"], st["rstd"], st["d_normed"], st["d_residual"],
                                 st["d_block"], st["d_pre_weight"], d_post_weight=st["d_post_weight"],
                                 d_gate=st["d_gate"], d_stream=st["d_stream"], post_norm=case["post"],
                                 post_weight=st["post_weight"], pre_weight=st["pre_weight"], gate=st["gate"],
                                 residual_scale=RESIDUAL_SCALE, branch_scale=BRANCH_SCALE, eps=EPS,
                                 workspace=st["workspace"])
        return _given(d_residual=st["d_residual"], d_block=st["d_block"], d_pre_weight=st["d_pre_weight"],
                      d_post_weight=st["d_post_weight"], d_gate=st["d_gate"])
    dtype, h = st["d_normed"].dtype, case["cols"]
    if case["ckpt"]:
        a, s = _decode8(*st["block8"]), _decode8(*st["stream8"])
    else:
        a, s = st["block"].float(), st["stream"].float()
    ra, r = st["rstd"][0][:, None], st["rstd"][1][:, None]
    dy = st["d_normed"].float()
    wdy = dy * st["pre_weight"].float()
    ds = st["d_stream"].float() + r * wdy - s * (r ** 3 / h * (wdy * s).sum(1, keepdim=True))
    g = 1.0 if st["gate"] is None else st["gate"].float()
    dn = BRANCH_SCALE * g * ds
    if case["post"]:
        wpost = st["post_weight"].float()
        n = a * ra * wpost
        wdn = dn * wpost
        da = ra * wdn - a * (ra ** 3 / h * (wdn * a).sum(1, keepdim=True))
        d_post = (dn * (a * ra)).sum(0)
    else:
        n, da, d_post = a, dn, None
    d_gate = None
    if st["gate"] is not None:
        full = BRANCH_SCALE * ds * n
        d_gate = {"scalar": lambda: full.sum().reshape(1), "channel": lambda: full.sum(0),
                  "token": lambda: full.sum(1, keepdim=True)}[case["gate"]]()
    return _given(d_residual=(RESIDUAL_SCALE * ds).to(dtype), d_block=da.to(dtype), d_pre_weight=(dy * (s * r)).sum(0),
                  d_post_weight=d_post, d_gate=d_gate)


def _run_ckpt(st):
    if own:
        import tile_level_collective_gb300 as ptoc
        ptoc.checkpoint8(st["x"], st["ckpt"])
        ptoc.restore8(st["ckpt"], st["out"])
        return st["out"]
    return _decode8(*_encode8(st["x"].float())).to(st["x"].dtype)


def _route(logits, bias, case):
    """Ids (descending, ties to the lowest index) and weights of the chosen experts."""
    if case["score"] == "softmax":
        key, score = logits, torch.softmax(logits, 1)
    else:
        score = torch.sigmoid(logits)
        key = score if bias is None else score + bias.to(score.dtype)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :case["top_k"]]
    w = score.gather(1, ids)
    return ids, 2.5 * w / w.sum(1, keepdim=True)


def _run_moe(st):
    case = st["case"]
    if own:
        st["layer"](st["x"], st["y"], ids=st["ids"], weights=st["weights"], workspace=st["workspace"])
        return dict(y=st["y"], ids=st["ids"], weights=st["weights"])
    x, i = st["x"].float(), case["inter"]
    ids, w = _route(x @ st["router"].float().t(), st["bias"], case)
    y = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        if not case["first"] <= e < case["first"] + case["local"]:
            continue
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        gu = x[token] @ st["w_in"][e - case["first"]].float().t()
        g, u = gu[:, :i], gu[:, i:]
        h = g * torch.sigmoid(g) * u
        y[token] += w[token, slot][:, None] * (h @ st["w_out"][e - case["first"]].float().t())
    return dict(y=y.to(st["x"].dtype), ids=ids.to(torch.int32), weights=w)


# ---- the work that cannot be avoided -------------------------------------------

def work(case):
    op, es = case["op"], _size(case["dtype"])
    if op == "moe":
        t, h, i, e, k = case["tokens"], case["hidden"], case["inter"], case["experts"], case["top_k"]
        # the experts held here that at least one token is expected to choose
        active = case["local"] * (1 - (1 - k / e) ** t)
        pairs = t * k * case["local"] / e
        return dict(bytes=int(es * (active * 3 * h * i + e * h + 2 * t * h) + 8 * t * k),
                    flops=int(2 * t * e * h + pairs * 6 * h * i))
    n = case["rows"] * case["cols"]
    blocks = case["rows"] * ((case["cols"] + BLOCK - 1) // BLOCK)
    if op == "checkpoint":
        return dict(bytes=2 * es * n + 2 * (n + blocks), flops=4 * n)
    per_gate = {"none": 0, "scalar": 1, "channel": case["cols"], "token": case["rows"]}[case["gate"]]
    if op == "norm":
        extra = 2 * (n + blocks) if case["ckpt"] else 0
        return dict(bytes=es * (n * (case["parts"] + 3) + 2 * case["cols"] + per_gate) + extra + 8 * case["rows"],
                    flops=n * (case["parts"] + 10))
    saved = 2 * (n + blocks) if case["ckpt"] else 2 * n * es
    return dict(bytes=es * (4 * n + 2 * case["cols"] + per_gate) + saved + 4 * (2 * case["cols"] + per_gate)
                + 8 * case["rows"], flops=24 * n)


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    f = torch.float64
    if case["op"] == "moe":
        return _exact_moe(st, case)
    if case["op"] == "checkpoint":
        x = st["x"].to(f)
        out = torch.empty_like(x)
        for c in range(0, case["cols"], BLOCK):
            b = x[:, c:c + BLOCK]
            top = b.abs().amax(1, keepdim=True)
            _, e = torch.frexp(top / 127)                         # top / 127 = m * 2^e with 0.5 <= m < 1
            e = e.to(f)
            e = torch.where(top / 127 <= torch.exp2(e - 1), e - 1, e)
            e = torch.where(top == 0, torch.zeros_like(e), e)
            out[:, c:c + BLOCK] = torch.round(b / torch.exp2(e)) * torch.exp2(e)
        return out

    h, step = case["cols"], 2048
    wpre = st["pre_weight"].to(f)
    wpost = st["post_weight"].to(f) if case["post"] else None

    def gate_of(lo, hi):
        if st["gate"] is None:
            return torch.ones((), dtype=f, device="cuda")
        return st["gate"][lo:hi].to(f) if case["gate"] == "token" else st["gate"].to(f)

    if case["op"] == "norm":
        parts = dict(stream=[], normed=[], rstd=[])
        for lo in range(0, case["rows"], step):
            a = sum(p[lo:lo + step].to(f) for p in st["parts"])
            ra = (a.square().mean(1, keepdim=True) + EPS) ** -0.5 if case["post"] else torch.ones_like(a[:, :1])
            n = a * ra * wpost if case["post"] else a
            s = RESIDUAL_SCALE * st["x"][lo:lo + step].to(f) + BRANCH_SCALE * gate_of(lo, lo + step) * n
            r = (s.square().mean(1, keepdim=True) + EPS) ** -0.5
            parts["stream"].append(s)
            parts["normed"].append(s * r * wpre)
            parts["rstd"].append(torch.cat([ra, r], 1))
        out = {k: torch.cat(v) for k, v in parts.items()}
        out["rstd"] = out["rstd"].t().contiguous()
        if case["ckpt"]:
            # codes of rounded sums: no value of their own in 64 bits
            out["block_ckpt"] = out["stream_ckpt"] = None
        return out

    parts = dict(d_residual=[], d_block=[])
    d_pre = torch.zeros(h, dtype=f, device="cuda")
    d_post = torch.zeros(h, dtype=f, device="cuda")
    gates = []
    for lo in range(0, case["rows"], step):
        hi = lo + step
        if case["ckpt"]:
            a = _decode8(st["block8"][0][lo:hi], st["block8"][1][lo:hi], f)
            s = _decode8(st["stream8"][0][lo:hi], st["stream8"][1][lo:hi], f)
        else:
            a, s = st["block"][lo:hi].to(f), st["stream"][lo:hi].to(f)
        ra, r = st["rstd"][0, lo:hi, None].to(f), st["rstd"][1, lo:hi, None].to(f)
        dy = st["d_normed"][lo:hi].to(f)
        # the gradient of s / sqrt(mean(s^2) + eps), with the saved statistic
        shat = s * r
        up = dy * wpre
        ds = st["d_stream"][lo:hi].to(f) + r * (up - shat * (up * shat).mean(1, keepdim=True))
        d_pre += (dy * shat).sum(0)
        dn = BRANCH_SCALE * gate_of(lo, hi) * ds
        n = a
        if case["post"]:
            ahat = a * ra
            n = ahat * wpost
            d_post += (dn * ahat).sum(0)
            up = dn * wpost
            parts["d_block"].append(ra * (up - ahat * (up * ahat).mean(1, keepdim=True)))
        else:
            parts["d_block"].append(dn)
        parts["d_residual"].append(RESIDUAL_SCALE * ds)
        gates.append({"none": lambda: None, "scalar": lambda: (BRANCH_SCALE * ds * n).sum().reshape(1),
                      "channel": lambda: (BRANCH_SCALE * ds * n).sum(0),
                      "token": lambda: (BRANCH_SCALE * ds * n).sum(1, keepdim=True)}[case["gate"]]())
    d_gate = None
    if case["gate"] == "token":
        d_gate = torch.cat(gates)
    elif case["gate"] != "none":
        d_gate = sum(gates)
    return _given(d_residual=torch.cat(parts["d_residual"]), d_block=torch.cat(parts["d_block"]), d_pre_weight=d_pre,
                  d_post_weight=d_post if case["post"] else None, d_gate=d_gate)


def _exact_moe(st, case):
    f = torch.float64
    x, i = st["x"].to(f), case["inter"]
    logits = torch.einsum("th,eh->te", x, st["router"].to(f))
    if case["score"] == "softmax":
        z = torch.exp(logits - logits.amax(1, keepdim=True))
        score = z / z.sum(1, keepdim=True)
        key = logits
    else:
        score = 1 / (1 + torch.exp(-logits))
        key = score + st["bias"].to(f)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :case["top_k"]]
    w = torch.gather(score, 1, ids)
    w = 2.5 * w / w.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for local in range(case["local"]):
        chosen = ids == local + case["first"]
        token = torch.nonzero(chosen.any(1))[:, 0]
        if len(token) == 0:
            continue
        g = x[token] @ st["w_in"][local, :i].to(f).t()
        u = x[token] @ st["w_in"][local, i:].to(f).t()
        out = (g / (1 + torch.exp(-g)) * u) @ st["w_out"][local].to(f).t()
        y[token] += (w * chosen)[token].sum(1, keepdim=True) * out
    return dict(y=y, ids=ids.to(torch.int32), weights=w)
