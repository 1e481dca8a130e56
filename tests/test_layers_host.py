"""The layer operators without a GPU: the header, the exported symbols, and
every refusal. Each case here breaks a rule or is empty, so none can reach a
launch. Device addresses are fake and never dereferenced."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import tile_level_collective_gb300 as P
from conftest import ROOT
from test_c_abi import cuda_include

A, MB = 0x7F0000000000, 1 << 20


def at(i):
    return A + i * 64 * MB


def m(i, ld=64, off=0):
    return P.ptoc_matrix(at(i) + off, ld)


def k8(i, ld=64, ld_exps=2):
    return P.ptoc_ckpt8(at(i), ld, at(i) + 32 * MB, ld_exps)


def params(**kw):
    q = P.ptoc_block_norm_params(1, P.BF16, at(40), at(41), None, 0, 0, 1.0, 1.0, 1e-6)
    for name, v in kw.items():
        setattr(q, name, v)
    return q


def test_header_and_symbols():
    text = open(os.path.join(ROOT, "include", "ptoc_layers.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(ptoc_\w+)\s*\(", text)))
    assert names == ["ptoc_block_norm", "ptoc_block_norm_backward", "ptoc_block_norm_backward_workspace",
                     "ptoc_checkpoint8", "ptoc_moe_few_tokens", "ptoc_moe_few_tokens_workspace", "ptoc_restore8"]
    lib = ctypes.CDLL(P.LIB_PATH)
    for n in names:
        assert hasattr(lib, n) and hasattr(P, n), n


@pytest.mark.parametrize("lang,std,cc", [("c", "c99", "gcc"), ("c++", "c++17", "g++")])
def test_header_compiles_and_layouts_match(lang, std, cc, tmp_path):
    """The header is plain C, and the binding's structures have its layout."""
    src = tmp_path / "h.c"
    src.write_text('#include <stdio.h>\n#include "ptoc_layers.h"\nint main(void) {\n'
                   'printf("%d %d %d %d %d\\n", (int)sizeof(ptoc_matrix), (int)sizeof(ptoc_ckpt8), '
                   '(int)sizeof(ptoc_block_norm_params), (int)sizeof(ptoc_block_norm_saved), '
                   '(int)sizeof(ptoc_moe_params)); return 0; }\n')
    exe = tmp_path / "h"
    r = subprocess.run([cc, "-x", lang, "-std=" + std, "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), "-I", cuda_include(), "-o", str(exe), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    sizes = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert sizes == [ctypes.sizeof(t) for t in (P.ptoc_matrix, P.ptoc_ckpt8, P.ptoc_block_norm_params,
                                                P.ptoc_block_norm_saved, P.ptoc_moe_params)]


def ck(x=None, k=None, rows=8, cols=64, dt=P.BF16, call=P.ptoc_checkpoint8):
    x, k = x or m(0), k or k8(1)
    a = (x, k) if call is P.ptoc_checkpoint8 else (k, x)
    return call(*a, rows, cols, dt, stream=0, check=False)


@pytest.mark.parametrize("call", [P.ptoc_checkpoint8, P.ptoc_restore8])
def test_checkpoint_rejects(call):
    assert ck(call=call, dt=P.I32) == P.ERR_UNSUPPORTED
    assert ck(call=call, dt=9) == P.ERR_INVALID_ARG
    assert ck(call=call, rows=-1) == P.ERR_INVALID_ARG
    assert ck(call=call, x=m(0, 63)) == P.ERR_INVALID_ARG                       # pitch below cols
    assert ck(call=call, x=m(0, 64, 1)) == P.ERR_INVALID_ARG                    # misaligned
    assert ck(call=call, x=P.ptoc_matrix(None, 64)) == P.ERR_INVALID_ARG
    assert ck(call=call, k=k8(1, ld_exps=1)) == P.ERR_INVALID_ARG               # 64 columns: 2 exponents
    assert ck(call=call, k=P.ptoc_ckpt8(at(1), 64, None, 2)) == P.ERR_INVALID_ARG
    assert ck(call=call, k=P.ptoc_ckpt8(at(0) + 512, 64, at(2), 2)) == P.ERR_ALIAS
    assert ck(call=call, rows=2 ** 50, cols=2 ** 20, x=m(0, 2 ** 20), k=k8(1, 2 ** 20, 2 ** 15)) == P.ERR_INVALID_ARG
    far = dict(x=P.ptoc_matrix(1 << 40, 2 ** 33), k=P.ptoc_ckpt8(1 << 41, 2 ** 33, 1 << 42, 2 ** 28))
    assert ck(call=call, rows=1, cols=2 ** 33, **far) == P.ERR_UNSUPPORTED      # columns are counted in 32 bits
    assert ck(call=call, rows=2 ** 24, cols=2 ** 16, x=P.ptoc_matrix(1 << 50, 2 ** 16),
              k=P.ptoc_ckpt8(1 << 51, 2 ** 16, 1 << 52, 2 ** 11)) == P.ERR_UNSUPPORTED
    assert ck(call=call, rows=0) == P.OK and ck(call=call, cols=0) == P.OK


def bn(parts=None, ld=64, x=None, q=None, out=None, normed=None, block_out=None, bc=None, sc=None, rstd=None,
       rows=8, cols=64, dt=P.BF16):
    parts = [at(0), at(1)] if parts is None else parts
    return P.ptoc_block_norm(parts, ld, x or m(8), q or params(), out or m(9), normed, block_out, bc, sc, rstd, rows,
                             cols, dt, stream=0, check=False)


def test_block_norm_rejects():
    assert bn(parts=[]) == P.ERR_INVALID_ARG
    assert bn(parts=[at(0)] * 65) == P.ERR_INVALID_ARG
    assert bn(parts=[at(0), 0]) == P.ERR_INVALID_ARG
    assert bn(parts=[at(0), at(1) + 1]) == P.ERR_INVALID_ARG
    assert bn(ld=60) == P.ERR_INVALID_ARG
    assert bn(dt=P.I32) == P.ERR_UNSUPPORTED
    assert bn(dt=7) == P.ERR_INVALID_ARG
    assert bn(q=params(eps=0.0)) == P.ERR_INVALID_ARG
    assert bn(q=params(eps=float("nan"))) == P.ERR_INVALID_ARG
    assert bn(q=params(post_norm=2)) == P.ERR_INVALID_ARG
    assert bn(q=params(param_dtype=P.F16)) == P.ERR_INVALID_ARG                 # neither bf16 nor f32
    assert bn(q=params(gate=at(42), gate_col_stride=2)) == P.ERR_INVALID_ARG
    assert bn(q=params(gate=at(42), gate_row_stride=-1)) == P.ERR_INVALID_ARG
    assert bn(q=params(gate=at(42), gate_row_stride=8, gate_col_stride=1)) == P.ERR_INVALID_ARG   # rows overlap
    assert bn(q=params(pre_weight=at(41) + 1)) == P.ERR_INVALID_ARG
    assert bn(x=m(8, 32)) == P.ERR_INVALID_ARG
    assert bn(rstd=at(20) + 2) == P.ERR_INVALID_ARG
    assert bn(rows=4, cols=40000, ld=40000, x=m(8, 40000), out=m(9, 40000)) == P.ERR_UNSUPPORTED
    assert bn(out=m(0)) == P.ERR_ALIAS                                          # out over a part
    assert bn(out=m(8, 64, 128)) == P.ERR_ALIAS                                 # out over x, not the same matrix
    assert bn(normed=m(9)) == P.ERR_ALIAS                                       # two outputs
    assert bn(normed=m(40)) == P.ERR_ALIAS                                      # over a weight
    assert bn(rstd=at(9)) == P.ERR_ALIAS
    assert bn(bc=k8(10), sc=k8(10)) == P.ERR_ALIAS
    assert bn(q=params(gate=at(9), gate_col_stride=1)) == P.ERR_ALIAS
    assert bn(rows=0) == P.OK
    assert bn(rows=0, parts=[0, 0]) == P.OK                                     # an empty tensor has no address
    assert bn(cols=0, ld=0) == P.OK


def bb(saved=None, q=None, dy=None, du=None, dres=None, dblk=None, dpre=None, dpost=None, dgate=None, ws=None,
       nbytes=None, rows=8, cols=64, dt=P.BF16):
    if saved is None:
        saved = dict(block=m(0), stream=m(1))
    s = P.ptoc_block_norm_saved()
    for name, v in saved.items():
        setattr(s, name, v)
    s.rstd = at(2)
    need = P.ptoc_block_norm_backward_workspace(rows, cols)
    return P.ptoc_block_norm_backward(s, q or params(), dy or m(3), du, dres or m(4), dblk or m(5), dpre, dpost, dgate,
                                      at(30) if ws is None else ws, need if nbytes is None else nbytes, rows, cols,
                                      dt, stream=0, check=False)


def test_block_norm_backward_rejects():
    assert bb(saved=dict(block=m(0))) == P.ERR_INVALID_ARG                      # no stream
    assert bb(saved=dict(block=m(0), block_ckpt=k8(6), stream=m(1))) == P.ERR_INVALID_ARG   # both forms
    assert bb(dpost=at(20), q=params(post_norm=0)) == P.ERR_INVALID_ARG
    assert bb(dgate=at(20)) == P.ERR_INVALID_ARG                                # no gate
    assert bb(ws=at(30) + 64) == P.ERR_INVALID_ARG                              # workspace alignment
    assert bb(nbytes=P.ptoc_block_norm_backward_workspace(8, 64) - 1) == P.ERR_INVALID_ARG
    assert bb(ws=0) == P.ERR_INVALID_ARG
    assert bb(dt=P.I32) == P.ERR_UNSUPPORTED
    assert bb(dres=m(4, 32)) == P.ERR_INVALID_ARG
    assert bb(dres=m(3)) == P.ERR_ALIAS                                         # over dy
    assert bb(dblk=m(4)) == P.ERR_ALIAS
    assert bb(dpre=at(0)) == P.ERR_ALIAS                                        # over a saved matrix
    assert bb(dblk=m(1)) == P.ERR_ALIAS                                         # only the block may be replaced
    assert bb(ws=at(4)) == P.ERR_ALIAS
    assert bb(rows=2, cols=40000, dy=m(3, 40000), dres=m(4, 40000), dblk=m(5, 40000),
              saved=dict(block=m(0, 40000), stream=m(1, 40000))) == P.ERR_UNSUPPORTED
    assert bb(rows=0) == P.OK
    assert bb(cols=0) == P.OK


def moe_params(**kw):
    q = P.ptoc_moe_params(at(20), None, at(21), at(22), P.BF16, 8, 0, 8, 2, 0, 1, 1.0)
    for name, v in kw.items():
        setattr(q, name, v)
    return q


def moe(x=None, q=None, y=None, ids=None, w=None, ws=None, nbytes=None, tokens=4, hidden=64, inter=32, dt=P.BF16):
    q = q or moe_params()
    need = P.ptoc_moe_few_tokens_workspace(tokens, hidden, inter, q.experts, q.top_k)
    return P.ptoc_moe_few_tokens(x or m(0), q, y or m(1), ids, w, at(30) if ws is None else ws,
                                 need if nbytes is None else nbytes, tokens, hidden, inter, dt, stream=0, check=False)


def test_moe_rejects():
    for bad in (dict(router=None), dict(w_in=None), dict(experts=0), dict(first_expert=-1), dict(local_experts=0),
                dict(first_expert=4, local_experts=5), dict(top_k=0), dict(top_k=9), dict(score=2),
                dict(renormalize=3), dict(router_dtype=P.F16), dict(router=at(20) + 1), dict(bias=at(23) + 2)):
        assert moe(q=moe_params(**bad)) == P.ERR_INVALID_ARG, bad
    assert moe(dt=P.F32) == P.ERR_UNSUPPORTED
    assert moe(dt=P.I32) == P.ERR_UNSUPPORTED
    assert moe(dt=12) == P.ERR_INVALID_ARG
    assert moe(tokens=65) == P.ERR_UNSUPPORTED
    assert moe(q=moe_params(experts=2000, local_experts=8)) == P.ERR_UNSUPPORTED
    assert moe(q=moe_params(experts=64, top_k=17)) == P.ERR_UNSUPPORTED
    assert moe(tokens=-1) == P.ERR_INVALID_ARG
    assert moe(hidden=0) == P.ERR_INVALID_ARG
    assert moe(x=m(0, 32)) == P.ERR_INVALID_ARG
    assert moe(nbytes=16) == P.ERR_INVALID_ARG
    assert moe(ws=at(30) + 128) == P.ERR_INVALID_ARG
    assert moe(ids=at(5) + 2) == P.ERR_INVALID_ARG
    assert moe(y=m(0)) == P.ERR_ALIAS
    assert moe(y=m(21)) == P.ERR_ALIAS
    assert moe(ids=at(1)) == P.ERR_ALIAS
    assert moe(ws=at(21)) == P.ERR_ALIAS
    assert moe(tokens=0) == P.OK
    assert P.ptoc_moe_few_tokens_workspace(65, 64, 32, 8, 2) == 0


def t(rows=4, cols=64, dtype=torch.bfloat16):
    return torch.zeros(rows, cols, dtype=dtype)


def test_conveniences_refuse_what_the_calls_cannot_describe():
    for kw in (dict(residual=t(4, 32)), dict(residual=t(dtype=torch.float32)), dict(parts=[t(), t(5)]),
               dict(gate=torch.zeros(3, dtype=torch.bfloat16)), dict(gate=torch.zeros(4, 1)[:, 0]),
               dict(gate=torch.zeros(64, 4, dtype=torch.bfloat16).t()),
               dict(pre_weight=torch.zeros(64), post_weight=torch.zeros(64, dtype=torch.bfloat16)),
               dict(pre_weight=torch.zeros(128, dtype=torch.bfloat16)[::2]), dict(rstd=torch.zeros(4)),
               dict(stream_ckpt=P.Checkpoint8(4, 32, device="cpu")),
               dict(post_weight=torch.zeros(64, dtype=torch.bfloat16), post_norm=False),
               dict(normed=t(4, 128)[:, ::2])):
        args = dict(dict(parts=[t()], residual=t()), **kw)
        with pytest.raises(ValueError):
            P.block_norm(args.pop("parts"), args.pop("residual"), t(), **args)
    rstd, ws = torch.zeros(2, 4), torch.zeros(1 << 20, dtype=torch.uint8)
    for kw in (dict(d_pre_weight=torch.zeros(64, dtype=torch.bfloat16)), dict(d_gate=torch.zeros(64)),
               dict(block=t(4, 32)), dict(d_block=t(dtype=torch.float32))):
        args = dict(dict(block=t(), d_block=t()), **kw)
        with pytest.raises(ValueError):
            P.block_norm_backward(args.pop("block"), t(), rstd, t(), t(), args.pop("d_block"), workspace=ws, **args)
    with pytest.raises(ValueError):
        P.Checkpoint8.of(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 3, dtype=torch.uint8))
    with pytest.raises(ValueError):
        P.checkpoint8(t(), P.Checkpoint8(5, 64, device="cpu"))
    h = torch.bfloat16
    with pytest.raises(ValueError):
        P.MoeLayer(torch.zeros(8, 64, dtype=h), torch.zeros(8, 60, 64, dtype=h), torch.zeros(8, 64, 32, dtype=h), 2)
    with pytest.raises(ValueError):
        P.MoeLayer(torch.zeros(8, 64, dtype=h), torch.zeros(8, 64, 64, dtype=h), torch.zeros(8, 64, 32, dtype=h), 2,
                   score="tanh")
    layer = P.MoeLayer(torch.zeros(8, 64, dtype=h), torch.zeros(8, 64, 64, dtype=h), torch.zeros(8, 64, 32, dtype=h), 2)
    for bad in (dict(x=t(4, 32)), dict(x=t(dtype=torch.float16)), dict(y=t(3)), dict(ids=torch.zeros(4, 2))):
        args = dict(dict(x=t(), y=t(), ids=None), **bad)
        with pytest.raises(ValueError):
            layer(args["x"], args["y"], ids=args["ids"], workspace=ws)
