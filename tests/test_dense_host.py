"""The dense block's operators without a GPU: the header, the exported symbols,
and every refusal. Each case here breaks a rule or is empty, so none can reach a
launch. Device addresses are fake and never dereferenced."""
import ctypes
import functools
import os
import re
import subprocess

import pytest
import torch

import tile_level_collective_gb300 as P
from conftest import ROOT
from test_c_abi import cuda_include

A, MB = 0x7F0000000000, 1 << 20
BAD, UNS, ALIAS = P.ERR_INVALID_ARG, P.ERR_UNSUPPORTED, P.ERR_ALIAS


def at(i):
    return A + i * 64 * MB


def m(i, ld=64, off=0):
    return P.ptoc_matrix(at(i) + off, ld)


def test_header_and_symbols():
    text = open(os.path.join(ROOT, "include", "ptoc_dense.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(ptoc_\w+)\s*\(", text)))
    assert names == ["ptoc_clip_gradients", "ptoc_clip_gradients_workspace", "ptoc_gated_ffn",
                     "ptoc_gated_ffn_backward", "ptoc_gated_ffn_backward_workspace", "ptoc_gated_ffn_workspace",
                     "ptoc_layer_norm", "ptoc_layer_norm_backward", "ptoc_layer_norm_backward_workspace"]
    lib = ctypes.CDLL(P.LIB_PATH)
    for n in names:
        assert hasattr(lib, n) and hasattr(P, n), n
    limits = dict(re.findall(r"#define (PTOC_\w+_MAX_\w+) (\d+)", text))
    assert {k: int(v) for k, v in limits.items()} == {
        "PTOC_FFN_MAX_TOKENS": P.FFN_MAX_TOKENS, "PTOC_FFN_MAX_WIDTH": P.FFN_MAX_WIDTH,
        "PTOC_CLIP_MAX_GRADIENTS": P.CLIP_MAX_GRADIENTS}


@pytest.mark.parametrize("lang,std,cc", [("c", "c99", "gcc"), ("c++", "c++17", "g++")])
def test_header_compiles_and_layouts_match(lang, std, cc, tmp_path):
    """The header is plain C, and the binding's structures have its layout."""
    src = tmp_path / "h.c"
    src.write_text('#include <stdio.h>\n#include "ptoc_dense.h"\nint main(void) {\n'
                   'printf("%d %d %d\\n", (int)sizeof(ptoc_layer_norm_params), (int)sizeof(ptoc_gated_ffn_params), '
                   '(int)sizeof(ptoc_gradient)); return 0; }\n')
    exe = tmp_path / "h"
    r = subprocess.run([cc, "-x", lang, "-std=" + std, "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), "-I", cuda_include(), "-o", str(exe), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    sizes = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert sizes == [ctypes.sizeof(t) for t in (P.ptoc_layer_norm_params, P.ptoc_gated_ffn_params, P.ptoc_gradient)]


# ---- layer norm ------------------------------------------------------------------------

def params(**kw):
    q = P.ptoc_layer_norm_params(at(40), at(41), P.BF16, 1e-5)
    for name, v in kw.items():
        setattr(q, name, v)
    return q


def ln(parts=None, ld=64, x=None, q=None, out=None, normed=None, stats=None, rows=8, cols=64, dt=P.BF16):
    parts = [at(0), at(1)] if parts is None else parts
    return P.ptoc_layer_norm(parts, ld, x, q or params(), out, normed or m(9), stats, rows, cols, dt, stream=0,
                             check=False)


def test_layer_norm_rejects():
    assert ln(parts=[]) == BAD
    assert ln(parts=[at(0)] * 65) == BAD
    assert ln(parts=[at(0), 0]) == BAD
    assert ln(parts=[at(0), at(1) + 1]) == BAD
    assert ln(ld=60) == BAD
    assert ln(dt=P.I32) == UNS
    assert ln(dt=7) == BAD
    assert ln(rows=-1) == BAD
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert ln(q=params(eps=eps)) == BAD
    assert ln(q=params(param_dtype=P.F16)) == BAD                               # neither bf16 nor f32
    assert ln(q=params(weight=at(41) + 1)) == BAD
    assert ln(q=params(bias=at(41) + 1)) == BAD
    assert ln(x=m(8, 32)) == BAD
    assert ln(normed=P.ptoc_matrix(None, 64)) == BAD
    assert ln(stats=at(20) + 2) == BAD
    assert ln(rows=4, cols=40000, ld=40000, normed=m(9, 40000)) == UNS
    assert ln(rows=2 ** 48, cols=2 ** 14, ld=2 ** 14, normed=m(9, 2 ** 14)) == BAD      # past the address space
    assert ln(normed=m(0)) == ALIAS                                             # over a part
    assert ln(x=m(8), out=m(8, 64, 128)) == ALIAS                               # over x, not the same matrix
    assert ln(x=m(8), out=m(9)) == ALIAS                                        # two outputs
    assert ln(x=m(9)) == ALIAS                                                  # normed over x
    assert ln(normed=m(40)) == ALIAS and ln(normed=m(41)) == ALIAS              # over the weight, the bias
    assert ln(stats=at(9)) == ALIAS and ln(stats=at(0)) == ALIAS
    assert ln(rows=0) == P.OK and ln(rows=0, parts=[0, 0]) == P.OK
    assert ln(cols=0, ld=0) == P.OK


def lb(s=None, stats=at(2), q=None, dy=None, du=None, dx=None, dw=None, db=None, ws=None, nbytes=None, rows=8,
       cols=64, dt=P.BF16):
    need = P.ptoc_layer_norm_backward_workspace(rows, cols)
    return P.ptoc_layer_norm_backward(s or m(1), stats, q or params(), dy or m(3), du, dx or m(4), dw, db,
                                      at(30) if ws is None else ws, need if nbytes is None else nbytes, rows, cols,
                                      dt, stream=0, check=False)


def test_layer_norm_backward_rejects():
    assert P.ptoc_layer_norm_backward_workspace(8, 64) == 8 * 2 * 64 * 4
    assert P.ptoc_layer_norm_backward_workspace(0, 64) == 0
    assert P.ptoc_layer_norm_backward_workspace(8, 40000) == 0
    assert lb(stats=None) == BAD
    assert lb(ws=0) == BAD and lb(ws=at(30) + 64) == BAD                        # absent, misaligned
    assert lb(nbytes=P.ptoc_layer_norm_backward_workspace(8, 64) - 1) == BAD
    assert lb(dt=P.I32) == UNS and lb(dt=-1) == BAD
    assert lb(s=m(1, 63)) == BAD and lb(dy=m(3, 64, 1)) == BAD
    assert lb(q=params(param_dtype=P.F16)) == BAD
    assert lb(dw=at(20) + 2) == BAD and lb(db=at(20) + 1) == BAD
    assert lb(rows=2, cols=40000, s=m(1, 40000), dy=m(3, 40000), dx=m(4, 40000)) == UNS
    assert lb(dx=m(1)) == ALIAS                                                 # over the stream
    assert lb(dx=m(3, 64, 256)) == ALIAS                                        # over dy, not the same matrix
    assert lb(du=m(5), dx=m(5, 64, 256)) == ALIAS
    assert lb(dx=m(30)) == ALIAS                                                # over the workspace
    assert lb(dw=at(6), db=at(6)) == ALIAS and lb(dw=at(40)) == ALIAS and lb(db=at(2)) == ALIAS


# ---- the gated feed-forward block -------------------------------------------------------

def fp(**kw):
    q = P.ptoc_gated_ffn_params(m(20, 64), m(21, 32), 0)
    for name, v in kw.items():
        setattr(q, name, v)
    return q


def ffn(x=None, q=None, y=None, pre=None, ws=None, nbytes=None, tokens=8, hidden=64, inter=32, dt=P.BF16):
    need = P.ptoc_gated_ffn_workspace(tokens, hidden, inter)
    return P.ptoc_gated_ffn(x or m(0), q or fp(), y or m(1), pre, at(30) if ws is None else ws,
                            need if nbytes is None else nbytes, tokens, hidden, inter, dt, stream=0, check=False)


SIZES = [dict(tokens=-1), dict(hidden=0), dict(inter=0)]
FAR = [dict(tokens=P.FFN_MAX_TOKENS + 1), dict(hidden=P.FFN_MAX_WIDTH + 1), dict(inter=P.FFN_MAX_WIDTH + 1)]


def test_gated_ffn_rejects():
    assert ffn(dt=P.F32) == UNS and ffn(dt=P.I32) == UNS and ffn(dt=5) == BAD
    for sizes in SIZES:
        assert ffn(**sizes) == BAD
    for sizes in FAR:
        assert ffn(**sizes) == UNS
        assert P.ptoc_gated_ffn_workspace(**dict(dict(tokens=8, hidden=64, inter=32), **sizes)) == 0
    assert ffn(q=fp(act=2)) == BAD and ffn(q=fp(act=-1)) == BAD
    assert ffn(q=fp(w_in=m(20, 63))) == BAD and ffn(q=fp(w_out=m(21, 31))) == BAD
    assert ffn(q=fp(w_in=P.ptoc_matrix(None, 64))) == BAD and ffn(q=fp(w_out=m(21, 32, 1))) == BAD
    assert ffn(x=m(0, 60)) == BAD and ffn(y=m(1, 64, 1)) == BAD and ffn(pre=m(2, 63)) == BAD
    assert ffn(x=P.ptoc_matrix(None, 64)) == BAD
    assert ffn(ws=0) == BAD and ffn(ws=at(30) + 128) == BAD
    assert ffn(nbytes=P.ptoc_gated_ffn_workspace(8, 64, 32) - 1) == BAD
    for i in (0, 20, 21, 30):                                                   # x, the weights, the workspace
        assert ffn(y=m(i)) == ALIAS and ffn(pre=m(i)) == ALIAS
    assert ffn(pre=m(1)) == ALIAS
    assert ffn(tokens=0) == P.OK and ffn(tokens=0, ws=0, nbytes=0, x=P.ptoc_matrix(None, 64)) == P.OK


def fb(x=None, pre=None, q=None, dy=None, dx=None, din=None, dout=None, ws=None, nbytes=None, tokens=8, hidden=64,
       inter=32, dt=P.BF16):
    need = P.ptoc_gated_ffn_backward_workspace(tokens, hidden, inter)
    return P.ptoc_gated_ffn_backward(x or m(0), pre or m(1), q or fp(), dy or m(2), dx, din, dout,
                                     at(30) if ws is None else ws, need if nbytes is None else nbytes, tokens, hidden,
                                     inter, dt, stream=0, check=False)


def test_gated_ffn_backward_rejects():
    assert fb(dx=m(3), dt=P.F32) == UNS and fb(dx=m(3), dt=9) == BAD
    for sizes in SIZES:
        assert fb(dx=m(3), **sizes) == BAD
    for sizes in FAR:
        assert fb(dx=m(3), **sizes) == UNS
    assert fb(q=fp(act=7), dx=m(3)) == BAD
    assert fb(pre=m(1, 63), dx=m(3)) == BAD and fb(dy=m(2, 32), dx=m(3)) == BAD
    assert fb(dx=m(3, 32)) == BAD and fb(din=m(4, 32)) == BAD and fb(dout=m(5, 16)) == BAD
    assert fb(dx=m(3), ws=0) == BAD and fb(dx=m(3), ws=at(30) + 8) == BAD
    assert fb(dx=m(3), nbytes=P.ptoc_gated_ffn_backward_workspace(8, 64, 32) - 1) == BAD
    for i in (0, 1, 2, 20, 21, 30):                                             # inputs, the workspace
        assert fb(dx=m(i)) == ALIAS and fb(din=m(i)) == ALIAS and fb(dout=m(i)) == ALIAS
    assert fb(dx=m(3), din=m(3)) == ALIAS and fb(din=m(4), dout=m(4)) == ALIAS
    assert fb() == P.OK                                                         # nothing is asked for
    assert fb(tokens=0, dx=m(3), ws=0, nbytes=0) == P.OK


# ---- the gradients' norm -----------------------------------------------------------------

def g(i, rows=4, cols=64, ld=64, out=None, ld_out=64, dt=P.BF16, off=0):
    return P.ptoc_gradient(at(i) + off, out, ld, ld_out, rows, cols, dt)


def clip(*grads, max_norm=1.0, result=at(50), ws=at(51), nbytes=None):
    need = P.ptoc_clip_gradients_workspace(len(grads))
    return P.ptoc_clip_gradients(list(grads), max_norm, result, ws, need if nbytes is None else nbytes, stream=0,
                                 check=False)


def test_clip_gradients_rejects():
    for norm in (0.0, -1.0, float("nan"), float("-inf")):
        assert clip(g(0), max_norm=norm) == BAD
    assert clip(g(0), result=0) == BAD and clip(g(0), result=at(50) + 2) == BAD
    assert clip(g(0), ws=0) == BAD and clip(g(0), ws=at(51) + 128) == BAD
    assert clip(g(0), nbytes=P.ptoc_clip_gradients_workspace(1) - 1) == BAD
    assert clip(g(0, dt=P.I32)) == UNS and clip(g(0, dt=8)) == BAD
    assert clip(g(0, rows=-1)) == BAD and clip(g(0, ld=63)) == BAD and clip(g(0, off=1)) == BAD
    assert clip(g(0, out=at(1), ld_out=60)) == BAD and clip(g(0, out=at(1) + 1)) == BAD
    assert clip(P.ptoc_gradient(None, None, 64, 64, 4, 64, P.BF16)) == BAD
    assert clip(g(0), g(0)) == ALIAS                                            # the same gradient twice
    assert clip(g(0), g(0, off=256)) == ALIAS                                   # its second half too
    assert clip(g(0, out=at(1)), g(2, out=at(1))) == ALIAS                      # two outs
    assert clip(g(0, out=at(2)), g(2)) == ALIAS                                 # an out over another gradient
    assert clip(g(0, out=at(0) + 128)) == ALIAS                                 # over its own, not the same matrix
    assert clip(g(0, ld=128, out=at(0), ld_out=64)) == ALIAS
    assert clip(g(0), result=at(0) + 16) == ALIAS and clip(g(0), ws=at(0)) == ALIAS
    assert clip(g(0), result=at(51)) == ALIAS
    assert clip(P.ptoc_gradient(1 << 50, None, 64, 64, 2 ** 40, 64, P.BF16)) == UNS     # 2^46 elements
    assert P.ptoc_clip_gradients_workspace(P.CLIP_MAX_GRADIENTS + 1) == 0
    assert clip(*[g(0, rows=0)] * (P.CLIP_MAX_GRADIENTS + 1), nbytes=1 << 30) == UNS
    assert P.ptoc_clip_gradients([g(0)], 1.0, at(50), None, 0, stream=0, check=False) == BAD


# ---- the binding's own refusals --------------------------------------------------------------

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def block(h=64, i=32, dtype=torch.bfloat16):
    return P.GatedFfn(t(2 * i, h, dtype=dtype), t(h, i, dtype=dtype))


def test_host_tensors_are_refused():
    """Every convenience, with arguments that are right but for their memory."""
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    x, stats, res = t(4, 64), torch.zeros(2, 4), torch.zeros(2)
    for call in (lambda: P.layer_norm([x], t(4, 64)), lambda: P.layer_norm_backward(x, stats, x, x, workspace=ws),
                 lambda: block()(x, t(4, 64), workspace=ws),
                 lambda: block().backward(x, t(4, 64), x, d_x=t(4, 64), workspace=ws),
                 lambda: P.Gradients([x]).clip(1.0, res, workspace=ws),
                 lambda: P.Gradients([]).clip(1.0, res, workspace=ws),
                 lambda: P.Gradients([x]).clip(1.0, res, workspace=ws, stream=0)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_layouts_are_refused():
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    x, stats = t(4, 64), torch.zeros(2, 4)
    f = block()
    calls = [lambda: P.layer_norm([], x), lambda: P.layer_norm([x, t(4, 63)], x),
             lambda: P.layer_norm([x], t(4, 64, dtype=torch.float16)), lambda: P.layer_norm([x], t(64, 4).t()),
             lambda: P.layer_norm([x], x, weight=t(63)), lambda: P.layer_norm([x], x, weight=t(64), bias=torch.zeros(64)),
             lambda: P.layer_norm([x], x, weight=t(64, dtype=torch.float16)),
             lambda: P.layer_norm([x], x, stats=torch.zeros(4, 2)),
             lambda: P.layer_norm_backward(x, stats[:, :3], x, x, workspace=ws),
             lambda: P.layer_norm_backward(x, stats, x, x, t(64), workspace=ws),
             lambda: P.GatedFfn(t(63, 64), t(64, 32)), lambda: P.GatedFfn(t(64, 64), t(64, 32), act="relu"),
             lambda: block(dtype=torch.float32), lambda: P.GatedFfn(t(64, 64), t(64, 32, dtype=torch.float16)),
             lambda: P.GatedFfn(t(64, 64).t(), t(64, 32)),
             lambda: f(t(4, 63), x, workspace=ws), lambda: f(x, t(3, 64), workspace=ws),
             lambda: f(x, x, pre=t(4, 63), workspace=ws), lambda: f(x, x, workspace=ws[::2]),
             lambda: f(t(4, 64, dtype=torch.float16), x, workspace=ws),
             lambda: f.backward(x, None, x, workspace=ws), lambda: f.backward(x, t(4, 64), None, workspace=ws),
             lambda: f.backward(x, t(4, 64), x, d_w_in=t(64, 63), workspace=ws),
             lambda: f.backward(x, t(4, 64), x, d_w_out=t(32, 64), workspace=ws),
             lambda: P.Gradients([x], []), lambda: P.Gradients([x], [t(4, 63)]),
             lambda: P.Gradients([x], [t(4, 64, dtype=torch.float16)]), lambda: P.Gradients([t(64, 4).t()]),
             lambda: P.Gradients([t(2, 4, 64)[:, :, :8]]),
             lambda: P.Gradients([x]).clip(1.0, torch.zeros(3), workspace=ws),
             lambda: P.Gradients([x]).clip(1.0, t(2), workspace=ws)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)
    with pytest.raises(TypeError):
        P.Gradients([torch.zeros(4, dtype=torch.float64)])


def test_weights_and_gradients_are_followed():
    f = block()
    before = f._params()
    f.w_in.data = t(64, 80)[:, :64]
    assert f._params() != before and f._params() == f._packed
    f.w_in.data = t(64, 48)
    with pytest.raises(ValueError, match="w_in"):
        f._params()
    grads = [t(4, 64), torch.zeros(7)]
    s = P.Gradients(grads)
    before = s._pack()
    assert s._pack() is before
    grads[1].data = torch.zeros(9)
    assert s._pack() != before and len(s._packed) == 2 * ctypes.sizeof(P.ptoc_gradient)


def test_gradient_layouts():
    """Packed tensors are one row; a packed one beside one with gaps keeps its rows."""
    wide = t(4, 70)[:, :64]

    def rows(grads, outs=None):
        raw = P.Gradients(grads, outs)._packed
        return [(q.ld, q.ld_out, q.rows, q.cols) for q in (P.ptoc_gradient * len(grads)).from_buffer_copy(raw)]

    assert rows([t(4, 64), t(2, 3, 5), wide, torch.tensor(1.0)]) == [(256, 256, 1, 256), (30, 30, 1, 30),
                                                                     (70, 70, 4, 64), (1, 1, 1, 1)]
    assert rows([wide, t(4, 64), wide], [t(4, 64), wide, t(4, 90)[:, :64]]) == [(70, 64, 4, 64), (64, 70, 4, 64),
                                                                                (70, 90, 4, 64)]


def test_gated_ffn_parts():
    """Two numbers for what passes between the products: the binding's choice, other numbers, and twice the workspace."""
    two = fp(parts=2)
    for call, need in ((ffn, P.ptoc_gated_ffn_workspace(8, 64, 32)),
                       (functools.partial(fb, dx=m(3)), P.ptoc_gated_ffn_backward_workspace(8, 64, 32))):
        assert call(q=fp(parts=3)) == BAD and call(q=fp(parts=-1)) == BAD
        assert call(q=two, nbytes=2 * need - 1) == BAD
        # the workspace is as long as that: its second half is not another operand's
        assert call(q=two, nbytes=2 * need, ws=at(0) - 2 * need + 256, x=m(0)) == ALIAS
    w_in, w_out = t(64, 64), t(64, 32)
    one = P.GatedFfn(w_in, w_out)
    both = P.GatedFfn(w_in, w_out, parts=2)
    assert P.ptoc_gated_ffn_params.from_buffer_copy(one._params()).parts == 1
    assert P.ptoc_gated_ffn_params.from_buffer_copy(both._params()).parts == 2
    for name in ("workspace", "backward_workspace"):
        assert getattr(both, name)(8).numel() == 2 * getattr(one, name)(8).numel()
    for parts in (0, 3, None):
        with pytest.raises(ValueError, match="parts"):
            P.GatedFfn(w_in, w_out, parts=parts)


def test_header_offsets_match(tmp_path):
    """Members whose place a size does not tell."""
    src, exe = tmp_path / "o.c", tmp_path / "o"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ptoc_dense.h"\nint main(void) {\n'
                   'printf("%d %d %d\\n", (int)offsetof(ptoc_gated_ffn_params, act), '
                   '(int)offsetof(ptoc_gated_ffn_params, parts), (int)offsetof(ptoc_gradient, dtype)); return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), "-I",
                    cuda_include(), "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out] == [P.ptoc_gated_ffn_params.act.offset, P.ptoc_gated_ffn_params.parts.offset,
                                     P.ptoc_gradient.dtype.offset]
