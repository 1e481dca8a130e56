"""Binding of the layer operators declared in ``include/ptoc_layers.h``: the
norms around a block whose output is spread over N windows, 8-bit activation
checkpoints, and a mixture-of-experts layer for a few tokens.

The C names take the C arguments; ``block_norm``, ``block_norm_backward``,
``checkpoint8``, ``restore8`` and ``MoeLayer`` infer sizes, pitches and types
from torch tensors and refuse (ValueError) what the C calls cannot describe.
Outputs and workspaces belong to the caller; nothing is allocated in a call.

    import torch, tile_level_collective_gb300 as ptoc

    # one decode step of a tensor-parallel model: the ranks' partial outputs of
    # a block are summed, normed, gated and added to the residual stream, and
    # the next block's input is normed, in one launch
    ptoc.block_norm(parts, residual, out, normed, post_weight=w_post,
                    pre_weight=w_pre, gate=gate, residual_scale=0.9)
    # this rank's experts on the normed tokens; y is its part of the next sum
    layer = ptoc.MoeLayer(router, w_in, w_out, top_k=8, experts=128, first_expert=32)
    layer(normed, y, workspace=layer.workspace(64))
"""
import ctypes

from . import (F32, _addr, _done, _group, _lib, _rows_cols_ld, _same_layout, _stream, _vp, _i64, _G, dtype_code)

CKPT_BLOCK = 32
NORM_MAX_COLS = 32768
MOE_MAX_TOKENS, MOE_MAX_EXPERTS, MOE_MAX_TOP_K = 64, 1024, 16
SCORES = {"softmax": 0, "sigmoid": 1}

_i32, _f32, _size_t = ctypes.c_int32, ctypes.c_float, ctypes.c_size_t


class ptoc_matrix(ctypes.Structure):
    _fields_ = [("data", _vp), ("ld", _i64)]


class ptoc_ckpt8(ctypes.Structure):
    _fields_ = [("codes", _vp), ("ld_codes", _i64), ("exps", _vp), ("ld_exps", _i64)]


class ptoc_block_norm_params(ctypes.Structure):
    _fields_ = [("post_norm", _i32), ("param_dtype", _i32), ("post_weight", _vp), ("pre_weight", _vp), ("gate", _vp),
                ("gate_row_stride", _i64), ("gate_col_stride", _i64), ("residual_scale", _f32),
                ("branch_scale", _f32), ("eps", _f32)]


class ptoc_block_norm_saved(ctypes.Structure):
    _fields_ = [("block", ctypes.POINTER(ptoc_matrix)), ("block_ckpt", ctypes.POINTER(ptoc_ckpt8)),
                ("stream", ctypes.POINTER(ptoc_matrix)), ("stream_ckpt", ctypes.POINTER(ptoc_ckpt8)), ("rstd", _vp)]


class ptoc_moe_params(ctypes.Structure):
    _fields_ = [("router", _vp), ("bias", _vp), ("w_in", _vp), ("w_out", _vp), ("router_dtype", _i32),
                ("experts", _i32), ("first_expert", _i32), ("local_experts", _i32), ("top_k", _i32), ("score", _i32),
                ("renormalize", _i32), ("scale", _f32)]


_M, _K = ctypes.POINTER(ptoc_matrix), ctypes.POINTER(ptoc_ckpt8)
_N, _S, _E = (ctypes.POINTER(t) for t in (ptoc_block_norm_params, ptoc_block_norm_saved, ptoc_moe_params))
_lib.ptoc_checkpoint8.argtypes = [_M, _K, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_restore8.argtypes = [_K, _M, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_block_norm.argtypes = [_G, _i64, _M, _N, _M, _M, _M, _K, _K, _vp, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_block_norm_backward.argtypes = [_S, _N, _M, _M, _M, _M, _vp, _vp, _vp, _vp, _size_t, _i64, _i64,
                                          ctypes.c_int, _vp]
_lib.ptoc_block_norm_backward_workspace.argtypes = [_i64, _i64]
_lib.ptoc_moe_few_tokens.argtypes = [_M, _E, _M, _vp, _vp, _vp, _size_t, _i64, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_moe_few_tokens_workspace.argtypes = [_i64, _i64, _i64, _i32, _i32]
for _f in ("ptoc_checkpoint8", "ptoc_restore8", "ptoc_block_norm", "ptoc_block_norm_backward", "ptoc_moe_few_tokens"):
    getattr(_lib, _f).restype = ctypes.c_int
for _f in ("ptoc_block_norm_backward_workspace", "ptoc_moe_few_tokens_workspace"):
    getattr(_lib, _f).restype = _size_t


def _ref(x):
    return None if x is None else ctypes.byref(x)


# ---- the C calls (structures and addresses as the header declares them) -----------

def ptoc_checkpoint8(x, out, rows, cols, dtype, stream=None, check=True):
    st = _lib.ptoc_checkpoint8(_ref(x), _ref(out), rows, cols, int(dtype), _stream(stream))
    return _done(st, "ptoc_checkpoint8", check)


def ptoc_restore8(ckpt, x, rows, cols, dtype, stream=None, check=True):
    st = _lib.ptoc_restore8(_ref(ckpt), _ref(x), rows, cols, int(dtype), _stream(stream))
    return _done(st, "ptoc_restore8", check)


def ptoc_block_norm(parts, ld_parts, x, params, out, normed, block_out, block_ckpt, stream_ckpt, rstd, rows, cols,
                    dtype, stream=None, check=True):
    g, keep = _group(parts)
    st = _lib.ptoc_block_norm(ctypes.byref(g), ld_parts, _ref(x), _ref(params), _ref(out), _ref(normed),
                              _ref(block_out), _ref(block_ckpt), _ref(stream_ckpt), _addr(rstd), rows, cols,
                              int(dtype), _stream(stream))
    return _done(st, "ptoc_block_norm", check)


def ptoc_block_norm_backward(saved, params, dy, du, d_residual, d_block, d_pre_weight, d_post_weight, d_gate,
                             workspace, workspace_bytes, rows, cols, dtype, stream=None, check=True):
    st = _lib.ptoc_block_norm_backward(_ref(saved), _ref(params), _ref(dy), _ref(du), _ref(d_residual), _ref(d_block),
                                       _addr(d_pre_weight), _addr(d_post_weight), _addr(d_gate), _addr(workspace),
                                       workspace_bytes, rows, cols, int(dtype), _stream(stream))
    return _done(st, "ptoc_block_norm_backward", check)


def ptoc_block_norm_backward_workspace(rows, cols):
    """Bytes of workspace that ptoc_block_norm_backward needs."""
    return _lib.ptoc_block_norm_backward_workspace(rows, cols)


def ptoc_moe_few_tokens(x, params, y, ids, weights, workspace, workspace_bytes, tokens, hidden, inter, dtype,
                        stream=None, check=True):
    st = _lib.ptoc_moe_few_tokens(_ref(x), _ref(params), _ref(y), _addr(ids), _addr(weights), _addr(workspace),
                                  workspace_bytes, tokens, hidden, inter, int(dtype), _stream(stream))
    return _done(st, "ptoc_moe_few_tokens", check)


def ptoc_moe_few_tokens_workspace(tokens, hidden, inter, experts, top_k):
    """Bytes of workspace that ptoc_moe_few_tokens needs (0 for sizes it does not take)."""
    return _lib.ptoc_moe_few_tokens_workspace(tokens, hidden, inter, experts, top_k)


# ---- shape-inferring conveniences over torch tensors -------------------------------

def _matrix(t):
    """A 2-D tensor as a ptoc_matrix. A single row may have any row stride."""
    rows, cols, ld = _rows_cols_ld(t)
    return ptoc_matrix(t.data_ptr(), max(ld, cols) if rows <= 1 else ld)


def _like(t, ref, what):
    if tuple(t.shape) != tuple(ref.shape) or t.dtype != ref.dtype or t.device != ref.device:
        raise ValueError("%s: needs the shape, dtype and device of the activations" % what)


def _packed(t, shape, dtype, device, what):
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError("%s: expected a packed %s tensor of shape %s on %s" % (what, dtype, tuple(shape), device))
    return t


def _workspace(nbytes, device):
    import torch
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


class Checkpoint8:
    """Storage of a [rows, cols] activation in 8 bits: ``codes`` (int8) and
    ``exps`` (uint8, one for every 32 columns), both with padded pitches."""

    def __init__(self, rows, cols, device="cuda"):
        import torch
        blocks = (cols + CKPT_BLOCK - 1) // CKPT_BLOCK
        self.cols = cols
        self.codes = torch.empty(rows, blocks * CKPT_BLOCK, dtype=torch.int8, device=device)[:, :cols]
        self.exps = torch.empty(rows, blocks, dtype=torch.uint8, device=device)

    @classmethod
    def of(cls, codes, exps, cols=None):
        """A checkpoint over given codes [rows, cols] and exponent bytes."""
        import torch
        k = cls.__new__(cls)
        k.cols = codes.shape[1] if cols is None else cols
        if codes.dtype != torch.int8 or exps.dtype != torch.uint8 or codes.device != exps.device:
            raise ValueError("checkpoint: expected int8 codes and uint8 exponents on one device")
        if tuple(codes.shape) != (codes.shape[0], k.cols) or \
                tuple(exps.shape) != (codes.shape[0], (k.cols + CKPT_BLOCK - 1) // CKPT_BLOCK):
            raise ValueError("checkpoint: expected codes [rows, cols] and exponents [rows, ceil(cols / 32)]")
        k.codes, k.exps = codes, exps
        return k

    @property
    def shape(self):
        return tuple(self.codes.shape)

    def c(self):
        m, e = _matrix(self.codes), _matrix(self.exps)
        return ptoc_ckpt8(m.data, m.ld, e.data, e.ld)


def _ckpt(k, ref, what):
    if k is None:
        return None
    if k.shape != tuple(ref.shape) or k.codes.device != ref.device:
        raise ValueError("%s: the checkpoint needs the shape and device of the activations" % what)
    return k.c()


def checkpoint8(x, ckpt, stream=None):
    """ckpt = x [rows, cols] in 8 bits."""
    return ptoc_checkpoint8(_matrix(x), _ckpt(ckpt, x, "checkpoint8"), x.shape[0], x.shape[1], dtype_code(x),
                            stream=stream)


def restore8(ckpt, x, stream=None):
    """x [rows, cols] = the values that the checkpoint holds."""
    return ptoc_restore8(_ckpt(ckpt, x, "restore8"), _matrix(x), x.shape[0], x.shape[1], dtype_code(x), stream=stream)


def _gate_strides(gate, rows, cols):
    """Row and column stride of a gate that broadcasts to [rows, cols]: a
    scalar, [cols], [1, cols], [rows, 1] or [rows, cols]."""
    if gate.dim() > 2:
        raise ValueError("gate: expected at most 2 dimensions")
    shape = (1,) * (2 - gate.dim()) + tuple(gate.shape)
    stride = (0,) * (2 - gate.dim()) + tuple(gate.stride())
    if shape[0] not in (1, rows) or shape[1] not in (1, cols):
        raise ValueError("gate: shape %s does not broadcast to [%d, %d]" % (tuple(gate.shape), rows, cols))
    rs = stride[0] if shape[0] > 1 else 0
    cs = stride[1] if shape[1] > 1 else 0
    if shape[0] > 1 and rs < 1 or cs not in (0, 1) or shape[1] > 1 and cs != 1:
        raise ValueError("gate: needs packed columns and its own rows")
    return rs, cs


def _norm_params(ref, post_norm, post_weight, pre_weight, gate, residual_scale, branch_scale, eps):
    import torch
    rows, cols = ref.shape
    given = [t for t in (post_weight if post_norm else None, pre_weight, gate) if t is not None]
    kind = given[0].dtype if given else ref.dtype
    for t in given:
        if t.dtype != kind or kind not in (ref.dtype, torch.float32) or t.device != ref.device:
            raise ValueError("block_norm: weights and gate need one dtype (the activations' or float32) and their device")
    for t, what in ((post_weight, "post_weight"), (pre_weight, "pre_weight")):
        _packed(t, (cols,), t.dtype if t is not None else None, ref.device, what)
    if post_weight is not None and not post_norm:
        raise ValueError("block_norm: post_weight without the norm after the block")
    rs, cs = _gate_strides(gate, rows, cols) if gate is not None else (0, 0)
    return ptoc_block_norm_params(int(bool(post_norm)), dtype_code(given[0]) if given else dtype_code(ref),
                                  _addr(post_weight), _addr(pre_weight), _addr(gate), rs, cs, residual_scale,
                                  branch_scale, eps)


def block_norm(parts, residual, out, normed=None, *, post_norm=True, post_weight=None, pre_weight=None, gate=None,
               residual_scale=1.0, branch_scale=1.0, eps=1e-6, block_out=None, block_ckpt=None, stream_ckpt=None,
               rstd=None, stream=None):
    """out = residual_scale * residual + branch_scale * gate * norm(sum of parts);
    normed = norm(out) * pre_weight. ``out`` may be ``residual``. ``gate``
    broadcasts to the activations; ``rstd`` is float32 [2, rows]."""
    import torch
    rows, cols, ld = _same_layout(parts, "block_norm")
    if rows <= 1:
        ld = max(ld, cols)
    for t, what in ((residual, "residual"), (out, "out"), (normed, "normed"), (block_out, "block_out")):
        if t is not None:
            _like(t, parts[0], what)
    _packed(rstd, (2, rows), torch.float32, out.device, "rstd")
    p = _norm_params(out, post_norm, post_weight, pre_weight, gate, residual_scale, branch_scale, eps)
    return ptoc_block_norm(parts, ld, _matrix(residual), p, _matrix(out), None if normed is None else _matrix(normed),
                           None if block_out is None else _matrix(block_out), _ckpt(block_ckpt, out, "block_ckpt"),
                           _ckpt(stream_ckpt, out, "stream_ckpt"), rstd, rows, cols, dtype_code(out), stream=stream)


def block_norm_backward_workspace(rows, cols, device="cuda"):
    """A workspace tensor for block_norm_backward on [rows, cols] activations."""
    return _workspace(ptoc_block_norm_backward_workspace(rows, cols), device)


def block_norm_backward(block, saved_stream, rstd, d_normed, d_residual, d_block, d_pre_weight=None, *,
                        d_post_weight=None, d_gate=None, d_stream=None, post_norm=True, post_weight=None,
                        pre_weight=None, gate=None, residual_scale=1.0, branch_scale=1.0, eps=1e-6, workspace,
                        stream=None):
    """Gradients of block_norm. ``block`` and ``saved_stream`` are the forward
    pass's block output and stream, as tensors or Checkpoint8; ``d_stream`` is
    the gradient that reaches the stream from later layers. ``d_block`` is the
    gradient of every part. Weight and gate gradients are float32, the gate's
    in the gate's shape."""
    import torch
    ref = d_normed
    rows, cols, _ = _rows_cols_ld(ref)
    for t, what in ((d_residual, "d_residual"), (d_block, "d_block"), (d_stream, "d_stream")):
        if t is not None:
            _like(t, ref, what)
    _packed(rstd, (2, rows), torch.float32, ref.device, "rstd")
    for t, what in ((d_pre_weight, "d_pre_weight"), (d_post_weight, "d_post_weight")):
        _packed(t, (cols,), torch.float32, ref.device, what)
    if d_gate is not None:
        if gate is None:
            raise ValueError("block_norm_backward: d_gate without a gate")
        _packed(d_gate, gate.shape, torch.float32, ref.device, "d_gate")
    p = _norm_params(ref, post_norm, post_weight, pre_weight, gate, residual_scale, branch_scale, eps)
    s = ptoc_block_norm_saved()
    keep = []
    for t, what in ((block, "block"), (saved_stream, "stream")):
        if isinstance(t, Checkpoint8):
            keep.append(_ckpt(t, ref, what))
            setattr(s, what + "_ckpt", ctypes.pointer(keep[-1]))
        else:
            _like(t, ref, what)
            keep.append(_matrix(t))
            setattr(s, what, ctypes.pointer(keep[-1]))
    s.rstd = rstd.data_ptr()
    return ptoc_block_norm_backward(s, p, _matrix(d_normed), None if d_stream is None else _matrix(d_stream),
                                    _matrix(d_residual), _matrix(d_block), d_pre_weight, d_post_weight, d_gate,
                                    workspace, workspace.numel() * workspace.element_size(), rows, cols,
                                    dtype_code(ref), stream=stream)


class MoeLayer:
    """A mixture-of-experts layer over given weights: ``router`` [experts,
    hidden], ``w_in`` [local, 2 * inter, hidden] (gate rows, then up rows) and
    ``w_out`` [local, hidden, inter], where ``local`` counts the experts held
    here, from ``first_expert`` on. The weights are used in place."""

    def __init__(self, router, w_in, w_out, top_k, *, bias=None, first_expert=0, score="softmax", renormalize=True,
                 scale=1.0):
        import torch
        if w_in.dim() != 3 or w_out.dim() != 3 or router.dim() != 2:
            raise ValueError("MoeLayer: expected router [experts, hidden], w_in [local, 2 * inter, hidden] and "
                             "w_out [local, hidden, inter]")
        local, hidden, inter = w_out.shape
        device = w_in.device
        _packed(w_in, (local, 2 * inter, hidden), w_in.dtype, device, "w_in")
        _packed(w_out, (local, hidden, inter), w_in.dtype, device, "w_out")
        if router.dtype not in (w_in.dtype, torch.float32):
            raise ValueError("MoeLayer: the router needs the experts' dtype or float32")
        _packed(router, (router.shape[0], hidden), router.dtype, device, "router")
        _packed(bias, (router.shape[0],), torch.float32, device, "bias")
        if score not in SCORES:
            raise ValueError("MoeLayer: score is one of %s" % sorted(SCORES))
        self.router, self.w_in, self.w_out, self.bias = router, w_in, w_out, bias
        self.hidden, self.inter, self.experts, self.top_k = hidden, inter, router.shape[0], top_k
        self.params = ptoc_moe_params(_addr(router), _addr(bias), _addr(w_in), _addr(w_out), dtype_code(router),
                                      self.experts, first_expert, local, top_k, SCORES[score], int(bool(renormalize)),
                                      scale)

    def workspace(self, tokens):
        """A workspace tensor for calls of up to `tokens` tokens."""
        n = ptoc_moe_few_tokens_workspace(tokens, self.hidden, self.inter, self.experts, self.top_k)
        return _workspace(n, self.w_in.device)

    def __call__(self, x, y, *, ids=None, weights=None, workspace, stream=None):
        """y [tokens, hidden] = the held experts' part of the layer's output
        for x; ids (int32) and weights (float32) [tokens, top_k] are optional
        outputs."""
        import torch
        tokens, hidden, _ = _rows_cols_ld(x)
        if hidden != self.hidden or x.dtype != self.w_in.dtype or x.device != self.w_in.device:
            raise ValueError("MoeLayer: x needs the weights' width, dtype and device")
        _like(y, x, "y")
        _packed(ids, (tokens, self.top_k), torch.int32, x.device, "ids")
        _packed(weights, (tokens, self.top_k), torch.float32, x.device, "weights")
        return ptoc_moe_few_tokens(_matrix(x), self.params, _matrix(y), ids, weights, workspace,
                                   workspace.numel() * workspace.element_size(), tokens, hidden, self.inter,
                                   dtype_code(x), stream=stream)
