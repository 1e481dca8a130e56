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
import struct

from . import OK, F16, F32, BF16, PtocError, _addr, _done, _group, _lib, _stream, _vp, _i64

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
    _fields_ = [("block", ptoc_matrix), ("stream", ptoc_matrix), ("block_ckpt", ptoc_ckpt8),
                ("stream_ckpt", ptoc_ckpt8), ("rstd", _vp)]


class ptoc_moe_params(ctypes.Structure):
    _fields_ = [("router", _vp), ("bias", _vp), ("w_in", _vp), ("w_out", _vp), ("router_dtype", _i32),
                ("experts", _i32), ("first_expert", _i32), ("local_experts", _i32), ("top_k", _i32), ("score", _i32),
                ("renormalize", _i32), ("scale", _f32)]


# Structure arguments are declared as addresses: the C-name calls below pass
# structures by reference, the conveniences pass their packed bytes.
_lib.ptoc_checkpoint8.argtypes = [_vp, _vp, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_restore8.argtypes = [_vp, _vp, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_block_norm.argtypes = [_vp, _i64] + [_vp] * 8 + [_i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_block_norm_backward.argtypes = [_vp] * 10 + [_size_t, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_block_norm_backward_workspace.argtypes = [_i64, _i64]
_lib.ptoc_moe_few_tokens.argtypes = [_vp] * 6 + [_size_t, _i64, _i64, _i64, ctypes.c_int, _vp]
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
# They run for every layer of every step, and a small call's kernel is shorter
# than a careless check of its arguments: each tensor's layout is read once,
# and the C structures are packed as bytes.

_matrix_bytes = struct.Struct("Pq").pack
_ckpt_bytes = struct.Struct("PqPq").pack
_params_bytes = struct.Struct("iiPPPqqfff4x").pack
_saved_bytes = struct.Struct("PqPqPqPqPqPqP").pack
assert struct.calcsize("iiPPPqqfff4x") == ctypes.sizeof(ptoc_block_norm_params)
_group_bytes = struct.Struct("Pii").pack
_array_types = {}
_codes = {}
_raw_stream = _current_device = _one_device = None


def _torch_names():
    """Fill what depends on torch, which the package imports on first use."""
    import torch
    global _raw_stream, _current_device, _one_device, _float32, _int32
    _float32, _int32 = torch.float32, torch.int32
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _one_device = torch.cuda.device_count() == 1
    _codes.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})     # last: tells that all is there


def _code(dtype):
    if not _codes:
        _torch_names()
    code = _codes.get(dtype)
    if code is None:
        raise TypeError("unsupported dtype %s" % dtype)
    return code


def _stream_of(stream, device):
    """The given stream, or torch's current one on the tensors' device (an
    index; -1 for the host's memory). The kernels run on the current device:
    tensors elsewhere are refused (last, after every check of the layouts)."""
    if device < 0:
        raise ValueError("expected tensors on a CUDA device")
    if not _one_device and device != _current_device():
        raise ValueError("the tensors' device cuda:%d is not the current one" % device)
    return _raw_stream(device) if stream is None else _stream(stream)


def _call(status, where):
    if status != OK:
        raise PtocError(status, where)
    return status


def _pitch(t, rows, cols, what):
    """The row pitch of a [rows, cols] tensor. A single row may have any row stride."""
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError("%s: rows must be contiguous (stride(1) == 1)" % what)
    return ld if rows > 1 or ld > cols else cols


def _first(t, what):
    """Shape, rows, columns, dtype and device index of the tensor that the others must match."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s: expected a 2-D tensor" % what)
    return shape, shape[0], shape[1], t.dtype, t.get_device()


def _like(t, kind, what):
    """A matrix argument of the activations' kind (_first's answer), packed for C; None stays None."""
    if t is None:
        return None
    shape, rows, cols, dtype, device = kind
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        raise ValueError("%s: needs the shape, dtype and device of the activations" % what)
    return _matrix_bytes(t.data_ptr(), _pitch(t, rows, cols, what))


def _packed(t, shape, dtype, device, what):
    """The address of a packed tensor argument; None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: expected a packed %s tensor of shape %s on the activations' device" %
                         (what, dtype, tuple(shape)))
    return t.data_ptr()


def _workspace(nbytes, device):
    import torch
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _space(workspace, device):
    """Address and bytes of a workspace argument."""
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace: expected a packed tensor on the activations' device")
    return workspace.data_ptr(), workspace.nbytes


class Checkpoint8:
    """Storage of a [rows, cols] activation in 8 bits: ``codes`` (int8) and
    ``exps`` (uint8, one for every 32 columns), both with padded pitches."""

    def __init__(self, rows, cols, device="cuda"):
        import torch
        blocks = (cols + CKPT_BLOCK - 1) // CKPT_BLOCK
        self._hold(torch.empty(rows, blocks * CKPT_BLOCK, dtype=torch.int8, device=device)[:, :cols],
                   torch.empty(rows, blocks, dtype=torch.uint8, device=device), cols)

    @classmethod
    def of(cls, codes, exps, cols=None):
        """A checkpoint over given codes [rows, cols] and exponent bytes."""
        cols = codes.shape[-1] if cols is None else cols
        k = cls.__new__(cls)
        k._hold(codes, exps, cols)
        return k

    def _hold(self, codes, exps, cols):
        import torch
        if codes.dtype != torch.int8 or exps.dtype != torch.uint8 or codes.device != exps.device:
            raise ValueError("checkpoint: expected int8 codes and uint8 exponents on one device")
        if codes.dim() != 2 or codes.shape[1] != cols or \
                tuple(exps.shape) != (codes.shape[0], (cols + CKPT_BLOCK - 1) // CKPT_BLOCK):
            raise ValueError("checkpoint: expected codes [rows, cols] and exponents [rows, ceil(cols / 32)]")
        self.codes, self.exps = codes, exps
        self.shape, self.device = codes.shape, codes.get_device()
        self.c = (codes.data_ptr(), _pitch(codes, *codes.shape, "codes"), exps.data_ptr(),
                  _pitch(exps, *exps.shape, "exps"))
        self.packed = _ckpt_bytes(*self.c)


def _ckpt(k, kind, what):
    if k is None:
        return None
    if k.shape != kind[0] or k.device != kind[4]:
        raise ValueError("%s: the checkpoint needs the shape and device of the activations" % what)
    c = k.c
    if k.codes.data_ptr() != c[0] or k.exps.data_ptr() != c[2]:
        # its tensors have got other storage
        k._hold(k.codes, k.exps, kind[2])
        if k.shape != kind[0] or k.device != kind[4]:
            raise ValueError("%s: the checkpoint's tensors were replaced by others of another kind" % what)
    return k.packed


def checkpoint8(x, ckpt, stream=None):
    """ckpt = x [rows, cols] in 8 bits."""
    kind = _first(x, "checkpoint8")
    shape, rows, cols, dtype, device = kind
    code = _code(dtype)
    st = _lib.ptoc_checkpoint8(_like(x, kind, "checkpoint8"), _ckpt(ckpt, kind, "checkpoint8"), rows, cols, code,
                               _stream_of(stream, device))
    return _call(st, "ptoc_checkpoint8")


def restore8(ckpt, x, stream=None):
    """x [rows, cols] = the values that the checkpoint holds."""
    kind = _first(x, "restore8")
    shape, rows, cols, dtype, device = kind
    code = _code(dtype)
    st = _lib.ptoc_restore8(_ckpt(ckpt, kind, "restore8"), _like(x, kind, "restore8"), rows, cols, code,
                            _stream_of(stream, device))
    return _call(st, "ptoc_restore8")


def _gate_strides(gate, rows, cols):
    """Row and column stride of a gate that broadcasts to [rows, cols]: a
    scalar, [cols], [1, cols], [rows, 1] or [rows, cols]."""
    d = gate.dim()
    if d > 2:
        raise ValueError("gate: expected at most 2 dimensions")
    shape, stride = gate.shape, gate.stride()
    across = shape[d - 1] if d > 0 else 1
    down = shape[0] if d > 1 else 1
    if down not in (1, rows) or across not in (1, cols):
        raise ValueError("gate: shape %s does not broadcast to [%d, %d]" % (tuple(shape), rows, cols))
    rs = stride[0] if down > 1 else 0
    cs = stride[d - 1] if across > 1 else 0
    if down > 1 and rs < 1 or across > 1 and cs != 1:
        raise ValueError("gate: needs packed columns and its own rows")
    return rs, cs


def _norm_params(kind, post_norm, post_weight, pre_weight, gate, residual_scale, branch_scale, eps):
    shape, rows, cols, dtype, device = kind
    if post_weight is not None and not post_norm:
        raise ValueError("block_norm: post_weight without the norm after the block")
    params = None
    for t in (post_weight, pre_weight, gate):
        if t is not None:
            if params is None:
                params = t.dtype
            if t.dtype is not params or (params is not dtype and params is not _float32) or t.get_device() != device:
                raise ValueError("block_norm: weights and gate need one dtype (the activations' or float32) and their "
                                 "device")
    rs, cs = _gate_strides(gate, rows, cols) if gate is not None else (0, 0)
    columns = (cols,)
    return _params_bytes(1 if post_norm else 0, _codes[dtype if params is None else params],
                         _packed(post_weight, columns, params, device, "post_weight") or 0,
                         _packed(pre_weight, columns, params, device, "pre_weight") or 0,
                         0 if gate is None else gate.data_ptr(), rs, cs, residual_scale, branch_scale, eps)


def block_norm(parts, residual, out, normed=None, *, post_norm=True, post_weight=None, pre_weight=None, gate=None,
               residual_scale=1.0, branch_scale=1.0, eps=1e-6, block_out=None, block_ckpt=None, stream_ckpt=None,
               rstd=None, stream=None):
    """out = residual_scale * residual + branch_scale * gate * norm(sum of parts);
    normed = norm(out) * pre_weight. ``out`` may be ``residual``. ``gate``
    broadcasts to the activations; ``rstd`` is float32 [2, rows]."""
    n = len(parts)
    if n == 0:
        raise ValueError("block_norm: expected at least one part")
    first = parts[0]
    kind = _first(first, "parts")
    shape, rows, cols, dtype, device = kind
    code = _code(dtype)
    ld = _pitch(first, rows, cols, "parts")
    pointers = [first.data_ptr()]
    if n > 1:
        strides = first.stride()
        for t in parts[1:]:
            if t.dtype is not dtype or t.get_device() != device or t.shape != shape or t.stride() != strides:
                raise ValueError("block_norm: every part needs the same shape, strides, dtype and device")
            pointers.append(t.data_ptr())
    array = _array_types.get(n)
    if array is None:
        array = _array_types[n] = ctypes.c_void_p * n
    group = array(*pointers)
    p = _norm_params(kind, post_norm, post_weight, pre_weight, gate, residual_scale, branch_scale, eps)
    st = _lib.ptoc_block_norm(
        _group_bytes(ctypes.addressof(group), n, 0), ld, _like(residual, kind, "residual"), p, _like(out, kind, "out"),
        _like(normed, kind, "normed"), _like(block_out, kind, "block_out"), _ckpt(block_ckpt, kind, "block_ckpt"),
        _ckpt(stream_ckpt, kind, "stream_ckpt"), _packed(rstd, (2, rows), _float32, device, "rstd"), rows, cols, code,
        _stream_of(stream, device))
    return _call(st, "ptoc_block_norm")


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
    kind = _first(d_normed, "d_normed")
    shape, rows, cols, dtype, device = kind
    code = _code(dtype)
    if d_gate is not None and gate is None:
        raise ValueError("block_norm_backward: d_gate without a gate")
    p = _norm_params(kind, post_norm, post_weight, pre_weight, gate, residual_scale, branch_scale, eps)
    held = [(0, 0), (0, 0), (0, 0, 0, 0), (0, 0, 0, 0)]           # block, stream, their checkpoints
    for i, (t, what) in enumerate(((block, "block"), (saved_stream, "stream"))):
        if isinstance(t, Checkpoint8):
            _ckpt(t, kind, what)
            held[2 + i] = t.c
        else:
            _like(t, kind, what)
            held[i] = (t.data_ptr(), _pitch(t, rows, cols, what))
    columns = (cols,)
    s = _saved_bytes(*held[0], *held[1], *held[2], *held[3],
                     _packed(rstd, (2, rows), _float32, device, "rstd") or 0)
    space, nbytes = _space(workspace, device)
    st = _lib.ptoc_block_norm_backward(
        s, p, _like(d_normed, kind, "d_normed"), _like(d_stream, kind, "d_stream"),
        _like(d_residual, kind, "d_residual"), _like(d_block, kind, "d_block"),
        _packed(d_pre_weight, columns, _float32, device, "d_pre_weight"),
        _packed(d_post_weight, columns, _float32, device, "d_post_weight"),
        _packed(d_gate, None if gate is None else gate.shape, _float32, device, "d_gate"), space, nbytes, rows, cols,
        code, _stream_of(stream, device))
    return _call(st, "ptoc_block_norm_backward")


class MoeLayer:
    """A mixture-of-experts layer over given weights: ``router`` [experts,
    hidden], ``w_in`` [local, 2 * inter, hidden] (gate rows, then up rows) and
    ``w_out`` [local, hidden, inter], where ``local`` counts the experts held
    here, from ``first_expert`` on. The weights are used in place, where they
    are at each call."""

    def __init__(self, router, w_in, w_out, top_k, *, bias=None, first_expert=0, score="softmax", renormalize=True,
                 scale=1.0):
        if w_in.dim() != 3 or w_out.dim() != 3 or router.dim() != 2:
            raise ValueError("MoeLayer: expected router [experts, hidden], w_in [local, 2 * inter, hidden] and "
                             "w_out [local, hidden, inter]")
        local, hidden, inter = w_out.shape
        dtype, device = w_in.dtype, w_in.get_device()
        self.code = _code(dtype)
        if score not in SCORES:
            raise ValueError("MoeLayer: score is one of %s" % sorted(SCORES))
        if router.dtype not in (dtype, _float32):
            raise ValueError("MoeLayer: the router needs the experts' dtype or float32")
        self.router, self.w_in, self.w_out, self.bias = router, w_in, w_out, bias
        self.dtype, self.device = dtype, w_in.device
        self._kind = (dtype, device)
        self.hidden, self.inter, self.experts, self.top_k = hidden, inter, router.shape[0], top_k
        self._shapes = ((self.experts, hidden), (self.experts,), (local, 2 * inter, hidden), (local, hidden, inter))
        self._router_dtype = router.dtype
        self.params = ptoc_moe_params(None, None, None, None, _code(router.dtype), self.experts, first_expert, local,
                                      top_k, SCORES[score], int(bool(renormalize)), scale)
        self._at = None
        self._weights()

    def _weights(self):
        """The C parameters. The weights may have got other storage since the
        last call."""
        bias = self.bias
        at = (self.router.data_ptr(), bias if bias is None else bias.data_ptr(), self.w_in.data_ptr(),
              self.w_out.data_ptr())
        if at != self._at:
            self._take(at)
        return self.params

    def _take(self, at):
        dtype, device = self._kind
        router, bias, w_in, w_out = self._shapes
        _packed(self.router, router, self._router_dtype, device, "router")
        _packed(self.bias, bias, _float32, device, "bias")
        _packed(self.w_in, w_in, dtype, device, "w_in")
        _packed(self.w_out, w_out, dtype, device, "w_out")
        q = self.params
        q.router, q.bias, q.w_in, q.w_out = self._at = at

    def workspace(self, tokens):
        """A workspace tensor for calls of up to `tokens` tokens."""
        n = ptoc_moe_few_tokens_workspace(tokens, self.hidden, self.inter, self.experts, self.top_k)
        return _workspace(n, self.device)

    def __call__(self, x, y, *, ids=None, weights=None, workspace, stream=None):
        """y [tokens, hidden] = the held experts' part of the layer's output
        for x; ids (int32) and weights (float32) [tokens, top_k] are optional
        outputs."""
        kind = _first(x, "x")
        shape, tokens, hidden, dtype, device = kind
        if (dtype, device) != self._kind or hidden != self.hidden:
            raise ValueError("MoeLayer: x needs the weights' width, dtype and device")
        choice = (tokens, self.top_k)
        space, nbytes = _space(workspace, device)
        st = _lib.ptoc_moe_few_tokens(
            _like(x, kind, "x"), ctypes.byref(self._weights()), _like(y, kind, "y"),
            _packed(ids, choice, _int32, device, "ids"), _packed(weights, choice, _float32, device, "weights"),
            space, nbytes, tokens, hidden, self.inter, self.code, _stream_of(stream, device))
        return _call(st, "ptoc_moe_few_tokens")
