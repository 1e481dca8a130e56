"""Binding of the dense block's operators declared in ``include/ptoc_dense.h``:
layer norm of a sum of windows, the gated feed-forward block, both with their
backward pass, and the global norm of the gradients with clipping.

The C names take the C arguments; ``layer_norm``, ``layer_norm_backward``,
``GatedFfn`` and ``Gradients`` infer sizes, pitches and types from torch tensors
and refuse (ValueError) what the C calls cannot describe. Outputs and workspaces
belong to the caller; nothing is allocated on the device in a call. While a call
is being made, no other thread may put work on its stream that writes its tensors
or uses its workspace (a call is several launches).

    import torch, tile_level_collective_gb300 as ptoc

    # the end of one block and the start of the next: the ranks' partial outputs
    # are summed, added to the residual stream, and normed, in one launch
    ptoc.layer_norm(parts, normed, residual=x, out=x, weight=w, bias=b, stats=stats)
    # this rank's slice of a dense block; y is its part of the next sum
    ffn = ptoc.GatedFfn(w_in, w_out)
    ffn(normed, y, pre=pre, workspace=ffn.workspace(tokens))
    ffn.backward(normed, pre, d_y, d_x=d_x, d_w_in=d_w_in, d_w_out=d_w_out,
                 workspace=ffn.backward_workspace(tokens))
    # the norm of every gradient together, and the gradients scaled to at most 1
    grads = ptoc.Gradients([d_w_in, d_w_out, d_w, d_b])
    grads.clip(1.0, result, workspace=grads.workspace())
"""
import ctypes
import struct

from . import F16, BF16, _addr, _done, _group, _lib, _stream, _vp, _i64
from . import layers as _layers
from .layers import (_array_types, _call, _code, _codes, _f32, _first, _group_bytes, _i32, _like, _matrix_bytes, _packed,
                     _pitch, _ref, _size_t, _space, _stream_of, _workspace, ptoc_matrix)

ACTIVATIONS = {"silu": 0, "gelu": 1}
FFN_MAX_TOKENS, FFN_MAX_WIDTH = 4194304, 262144
CLIP_MAX_GRADIENTS = 65536


class ptoc_layer_norm_params(ctypes.Structure):
    _fields_ = [("weight", _vp), ("bias", _vp), ("param_dtype", _i32), ("eps", _f32)]


class ptoc_gated_ffn_params(ctypes.Structure):
    _fields_ = [("w_in", ptoc_matrix), ("w_out", ptoc_matrix), ("act", _i32), ("parts", _i32)]


class ptoc_gradient(ctypes.Structure):
    _fields_ = [("data", _vp), ("out", _vp), ("ld", _i64), ("ld_out", _i64), ("rows", _i64), ("cols", _i64),
                ("dtype", _i32)]


_lib.ptoc_layer_norm.argtypes = [_vp, _i64] + [_vp] * 5 + [_i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_layer_norm_backward.argtypes = [_vp] * 9 + [_size_t, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_layer_norm_backward_workspace.argtypes = [_i64, _i64]
_lib.ptoc_gated_ffn.argtypes = [_vp] * 5 + [_size_t, _i64, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_gated_ffn_workspace.argtypes = [_i64, _i64, _i64]
_lib.ptoc_gated_ffn_backward.argtypes = [_vp] * 8 + [_size_t, _i64, _i64, _i64, ctypes.c_int, _vp]
_lib.ptoc_gated_ffn_backward_workspace.argtypes = [_i64, _i64, _i64]
_lib.ptoc_clip_gradients.argtypes = [_vp, _i32, _f32, _vp, _vp, _size_t, _vp]
_lib.ptoc_clip_gradients_workspace.argtypes = [_i32]
for _f in ("ptoc_layer_norm", "ptoc_layer_norm_backward", "ptoc_gated_ffn", "ptoc_gated_ffn_backward",
           "ptoc_clip_gradients"):
    getattr(_lib, _f).restype = ctypes.c_int
for _f in ("ptoc_layer_norm_backward_workspace", "ptoc_gated_ffn_workspace", "ptoc_gated_ffn_backward_workspace",
           "ptoc_clip_gradients_workspace"):
    getattr(_lib, _f).restype = _size_t


# ---- the C calls (structures and addresses as the header declares them) -----------

def ptoc_layer_norm(parts, ld_parts, x, params, out, normed, stats, rows, cols, dtype, stream=None, check=True):
    g, keep = _group(parts)
    st = _lib.ptoc_layer_norm(ctypes.byref(g), ld_parts, _ref(x), _ref(params), _ref(out), _ref(normed), _addr(stats),
                              rows, cols, int(dtype), _stream(stream))
    return _done(st, "ptoc_layer_norm", check)


def ptoc_layer_norm_backward_workspace(rows, cols):
    """Bytes of workspace that ptoc_layer_norm_backward needs."""
    return _lib.ptoc_layer_norm_backward_workspace(rows, cols)


def ptoc_layer_norm_backward(s, stats, params, dy, du, dx, d_weight, d_bias, workspace, workspace_bytes, rows, cols,
                             dtype, stream=None, check=True):
    st = _lib.ptoc_layer_norm_backward(_ref(s), _addr(stats), _ref(params), _ref(dy), _ref(du), _ref(dx),
                                       _addr(d_weight), _addr(d_bias), _addr(workspace), workspace_bytes, rows, cols,
                                       int(dtype), _stream(stream))
    return _done(st, "ptoc_layer_norm_backward", check)


def ptoc_gated_ffn_workspace(tokens, hidden, inter):
    """Bytes of workspace that ptoc_gated_ffn needs (0 for sizes it does not take)."""
    return _lib.ptoc_gated_ffn_workspace(tokens, hidden, inter)


def ptoc_gated_ffn(x, params, y, pre, workspace, workspace_bytes, tokens, hidden, inter, dtype, stream=None,
                   check=True):
    st = _lib.ptoc_gated_ffn(_ref(x), _ref(params), _ref(y), _ref(pre), _addr(workspace), workspace_bytes, tokens,
                             hidden, inter, int(dtype), _stream(stream))
    return _done(st, "ptoc_gated_ffn", check)


def ptoc_gated_ffn_backward_workspace(tokens, hidden, inter):
    """Bytes of workspace that ptoc_gated_ffn_backward needs (0 for sizes it does not take)."""
    return _lib.ptoc_gated_ffn_backward_workspace(tokens, hidden, inter)


def ptoc_gated_ffn_backward(x, pre, params, dy, dx, d_w_in, d_w_out, workspace, workspace_bytes, tokens, hidden, inter,
                            dtype, stream=None, check=True):
    st = _lib.ptoc_gated_ffn_backward(_ref(x), _ref(pre), _ref(params), _ref(dy), _ref(dx), _ref(d_w_in),
                                      _ref(d_w_out), _addr(workspace), workspace_bytes, tokens, hidden, inter,
                                      int(dtype), _stream(stream))
    return _done(st, "ptoc_gated_ffn_backward", check)


def ptoc_clip_gradients_workspace(count):
    """Bytes of workspace that ptoc_clip_gradients needs."""
    return _lib.ptoc_clip_gradients_workspace(count)


def ptoc_clip_gradients(grads, max_norm, result, workspace, workspace_bytes, stream=None, check=True):
    """``grads``: a list of ptoc_gradient."""
    array = (ptoc_gradient * max(len(grads), 1))(*grads)
    st = _lib.ptoc_clip_gradients(array, len(grads), max_norm, _addr(result), _addr(workspace), workspace_bytes,
                                  _stream(stream))
    return _done(st, "ptoc_clip_gradients", check)


# ---- layer norm over torch tensors --------------------------------------------------

_norm_bytes = struct.Struct("PPif").pack
_ffn_bytes = struct.Struct("PqPqii").pack
_gradient_bytes = struct.Struct("PPqqqqi4x").pack
assert struct.calcsize("PPif") == ctypes.sizeof(ptoc_layer_norm_params)
assert struct.calcsize("PqPqii") == ctypes.sizeof(ptoc_gated_ffn_params)
assert struct.calcsize("PPqqqqi4x") == ctypes.sizeof(ptoc_gradient)


def _norm_params(kind, weight, bias, eps):
    shape, rows, cols, dtype, device = kind
    params = None
    for t in (weight, bias):
        if t is not None:
            if params is None:
                params = t.dtype
            if t.dtype is not params or (params is not dtype and params is not _layers._float32):
                raise ValueError("layer_norm: weight and bias need one dtype, the activations' or float32")
    columns = (cols,)
    return _norm_bytes(_packed(weight, columns, params, device, "weight") or 0,
                       _packed(bias, columns, params, device, "bias") or 0,
                       _codes[dtype if params is None else params], eps)


def layer_norm(parts, normed, *, residual=None, out=None, weight=None, bias=None, eps=1e-5, stats=None, stream=None):
    """out = residual + sum of parts; normed = its layer norm, times weight, plus
    bias. ``out`` may be ``residual``; ``stats`` is float32 [2, rows] (mean, then
    1 / standard deviation)."""
    n = len(parts)
    if n == 0:
        raise ValueError("layer_norm: expected at least one part")
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
                raise ValueError("layer_norm: every part needs the same shape, strides, dtype and device")
            pointers.append(t.data_ptr())
    array = _array_types.get(n)
    if array is None:
        array = _array_types[n] = ctypes.c_void_p * n
    group = array(*pointers)
    st = _lib.ptoc_layer_norm(
        _group_bytes(ctypes.addressof(group), n, 0), ld, _like(residual, kind, "residual"),
        _norm_params(kind, weight, bias, eps), _like(out, kind, "out"), _like(normed, kind, "normed"),
        _packed(stats, (2, rows), _layers._float32, device, "stats"), rows, cols, code, _stream_of(stream, device))
    return _call(st, "ptoc_layer_norm")


def layer_norm_backward_workspace(rows, cols, device="cuda"):
    """A workspace tensor for layer_norm_backward on [rows, cols] activations."""
    return _workspace(ptoc_layer_norm_backward_workspace(rows, cols), device)


def layer_norm_backward(saved_stream, stats, d_normed, d_x, d_weight=None, d_bias=None, *, d_stream=None, weight=None,
                        workspace, stream=None):
    """Gradients of layer_norm from its ``out`` (without a residual: the sum of
    the parts) and ``stats``. ``d_stream`` is the gradient that reaches the
    stream from later layers; ``d_x`` is the gradient of the residual and of
    every part. The weight's and the bias' gradients are float32."""
    kind = _first(d_normed, "d_normed")
    shape, rows, cols, dtype, device = kind
    code = _code(dtype)
    columns, f32 = (cols,), _layers._float32
    params = _norm_params(kind, weight, None, 1.0)
    space, nbytes = _space(workspace, device)
    st = _lib.ptoc_layer_norm_backward(
        _like(saved_stream, kind, "saved_stream"), _packed(stats, (2, rows), f32, device, "stats"), params,
        _like(d_normed, kind, "d_normed"), _like(d_stream, kind, "d_stream"), _like(d_x, kind, "d_x"),
        _packed(d_weight, columns, f32, device, "d_weight"), _packed(d_bias, columns, f32, device, "d_bias"), space,
        nbytes, rows, cols, code, _stream_of(stream, device))
    return _call(st, "ptoc_layer_norm_backward")


# ---- the gated feed-forward block ---------------------------------------------------

def _matrix(t, rows, cols, dtype, device, what):
    """A [rows, cols] matrix argument, packed for C; None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or t.shape != (rows, cols):
        raise ValueError("%s: expected a %s tensor of shape %s on the weights' device" % (what, dtype, (rows, cols)))
    return _matrix_bytes(t.data_ptr(), _pitch(t, rows, cols, what))


class GatedFfn:
    """A gated feed-forward block over given weights: ``w_in`` [2 * inter,
    hidden] (gate rows, then up rows) and ``w_out`` [hidden, inter], in float16
    or bfloat16, with rows at any pitch. ``act`` is "silu" or "gelu". The weights
    are used in place, where they are at each call. ``parts`` = 2: what passes
    between the products (act(g) * u, and the gradients of g and u) is held in two
    numbers of the weights' dtype instead of one, for 1.35 times the time forward
    and 1.6 to 2.4 times backward."""

    def __init__(self, w_in, w_out, act="silu", parts=1):
        if w_in.dim() != 2 or w_out.dim() != 2 or w_in.shape != (2 * w_out.shape[1], w_out.shape[0]):
            raise ValueError("GatedFfn: expected w_in [2 * inter, hidden] and w_out [hidden, inter]")
        if act not in ACTIVATIONS:
            raise ValueError("GatedFfn: act is one of %s" % sorted(ACTIVATIONS))
        if parts not in (1, 2):
            raise ValueError("GatedFfn: parts is 1 or 2")
        self.hidden, self.inter = w_out.shape
        self.w_in, self.w_out, self.act, self.parts = w_in, w_out, act, int(parts)
        self.dtype, self.device = w_in.dtype, w_in.device
        self.code = _code(self.dtype)
        if self.code not in (F16, BF16):
            raise ValueError("GatedFfn: the weights need float16 or bfloat16")
        self._kind = (w_in.dtype, w_in.get_device())
        self._at = None
        self._params()

    def _params(self):
        """The C parameters. The weights may have got other storage since the
        last call."""
        at = (self.w_in.data_ptr(), self.w_out.data_ptr(), self.w_in.stride(), self.w_out.stride(), self.w_in.shape,
              self.w_out.shape, self.w_in.dtype, self.w_out.dtype, self.act, self.parts)
        if at != self._at:
            dtype, device = self._kind
            for t, rows, cols, what in ((self.w_in, 2 * self.inter, self.hidden, "w_in"),
                                        (self.w_out, self.hidden, self.inter, "w_out")):
                _matrix(t, rows, cols, dtype, device, what)
            self._packed = _ffn_bytes(at[0], _pitch(self.w_in, 2 * self.inter, self.hidden, "w_in"), at[1],
                                      _pitch(self.w_out, self.hidden, self.inter, "w_out"), ACTIVATIONS[self.act],
                                      self.parts)
            self._at = at
        return self._packed

    def workspace(self, tokens):
        """A workspace tensor for calls of up to `tokens` tokens."""
        return _workspace(self.parts * ptoc_gated_ffn_workspace(tokens, self.hidden, self.inter), self.device)

    def backward_workspace(self, tokens):
        """A workspace tensor for backward passes of up to `tokens` tokens."""
        return _workspace(self.parts * ptoc_gated_ffn_backward_workspace(tokens, self.hidden, self.inter),
                          self.device)

    def _tokens(self, x):
        kind = _first(x, "x")
        shape, tokens, hidden, dtype, device = kind
        if (dtype, device) != self._kind or hidden != self.hidden:
            raise ValueError("GatedFfn: x needs the weights' width, dtype and device")
        return kind

    def __call__(self, x, y, *, pre=None, workspace, stream=None):
        """y [tokens, hidden] = the block's output for x; ``pre`` [tokens, 2 *
        inter], an optional output, is what the backward pass reads."""
        kind = self._tokens(x)
        shape, tokens, hidden, dtype, device = kind
        space, nbytes = _space(workspace, device)
        st = _lib.ptoc_gated_ffn(
            _like(x, kind, "x"), self._params(), _like(y, kind, "y"),
            _matrix(pre, tokens, 2 * self.inter, dtype, device, "pre"), space, nbytes, tokens, hidden, self.inter,
            self.code, _stream_of(stream, device))
        return _call(st, "ptoc_gated_ffn")

    def backward(self, x, pre, d_y, *, d_x=None, d_w_in=None, d_w_out=None, workspace, stream=None):
        """The gradients that are asked for, in the weights' dtype."""
        kind = self._tokens(x)
        shape, tokens, hidden, dtype, device = kind
        inter = self.inter
        space, nbytes = _space(workspace, device)
        if pre is None or d_y is None:
            raise ValueError("GatedFfn: the backward pass needs pre and d_y")
        st = _lib.ptoc_gated_ffn_backward(
            _like(x, kind, "x"), _matrix(pre, tokens, 2 * inter, dtype, device, "pre"), self._params(),
            _like(d_y, kind, "d_y"), _like(d_x, kind, "d_x"),
            _matrix(d_w_in, 2 * inter, hidden, dtype, device, "d_w_in"),
            _matrix(d_w_out, hidden, inter, dtype, device, "d_w_out"), space, nbytes, tokens, hidden, inter, self.code,
            _stream_of(stream, device))
        return _call(st, "ptoc_gated_ffn_backward")


# ---- the gradients' norm --------------------------------------------------------------

def _rows_of(t, what):
    """Rows, columns and pitch of a gradient: packed tensors are one row."""
    if t.is_contiguous():
        n = t.numel()
        return 1, n, n
    if t.dim() != 2:
        raise ValueError("%s: expected a packed tensor, or a 2-D one with contiguous rows" % what)
    rows, cols = t.shape
    return rows, cols, _pitch(t, rows, cols, what)


class Gradients:
    """A set of gradients (float32, float16 and bfloat16 together) whose global
    norm is taken and limited. Each is packed, or 2-D with contiguous rows.
    ``outs``: tensors of the same shapes and types that receive the scaled
    gradients; None: they are scaled in place. The tensors are used where they
    are at each call."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = None if outs is None else list(outs)
        if self.outs is not None and len(self.outs) != len(self.grads):
            raise ValueError("Gradients: expected an out for every gradient")
        if len(self.grads) > CLIP_MAX_GRADIENTS:
            raise ValueError("Gradients: at most %d" % CLIP_MAX_GRADIENTS)
        self._device = self.grads[0].get_device() if self.grads else None
        self._at = None
        self._pack()

    def _pack(self):
        at = [(t.data_ptr(), t.shape, t.stride(), t.dtype) for t in self.grads]
        if self.outs is not None:
            at += [(t.data_ptr(), t.shape, t.stride(), t.dtype) for t in self.outs]
        if at == self._at:
            return self._packed
        packed = []
        for i, t in enumerate(self.grads):
            o = t if self.outs is None else self.outs[i]
            if t.get_device() != self._device or o.get_device() != self._device:
                raise ValueError("Gradients: expected every tensor on one device")
            if o.shape != t.shape or o.dtype is not t.dtype:
                raise ValueError("Gradients: an out needs its gradient's shape and dtype")
            code = _code(t.dtype)
            rows, cols, ld = _rows_of(t, "Gradients")
            orows, ocols, ld_out = _rows_of(o, "Gradients")
            if orows != rows:                                    # one of them packed, the other with gaps
                rows, cols = t.shape
                ld = ld if orows == 1 else cols
                ld_out = cols if orows == 1 else ld_out
            packed.append(_gradient_bytes(t.data_ptr(), 0 if self.outs is None else o.data_ptr(), ld, ld_out, rows,
                                          cols, code))
        self._packed, self._at = b"".join(packed), at
        return self._packed

    def workspace(self):
        """A workspace tensor for calls on this set."""
        device = "cuda" if self._device is None else self.grads[0].device
        return _workspace(ptoc_clip_gradients_workspace(len(self.grads)), device)

    def clip(self, max_norm, result, *, workspace, stream=None):
        """Scale the set to a global norm of at most ``max_norm`` (infinity:
        the norm alone). ``result`` float32 [2]: the norm before, and the scale."""
        packed = self._pack()
        _code(result.dtype)
        device = result.get_device() if self._device is None else self._device
        at = _packed(result, (2,), _layers._float32, device, "result")
        space, nbytes = _space(workspace, device)
        st = _lib.ptoc_clip_gradients(packed, len(self.grads), max_norm, at, space, nbytes,
                                      _stream_of(stream, device))
        return _call(st, "ptoc_clip_gradients")
