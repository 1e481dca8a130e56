"""The layer operators' binding without a GPU: tensors that a kernel could not
use, first calls from several threads, tensors whose storage is replaced."""
import pytest
import torch

import tile_level_collective_gb300 as P
from tile_level_collective_gb300 import layers


def t(rows=4, cols=64, dtype=torch.bfloat16):
    return torch.zeros(rows, cols, dtype=dtype)


def moe_layer():
    h = torch.bfloat16
    return P.MoeLayer(torch.zeros(8, 64, dtype=h), torch.zeros(8, 64, 64, dtype=h), torch.zeros(8, 64, 32, dtype=h), 2)


# ---- where tensors live --------------------------------------------------------------

def test_host_tensors_are_refused():
    """Every convenience, with arguments that are right but for their memory:
    nothing reaches the library."""
    ws = torch.zeros(1 << 22, dtype=torch.uint8)
    k = P.Checkpoint8(4, 64, device="cpu")
    calls = [lambda: P.block_norm([t(), t()], t(), t()), lambda: P.checkpoint8(t(), k), lambda: P.restore8(k, t()),
             lambda: P.block_norm_backward(t(), t(), torch.zeros(2, 4), t(), t(), t(), workspace=ws),
             lambda: P.block_norm_backward(k, k, torch.zeros(2, 4), t(), t(), t(), workspace=ws, stream=0),
             lambda: moe_layer()(t(), t(), workspace=ws), lambda: moe_layer()(t(), t(), workspace=ws, stream=0)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_another_device_than_the_current_one_is_refused(monkeypatch):
    layers._code(torch.bfloat16)
    monkeypatch.setattr(layers, "_one_device", False)
    monkeypatch.setattr(layers, "_current_device", lambda: 0)
    monkeypatch.setattr(layers, "_raw_stream", lambda device: 1234)
    assert layers._stream_of(None, 0) == 1234
    for stream in (None, 0):
        with pytest.raises(ValueError, match="current"):
            layers._stream_of(stream, 1)


def test_workspaces_elsewhere_or_with_gaps_are_refused():
    ws = torch.zeros(256, dtype=torch.uint8)
    assert layers._space(ws, -1) == (ws.data_ptr(), 256)
    with pytest.raises(ValueError, match="workspace"):
        layers._space(ws, 0)                                     # a host tensor for tensors on device 0
    with pytest.raises(ValueError, match="workspace"):
        layers._space(ws[::2], -1)


# ---- the first call ------------------------------------------------------------------

def test_names_are_complete_before_the_first_code_is_seen(monkeypatch):
    """A second thread takes the codes as the sign that every name is set."""
    names = ("_float32", "_int32", "_raw_stream", "_current_device", "_one_device")
    layers._code(torch.bfloat16)
    seen = []

    class Codes(dict):
        def update(self, *a):
            seen.append([getattr(layers, n, None) is not None for n in names])
            super().update(*a)

    for n in names:
        monkeypatch.setattr(layers, n, None)
    monkeypatch.setattr(layers, "_codes", Codes())
    assert layers._code(torch.float16) == P.F16
    assert seen == [[True] * len(names)]


# ---- tensors whose storage is replaced -----------------------------------------------

def test_checkpoints_follow_their_tensors():
    k = P.Checkpoint8(4, 70, device="cpu")
    kind = (k.shape, 4, 70, torch.bfloat16, -1)
    packed = lambda: layers._ckpt(k, kind, "ckpt")
    assert packed() == layers._ckpt_bytes(k.codes.data_ptr(), 96, k.exps.data_ptr(), 3)
    k.codes.data = torch.zeros(4, 80, dtype=torch.int8)[:, :70]
    assert packed() == layers._ckpt_bytes(k.codes.data_ptr(), 80, k.exps.data_ptr(), 3)
    k.exps.data = torch.zeros(4, 8, dtype=torch.uint8)[:, :3]
    assert packed() == layers._ckpt_bytes(k.codes.data_ptr(), 80, k.exps.data_ptr(), 8)
    k.codes = torch.zeros(4, 64, dtype=torch.int8)                  # other columns than its exponents
    with pytest.raises(ValueError):
        packed()
    k.codes, k.exps = torch.zeros(3, 70, dtype=torch.int8), torch.zeros(3, 3, dtype=torch.uint8)
    with pytest.raises(ValueError):
        packed()


@pytest.mark.parametrize("name", ["router", "w_in", "w_out", "bias"])
def test_layers_follow_their_weights(name):
    h = torch.bfloat16
    w = dict(router=torch.zeros(8, 64, dtype=h), w_in=torch.zeros(8, 64, 64, dtype=h),
             w_out=torch.zeros(8, 64, 32, dtype=h), bias=torch.zeros(8))
    layer = P.MoeLayer(w["router"], w["w_in"], w["w_out"], 2, bias=w["bias"])
    at = lambda: {k: getattr(layer._weights(), k) for k in w}
    assert at() == {k: v.data_ptr() for k, v in w.items()}
    old = w[name].detach()
    w[name].data = torch.ones_like(old)
    assert at() == {k: v.data_ptr() for k, v in w.items()} and w[name].data_ptr() != old.data_ptr()
    for bad in (old[:4].clone(), old.double()):
        w[name].data = bad
        with pytest.raises(ValueError, match=name):
            layer._weights()
