"""The layer operators' binding without a GPU: tensors that a kernel could not
use, and first calls from several threads."""
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
    names = ("_float32", "_int32", "_raw_stream", "_current_device")
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
