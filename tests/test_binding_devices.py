"""The binding and a handle's device, without a GPU: stand-ins for tensors and for the library record what
would have been launched."""
import types

import pytest
import torch

from nvfp4_weight_only_route_b200 import tfmoe


class FakeTensor:
    """What the binding asks of a dense tensor, on any device."""

    def __init__(self, shape, device, dtype=torch.bfloat16):
        self.shape, self.device, self.dtype, self.is_cuda = tuple(shape), torch.device(device), dtype, True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


class FakeLibrary:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return tfmoe.OK
        return call


STREAM = types.SimpleNamespace(cuda_stream=77)


def _layer(device="cuda:0"):
    L = tfmoe.MoELayer.__new__(tfmoe.MoELayer)
    L.lib, L.handle, L.device = FakeLibrary(), None, torch.device(device)
    L.desc = tfmoe.LayerDesc(512, 256, 8, 2, 8, 0, 0, 0, 0, 1e-6)
    return L


def test_forward_decode_refuses_a_batch_on_another_device():
    """All tensors together on a device that is not the handle's: its kernel would run where the handle is."""
    here, there = [[FakeTensor((4, 512), d) for _ in range(4)] for d in ("cuda:0", "cuda:1")]
    gam = {d: FakeTensor((512,), d) for d in ("cuda:0", "cuda:1")}
    L = _layer()
    with pytest.raises(ValueError, match="x is on cuda:1, expected cuda:0"):
        L.forward_decode(there[0], residual=there[1], norm_w=gam["cuda:1"], out=there[2], out_norm=there[3], stream=STREAM)
    with pytest.raises(ValueError, match="x is on cuda:1"):
        L.forward_decode(there[0], out=here[0], stream=STREAM)
    assert L.lib.calls == []
    for kw in (dict(residual=there[1]), dict(norm_w=gam["cuda:1"], out_norm=here[3]), dict(norm_w=gam["cuda:0"], out_norm=there[3])):
        with pytest.raises(ValueError, match="expected cuda:0"):
            L.forward_decode(here[0], out=here[2], stream=STREAM, **kw)
    with pytest.raises(ValueError, match="out is on cuda:1"):
        L.forward_decode(here[0], out=there[2], stream=STREAM)
    assert L.lib.calls == []
    L.forward_decode(here[0], residual=here[1], norm_w=gam["cuda:0"], out=here[2], out_norm=here[3], stream=STREAM)
    assert [(n, a[-1]) for n, a in L.lib.calls] == [("tfmoe_forward_decode", 77)]
    L = _layer("cuda:1")                                # and a layer that lives on another device than the first
    L.forward_decode(there[0], out=there[2], stream=STREAM)
    assert len(L.lib.calls) == 1


def test_forward_decode_refuses_a_host_batch():
    L = _layer()
    with pytest.raises(ValueError, match="x is on cpu"):
        L.forward_decode(torch.zeros((4, 512), dtype=torch.bfloat16), stream=STREAM)
    assert L.lib.calls == []


@pytest.mark.parametrize("kind,call", [("MoELayer", "tfmoe_sync_status"), ("Linear", "tfmoe_linear_sync_status")])
def test_sync_status_waits_for_the_stream_its_forward_ran_on(kind, call, monkeypatch):
    """forward and forward_decode take the current stream of the handle's device, which need not be the current
    device; sync_status has to wait for the same one."""
    monkeypatch.setattr(tfmoe, "_current_stream", lambda device: 100 + device.index)
    cls = getattr(tfmoe, kind)
    h = cls.__new__(cls)
    h.lib, h.handle, h.device = FakeLibrary(), None, torch.device("cuda:1")
    assert h.sync_status() == tfmoe.OK and h.sync_status(stream=STREAM) == tfmoe.OK
    assert [(n, a[-1]) for n, a in h.lib.calls] == [(call, 101), (call, 77)]
