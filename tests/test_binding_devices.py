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


class Strided(FakeTensor):
    def is_contiguous(self):
        return False

    def stride(self):
        return (1, self.shape[0])


def _linear(activation="none", has_bias=False):
    lin = tfmoe.Linear.__new__(tfmoe.Linear)
    lin.lib, lin.handle, lin.device, lin._widths = FakeLibrary(), None, torch.device("cuda:0"), (64, 48)
    lin.desc = tfmoe.LinearDesc(64, 48, 4, tfmoe.ACTIVATIONS.index(activation), int(has_bias), 0)
    return lin


def _weights(prefixes=("",), bias=None):
    w = {}
    for p in prefixes:
        w.update({p + "codes": FakeTensor((48, 32), "cuda:0", torch.uint8), p + "scales": FakeTensor((48, 4), "cuda:0", torch.uint8),
                  p + "global": FakeTensor((1,), "cuda:0", torch.float32)})
    if bias:
        w["bias"] = FakeTensor((bias,), "cuda:0", torch.float32)
    return w


@pytest.mark.parametrize("name,error,bad", [
    ("codes", ValueError, Strided((48, 32), "cuda:0", torch.uint8)), ("codes", ValueError, FakeTensor((32, 48), "cuda:0", torch.uint8)),
    ("codes", ValueError, FakeTensor((47, 32), "cuda:0", torch.uint8)), ("codes", TypeError, FakeTensor((48, 32), "cuda:0", torch.int32)),
    ("codes", ValueError, FakeTensor((48, 32), "cpu", torch.uint8)), ("codes", ValueError, FakeTensor((48, 32), "cuda:1", torch.uint8)),
    ("scales", TypeError, FakeTensor((48, 4), "cuda:0", torch.bfloat16)), ("scales", ValueError, FakeTensor((48, 3), "cuda:0", torch.uint8)),
    ("scales", ValueError, FakeTensor((), "cuda:0", torch.uint8)), ("global", TypeError, FakeTensor((1,), "cuda:0", torch.float64)),
    ("global", ValueError, FakeTensor((0,), "cuda:0", torch.float32)), ("global", ValueError, FakeTensor((1,), "cpu", torch.float32)),
    ("bias", TypeError, FakeTensor((96,), "cuda:0", torch.bfloat16)), ("bias", ValueError, FakeTensor((48,), "cuda:0", torch.float32)),
    ("up_codes", ValueError, FakeTensor((48, 16), "cuda:0", torch.uint8)), ("up_scales", ValueError, Strided((48, 4), "cuda:0", torch.uint8)),
    ("up_global", ValueError, FakeTensor((1,), "cuda:1", torch.float32)),
])
def test_load_weights_of_the_product_refuses_what_the_repack_would_misread(name, error, bad):
    lin = _linear("swiglu", has_bias=True)
    w = _weights(("", "up_"), bias=96)
    w[name] = bad
    with pytest.raises(error, match=name):
        lin.load_weights(w)
    assert lin.lib.calls == []


def test_load_weights_of_the_product_takes_what_it_reads():
    lin = _linear("swiglu", has_bias=True)
    lin.load_weights(_weights(("", "up_"), bias=96))
    w = _weights()
    w["scales"] = FakeTensor((48, 4), "cuda:0", torch.float8_e4m3fn)
    w["codes"] = FakeTensor((48 * 32,), "cuda:0", torch.uint8)          # flat
    w["global"] = FakeTensor((), "cuda:0", torch.float32)
    w["bias"] = torch.zeros(3)                                          # not read by a handle without a bias
    plain = _linear()
    plain.load_weights(w)
    assert [n for n, _ in lin.lib.calls + plain.lib.calls] == ["tfmoe_linear_load_weights"] * 2
    packed = _linear()                                                  # the bytes by their types' names
    packed.load_weights({**_weights(), "codes": FakeTensor((48, 32), "cuda:0", torch.float4_e2m1fn_x2)})
    assert len(packed.lib.calls) == 1
    given = plain.lib.calls[0][1][1]._obj
    assert given.codes == 4096 and given.bias is None and given.up_codes is None
    missing = _linear()
    missing.load_weights({"codes": w["codes"], "scales": w["scales"]})   # the library refuses a missing pointer
    assert getattr(missing.lib.calls[0][1][1]._obj, "global") is None
