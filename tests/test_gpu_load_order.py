"""load_weights runs after all work that was enqueued on the device before it, on any stream."""
import numpy as np
import pytest

import linear_reference as ref
from nvfp4_weight_only_route_b200 import synth
from test_gpu_decode import _check, _handle, _layer, _run

pytestmark = pytest.mark.gpu

DELAY = 40_000_000          # clocks: some 20 ms, far longer than a load


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_weight_only_route_b200 import build
    build.build()


def _dev(a):
    import torch
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def _late(new, into):
    """Fills the tensors `into` with `new` on a side stream, after a delay that the host does not wait for."""
    import torch
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(DELAY)
        for k, t in into.items():
            t.copy_(new[k])
    return s


def test_layer_weights_written_on_another_stream(oracle_mod):
    from nvfp4_weight_only_route_b200 import tfmoe
    shape, layer = _layer(512, 256, 8, 2, seed=96)
    x = synth.make_x(shape, 96, 3)
    L = _handle(_layer(512, 256, 8, 2, seed=97)[1], shape, 3)
    try:
        new = {k: v for k, v in tfmoe.layer_to_device(layer).items() if v is not None}
        into = {k: v.new_zeros(v.shape) for k, v in new.items()}
        s = _late(new, into)
        assert not s.query()
        L.load_weights(into)
        _check(oracle_mod, layer, shape, x, _run(L, x))
    finally:
        L.close()


def test_layer_weights_replaced_under_a_forward(oracle_mod):
    """A forward that waits on its stream still reads the weights that were loaded when it was called."""
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    shape, old = _layer(512, 256, 8, 2, seed=98)
    new = _layer(512, 256, 8, 2, seed=99)[1]
    x = synth.make_x(shape, 98, 3)
    L = _handle(old, shape, 3)
    try:
        xd, want = _dev(x), L.forward(_dev(x))
        out, s, other = torch.empty_like(want), torch.cuda.Stream(), tfmoe.layer_to_device(new)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(DELAY)
        L.forward(xd, out=out, stream=s)
        L.load_weights(other)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        _check(oracle_mod, new, shape, x, _run(L, x))
    finally:
        L.close()


def test_product_weights_written_on_another_stream():
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    rng = np.random.default_rng(100)
    K, N, T = 512, 300, 3
    w = ref.make_weights(rng, K, N, bias=True)
    x = ref.bf16_bits(rng.standard_normal((T, K)))
    lin = tfmoe.Linear(K, N, max_tokens=T, has_bias=True, out_fp32=True)
    try:
        new = {k: _dev(v) for k, v in w.items()}
        into = {k: torch.zeros_like(v) for k, v in new.items()}
        s = _late(new, into)
        assert not s.query()
        lin.load_weights(into)
        got = lin.forward(_dev(x))
        assert lin.sync_status() == 0
        ref.check(got.double().cpu().numpy(), *ref.linear64(x, w, fp32=True))
    finally:
        lin.close()
