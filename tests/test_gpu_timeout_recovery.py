"""After a wait that gave up, tfmoe_sync_status / tfmoe_linear_sync_status make the same handle usable again.

TFMOE_FLAG_TEST_TIMEOUT makes one thread of a handle's first call wait 1 ms for something that nothing does;
every other wait of that call then ends by the abort flag, and the call returns.
"""
import numpy as np
import pytest

import linear_reference as ref
from nvfp4_weight_only_route_b200 import synth
from test_gpu_decode import _check, _handle, _layer, _run

pytestmark = pytest.mark.gpu

STREAM, MMA = 0x1, 0x2


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


@pytest.mark.parametrize("H,I,E,k,m,T", [(256, 128, 8, 2, 0, 1), (512, 256, 16, 4, 1, 8), (2048, 768, 64, 8, 0, 12)])
def test_decode_on_the_handle_that_timed_out(oracle_mod, H, I, E, k, m, T):
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    shape, layer = _layer(H, I, E, k, m, seed=91)
    x = synth.make_x(shape, 91, T)
    L = _handle(layer, shape, T, m, flags=tfmoe.FLAG_TEST_TIMEOUT)
    s = torch.cuda.Stream()                                # does not wait for the legacy stream
    try:
        xd, out = _dev(x), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        L.forward_decode(xd, out=out, stream=s)
        assert L.sync_status(s) == tfmoe.ERR_TIMEOUT
        L.forward_decode(xd, out=out, stream=s)            # at once, on the same stream
        assert L.sync_status(s) == 0
        first = out.view(torch.int16).clone()
        _check(oracle_mod, layer, shape, x, _run(L, x), m)
        for _ in range(20):
            L.forward_decode(xd, out=out, stream=s)
        assert L.sync_status(s) == 0 and torch.equal(out.view(torch.int16), first)
    finally:
        L.close()


@pytest.mark.parametrize("T,K,N,act,flags", [
    (3, 2688, 130, "none", STREAM),         # row tiles cut by many CTAs
    (1, 128, 30000, "none", STREAM),        # several whole row tiles a CTA
    (16, 1040, 600, "swiglu", STREAM),
    (5, 2688, 130, "silu", MMA),            # split reductions
    (3, 64, 200, "none", MMA),              # one stage
    (400, 1024, 9000, "none", MMA),         # several tiles a CTA, none split
    (400, 1024, 4500, "swiglu", MMA),
])
def test_product_on_the_handle_that_timed_out(T, K, N, act, flags):
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    rng = np.random.default_rng(92)
    w = ref.make_weights(rng, K, N, gated=act == "swiglu")
    x = ref.bf16_bits(rng.standard_normal((T, K)))
    lin = tfmoe.Linear(K, N, max_tokens=T, activation=act, out_fp32=True, flags=flags | tfmoe.FLAG_TEST_TIMEOUT)
    s = torch.cuda.Stream()
    try:
        lin.load_weights({k: _dev(v) for k, v in w.items() if v is not None})
        xd, out = _dev(x), torch.empty((T, N), device="cuda")
        torch.cuda.synchronize()
        lin.forward(xd, out=out, stream=s)
        assert lin.sync_status(s) == tfmoe.ERR_TIMEOUT
        lin.forward(xd, out=out, stream=s)
        assert lin.sync_status(s) == 0
        ref.check(out.double().cpu().numpy(), *ref.linear64(x, w, act, fp32=True))
        first = out.clone()
        for _ in range(20):
            lin.forward(xd, out=out, stream=s)
        assert lin.sync_status(s) == 0 and torch.equal(out, first)
    finally:
        lin.close()
