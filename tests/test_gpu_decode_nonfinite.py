"""Non-finite activations in tfmoe_forward_decode: the routing is tfmoe_forward's, bit for bit.

A logit is the sum of the products x w, so an infinity in x makes it infinite, or NaN where it meets a
zero weight or the opposite infinity, whatever the size of the router's weights; a NaN makes it NaN.
Both paths sum in 64 bits, where no product of finite bf16 values overflows, so which entries are
non-finite does not depend on the order of the sum, and the finite ones are exact in both.
"""
import numpy as np
import pytest

from nvfp4_weight_only_route_b200 import synth

pytestmark = pytest.mark.gpu

INF, NEG_INF, NAN, NEG_NAN = 0x7F80, 0xFF80, 0x7FC0, 0xFFC0


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_weight_only_route_b200 import build
    build.build()


def _layer(H, I, E, k, router_std, seed):
    shape = synth.custom_shape(H, I, E, k, global_scale=0.02, router_std=router_std)
    return shape, synth.make_layer(shape, seed)


def _handle(layer, shape, T, flags=0):
    from nvfp4_weight_only_route_b200 import tfmoe
    L = tfmoe.MoELayer(shape.H, shape.I, shape.E, shape.k, T, has_router_bias=layer.get("router_bias") is not None, flags=flags)
    L.load_weights(tfmoe.layer_to_device(layer))
    return L


def _dev(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()


def _routing(L, run, x):
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    T, k, E = x.shape[0], L.desc.top_k, L.desc.num_experts
    out = run(_dev(x))
    out = out[0] if isinstance(out, tuple) else out
    assert L.sync_status() == 0, tfmoe.last_error()
    one = lambda b, dt, n: L.buffer_tensor(b, dt, (T, n)).cpu().numpy()
    return (one(tfmoe.BUF_LOGITS, torch.float32, E), one(tfmoe.BUF_TOPK_IDS, torch.int32, k),
            one(tfmoe.BUF_TOPK_WEIGHTS, torch.float32, k), out.float().cpu().numpy())


@pytest.mark.parametrize("router_std", [0.02, 1.0])
@pytest.mark.parametrize("H,E,k,T", [(256, 8, 2, 6), (2048, 128, 8, 6), (512, 200, 5, 16)])
def test_same_routing_as_the_chain(H, E, k, T, router_std):
    shape, layer = _layer(H, 128, E, k, router_std, seed=83)
    layer["router_w"][1, 7] = 0                        # an infinity there is NaN for expert 1
    x = synth.make_x(shape, 83, T)
    x[1, 3], x[2, H - 1], x[3, 7], x[4, 7] = INF, NEG_INF, NAN, INF
    x[5, 0], x[5, H // 2] = INF, NEG_INF
    if T > 6:
        x[9, 100] = NEG_NAN
    L = _handle(layer, shape, T)
    try:
        want, got = _routing(L, L.forward, x), _routing(L, L.forward_decode, x)
    finally:
        L.close()
    finite = [t for t in range(T) if t not in (1, 2, 3, 4, 5, 9)]
    assert not np.isfinite(want[0][1:6]).any() and np.isfinite(want[0][finite]).all()
    for w, g in zip(want[:3], got[:3]):
        assert np.array_equal(w.view(np.int32), g.view(np.int32))
    assert np.isfinite(got[3][finite]).all() and not np.isfinite(got[3][1:6]).any()


@pytest.mark.parametrize("value", [INF, NEG_INF, NAN])
def test_debug_word_whatever_the_size_of_the_router_weights(value):
    from nvfp4_weight_only_route_b200 import tfmoe
    shape, layer = _layer(256, 128, 8, 2, 0.02, seed=84)
    x = synth.make_x(shape, 84, 2)
    x[1, 3] = value
    L = _handle(layer, shape, 2, flags=tfmoe.FLAG_DEBUG_CHECKS)
    try:
        L.forward_decode(_dev(synth.make_x(shape, 84, 2)))
        assert L.sync_status() == 0
        L.forward_decode(_dev(x))
        assert L.sync_status() == tfmoe.ERR_DEVICE
        assert L.sync_status() == 0
    finally:
        L.close()
