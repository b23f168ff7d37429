"""Token rows whose elements lie further apart than one f16 row can hold.

The few-token kernels keep a token row as f16 times a power of two, which is exact while the row's
elements lie within 2^31 of one another. With an outlier 2^40 times the others the row has to be
summed without that rounding: where the outlier meets zero weights, the others are the whole result.
The references and bounds are those of the other tests (no allowance for x: it is exact).
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


def _product(T, K, N, x, w, act, flags, fp32=True, residual=None, in_place=False):
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    lin = tfmoe.Linear(K, N, max_tokens=T, activation=act, has_bias=w.get("bias") is not None, out_fp32=fp32, flags=flags)
    try:
        lin.load_weights({k: _dev(v) for k, v in w.items() if v is not None})
        r = None if residual is None else _dev(residual).view(torch.bfloat16)
        out = lin.forward(_dev(x), residual=r, out=r if in_place else None)
        assert lin.sync_status() == 0, tfmoe.last_error()
        again = None if in_place else lin.forward(_dev(x), residual=r)
        bits = torch.int32 if fp32 else torch.int16
        assert again is None or torch.equal(out.view(bits), again.view(bits))
        return out.double().cpu().numpy()
    finally:
        lin.close()


def _outlier_case(T, K, N, act, seed, bias=False, columns=(0,)):
    """Blocks of zero weights at `columns`, and there in every other row of x an element 2^40 times the rest."""
    rng = np.random.default_rng(seed)
    w = ref.make_weights(rng, K, N, gated=act == "swiglu", bias=bias)
    xf = rng.standard_normal((T, K))
    for c in columns:
        for p in ("", "up_") if act == "swiglu" else ("",):
            w[p + "scales"][:, c // 16] = 0
        xf[::2, c] = 2.0 ** 40
    return ref.bf16_bits(xf), w


@pytest.mark.parametrize("regime", [STREAM, MMA])
@pytest.mark.parametrize("T,K,N,act", [(1, 16, 40, "none"), (1, 320, 200, "none"), (3, 208, 130, "silu"), (8, 4096, 300, "none"),
                                       (9, 1040, 520, "swiglu"), (16, 704, 520, "none"), (16, 4096, 24000, "none")])
def test_outlier_over_zero_weights(T, K, N, act, regime):
    columns = {0, K // 2 // 16 * 16, K - 1}
    x, w = _outlier_case(T, K, N, act, 61, bias=N < 1000, columns=columns if K > 16 else (3,))
    ref.check(_product(T, K, N, x, w, act, regime), *ref.linear64(x, w, act, fp32=True))


@pytest.mark.parametrize("T,K,N", [(2, 128, 20000), (2, 2048, 129), (16, 256, 19000)])
def test_residual_in_place_of_wide_rows(T, K, N):
    """Whole and cut row tiles: every output is finished once, from the residual as it was."""
    x, w = _outlier_case(T, K, N, "none", 62)
    r = ref.bf16_bits(np.random.default_rng(63).standard_normal((T, N)))
    got = _product(T, K, N, x, w, "none", STREAM, fp32=False, residual=r, in_place=True)
    ref.check(got, *ref.linear64(x, w, "none", r))


@pytest.mark.parametrize("apart", [28, 31, 32, 39, 60, 120])
@pytest.mark.parametrize("top", [2.0 ** 100, 1.0, 2.0 ** -60])
def test_every_distance(apart, top):
    """Elements `apart` binary orders below the largest, all eight significant bits in use, down to subnormals."""
    T, K, N = 4, 192, 140
    rng = np.random.default_rng(64)
    w = ref.make_weights(rng, K, N)
    w["scales"][:, 0] = 0
    xf = (129 + 2 * rng.integers(0, 63, (T, K))) / 128 * rng.choice([-1.0, 1.0], (T, K)) * top * 2.0 ** -apart
    xf[:, 5] = top
    xf[1, 5] = 0                                   # a narrow row beside them
    x = ref.bf16_bits(xf)
    got, (want, bound) = _product(T, K, N, x, w, "none", STREAM), ref.linear64(x, w, "none", fp32=True)
    ref.check(got, want, bound + 2.0 ** -133)      # sums of a few subnormal steps


def test_nonfinite_row_beside_a_wide_one():
    T, K, N = 3, 192, 140
    x, w = _outlier_case(T, K, N, "none", 65)
    x[1, 7] = 0x7F80
    got = _product(T, K, N, x, w, "none", STREAM)
    with np.errstate(invalid="ignore"):
        want, bound = ref.linear64(x, w, "none", fp32=True)
    assert not np.isfinite(got[1]).any()
    ref.check(got[[0, 2]], want[[0, 2]], bound[[0, 2]])


@pytest.mark.parametrize("H,I,E,k,m,T", [(512, 256, 8, 2, 0, 1), (512, 256, 16, 4, 1, 5), (2048, 768, 32, 4, 0, 8), (512, 192, 12, 3, 2, 16)])
def test_layer_with_an_outlier_channel(oracle_mod, H, I, E, k, m, T):
    """A channel of x 2^40 times the others, which no expert's gate or up matrix reads."""
    shape, layer = _layer(H, I, E, k, m, seed=66)
    c = 7
    for p in ("",) + (("shared_",) if m else ()):
        for n in ("gate", "up"):
            layer[f"{p}{n}_scales"][..., c // 16] = 0
    layer["router_w"][:, c // 16 * 16:c // 16 * 16 + 16] = 0
    x = synth.make_x(shape, 66, T)
    x[::2, c] = ref.bf16_bits(np.full(1, 2.0 ** 40))[0]
    L = _handle(layer, shape, T, m)
    try:
        _check(oracle_mod, layer, shape, x, _run(L, x), m)
        narrow = synth.make_x(shape, 67, T)
        _check(oracle_mod, layer, shape, narrow, _run(L, narrow), m)
    finally:
        L.close()
