"""Exact GELU in its negative tail, where y (1 + erf(y / sqrt 2)) / 2 cancels if it is summed as written.

x = 0 makes the argument the bias itself, exactly. With u = 2^-24 and f = y Phi(y): the tail Phi(-|y|) is a product
of an exponential (4 u, its argument's rounding put back), a reciprocal (2 u, and as much again through the
polynomial's argument), the polynomial (a fit within u, six roundings of its larger terms) and two more roundings;
1 - tail has no more of an error than the tail, and the last product rounds once: 20 u of |f| in all, and
2^-149 (2 |y| + 1) where the exponential or the tail is subnormal. For a bf16 output the polynomial is a
coarser fit (2^-16.9, 140 u) and the exponential the approximate one, whose argument is off by 2 u y^2: u (2 y^2 + 164).
The streaming regime always takes the finer form. Then the output's rounding, u or 2^-8 of the value.
"""
import math

import numpy as np
import pytest

import linear_reference as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_weight_only_route_b200 import build
    build.build()


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("T,flags", [(3, 0x1), (16, 0x1), (3, 0x2), (70, 0)])
def test_gelu_keeps_its_precision_for_negative_arguments(T, flags, fp32):
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    K, N = 512, 700
    rng = np.random.default_rng(51)
    w = ref.make_weights(rng, K, N)
    y = np.linspace(-13.5, 8.0, N).astype(np.float32)
    y[:4] = [0.0, -0.0, -1e-30, -5.5]
    lin = tfmoe.Linear(K, N, max_tokens=T, activation="gelu", has_bias=True, out_fp32=fp32, flags=flags)
    try:
        lin.load_weights({**{k: torch.from_numpy(v).cuda() for k, v in w.items() if v is not None}, "bias": torch.from_numpy(y).cuda()})
        got = lin.forward(torch.zeros((T, K), dtype=torch.bfloat16, device="cuda"))
        assert lin.sync_status() == 0
        got = got.double().cpu().numpy()
    finally:
        lin.close()
    y = y.astype(np.float64)
    f = np.array([0.5 * v * math.erfc(-v / math.sqrt(2)) for v in y])
    err = np.abs(f) * U * (20 if fp32 or flags == 0x1 else 2 * y * y + 164) + 2.0 ** -149 * (2 * np.abs(y) + 1)
    # the output's own rounding: half a step of the value, or of the smallest subnormal
    err += (U if fp32 else 2.0 ** -8) * (np.abs(f) + err) + (2.0 ** -150 if fp32 else 2.0 ** -134)
    ref.check(got, np.tile(f, (T, 1)), np.tile(err, (T, 1)))


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("flags", [0x1, 0x2])
def test_gelu_at_the_ends_of_its_range(flags, fp32):
    """Infinities as y Phi(y) in IEEE arithmetic gives them (-inf times 0 is NaN), NaN, and values whose square overflows."""
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    K, y = 64, np.array([np.inf, -np.inf, np.nan, 3e38, -3e38, 1e20, -1e20, 100.0, -100.0, -0.0], np.float32)
    w = ref.make_weights(np.random.default_rng(52), K, len(y))
    lin = tfmoe.Linear(K, len(y), max_tokens=2, activation="gelu", has_bias=True, out_fp32=fp32, flags=flags)
    try:
        lin.load_weights({**{k: torch.from_numpy(v).cuda() for k, v in w.items() if v is not None}, "bias": torch.from_numpy(y).cuda()})
        got = lin.forward(torch.zeros((2, K), dtype=torch.bfloat16, device="cuda"))
        assert lin.sync_status() == 0
        want = torch.tensor([np.inf, np.nan, np.nan, 3e38, 0, 1e20, 0, 100, 0, 0], dtype=torch.float32).to(got.dtype)
        assert torch.equal(got.cpu().nan_to_num(nan=7.0, posinf=8.0), want.nan_to_num(nan=7.0, posinf=8.0).expand(2, -1))
    finally:
        lin.close()
