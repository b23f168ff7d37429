"""Long reductions, exactly: whatever the order of the sum, no term may be missing.

The bound for fp32 sums of K terms grows with K and passes the size of the result at tens of thousands of
terms. So here x is a small whole number, the scales are 1 and the multiplier is 1: every product is a multiple
of 1/2 of at most 12, every partial sum of up to 65536 of them one of at most 2^20 (21 bits), and fp32
holds all of them in any order. The output has to be equal.
"""
import numpy as np
import pytest

import linear_reference as ref

pytestmark = pytest.mark.gpu

STREAM, MMA = 0x1, 0x2


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_weight_only_route_b200 import build
    build.build()


@pytest.mark.parametrize("T,K,N,flags", [
    (1, 65536, 130, STREAM), (1, 65536, 130, MMA), (16, 65536, 130, 0), (16, 65536, 1, MMA), (40, 65536, 257, 0),
    (1, 16400, 700, STREAM), (3, 16400, 700, STREAM), (3, 16400, 700, MMA), (8, 11008, 4096, 0), (5, 11008, 4096, STREAM), (1, 14336, 4096, 0),
    (16, 4096, 11008, STREAM), (8, 11008, 4096, MMA), (200, 11008, 600, 0), (300, 14336, 1000, 0), (5, 4112, 40, STREAM),
])
def test_no_term_of_a_long_sum_is_lost(T, K, N, flags):
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    rng = np.random.default_rng(K + T)
    x = rng.integers(-2, 3, (T, K)).astype(np.float32)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    lin = tfmoe.Linear(K, N, max_tokens=T, out_fp32=True, flags=flags)
    try:
        lin.load_weights({"codes": torch.from_numpy(codes).cuda(), "scales": torch.full((N, K // 16), 0x38, dtype=torch.uint8, device="cuda"),
                          "global": torch.ones(1, device="cuda")})
        got = lin.forward(torch.from_numpy(x).to(torch.bfloat16).cuda())
        assert lin.sync_status() == 0, tfmoe.last_error()
        got = got.cpu().numpy()
    finally:
        lin.close()
    w = np.empty((N, K), np.float32)
    w[:, 0::2], w[:, 1::2] = ref.E2M1[codes & 15], ref.E2M1[codes >> 4]
    assert np.array_equal(got, x @ w.T)          # exact in fp32 as well, by the same argument
