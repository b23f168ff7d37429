"""Linear.load_weights on real tensors: refusals leave the loaded weights alone."""
import numpy as np
import pytest

import linear_reference as ref

pytestmark = pytest.mark.gpu


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


def test_refused_weights_leave_the_loaded_ones():
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    rng = np.random.default_rng(41)
    K, N, T = 128, 96, 3
    w = ref.make_weights(rng, K, N, bias=True)
    x = ref.bf16_bits(rng.standard_normal((T, K)))
    d = {k: _dev(v) for k, v in w.items()}
    lin = tfmoe.Linear(K, N, max_tokens=T, has_bias=True, out_fp32=True)
    try:
        lin.load_weights({**d, "scales": d["scales"].view(torch.float8_e4m3fn)})
        bad = [(ValueError, {"codes": d["codes"].t()}), (ValueError, {"codes": d["codes"].cpu()}),
               (ValueError, {"codes": d["codes"][:-1]}), (ValueError, {"scales": d["scales"].t().contiguous()}),
               (TypeError, {"global": d["global"].double()}), (TypeError, {"bias": d["bias"].bfloat16()}),
               (ValueError, {"bias": d["bias"][:-1]}), (ValueError, {"codes": torch.cat([d["codes"]] * 2, 1)[:, :K // 2]})]
        for error, change in bad:
            with pytest.raises(error):
                lin.load_weights({**d, **change})
        with pytest.raises(tfmoe.TfmoeError):
            lin.load_weights({k: v for k, v in d.items() if k != "global"})
        got = lin.forward(_dev(x).view(torch.bfloat16))
        assert lin.sync_status() == 0
        ref.check(got.cpu().numpy(), *ref.linear64(x, w, fp32=True))
    finally:
        lin.close()
