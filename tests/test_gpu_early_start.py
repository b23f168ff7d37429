"""The product after a kernel that lets its successor start early and then runs on for longer than the kernels' limit
on a wait (2 s): the time before the product's own turn does not count."""
import ctypes

import numpy as np
import pytest

import linear_reference as ref

pytestmark = pytest.mark.gpu

STREAM, MMA = 0x1, 0x2
RUN_ON_NS = 2_600_000_000

SOURCE = r"""
extern "C" __global__ void run_on(unsigned long long ns) {
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    do {
        __nanosleep(1000);
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    } while (t - t0 < ns);
}
"""


@pytest.fixture(scope="module")
def run_on():
    """Launches one warp that triggers its dependents at once and ends RUN_ON_NS later."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from cuda.bindings import driver, nvrtc
    from nvfp4_weight_only_route_b200 import build
    build.build()
    torch.cuda.init()
    torch.zeros(1, device="cuda")

    def ok(r):
        assert int(r[0]) == 0, r[0]
        return r[1] if len(r) == 2 else r[1:]

    prog = ok(nvrtc.nvrtcCreateProgram(SOURCE.encode(), b"run_on.cu", 0, [], []))
    assert int(nvrtc.nvrtcCompileProgram(prog, 1, [b"--gpu-architecture=sm_100a"])[0]) == 0
    image = b" " * ok(nvrtc.nvrtcGetCUBINSize(prog))
    assert int(nvrtc.nvrtcGetCUBIN(prog, image)[0]) == 0
    module = ok(driver.cuModuleLoadData(image))
    kernel = ok(driver.cuModuleGetFunction(module, b"run_on"))

    def launch(stream):
        ns = ctypes.c_ulonglong(RUN_ON_NS)
        args = (ctypes.c_void_p * 1)(ctypes.addressof(ns))
        r = driver.cuLaunchKernel(kernel, 1, 1, 1, 32, 1, 1, 0, stream.cuda_stream, ctypes.addressof(args), 0)
        assert int(r[0]) == 0, r[0]

    yield launch
    torch.cuda.synchronize()
    driver.cuModuleUnload(module)


@pytest.mark.parametrize("T,K,N,flags", [(3, 2688, 4000, STREAM), (3, 2688, 200, MMA), (300, 1024, 9000, MMA)])
def test_the_time_of_the_kernel_before_does_not_count(run_on, T, K, N, flags):
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    rng = np.random.default_rng(95)
    w = ref.make_weights(rng, K, N)
    x = ref.bf16_bits(rng.standard_normal((T, K)))
    lin = tfmoe.Linear(K, N, max_tokens=T, out_fp32=True, flags=flags)
    try:
        lin.load_weights({k: torch.from_numpy(v).cuda() for k, v in w.items() if v is not None})
        xd, out = torch.from_numpy(x.view(np.int16)).cuda(), torch.empty((T, N), device="cuda")
        lin.forward(xd, out=out)                 # the kernel is loaded
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        run_on(s)
        lin.forward(xd, out=out.zero_(), stream=s)
        assert lin.sync_status(s) == 0, tfmoe.last_error()
        ref.check(out.double().cpu().numpy(), *ref.linear64(x, w, fp32=True))
    finally:
        lin.close()
