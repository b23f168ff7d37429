"""The NVFP4 matrix product on the GPU (tfmoe_linear_*) against its 64-bit reference, within the
bound that linear_reference.py derives."""
import numpy as np
import pytest

import linear_reference as ref

pytestmark = pytest.mark.gpu

FORCE = {"auto": 0, "stream": 0x1, "mma": 0x2}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_weight_only_route_b200 import build
    build.build()


def _torch():
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    return torch, tfmoe


def _dev(a):
    import torch
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def _make(w, K, N, T, act="none", fp32=False, flags=0):
    _, tfmoe = _torch()
    lin = tfmoe.Linear(K, N, max_tokens=max(T, 1), activation=act, has_bias=w.get("bias") is not None, out_fp32=fp32,
                       flags=flags)
    lin.load_weights({k: None if v is None else _dev(v) for k, v in w.items()})
    return lin


def _bits(t):
    torch, _ = _torch()
    return t.cpu().numpy() if t.dtype == torch.float32 else t.view(torch.int16).cpu().numpy().view(np.uint16)


def _values(t):
    b = _bits(t)
    return b.astype(np.float64) if b.dtype == np.float32 else ref.bf16_to_f64(b)


def _case(T, K, N, act="none", bias=False, residual=False, fp32=False, flags=0, seed=0, x=None, w=None):
    torch, tfmoe = _torch()
    rng = np.random.default_rng(seed + 1000 * T + K + N)
    if w is None:
        w = ref.make_weights(rng, K, N, gated=act == "swiglu", bias=bias)
    if x is None:
        x = ref.bf16_bits(rng.standard_normal((T, K)))
    r = ref.bf16_bits(rng.standard_normal((T, N))) if residual else None
    lin = _make(w, K, N, T, act, fp32, flags)
    try:
        got = lin.forward(_dev(x), residual=None if r is None else _dev(r))
        assert lin.sync_status() == 0, tfmoe.last_error()
        assert lin.last_launch_count() >= 1
        got = _values(got)
    finally:
        lin.close()
    want, bound = ref.linear64(x, w, act, r, fp32)
    ref.check(got, want, bound)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("T,regime", [(3, "auto"), (16, "stream"), (5, "mma"), (40, "auto")])
def test_activations_bias_residual(act, T, regime):
    _case(T, 320, 200, act, bias=True, residual=True, flags=FORCE[regime])
    _case(T, 320, 200, act, bias=True, residual=True, fp32=True, flags=FORCE[regime])


@pytest.mark.parametrize("regime", ["stream", "mma"])
@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 128, 144, 208, 1024, 2688])
def test_reduction_lengths(K, regime):
    _case(2, K, 130, flags=FORCE[regime])
    _case(9, K, 70, "swiglu", fp32=True, flags=FORCE[regime])


@pytest.mark.parametrize("regime", ["stream", "mma"])
@pytest.mark.parametrize("N", [1, 2, 7, 63, 64, 127, 128, 129, 255, 1001])
def test_output_widths(N, regime):
    _case(3, 192, N, "silu", bias=True, residual=True, flags=FORCE[regime])
    _case(3, 192, N, "swiglu", bias=True, residual=True, flags=FORCE[regime])


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 255, 256, 257, 400, 513])
def test_token_counts(T):
    _case(T, 256, 264, residual=True)
    _case(T, 416, 136, "swiglu", bias=True, fp32=True)


@pytest.mark.parametrize("T", range(1, 17))
def test_every_small_batch_in_the_streaming_regime(T):
    _case(T, 704, 520, "none", fp32=True, flags=FORCE["stream"])


@pytest.mark.parametrize("T,K,N,act", [(1, 4096, 4096, "none"), (8, 2048, 2688, "swiglu"), (200, 4096, 2100, "none"),
                                       (700, 1536, 1300, "gelu"), (1300, 2048, 777, "swiglu")])
def test_larger_products(T, K, N, act):
    _case(T, K, N, act, residual=True)


def test_long_reduction_beyond_the_streaming_operands():
    """K = 65536: one row of x does not fit in shared memory sixteen times."""
    _case(16, 65536, 130, fp32=True)
    _case(1, 65536, 130, fp32=True)


def test_long_pieces_in_a_short_ring():
    """Row tiles of 64 column tiles, several per SM, with the ring of sixteen long token rows."""
    _case(16, 4096, 24000, fp32=True)


def test_wide_output_of_one_token():
    _case(1, 64, 40000, fp32=True)


@pytest.mark.parametrize("regime,T", [("stream", 4), ("mma", 4), ("auto", 70)])
def test_strided_rows_and_untouched_gaps(regime, T):
    """x, residual and out are columns of wider buffers; what lies between the rows stays as it was."""
    torch, tfmoe = _torch()
    K, N = 208, 150
    rng = np.random.default_rng(3)
    w = ref.make_weights(rng, K, N, bias=True)
    x, r = ref.bf16_bits(rng.standard_normal((T, K))), ref.bf16_bits(rng.standard_normal((T, N)))
    want, bound = ref.linear64(x, w, "silu", r)
    lin = _make(w, K, N, T, "silu", flags=FORCE[regime])
    try:
        xb = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
        xv = xb[:, 8:8 + K]
        xv.copy_(_dev(x).view(torch.bfloat16))
        rb = torch.full((T, N + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
        rv = rb[:, 1:1 + N]
        rv.copy_(_dev(r).view(torch.bfloat16))
        ob = torch.full((T + 2, N + 5), 7.0, dtype=torch.bfloat16, device="cuda")
        got = lin.forward(xv, residual=rv, out=ob[1:1 + T, 3:3 + N])
        assert lin.sync_status() == 0
        ref.check(_values(got.contiguous()), want, bound)
        keep = torch.ones_like(ob, dtype=torch.bool)
        keep[1:1 + T, 3:3 + N] = False
        assert bool((ob[keep] == 7.0).all())
        # x and out as columns of one buffer
        wide = torch.zeros((T, 512), dtype=torch.bfloat16, device="cuda")
        wide[:, :K].copy_(_dev(x).view(torch.bfloat16))
        got = lin.forward(wide[:, :K], residual=rv, out=wide[:, K:K + N])
        assert lin.sync_status() == 0
        ref.check(_values(got.contiguous()), want, bound)
    finally:
        lin.close()


@pytest.mark.parametrize("T", [2, 90])
def test_residual_in_place(T):
    torch, _ = _torch()
    K, N = 128, 129
    rng = np.random.default_rng(4)
    w = ref.make_weights(rng, K, N)
    x, r = ref.bf16_bits(rng.standard_normal((T, K))), ref.bf16_bits(rng.standard_normal((T, N)))
    lin = _make(w, K, N, T)
    try:
        buf = _dev(r).view(torch.bfloat16)
        got = lin.forward(_dev(x), residual=buf, out=buf)
        assert got.data_ptr() == buf.data_ptr() and lin.sync_status() == 0
        ref.check(_values(got), *ref.linear64(x, w, "none", r))
    finally:
        lin.close()


@pytest.mark.parametrize("regime,T", [("stream", 7), ("mma", 7), ("auto", 60)])
def test_extreme_values(regime, T):
    """Wide activations, smallest and largest scales, zero rows, zero weights."""
    rng = np.random.default_rng(6)
    K, N = 256, 96
    w = ref.make_weights(rng, K, N)
    w["scales"][:, 0] = 0x01          # the smallest E4M3 subnormal
    w["scales"][:, 1] = 0x7E          # 448
    w["scales"][:, 2] = 0x00
    w["scales"][5] = 0x00             # a row of zeros
    w["codes"][6] = 0x80              # +-0 codes
    xf = rng.standard_normal((T, K)) * np.exp2(rng.integers(-10, 11, (T, K)))
    xf[0] = 0
    xf[1, :16] *= 2.0 ** 12
    xf[2] *= 2.0 ** 60
    xf[3] *= 2.0 ** -60
    _case(T, K, N, fp32=True, flags=FORCE[regime], x=ref.bf16_bits(xf), w=w)


@pytest.mark.parametrize("regime,T", [("stream", 12), ("mma", 12), ("auto", 40)])
def test_nonfinite_rows_stay_in_their_rows(regime, T):
    torch, _ = _torch()
    K, N = 192, 140
    rng = np.random.default_rng(8)
    w = ref.make_weights(rng, K, N)
    x = ref.bf16_bits(rng.standard_normal((T, K)))
    want, bound = ref.linear64(x, w)
    xb = x.copy()
    xb[1, 7] = 0x7FC0                 # NaN
    xb[4, 100] = 0x7F80               # +inf
    lin = _make(w, K, N, T, flags=FORCE[regime])
    try:
        got = _values(lin.forward(_dev(xb)))
        assert lin.sync_status() == 0
    finally:
        lin.close()
    rows = [t for t in range(T) if t not in (1, 4)]
    ref.check(got[rows], want[rows], bound[rows])
    assert np.isnan(got[1]).all()
    # inf times a weight is an infinity of its sign, or NaN where the weight is zero
    wcol = ref.decode(w["codes"], w["scales"])[:, 100]
    assert np.isnan(got[4][wcol == 0]).all()
    assert np.array_equal(got[4][wcol != 0], np.sign(wcol[wcol != 0]) * np.inf)


@pytest.mark.parametrize("T,K,N", [(1, 2048, 700), (16, 512, 300), (50, 512, 300), (300, 1024, 260)])
def test_equal_calls_give_equal_bits_and_graph_replay(T, K, N):
    torch, tfmoe = _torch()
    rng = np.random.default_rng(9)
    w = ref.make_weights(rng, K, N, gated=True)
    lin = _make(w, K, N, T, "swiglu")
    try:
        xs = [_dev(ref.bf16_bits(rng.standard_normal((T, K)))) for _ in range(3)]
        want = [_bits(lin.forward(x)) for x in xs]
        x, out = xs[0].clone(), torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        lin.forward(x, out=out)
        torch.cuda.synchronize()
        graphs = []
        for _ in range(2):             # two graphs share the handle's workspace, replayed in turn
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                lin.forward(x, out=out)
                lin.forward(x, out=out)
            graphs.append(g)
        for i in (1, 2, 0, 2):
            x.copy_(xs[i])
            graphs[i % 2].replay()
            torch.cuda.synchronize()
            assert np.array_equal(_bits(out), want[i])
        assert np.array_equal(_bits(lin.forward(xs[1])), want[1])       # an eager call between replays
        assert lin.sync_status() == 0
    finally:
        lin.close()


def test_other_stream_and_many_handles():
    """Two handles on two streams at once, many calls each."""
    torch, _ = _torch()
    rng = np.random.default_rng(10)
    lins, xs, wants, outs, streams = [], [], [], [], []
    for K, N, T in ((1024, 600, 4), (512, 900, 40)):
        w = ref.make_weights(rng, K, N)
        x = ref.bf16_bits(rng.standard_normal((T, K)))
        lins.append(_make(w, K, N, T))
        xs.append(_dev(x))
        wants.append(ref.linear64(x, w))
        outs.append([torch.empty((T, N), dtype=torch.bfloat16, device="cuda") for _ in range(30)])
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for i in range(30):
        for j in range(2):
            lins[j].forward(xs[j], out=outs[j][i], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        ref.check(_values(outs[j][0]), *wants[j])
        assert all(torch.equal(o, outs[j][0]) for o in outs[j])
        assert lins[j].sync_status() == 0
        lins[j].close()


def test_reloaded_weights_are_used():
    rng = np.random.default_rng(11)
    K, N, T = 128, 64, 3
    x = ref.bf16_bits(rng.standard_normal((T, K)))
    w1, w2 = ref.make_weights(rng, K, N), ref.make_weights(rng, K, N)
    lin = _make(w1, K, N, T)
    try:
        ref.check(_values(lin.forward(_dev(x))), *ref.linear64(x, w1))
        lin.load_weights({k: None if v is None else _dev(v) for k, v in w2.items()})
        ref.check(_values(lin.forward(_dev(x))), *ref.linear64(x, w2))
    finally:
        lin.close()


def test_refusals():
    torch, tfmoe = _torch()
    K, N, T = 128, 40, 4
    rng = np.random.default_rng(12)
    lib = tfmoe.load_library()
    fresh = tfmoe.Linear(K, N, T)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    fwd = lambda h, *a: lib.tfmoe_linear_forward(h.handle, *a)
    assert fwd(fresh, x.data_ptr(), K, T, None, 0, o.data_ptr(), N, s) == tfmoe.ERR_NOT_LOADED
    w = ref.make_weights(rng, K, N)
    with pytest.raises(tfmoe.TfmoeError):
        fresh.load_weights({k: None if v is None or k == "scales" else _dev(v) for k, v in w.items()})
    fresh.close()
    gated = tfmoe.Linear(K, N, T, activation="swiglu")
    with pytest.raises(tfmoe.TfmoeError):
        gated.load_weights({k: None if v is None else _dev(v) for k, v in w.items()})     # no up matrix
    gated.close()
    biased = tfmoe.Linear(K, N, T, has_bias=True)
    with pytest.raises(tfmoe.TfmoeError):
        biased.load_weights({k: None if v is None else _dev(v) for k, v in w.items()})
    biased.close()
    lin = _make(w, K, N, T)
    xp, op = x.data_ptr(), o.data_ptr()
    bad = [(None, K, T, None, 0, op, N), (xp, K, T, None, 0, None, N), (xp, K, T + 1, None, 0, op, N),
           (xp, K, -1, None, 0, op, N), (xp, K - 8, T, None, 0, op, N), (xp, K, T, None, 0, op, N - 1),
           (xp, K, T, op, N - 1, op, N), (xp + 2, K, T, None, 0, op, N), (xp, K + 4, T, None, 0, op, N),
           (xp, K, T, None, 0, op + 1, N), (xp, K, T, op + 1, N, op, N), (xp, K, T, None, 0, xp, N),
           (xp, K, T, op + 2, N, op, N), (xp, K, T, op, N, op, N + 1), (xp, 1 << 41, T, None, 0, op, N)]
    for a in bad:
        assert fwd(lin, *a, s) == tfmoe.ERR_INVALID_ARG, a
        assert tfmoe.last_error()
    assert fwd(lin, None, K, 0, None, 0, None, N, s) == tfmoe.OK and lin.last_launch_count() == 0
    for bad_x, err in ((x[:, :64], ValueError), (x.float(), TypeError), (x.t(), ValueError), (x.cpu(), ValueError),
                       (x[0], ValueError)):
        with pytest.raises(err):
            lin.forward(bad_x)
    with pytest.raises(tfmoe.TfmoeError):
        lin.forward(x[:1].expand(T, K))                    # row stride 0
    with pytest.raises(ValueError):
        lin.forward(x, residual=o[:2])
    with pytest.raises(TypeError):
        lin.forward(x, out=torch.zeros((T, N), device="cuda"))
    assert lin.forward(x[:0]).shape == (0, N)
    assert lin.sync_status() == 0
    lin.close()
    forced = _make(w, K, N, 17, flags=FORCE["stream"])
    with pytest.raises(tfmoe.TfmoeError) as e:
        forced.forward(torch.zeros((17, K), dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == tfmoe.ERR_UNSUPPORTED
    forced.close()


@pytest.mark.parametrize("regime,T,ld", [("stream", 5, 1 << 29), ("mma", 5, 1 << 29), ("auto", 260, 1 << 23)])
def test_row_offsets_beyond_32_bits(regime, T, ld):
    """Rows so far apart that the last ones' element offsets pass 2^31."""
    torch, tfmoe = _torch()
    K, N = 96, 40
    rng = np.random.default_rng(T)
    w = ref.make_weights(rng, K, N, bias=True)
    xb, rb = ref.bf16_bits(rng.standard_normal((T, K))), ref.bf16_bits(rng.standard_normal((T, N)))
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x = torch.empty((T - 1) * ld + K, **bf).as_strided((T, K), (ld, 1))
    out = torch.empty((T - 1) * ld + N, **bf).as_strided((T, N), (ld, 1))
    x.copy_(_dev(xb).view(torch.bfloat16))
    out.copy_(_dev(rb).view(torch.bfloat16))          # the residual, updated in place
    assert (T - 1) * ld >= 1 << 31
    lin = _make(w, K, N, T, flags=FORCE[regime])
    try:
        lin.forward(x, residual=out, out=out)
        assert lin.sync_status() == 0, tfmoe.last_error()
        want, bound = ref.linear64(xb, w, "none", rb)
        ref.check(_values(out.contiguous()), want, bound)
    finally:
        lin.close()
