"""The whole layer for a few tokens in one kernel (tfmoe_forward_decode) against the fp64 oracle.

Routing must match the oracle's bit for bit. The output is held to a bound derived from the
arithmetic rather than to the layer's general tolerance. With u = 2^-24 and the tensor core's
additions allowed two units each (4 u per term, as in linear_reference.py):

  G, U   off by at most 4 u (H + 2) S with S = |global| sum |x w|; x is exact in the kernel's operand
         unless it is more than 2^28 below its row's largest
  a      = silu(G) U: |silu'| <= 1.1, its evaluation (approximate exponential and reciprocal) good to
         32 u of max(|G|, |silu|), then rounded to 11 bits (2^-12 of the value, and 2^-39 of the row's
         largest where it would fall below the operand's normal range)
  y      the sums of a wd: error sum |da| |wd|, plus 4 u (I + 2) sum |a wd|
  out    the weights g within 2e-6 (the routing tests' bound), at most k + m + 1 additions, one
         rounding to bf16 (2^-8 of the value)

The 64-bit evaluation here keeps a unrounded: it is the unrounded layer. The oracle's own output
rounds a to bf16 and is checked with the layer's tolerance.
"""
import numpy as np
import pytest

import linear_reference as ref
from gpu_harness import bf16_to_f64, check_output
from nvfp4_weight_only_route_b200 import synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_weight_only_route_b200 import build
    build.build()


def _mods():
    import torch
    from nvfp4_weight_only_route_b200 import tfmoe
    return torch, tfmoe


def _layer(H, I, E, k, m=0, seed=0, zipf=False, shared_globals=(0.02, 0.03, 0.015)):
    shape = synth.custom_shape(H, I, E, k, global_scale=0.02, router_std=1.0, zipf_s=1.1 if zipf else None)
    layer = synth.make_layer(shape, seed)
    if m:
        layer.update(synth.make_shared(shape, seed, m * I))
        for name, v in zip(("gate", "up", "down"), shared_globals):
            layer[f"shared_{name}_global"] = np.full(1, v, np.float32)
    return shape, layer


def _handle(layer, shape, T, m=0, flags=0, eps=1e-6):
    _, tfmoe = _mods()
    L = tfmoe.MoELayer(shape.H, shape.I, shape.E, shape.k, T, has_router_bias=layer.get("router_bias") is not None,
                       flags=flags, shared_intermediate=m * shape.I, norm_eps=eps)
    L.load_weights(tfmoe.layer_to_device(layer))
    return L


def _dev(a):
    torch, _ = _mods()
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()


def _bits(t):
    torch, _ = _mods()
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _run(L, x, residual=None, norm_w=None, out=None):
    torch, tfmoe = _mods()
    T, kx = x.shape[0], L.desc.top_k + (L.desc.shared_intermediate // L.desc.intermediate)
    out, on = L.forward_decode(_dev(x), residual=_dev(residual), norm_w=_dev(norm_w), out=out)
    assert L.sync_status() == 0, tfmoe.last_error()
    assert L.last_launch_count() == 1
    return {"out": _bits(out), "out_norm": None if on is None else _bits(on),
            "ids": L.buffer_tensor(tfmoe.BUF_TOPK_IDS, torch.int32, (T, kx)).cpu().numpy(),
            "g": L.buffer_tensor(tfmoe.BUF_TOPK_WEIGHTS, torch.float32, (T, kx)).cpu().numpy(),
            "logits": L.buffer_tensor(tfmoe.BUF_LOGITS, torch.float32, (T, L.desc.num_experts)).cpu().numpy()}


def _ffn64(layer, x, prefix, e):
    """(y, bound) of one expert for the rows x, a unrounded."""
    pick = (lambda n: layer[prefix + n]) if e is None else (lambda n: layer[prefix + n][e])
    one = lambda n: float(layer[prefix + n][0 if e is None else e])
    H, I = x.shape[1], pick("gate_codes").shape[0]

    def product(name):
        w = ref.decode(pick(name + "_codes"), pick(name + "_scales"))
        g = one(name + "_global")
        return x @ w.T * g, 4 * U * (H + 2) * (np.abs(x) @ np.abs(w).T * abs(g))

    (G, dG), (Up, dU) = product("gate"), product("up")
    with np.errstate(over="ignore"):
        f = G / (1 + np.exp(-G))
    df = 1.1 * dG + 32 * U * np.maximum(np.abs(G), np.abs(f))
    a = f * Up
    da = df * np.abs(Up) + np.abs(f) * dU + df * dU + U * np.abs(a)
    da = da + 2.0 ** -12 * (np.abs(a) + da) + 2.0 ** -39 * np.max(np.abs(a) + da, axis=1, keepdims=True)
    wd = np.abs(ref.decode(pick("down_codes"), pick("down_scales")))
    y = a @ ref.decode(pick("down_codes"), pick("down_scales")).T * one("down_global")
    g = abs(one("down_global"))
    return y, da @ wd.T * g + 4 * U * (I + 2) * ((np.abs(a) + da) @ wd.T * g), (np.abs(a) + da) @ wd.T * g


def _layer64(layer, x_bits, ids, g, m, residual):
    """(out, bound) of the unrounded layer for a given routing."""
    x = bf16_to_f64(x_bits)
    T, k = ids.shape[0], ids.shape[1] - m
    out, err = np.zeros_like(x), np.zeros_like(x)
    for e in np.unique(ids[:, :k]):
        t, s = np.nonzero(ids[:, :k] == e)
        y, dy, mag = _ffn64(layer, x[t], "", int(e))
        w = g[t, s].astype(np.float64)[:, None]
        np.add.at(out, t, w * y)
        np.add.at(err, t, w * dy + 2e-6 * mag + 16 * U * w * mag)
    if m:
        y, dy, mag = _ffn64(layer, x, "shared_", None)
        out += y
        err += dy + 16 * U * mag
    if residual is not None:
        out += bf16_to_f64(residual)
    err += (k + m + 2) * U * (np.abs(out) + err)
    return out, err + 2.0 ** -8 * (np.abs(out) + err) + 2.0 ** -130


def _check(oracle_mod, layer, shape, x, got, m=0, residual=None, norm_w=None, eps=1e-6, oracle_out=True):
    T, k, E = x.shape[0], shape.k, shape.E
    o = oracle_mod.forward(layer, x, top_k=k, intermediates=True, residual=residual, norm_w=norm_w, eps=eps)
    assert np.array_equal(got["ids"][:, :k], o["ids"])
    assert np.array_equal(got["ids"][:, k:], np.tile(E + np.arange(m), (T, 1)))
    assert np.array_equal(got["logits"], o["logits"])
    assert np.max(np.abs(got["g"][:, :k] - o["g"])) <= 2e-6 and np.all(got["g"][:, k:] == 1.0)
    # the oracle's weights are the reference: the bound allows 2e-6 for the kernel's
    g = np.concatenate([o["g"], np.ones((T, m))], axis=1)
    want, bound = _layer64(layer, x, got["ids"], g, m, residual)
    ref.check(bf16_to_f64(got["out"]), want, bound)
    if oracle_out:
        check_output(got["out"], o)
    if norm_w is not None:
        wn = oracle_mod.rms_norm(got["out"], norm_w, eps)
        assert np.mean(got["out_norm"] == wn) >= 0.9999
        gv, wv = bf16_to_f64(got["out_norm"]), bf16_to_f64(wn)
        assert np.all(np.abs(gv - wv) <= 2.0 ** -7 * np.abs(wv) + 1e-30)


@pytest.mark.parametrize("H,I,E,k,m,T", [
    (128, 64, 4, 1, 0, 1),        # one unit more than nothing: most CTAs have no work
    (128, 64, 1, 1, 0, 1),
    (128, 64, 4, 4, 0, 16),       # k == E, every token in every expert
    (256, 320, 5, 2, 0, 3),
    (384, 192, 6, 3, 2, 7),       # odd column tiles, a shared expert of two slots
    (384, 192, 6, 3, 0, 16),
    (512, 1024, 8, 2, 0, 4),
    (640, 448, 40, 10, 1, 11),
    (2048, 768, 128, 8, 0, 1),
    (2048, 768, 128, 8, 0, 8),
    (1024, 2688, 16, 4, 0, 5),
    (256, 64, 250, 26, 6, 16),    # 32 slots per token, 512 pairs
    (4096, 384, 56, 8, 0, 14),    # long row tiles, several per SM, in the short ring of long token rows
])
def test_shapes(oracle_mod, H, I, E, k, m, T):
    shape, layer = _layer(H, I, E, k, m, seed=70 + T)
    x = synth.make_x(shape, 70 + T, T)
    L = _handle(layer, shape, T, m)
    try:
        assert L.decode_max_tokens() == T
        _check(oracle_mod, layer, shape, x, _run(L, x), m)
    finally:
        L.close()


def test_long_rows_that_leave_a_short_ring(oracle_mod):
    """Up to 8 tokens of rows so long that the ring keeps 3 slots (the kernel for two tiles), and 4."""
    for T, H in ((8, 8704), (7, 8704), (8, 8192), (9, 8192)):
        shape, layer = _layer(H, 64, 3, 2, seed=T + H)
        x = synth.make_x(shape, T, T)
        L = _handle(layer, shape, T)
        try:
            assert L.decode_max_tokens() == T
            _check(oracle_mod, layer, shape, x, _run(L, x))
        finally:
            L.close()


@pytest.mark.parametrize("T", range(1, 17))
def test_every_batch_with_one_handle(oracle_mod, T):
    """A handle made for 16 tokens serves fewer."""
    shape, layer = _layer(512, 256, 24, 4, 1, seed=71, zipf=True)
    L = _handle(layer, shape, 16, 1)
    try:
        x = synth.make_x(shape, 71, T)
        _check(oracle_mod, layer, shape, x, _run(L, x), 1)
    finally:
        L.close()


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("in_place", [False, True])
def test_residual_and_norm(oracle_mod, T, in_place):
    shape, layer = _layer(1024, 320, 12, 3, 1, seed=72)
    x, res = synth.make_x(shape, 72, T), synth.make_residual(shape, 72, T)
    gam = synth.make_norm_weight(shape, 72)
    L = _handle(layer, shape, T, 1, eps=1e-5)
    torch, _ = _mods()
    try:
        if in_place:
            buf = _dev(res).view(torch.bfloat16)
            out, on = L.forward_decode(_dev(x), residual=buf, norm_w=_dev(gam), out=buf)
            assert L.sync_status() == 0 and out.data_ptr() == buf.data_ptr()
            got = _run(L, x, res, gam)
            assert np.array_equal(got["out"], _bits(out)) and np.array_equal(got["out_norm"], _bits(on))
        else:
            got = _run(L, x, res, gam)
            plain = _run(L, x, res)           # the same out without the norm
            assert plain["out_norm"] is None and np.array_equal(plain["out"], got["out"])
        _check(oracle_mod, layer, shape, x, got, 1, res, gam, 1e-5)
    finally:
        L.close()


def test_all_tokens_on_one_expert_and_ties(oracle_mod):
    """Equal router rows: every token takes the k lowest experts; 16 tokens fill both column tiles."""
    shape, layer = _layer(256, 128, 9, 2, 0, seed=73)
    layer["router_w"][:] = layer["router_w"][:1]
    x = synth.make_x(shape, 73, 16)
    L = _handle(layer, shape, 16)
    try:
        got = _run(L, x)
        assert np.array_equal(got["ids"], np.tile([0, 1], (16, 1)))
        _check(oracle_mod, layer, shape, x, got)
    finally:
        L.close()


def test_zero_rows_and_extreme_activations(oracle_mod):
    """A padded batch's zero rows, tiny and huge rows, subnormal inputs and weights."""
    shape, layer = _layer(256, 128, 16, 3, 0, seed=74)
    rng = np.random.default_rng(74)
    xf = rng.standard_normal((8, 256)).astype(np.float32)
    xf[1] = 0
    xf[2] *= np.float32(2.0 ** 20)
    xf[3] *= np.float32(2.0 ** -40)
    xf[4, ::3] *= np.float32(2.0 ** 12)
    xf[5, 7] = np.float32(2.0 ** -130)
    x = ref.bf16_bits(xf)
    layer["gate_scales"][:, :, 3] = 0x01
    layer["down_scales"][:, 5] = 0x00
    L = _handle(layer, shape, 8)
    try:
        got = _run(L, x)
        # (the general tolerance's 1e-3 makes no sense beside rows of 1e12; the derived bound does)
        _check(oracle_mod, layer, shape, x, got, oracle_out=False)
        assert np.all(bf16_to_f64(got["out"][1]) == 0)
    finally:
        L.close()


def test_router_exact_for_extreme_exponents(oracle_mod):
    """Products of router weights and activations beyond fp32's range in both directions."""
    shape, layer = _layer(256, 64, 12, 3, 0, seed=75)
    rng = np.random.default_rng(75)
    w = rng.standard_normal((12, 256)) * np.exp2(rng.integers(-70, 30, (12, 256)))
    layer["router_w"] = ref.bf16_bits(w)
    xf = rng.standard_normal((6, 256)) * np.exp2(rng.integers(-70, 30, (6, 256)))
    x = ref.bf16_bits(xf)
    L = _handle(layer, shape, 6)
    try:
        torch, tfmoe = _mods()
        L.forward_decode(_dev(x))
        assert L.sync_status() == 0
        o = oracle_mod.forward(layer, x, top_k=3, intermediates=True)
        ids = L.buffer_tensor(tfmoe.BUF_TOPK_IDS, torch.int32, (6, 3)).cpu().numpy()
        assert np.array_equal(L.buffer_tensor(tfmoe.BUF_LOGITS, torch.float32, (6, 12)).cpu().numpy(), o["logits"])
        assert np.array_equal(ids, o["ids"])
    finally:
        L.close()


def test_nonfinite_rows_stay_in_their_rows(oracle_mod):
    shape, layer = _layer(256, 128, 8, 2, 1, seed=76)
    x = synth.make_x(shape, 76, 10)
    L = _handle(layer, shape, 10, 1)
    try:
        good = _run(L, x)
        bad = x.copy()
        bad[2, 5] = 0x7FC0
        bad[7, 100] = 0x7F80
        got = _run(L, bad)
        rows = [t for t in range(10) if t not in (2, 7)]
        assert np.array_equal(got["ids"][rows], good["ids"][rows])
        want, bound = _layer64(layer, x, good["ids"], good["g"].astype(np.float64), 1, None)
        ref.check(bf16_to_f64(got["out"])[rows], want[rows], bound[rows])
        assert not np.isfinite(bf16_to_f64(got["out"][2])).any()
        assert not np.isfinite(bf16_to_f64(got["out"][7])).any()
    finally:
        L.close()


def test_same_routing_and_close_output_as_the_chain(oracle_mod):
    torch, tfmoe = _mods()
    s = synth.SHAPES[1]
    layer = synth.make_layer(s, 1)
    L = _handle(layer, s, 8)
    try:
        x = synth.make_x(s, 1, 8)
        chain = L.forward(_dev(x))
        assert L.sync_status() == 0
        ids = L.buffer_tensor(tfmoe.BUF_TOPK_IDS, torch.int32, (8, 8)).cpu().numpy()
        g = L.buffer_tensor(tfmoe.BUF_TOPK_WEIGHTS, torch.float32, (8, 8)).cpu().numpy()
        logits = L.buffer_tensor(tfmoe.BUF_LOGITS, torch.float32, (8, 128)).cpu().numpy()
        got = _run(L, x)
        assert np.array_equal(got["ids"], ids) and np.array_equal(got["g"], g) and np.array_equal(got["logits"], logits)
        # no stage of the chain can be replayed after it
        assert L.lib.tfmoe_forward_stage(L.handle, 7, _dev(x).data_ptr(), 8, chain.data_ptr(), None) == tfmoe.ERR_INVALID_ARG
        again = L.forward(_dev(x))
        assert L.sync_status() == 0 and np.array_equal(_bits(again), _bits(chain))
    finally:
        L.close()


@pytest.mark.parametrize("T,H,I,E,k", [(1, 2048, 768, 128, 8), (8, 512, 256, 32, 4), (16, 512, 256, 6, 3)])
def test_equal_calls_give_equal_bits_and_graph_replay(T, H, I, E, k):
    torch, tfmoe = _mods()
    shape, layer = _layer(H, I, E, k, 0, seed=77)
    L = _handle(layer, shape, T)
    try:
        xs = [_dev(synth.make_x(shape, 77, T, stream=i)) for i in range(3)]
        gam = _dev(synth.make_norm_weight(shape, 77))
        want = [tuple(_bits(v) for v in L.forward_decode(x, norm_w=gam)) for x in xs]
        x, out, on = xs[0].clone(), torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), \
            torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                L.forward_decode(x, norm_w=gam, out=out, out_norm=on)
                L.forward_decode(x, norm_w=gam, out=out, out_norm=on)
            graphs.append(g)
        for n in range(6):
            x.copy_(xs[n % 3])
            graphs[n % 2].replay()
            torch.cuda.synchronize()
            assert np.array_equal(_bits(out), want[n % 3][0]) and np.array_equal(_bits(on), want[n % 3][1])
        for n in range(200):                 # many calls back to back, with and without the norm
            L.forward_decode(xs[n % 3], norm_w=gam if n % 2 else None, out=out, out_norm=on if n % 2 else None)
        assert np.array_equal(_bits(out), want[199 % 3][0])
        assert L.sync_status() == 0
    finally:
        L.close()


def test_two_handles_on_two_streams():
    torch, tfmoe = _mods()
    hs, xs, outs, wants, streams = [], [], [], [], []
    for i in range(2):
        shape, layer = _layer(512, 256, 16, 4, 0, seed=78 + i)
        hs.append(_handle(layer, shape, 4))
        xs.append(_dev(synth.make_x(shape, 78, 4)))
        outs.append([torch.empty((4, 512), dtype=torch.bfloat16, device="cuda") for _ in range(20)])
        wants.append(_bits(hs[i].forward_decode(xs[i])[0]))
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for n in range(20):
        for i in range(2):
            hs[i].forward_decode(xs[i], out=outs[i][n], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(np.array_equal(_bits(o), wants[i]) for o in outs[i])
        assert hs[i].sync_status() == 0
        hs[i].close()


def test_timeout_is_reported_and_the_handle_recovers(oracle_mod):
    """One thread waits 1 ms on a barrier that nothing completes and takes the timeout path."""
    torch, tfmoe = _mods()
    shape, layer = _layer(256, 128, 8, 2, 0, seed=79)
    x = synth.make_x(shape, 79, 4)
    L = _handle(layer, shape, 4, flags=tfmoe.FLAG_TEST_TIMEOUT)
    try:
        L.forward_decode(_dev(x))
        assert L.sync_status() == tfmoe.ERR_TIMEOUT
        assert L.sync_status() == 0
    finally:
        L.close()
    L = _handle(layer, shape, 4)
    try:
        _check(oracle_mod, layer, shape, x, _run(L, x))
    finally:
        L.close()


def test_nonfinite_logit_sets_the_debug_word():
    _, tfmoe = _mods()
    shape, layer = _layer(256, 128, 8, 2, 0, seed=80)
    x = synth.make_x(shape, 80, 2)
    x[1, 3] = 0x7F80
    L = _handle(layer, shape, 2, flags=tfmoe.FLAG_DEBUG_CHECKS)
    try:
        L.forward_decode(_dev(x))
        assert L.sync_status() == tfmoe.ERR_DEVICE
        assert L.sync_status() == 0
    finally:
        L.close()


def test_refusals():
    torch, tfmoe = _mods()
    lib = tfmoe.load_library()
    shape, layer = _layer(512, 256, 8, 2, 0, seed=81)
    fresh = tfmoe.MoELayer(512, 256, 8, 2, 4)
    x = torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")
    o, n = torch.zeros_like(x), torch.zeros_like(x)
    s = torch.cuda.current_stream().cuda_stream
    call = lambda h, *a: lib.tfmoe_forward_decode(h.handle, *a, s)
    xp, op, np_ = x.data_ptr(), o.data_ptr(), n.data_ptr()
    assert call(fresh, xp, 4, None, None, op, None) == tfmoe.ERR_NOT_LOADED
    fresh.close()
    L = _handle(layer, shape, 40)
    assert L.decode_max_tokens() == 16
    for a in [(None, 4, None, None, op, None), (xp, 4, None, None, None, None), (xp, 41, None, None, op, None),
              (xp, -1, None, None, op, None), (xp + 2, 4, None, None, op, None), (xp, 4, None, None, xp, None),
              (xp, 4, op + 16, None, op, None), (xp, 4, None, np_, op, None), (xp, 4, None, np_, op, op),
              (xp, 4, None, xp, op, xp)]:
        assert call(L, *a) == tfmoe.ERR_INVALID_ARG, a
    big = torch.zeros((17, 512), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tfmoe.TfmoeError) as e:
        L.forward_decode(big)
    assert e.value.status == tfmoe.ERR_UNSUPPORTED
    assert call(L, None, 0, None, None, None, None) == tfmoe.OK and L.last_launch_count() == 0
    L.close()
    # rows too long for sixteen tokens: the limit says so and one token still runs
    wide = tfmoe.MoELayer(8192, 64, 2, 1, 16)
    lim = wide.decode_max_tokens()
    assert 1 <= lim < 16
    wide.close()


def test_the_binding_refuses_what_the_kernel_would_misread():
    """Strided, narrow, mistyped or misplaced tensors: an error, and nothing written."""
    torch, _ = _mods()
    shape, layer = _layer(512, 256, 8, 2, seed=95)
    L = _handle(layer, shape, 8)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, wide = torch.zeros((4, 512), **bf), torch.zeros((4, 1024), **bf)
    out = torch.full((4, 512), 7.0, **bf)
    try:
        for error, kw in ((ValueError, dict(x=wide[:, :512])), (ValueError, dict(x=wide)), (ValueError, dict(x=x, T=5)),
                          (TypeError, dict(x=x.half())), (ValueError, dict(x=x, residual=wide[:, ::2])),
                          (ValueError, dict(x=x, residual=x[:3].clone())), (ValueError, dict(x=x, norm_w=x[0, :256])),
                          (TypeError, dict(x=x, norm_w=x[0].float())), (ValueError, dict(x=x, residual=torch.zeros((4, 512), dtype=torch.bfloat16)))):
            with pytest.raises(error):
                L.forward_decode(out=out, **kw)
        with pytest.raises(ValueError):
            L.forward_decode(x, out=wide[:, :512])
        with pytest.raises(TypeError):
            L.forward_decode(x, out=torch.zeros((4, 512), device="cuda"))
        assert L.sync_status() == 0 and bool((out == 7.0).all()) and not wide.any()
        L.forward_decode(x, T=2, out=out)              # the first rows of a larger batch
        assert L.sync_status() == 0 and not out[:2].any() and bool((out[2:] == 7.0).all())
    finally:
        L.close()
