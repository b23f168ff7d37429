"""The operators of a decode step run together, as a model would: a mixture-of-experts layer (with
residual and RMS norm), a second block on its two outputs (dense feed-forward of two matrix products,
or another layer), and the fp32 logits of a vocabulary. Each is held to the 64-bit bound of its own
tests on the inputs that it really got; a captured graph of the whole step gives the eager bits."""
import numpy as np
import pytest

import linear_reference as ref
import test_gpu_decode as dec
from gpu_harness import bf16_to_f64
from nvfp4_weight_only_route_b200 import synth

pytestmark = pytest.mark.gpu

H, I, E, K, M, F, V = 512, 256, 32, 4, 1, 640, 1001


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_weight_only_route_b200 import build
    build.build()


def _dev(a):
    import torch
    return None if a is None else torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


class Step:
    """o projection (+ residual) -> MoE layer (+ residual, norm) -> dense block (+ residual) -> MoE layer
    (+ residual, norm) -> logits; `max_tokens` sizes every handle."""

    def __init__(self, max_tokens):
        import torch
        from nvfp4_weight_only_route_b200 import tfmoe
        rng = np.random.default_rng(5)
        self.w = {"o": ref.make_weights(rng, H, H, spread=4), "up": ref.make_weights(rng, H, F, gated=True, spread=4),
                  "down": ref.make_weights(rng, F, H, spread=4), "head": ref.make_weights(rng, H, V, bias=True)}
        self.lin = {n: tfmoe.Linear(k, m, max_tokens, activation=a, has_bias=n == "head", out_fp32=n == "head")
                    for n, k, m, a in (("o", H, H, "none"), ("up", H, F, "swiglu"), ("down", F, H, "none"), ("head", H, V, "none"))}
        for n, lin in self.lin.items():
            lin.load_weights({k: _dev(v) for k, v in self.w[n].items()})
        self.layers = [dec._layer(H, I, E, K, M, seed=s) for s in (81, 82)]
        self.moe = [dec._handle(layer, shape, max_tokens, M) for shape, layer in self.layers]
        self.gamma = [synth.make_norm_weight(shape, 83 + i) for i, (shape, _) in enumerate(self.layers)]
        self.g = [_dev(g) for g in self.gamma]
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.t = {n: torch.zeros((max_tokens, F if n == "f" else H), **bf) for n in ("h1", "h2", "x2", "f", "h3", "h4", "x4")}
        self.t["logits"] = torch.zeros((max_tokens, V), dtype=torch.float32, device="cuda")

    def run(self, attn, x, h, decode=True):
        """attn, x, h: [T, H] attention output, MoE input and residual stream."""
        T, t = x.shape[0], {n: v[:x.shape[0]] for n, v in self.t.items()}
        forward = [(m.forward_decode if decode else m.forward_add_norm) for m in self.moe]
        self.lin["o"].forward(attn, residual=h, out=t["h1"])
        forward[0](x, residual=t["h1"], norm_w=self.g[0], out=t["h2"], out_norm=t["x2"], T=T)
        self.lin["up"].forward(t["x2"], out=t["f"])
        self.lin["down"].forward(t["f"], residual=t["h2"], out=t["h3"])
        forward[1](t["x2"], residual=t["h3"], norm_w=self.g[1], out=t["h4"], out_norm=t["x4"], T=T)
        self.lin["head"].forward(t["x4"], out=t["logits"])
        return t

    def status(self):
        return [m.sync_status() for m in self.moe] + [lin.sync_status() for lin in self.lin.values()]

    def close(self):
        for m in [*self.moe, *self.lin.values()]:
            m.close()


def _inputs(T, seed):
    rng = np.random.default_rng(seed)
    return [ref.bf16_bits(rng.standard_normal((T, H))) for _ in range(3)]


@pytest.mark.parametrize("T", [1, 5, 16])
def test_a_decode_step(oracle_mod, T):
    from nvfp4_weight_only_route_b200 import tfmoe
    import torch
    step = Step(16)
    try:
        attn, x, h = _inputs(T, T)
        t = step.run(_dev(attn), _dev(x), _dev(h))
        assert step.status() == [0] * 6, tfmoe.last_error()
        b = {n: (v.cpu().numpy() if v.dtype == torch.float32 else dec._bits(v)) for n, v in t.items()}
        for name, src, res, out in (("o", attn, h, "h1"), ("up", b["x2"], None, "f"), ("down", b["f"], b["h2"], "h3"),
                                    ("head", b["x4"], None, "logits")):
            want, bound = ref.linear64(src, step.w[name], "swiglu" if name == "up" else "none", res, name == "head")
            ref.check(b[out].astype(np.float64) if name == "head" else bf16_to_f64(b[out]), want, bound)
        for i, (src, res, out, norm) in enumerate(((x, b["h1"], "h2", "x2"), (b["x2"], b["h3"], "h4", "x4"))):
            shape, layer = step.layers[i]
            L = step.moe[i]
            got = {"out": b[out], "out_norm": b[norm],
                   "ids": L.buffer_tensor(tfmoe.BUF_TOPK_IDS, torch.int32, (T, K + M)).cpu().numpy(),
                   "g": L.buffer_tensor(tfmoe.BUF_TOPK_WEIGHTS, torch.float32, (T, K + M)).cpu().numpy(),
                   "logits": L.buffer_tensor(tfmoe.BUF_LOGITS, torch.float32, (T, E)).cpu().numpy()}
            dec._check(oracle_mod, layer, shape, src, got, M, res, step.gamma[i])
        for n, v in step.t.items():                  # rows past the batch
            assert not v[T:].any(), n
    finally:
        step.close()


def test_graphs_of_several_batches_share_the_handles():
    """Graphs captured for different batch sizes over the same handles, replayed in turn on one stream
    with new inputs, give the eager step's bits; a prefill between them changes nothing."""
    import torch
    step = Step(40)
    try:
        stream = torch.cuda.Stream()
        graphs, static = {}, {}
        with torch.cuda.stream(stream):
            for T in (1, 3, 16):
                static[T] = [_dev(a) for a in _inputs(T, 0)]
                step.run(*static[T])
                stream.synchronize()
                graphs[T] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graphs[T], stream=stream):
                    step.run(*static[T])
            for seed in range(1, 4):
                for T in (16, 1, 3):
                    new = _inputs(T, 10 * seed + T)
                    want = {n: v.clone() for n, v in step.run(*[_dev(a) for a in new]).items()}
                    if seed == 2:
                        step.run(*[_dev(a) for a in _inputs(40, seed)], decode=False)
                    for s, a in zip(static[T], new):
                        s.copy_(_dev(a))
                    for v in step.t.values():
                        v.zero_()
                    graphs[T].replay()
                    stream.synchronize()
                    for n, v in want.items():
                        assert torch.equal(step.t[n][:T], v), (T, seed, n)
                        assert not step.t[n][T:].any(), (T, seed, n)
        assert step.status() == [0] * 6
    finally:
        stream.synchronize()
        graphs.clear()
        step.close()
