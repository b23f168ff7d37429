"""Cases and plain forms of two operators of the NVFP4 (W4A16) library.

moe     the whole mixture-of-experts FFN layer for a few tokens (routing, SwiGLU experts, an
        optional shared expert, weighted sum, residual add, RMS norm) in one call
linear  a matrix product with NVFP4 weights and bias, activation and residual in its epilogue

Where `own` is false, run() computes them with elementary torch operations in 32 bits (the
router's logits in 64: the experts are chosen by comparing them). Where it is true, run() calls
the library.

NVFP4: element c of a row is an E2M1 code, in the low nibble of byte c/2 when c is even; one E4M3
scale per 16 consecutive elements of a row; one fp32 multiplier per matrix (per expert in `moe`).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")


def _moe(name, T, H, I, E, k, shared=0, bias=False, residual=False, norm=False, zero_rows=0):
    # shared: slots of width I of the shared expert; zero_rows: rows of a padded batch
    return {"name": name, "op": "moe", "T": T, "H": H, "I": I, "E": E, "k": k, "shared": shared, "bias": bias,
            "residual": residual, "norm": norm, "zero_rows": zero_rows}


def _linear(name, T, K, N, act="none", bias=False, residual=False, fp32=False, pad=0):
    # pad: elements between the end of a row of x, residual and out and the next row (a slice of a wider buffer)
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "act": act, "bias": bias, "residual": residual,
            "fp32": fp32, "pad": pad}


def listed():
    return [
        # one token through the tiny layer: the smallest call, all latency
        _moe("moe_tiny_t1", 1, 512, 1024, 8, 2),
        # single-stream decode of the decode layer
        _moe("moe_decode_t1", 1, 2048, 768, 128, 8),
        # eight streams decoded together
        _moe("moe_decode_t8", 8, 2048, 768, 128, 8),
        # the same step as a transformer block ends with it: shared expert, residual stream, next norm
        _moe("moe_decode_t8_block", 8, 2048, 768, 128, 8, shared=1, residual=True, norm=True),
        # thirteen streams in a batch padded to fourteen, biased router, the prefill layer's sizes
        _moe("moe_wide_t14_padded", 14, 4096, 1536, 128, 8, bias=True, residual=True, zero_rows=1),
        # single-stream decode of the large sparse layer: 4.8 GB of weights, of which 150 MB are read
        _moe("moe_sweep_t1", 1, 4096, 2688, 256, 8),
        # a projection back into the residual stream, one token
        _linear("linear_t1_residual", 1, 2048, 4096, residual=True),
        # an output head over an odd vocabulary, fp32 logits for eight streams
        _linear("linear_t8_head", 8, 4096, 32001, fp32=True),
        # the first half of a dense FFN for a full decode batch
        _linear("linear_t16_swiglu", 16, 4096, 2688, act="swiglu"),
        # a short prompt through a biased GELU projection, rows of a wider buffer
        _linear("linear_t100_gelu", 100, 1536, 4096, act="gelu_tanh", bias=True, pad=64),
        # a ragged prompt, odd width, everything in the epilogue
        _linear("linear_t601_odd", 601, 2688, 1001, act="silu", bias=True, residual=True),
        # the long prompt through the first half of a dense FFN
        _linear("linear_t7234_swiglu", 7234, 4096, 2688, act="swiglu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    if rng.random() < 0.5:
        E = rng.randint(4, 256)
        case = _moe("", rng.randint(1, 16), 128 * _log_int(rng, 2, 32), 64 * _log_int(rng, 1, 42), E,
                    rng.randint(1, min(10, E)), shared=rng.choice([0, 0, 1]), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, norm=rng.random() < 0.5)
        case["zero_rows"] = rng.randint(0, case["T"] - 1) if rng.random() < 0.25 else 0
        if case["shared"] and case["E"] == 256:
            case["E"] = 255
    else:
        case = _linear("", _log_int(rng, 1, 8192), 16 * _log_int(rng, 4, 256), _log_int(rng, 1, 6000),
                       act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                       fp32=rng.random() < 0.25, pad=8 * rng.choice([0, 0, 0, 1, 5]))
        while work(case)["flops"] > most:
            case["T"] = max(1, case["T"] // 2)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _codes(g, *shape):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)


def _scales(g, *shape):
    return torch.exp2(torch.rand(shape, device="cuda", generator=g) * 6 - 4).to(torch.float8_e4m3fn).view(torch.uint8)


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def _padded(t, pad):
    """The values of t as rows of a buffer that is `pad` elements wider."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = case["T"]
    s = {"case": case}
    if case["op"] == "moe":
        H, I, E = case["H"], case["I"], case["E"]
        w = {"router_w": _normal(g, E, H),
             "router_bias": _normal(g, E, dtype=torch.float32) if case["bias"] else None}
        for name, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I)):
            w[name + "_codes"] = _codes(g, E, rows, cols // 2)
            w[name + "_scales"] = _scales(g, E, rows, cols // 16)
            # per-expert multipliers that keep G, U and the layer's output of order one
            w[name + "_global"] = (0.5 + torch.rand(E, device="cuda", generator=g)) * (0.3 / math.sqrt(cols))
        Is = case["shared"] * I
        if Is:
            for name, rows, cols in (("gate", Is, H), ("up", Is, H), ("down", H, Is)):
                w["shared_" + name + "_codes"] = _codes(g, rows, cols // 2)
                w["shared_" + name + "_scales"] = _scales(g, rows, cols // 16)
                w["shared_" + name + "_global"] = torch.full((1,), 0.3 / math.sqrt(cols), device="cuda")
        s["w"] = w
        s["x"] = _normal(g, T, H)
        if case["zero_rows"]:
            s["x"][T - case["zero_rows"]:] = 0
        s["residual"] = _normal(g, T, H) if case["residual"] else None
        s["norm_w"] = (0.5 + torch.rand(H, device="cuda", generator=g)).bfloat16() if case["norm"] else None
    else:
        K, N = case["K"], case["N"]
        gated = case["act"] == "swiglu"
        w = {}
        for p in ("", "up_") if gated else ("",):
            w[p + "codes"] = _codes(g, N, K // 2)
            w[p + "scales"] = _scales(g, N, K // 16)
            w[p + "global"] = torch.full((1,), 0.3 / math.sqrt(K), device="cuda") * (0.8 if p else 1.0)
        w["bias"] = _normal(g, 2 * N if gated else N, std=0.5, dtype=torch.float32) if case["bias"] else None
        s["w"] = w
        s["x"] = _padded(_normal(g, T, K), case["pad"])
        s["residual"] = _padded(_normal(g, T, N), case["pad"]) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    T = case["T"]
    if own:
        from nvfp4_weight_only_route_b200 import tfmoe
        w = s.pop("w")
        if case["op"] == "moe":
            layer = tfmoe.MoELayer(case["H"], case["I"], case["E"], case["k"], max_tokens=T,
                                   has_router_bias=case["bias"], shared_intermediate=case["shared"] * case["I"],
                                   norm_eps=EPS)
            s["out"] = torch.empty_like(s["x"])
            s["out_norm"] = torch.empty_like(s["x"]) if case["norm"] else None
        else:
            layer = tfmoe.Linear(case["K"], case["N"], max_tokens=T, activation=case["act"], has_bias=case["bias"],
                                 out_fp32=case["fp32"])
            dtype = torch.float32 if case["fp32"] else torch.bfloat16
            s["out"] = _padded(torch.empty((T, case["N"]), dtype=dtype, device="cuda"), case["pad"])
        layer.load_weights(w)
        s["layer"] = layer
    else:
        s["e2m1"] = torch.tensor(E2M1, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _decode(codes, scales, table):
    """The matrix (or stack of matrices) without its multiplier, in 32 bits."""
    nib = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    v = table[nib.int()]
    sc = scales.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (sc.shape[-1], 16)) * sc.unsqueeze(-1)).flatten(-2)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_moe(s):
    case, w, x, table = s["case"], s["w"], s["x"], s["e2m1"]
    logits = (x.double() @ w["router_w"].double().T).float()
    if w["router_bias"] is not None:
        logits = logits + w["router_bias"]
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :case["k"]], ids[:, :case["k"]]
    e = torch.exp(top - top[:, :1])
    g = e / e.sum(1, keepdim=True)
    xf = x.float()
    out = torch.zeros_like(xf)
    for j in range(case["k"]):
        i = ids[:, j]
        gu = [torch.bmm(_decode(w[n + "_codes"][i], w[n + "_scales"][i], table), xf.unsqueeze(2)).squeeze(2)
              * w[n + "_global"][i].unsqueeze(1) for n in ("gate", "up")]
        a = _silu(gu[0]) * gu[1]
        y = torch.bmm(_decode(w["down_codes"][i], w["down_scales"][i], table), a.unsqueeze(2)).squeeze(2)
        out += y * (w["down_global"][i] * g[:, j]).unsqueeze(1)
    if case["shared"]:
        gu = [xf @ _decode(w["shared_%s_codes" % n], w["shared_%s_scales" % n], table).T * w["shared_%s_global" % n]
              for n in ("gate", "up")]
        a = _silu(gu[0]) * gu[1]
        out += a @ _decode(w["shared_down_codes"], w["shared_down_scales"], table).T * w["shared_down_global"]
    if s["residual"] is not None:
        out += s["residual"].float()
    out = out.bfloat16()
    if s["norm_w"] is None:
        return out
    o = out.float()                              # the norm is that of the rounded residual stream
    r = torch.rsqrt((o * o).mean(1, keepdim=True) + EPS)
    return out, (o * r * s["norm_w"].float()).bfloat16()


def _plain_linear(s):
    case, w, x, table = s["case"], s["w"], s["x"], s["e2m1"]
    act, N = case["act"], case["N"]
    xf = x.float()
    y = xf @ _decode(w["codes"], w["scales"], table).T * w["global"]
    if w["bias"] is not None:
        y = y + w["bias"][:N]
    if act == "relu":
        y = torch.clamp(y, min=0)
    elif act == "silu":
        y = _silu(y)
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    elif act == "swiglu":
        u = xf @ _decode(w["up_codes"], w["up_scales"], table).T * w["up_global"]
        if w["bias"] is not None:
            u = u + w["bias"][N:]
        y = _silu(y) * u
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y if case["fp32"] else y.bfloat16()


def run(state):
    case = state["case"]
    if not own:
        return _plain_moe(state) if case["op"] == "moe" else _plain_linear(state)
    if case["op"] == "moe":
        out, out_norm = state["layer"].forward_decode(state["x"], residual=state["residual"], norm_w=state["norm_w"],
                                                      out=state["out"], out_norm=state["out_norm"])
        return out if out_norm is None else (out, out_norm)
    return state["layer"].forward(state["x"], residual=state["residual"], out=state["out"])


# ------------------------------------------------------------------ work

def work(case):
    T = case["T"]
    if case["op"] == "moe":
        H, I, E, k, m = case["H"], case["I"], case["E"], case["k"], case["shared"]
        # distinct experts of T tokens that choose k of E each at random (rows of zeros choose the first k)
        live = T - case["zero_rows"]
        active = E * (1 - (1 - k / E) ** live)
        if case["zero_rows"]:
            active += k * (1 - k / E) ** live
        rows = 2 + (1 if case["residual"] else 0) + (1 if case["norm"] else 0)
        return {"bytes": int((active + m) * 3 * H * I * 0.5625 + E * H * 2 + rows * T * H * 2),
                "flops": 2 * T * (E * H + (k + m) * 3 * H * I)}
    K, N = case["K"], case["N"]
    mats = 2 if case["act"] == "swiglu" else 1
    out = N * (4 if case["fp32"] else 2) + (N * 2 if case["residual"] else 0)
    return {"bytes": int(mats * N * K * 0.5625 + T * (K * 2 + out) + (mats * N * 4 if case["bias"] else 0)),
            "flops": 2 * T * mats * N * K}


# ------------------------------------------------------------------ exact values

def _value_of_e4m3():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(b & 128, -v, v)


def _matrix64(codes, scales):
    """A row-major NVFP4 matrix in 64 bits, without its multiplier."""
    dev = codes.device
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=dev) / 2
    out = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device=dev)
    for half in (0, 1):
        c = (codes >> (4 * half)) & 15
        v = mag[(c & 7).long()]
        out[:, half::2] = torch.where(c > 7, -v, v)
    sc = torch.from_numpy(_value_of_e4m3()).to(dev)[scales.long()]
    return out.mul_(sc.repeat_interleave(16, dim=1))


def _ffn64(x, w, prefix, e=None):
    pick = (lambda n: w[prefix + n]) if e is None else (lambda n: w[prefix + n][e])
    one = lambda n: float(w[prefix + n][0 if e is None else e])
    G = x @ _matrix64(pick("gate_codes"), pick("gate_scales")).T * one("gate_global")
    U = x @ _matrix64(pick("up_codes"), pick("up_scales")).T * one("up_global")
    a = G * torch.sigmoid(G) * U
    return a @ _matrix64(pick("down_codes"), pick("down_scales")).T * one("down_global")


def exact(case, seed):
    s = _inputs(case, seed)
    x, w = s["x"].double(), s["w"]
    if case["op"] == "moe":
        k = case["k"]
        l = (x @ w["router_w"].double().T).float()
        if w["router_bias"] is not None:
            l = l + w["router_bias"]
        l = l.cpu().numpy()
        out = torch.zeros_like(x)
        chosen = {}                              # expert -> [(token, weight)]
        for t in range(case["T"]):
            order = sorted(range(case["E"]), key=lambda e: (-float(l[t, e]), e))[:k]
            p = np.exp(l[t, order].astype(np.float64) - float(l[t, order[0]]))
            for e, g in zip(order, p / p.sum()):
                chosen.setdefault(e, []).append((t, float(g)))
        for e, pairs in chosen.items():
            rows = [t for t, _ in pairs]
            g = torch.tensor([g for _, g in pairs], dtype=torch.float64, device=x.device)
            out[rows] += _ffn64(x[rows], w, "", e) * g[:, None]
        if case["shared"]:
            out += _ffn64(x, w, "shared_")
        if s["residual"] is not None:
            out += s["residual"].double()
        if s["norm_w"] is None:
            return out
        o = out.bfloat16().double()
        norm = o / torch.sqrt((o ** 2).mean(1, keepdim=True) + EPS) * s["norm_w"].double()
        return out, norm
    act, N = case["act"], case["N"]
    y = x @ _matrix64(w["codes"], w["scales"]).T * float(w["global"])
    if w["bias"] is not None:
        y += w["bias"][:N].double()
    if act == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif act == "silu":
        y = y * torch.sigmoid(y)
    elif act == "gelu":
        y = y * torch.special.ndtr(y)
    elif act == "gelu_tanh":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    elif act == "swiglu":
        u = x @ _matrix64(w["up_codes"], w["up_scales"]).T * float(w["up_global"])
        if w["bias"] is not None:
            u += w["bias"][N:].double()
        y = y * torch.sigmoid(y) * u
    if s["residual"] is not None:
        y += s["residual"].double()
    return y
