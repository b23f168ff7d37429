"""The NVFP4 matrix product with its epilogue in 64 bits, and the bound its GPU result is held to.

Both in numpy from the formula of include/tfmoe.h; nothing here comes from the CUDA path.

The bound. Products are exact; the sums are fp32 in some order, so a sum of K terms is off by at
most (K - 1) u S, u = 2^-24 and S = |global| sum |x w| (the standard bound for any order). The multiplier,
the bias and the residual round once each (u of their magnitude). An activation f moves an error d
of its argument by at most L d, with L = max |f'|: relu 1, silu 1.1, gelu 1.13, gelu_tanh 1.13,
and its own evaluation is good to 16 u of max(|y|, |f|) (expf and erff within 2 units, five more
roundings, argument errors of 2 u |2z| under the exponential where |z| matters, i.e. below 16 in
magnitude). The result is rounded to the output type: u for fp32, 2^-9 relative at most half a
step of bf16, i.e. 2^-8 of the value.
The tensor cores add products in groups whose order and alignment are not specified; the bound
allows each addition two units in the last place (as the router's bound does): 4 u per term
instead of u.
"""
import math

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
U = 2.0 ** -24


def e4m3_table():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def decode(codes, scales):
    """[N][K] fp64 matrix without its multiplier."""
    codes = np.asarray(codes)
    w = np.empty((codes.shape[0], codes.shape[1] * 2))
    w[:, 0::2] = E2M1[codes & 15]
    w[:, 1::2] = E2M1[codes >> 4]
    return w * np.repeat(e4m3_table()[np.asarray(scales)], 16, axis=1)


def bf16_to_f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


_erf = np.vectorize(math.erf, otypes=[float])


def _sigmoid(y):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-y))


def act64(y, name):
    """(f(y), Lipschitz constant)"""
    if name == "relu":
        return np.maximum(y, 0), 1.0
    if name == "silu":
        return y * _sigmoid(y), 1.1
    if name == "gelu":
        return 0.5 * y * (1 + _erf(y / math.sqrt(2))), 1.13
    if name == "gelu_tanh":
        return 0.5 * y * (1 + np.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))), 1.13
    return y, 1.0


def linear64(x_bits, w, act="none", residual_bits=None, fp32=False):
    """(value, bound) of every output. w: numpy arrays of tfmoe_linear_weights."""
    x = bf16_to_f64(x_bits)
    K = x.shape[1]

    def product(prefix, bias):
        m = decode(w[prefix + "codes"], w[prefix + "scales"])
        g = float(w[prefix + "global"][0])
        y = x @ m.T * g
        S = np.abs(x) @ np.abs(m).T * abs(g)
        err = 4 * U * (K + 2) * S
        if bias is not None:
            y = y + bias
            err = err + U * np.abs(y)
        return y, err

    bias = None if w.get("bias") is None else np.asarray(w["bias"], np.float64)
    N = np.asarray(w["codes"]).shape[0]
    y, err = product("", None if bias is None else bias[:N])
    if act == "swiglu":
        u, uerr = product("up_", None if bias is None else bias[N:])
        f, lip = act64(y, "silu")
        ferr = lip * err + 16 * U * np.maximum(np.abs(y), np.abs(f))
        y = f * u
        err = ferr * np.abs(u) + np.abs(f) * uerr + ferr * uerr + U * np.abs(y)
    else:
        f, lip = act64(y, act)
        err = lip * err + (0 if act in ("none", "relu") else 16 * U * np.maximum(np.abs(y), np.abs(f)))
        y = f
    if residual_bits is not None:
        y = y + bf16_to_f64(residual_bits)
        err = err + U * np.abs(y)
    half = 2.0 ** -24 if fp32 else 2.0 ** -8
    return y, err + half * (np.abs(y) + err) + 2.0 ** -130


def check(got, want, bound):
    err = np.abs(np.asarray(got, np.float64) - want)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} outputs outside the bound, first at "
                           f"{np.argwhere(bad)[0].tolist()}, worst err/bound {float(np.nanmax(err / bound)):.3f}")


def make_weights(rng, K, N, gated=False, bias=False, spread=6.0):
    """Random weights; block scales 2^U[-4, spread - 4]."""
    import torch
    w = {}
    for p in ("", "up_") if gated else ("",):
        w[p + "codes"] = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
        s = torch.from_numpy(np.exp2(rng.random((N, K // 16)) * spread - 4).astype(np.float32))
        w[p + "scales"] = s.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        w[p + "global"] = np.array([(0.5 + rng.random()) / math.sqrt(K)], np.float32)
    w["bias"] = rng.standard_normal(2 * N if gated else N).astype(np.float32) if bias else None
    return w


def bf16_bits(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
