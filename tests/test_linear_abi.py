"""tfmoe_linear_*: struct layout and every refusal that needs no GPU; the 64-bit reference of the
GPU tests against a direct evaluation."""
import ctypes
import math
import os
import subprocess
import tempfile

import numpy as np
import pytest

import linear_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tf():
    from nvfp4_weight_only_route_b200 import build, tfmoe
    build.build()
    tfmoe.load_library()
    return tfmoe


def test_struct_layout_matches_header(tf):
    fields = [("tfmoe_linear_desc", tf.LinearDesc), ("tfmoe_linear_weights", tf.LinearWeights)]
    lines = []
    for c_name, py in fields:
        lines.append(f'printf("%zu\\n", sizeof({c_name}));')
        lines += [f'printf("%zu\\n", offsetof({c_name}, {n}));' for n, _ in py._fields_]
    acts = ["NONE", "RELU", "SILU", "GELU", "GELU_TANH", "SWIGLU"]
    lines += [f'printf("%d\\n", (int)TFMOE_ACT_{a});' for a in acts] + ['printf("%u\\n", TFMOE_FLAG_OUT_FP32);']
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"tfmoe.h\"\nint main(void) {\n" + "\n".join(lines) + "\nreturn 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        got = [int(v) for v in subprocess.check_output([exe]).split()]
    want = []
    for _, py in fields:
        want += [ctypes.sizeof(py)] + [getattr(py, n).offset for n, _ in py._fields_]
    want += [tf.ACTIVATIONS.index(a.lower()) for a in acts] + [tf.FLAG_OUT_FP32]
    assert got == want


def _create(tf, **kw):
    d = dict(in_features=512, out_features=256, max_tokens=4, activation=0, has_bias=0, flags=0)
    d.update(kw)
    h = ctypes.c_void_p()
    return tf.load_library().tfmoe_linear_create(ctypes.byref(tf.LinearDesc(**d)), ctypes.byref(h)), h


@pytest.mark.parametrize("kw,status", [
    (dict(in_features=0), 1), (dict(in_features=-16), 1), (dict(in_features=24), 1), (dict(out_features=0), 1),
    (dict(max_tokens=0), 1), (dict(activation=6), 1), (dict(activation=-1), 1), (dict(flags=3), 1),
    (dict(flags=0x4), 1), (dict(flags=0x20), 1), (dict(in_features=65536 + 16), 5), (dict(out_features=(1 << 20) + 1), 5),
    (dict(max_tokens=(1 << 20) + 1), 5),
])
def test_create_rejects_bad_descriptors(tf, kw, status):
    st, h = _create(tf, **kw)
    assert st == status and not h.value and tf.last_error()


def test_null_arguments_and_injected_failure(tf, monkeypatch):
    lib = tf.load_library()
    h = ctypes.c_void_p()
    assert lib.tfmoe_linear_create(None, ctypes.byref(h)) == tf.ERR_INVALID_ARG
    assert lib.tfmoe_linear_create(ctypes.byref(tf.LinearDesc(512, 256, 4, 0, 0, 0)), None) == tf.ERR_INVALID_ARG
    assert lib.tfmoe_linear_load_weights(None, None) == tf.ERR_INVALID_ARG
    assert lib.tfmoe_linear_forward(None, None, 0, 1, None, 0, None, 0, None) == tf.ERR_INVALID_ARG
    assert lib.tfmoe_linear_sync_status(None, None) == tf.ERR_INVALID_ARG
    assert lib.tfmoe_linear_last_launch_count(None) == 0
    lib.tfmoe_linear_destroy(None)
    monkeypatch.setenv("TFMOE_FAIL_ALLOC", "1")
    st, h = _create(tf)
    assert st == tf.ERR_OOM and not h.value and "injected" in tf.last_error()


def test_unknown_activation_name(tf):
    with pytest.raises(ValueError):
        tf.Linear(64, 64, 1, activation="swish")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
def test_reference_against_direct_sums(act):
    """linear64 on a small case against scalar loops over the codes."""
    rng = np.random.default_rng(5)
    T, K, N = 2, 48, 3
    w = ref.make_weights(rng, K, N, gated=act == "swiglu", bias=True)
    x = ref.bf16_bits(rng.standard_normal((T, K)))
    r = ref.bf16_bits(rng.standard_normal((T, N)))
    got, bound = ref.linear64(x, w, act, r)
    xv, rv = ref.bf16_to_f64(x), ref.bf16_to_f64(r)

    def one(prefix, t, n, b):
        s = 0.0
        for k in range(K):
            byte = int(w[prefix + "codes"][n, k // 2])
            nib = byte >> 4 if k & 1 else byte & 15
            exp, man = (nib >> 1) & 3, nib & 1
            v = man * 0.5 if exp == 0 else (1 + man * 0.5) * 2.0 ** (exp - 1)
            sb = int(w[prefix + "scales"][n, k // 16])
            se, sm = (sb >> 3) & 15, sb & 7
            sv = sm * 2.0 ** -9 if se == 0 else (1 + sm / 8) * 2.0 ** (se - 7)
            s += float(xv[t, k]) * (-v if nib & 8 else v) * sv
        return s * float(w[prefix + "global"][0]) + float(b)

    for t in range(T):
        for n in range(N):
            y = one("", t, n, w["bias"][n])
            z = {"none": lambda: y, "relu": lambda: max(y, 0.0), "silu": lambda: y / (1 + math.exp(-y)),
                 "gelu": lambda: y * 0.5 * math.erfc(-y / math.sqrt(2)),
                 "gelu_tanh": lambda: y / (1 + math.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))),
                 "swiglu": lambda: y / (1 + math.exp(-y)) * one("up_", t, n, w["bias"][N + n])}[act]()
            assert abs(got[t, n] - (z + rv[t, n])) <= 1e-12 * (1 + abs(z))
    assert np.all(bound > 0)
