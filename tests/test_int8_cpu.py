"""8-bit activations without a GPU: hand-worked pins of the oracle's functions, and the entry
points' refusals (checked on the host before any HIP call)."""
import ctypes
import os

import numpy as np
import pytest

import oracle as O
from conftest import ROOT

LIB = os.path.join(ROOT, "post_weight_quantization_27_amd", "libpwq.so")


# ------------------------------------------------------------------ oracle
def test_token_codes_by_hand():
    # scale 2: quotients 127, 0.5, 1.5, -2.5 (ties to even: 0, 2, -2), 3.49 -> 3
    X = np.array([[254.0, 1.0, 3.0, -5.0, 6.98]], dtype=np.float32)
    q, s, n = O.quantize_tokens(X)
    assert s[0] == 2.0 and q.tolist() == [[127, 0, 2, -2, 3]] and n[0] == 130


def test_token_codes_of_special_rows():
    X = np.zeros((5, 4), dtype=np.float32)
    X[1, 2] = np.nan
    X[2, 0] = -np.inf
    X[3, 1] = 126.0 * 2.0 ** -120           # scale below 2^-120: counts as 0
    X[4, 1] = -127.0 * 2.0 ** -120          # scale 2^-120 exactly
    q, s, n = O.quantize_tokens(X)
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] == 0 and s[4] == np.float32(2.0 ** -120)
    assert not q[:4].any() and q[4].tolist() == [0, -127, 0, 0] and n.tolist() == [0, 0, 0, 0, -127]


def test_channel_scale_divides():
    X = np.array([[8.0, 2.0]], dtype=np.float32)
    q, s, _ = O.quantize_tokens(X, np.array([4.0, 0.5], dtype=np.float32))      # 2, 4
    assert s[0] == np.float32(4.0 / 127.0) and q.tolist() == [[64, 127]]        # 2 / s = 63.5 (ties to even)


def test_rms_norm_by_hand():
    h = np.array([[3.0, 4.0]])
    y = O.rms_norm(h, np.array([2.0, 1.0]), 0.0)                                # rms = sqrt(12.5)
    assert np.allclose(y, [[6.0 / np.sqrt(12.5), 4.0 / np.sqrt(12.5)]], rtol=1e-15)
    q, s, n = O.rms_norm_quantize(h, np.array([2.0, 1.0]), 0.0)
    assert q.tolist() == [[127, 85]] and n[0] == 212 and s[0] == np.float32(6.0 / np.sqrt(12.5) / 127.0)


def test_int8_product_by_hand():
    X = np.array([[1, -2, 3], [0, 0, 0]], dtype=np.int8)
    C = np.array([[4, 5, 6], [-128, 127, 1]], dtype=np.int8)
    sx, sw = np.array([0.5, np.nan], dtype=np.float32), np.array([2.0, 0.25], dtype=np.float16)
    Y = O.quantized_matmul_int8(X, sx, C, sw)
    assert Y[0].tolist() == [12.0, -379 * 0.125] and np.isnan(Y[1]).all()
    Z = O.quantized_matmul_int8(X, sx, np.array([[4, 5, 6], [255, 0, 1]], dtype=np.uint8), sw,
                                zeros=np.array([[5], [255]]))
    assert Z[0].tolist() == [-1 + 0 + 3, (0 + 510 - 762) * 0.125]


def test_int8_product_is_the_dequantized_product():
    rng = np.random.default_rng(5)
    W = rng.standard_normal((9, 40)).astype(np.float32)
    X = rng.standard_normal((6, 40)).astype(np.float32)
    q, s, n = O.quantize_tokens(X)
    for sym in (True, False):
        r = O.rtn(W, 8, 0, sym=sym)
        z = None if sym else r["zeros"]
        What = O.dequant(r["codes"], r["scales"], 0, zeros=z)
        want = (q * s.astype(np.float64)[:, None]) @ What.T
        got = O.quantized_matmul_int8(q, s, r["codes"], r["scales"], zeros=z)
        assert np.allclose(got, want, rtol=1e-12, atol=1e-14)
        # and near the product of what was quantized: half a step per factor
        assert np.max(np.abs(got - X @ W.T)) < 0.5


# ------------------------------------------------------------------ refusals
FAKE = ctypes.c_void_p(0x1000)      # aligned, never dereferenced: every call below is rejected first
ODD = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def P():
    if not os.path.exists(LIB):
        pytest.skip("libpwq.so not built")
    from post_weight_quantization_27_amd import pwq
    pwq.lib()
    return pwq


def _call(f, names, ok):
    def with_(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)
    return with_


def test_quantize_tokens_rejects(P):
    c = _call(P.lib().pwq_quantize_tokens, ["X", "xt", "T", "d", "ldx", "chan", "q", "ldq", "s", "sums", "stream"],
              [FAKE, P.PWQ_F16, 4, 256, 256, None, FAKE, 256, FAKE, None, None])
    assert c(xt=3) == P.PWQ_EDTYPE and c(xt=-1) == P.PWQ_EDTYPE
    for kw in ({"T": -1}, {"d": 0}, {"d": -4}, {"d": 65536, "ldx": 65536, "ldq": 65536}, {"ldx": 255}, {"ldq": 255},
               {"ldx": (1 << 30) + 1}, {"X": None}, {"q": None}, {"s": None}, {"X": ODD}, {"s": ODD}, {"sums": ODD},
               {"chan": ODD}):
        assert c(**kw) == P.PWQ_EINVAL, kw
    assert c(T=0, X=None, q=None, s=None) == P.PWQ_OK


def test_rms_norm_quantize_rejects(P):
    names = ["X", "xt", "T", "d", "ldx", "r", "ldr", "g", "gt", "eps", "h", "ldh", "q", "ldq", "s", "sums", "Y", "yt",
             "ldy", "stream"]
    c = _call(P.lib().pwq_rms_norm_quantize, names,
              [FAKE, P.PWQ_BF16, 4, 256, 256, FAKE, 256, FAKE, P.PWQ_F32, 1e-5, FAKE, 256, FAKE, 256, FAKE, FAKE, FAKE,
               P.PWQ_F16, 256, None])
    assert c(xt=7) == P.PWQ_EDTYPE and c(gt=7) == P.PWQ_EDTYPE and c(yt=7) == P.PWQ_EDTYPE
    for kw in ({"T": -1}, {"d": 0}, {"d": 65536, "ldx": 65536, "ldr": 65536, "ldh": 65536, "ldq": 65536, "ldy": 65536},
               {"ldx": 255}, {"ldr": 255}, {"ldh": 255}, {"ldq": 255}, {"ldy": 255}, {"eps": -1e-9},
               {"eps": float("nan")}, {"eps": float("inf")}, {"X": None}, {"q": None}, {"s": None},
               {"q": None, "s": None}, {"q": None, "s": None, "sums": None, "Y": None}, {"r": None}, {"X": ODD},
               {"r": ODD}, {"h": ODD}, {"g": ODD}, {"s": ODD}, {"sums": ODD}, {"Y": ODD}):
        assert c(**kw) == P.PWQ_EINVAL, kw
    assert c(T=0, X=None) == P.PWQ_OK


def test_quantized_matmul_int8_rejects(P):
    names = ["X", "T", "n", "ldx", "sx", "sums", "C", "sw", "z", "m", "Y", "yt", "ldy", "ws", "wsb", "stream"]
    c = _call(P.lib().pwq_quantized_matmul_int8, names,
              [FAKE, 4, 256, 256, FAKE, FAKE, FAKE, FAKE, FAKE, 64, FAKE, P.PWQ_F16, 64, FAKE, 1 << 40, None])
    assert c(yt=5) == P.PWQ_EDTYPE
    for kw in ({"T": -1}, {"m": -1}, {"n": 0}, {"n": 65536, "ldx": 65536}, {"ldx": 255}, {"ldy": 63}, {"X": None},
               {"sx": None}, {"sums": None}, {"C": None}, {"sw": None}, {"Y": None}, {"sx": ODD}, {"sums": ODD},
               {"sw": ODD}, {"z": ODD}, {"Y": ODD}, {"T": 1 << 30, "m": 1 << 30, "ldy": 1 << 30}):
        assert c(**kw) == P.PWQ_EINVAL, kw
    assert c(T=0, X=None) == P.PWQ_OK and c(m=0, C=None) == P.PWQ_OK
    size = P.lib().pwq_quantized_matmul_int8_workspace_size
    assert size(0, 256, 64) == 0 and size(4, 0, 64) == 0 and size(4, 65536, 64) == 0 and size(4, 256, -1) == 0
    # whatever the split of k: whole int32 sums of every output
    for T, n, m in ((1, 768, 768), (16, 28672, 8192), (333, 1601, 5003), (8192, 8192, 28672)):
        assert size(T, n, m) % (T * m * 4) == 0
    need = size(4, 65535, 64)
    if need:
        assert c(n=65535, ldx=65535, ws=None) == P.PWQ_EWORKSPACE
        assert c(n=65535, ldx=65535, wsb=need - 1) == P.PWQ_EWORKSPACE
        assert c(n=65535, ldx=65535, ws=ctypes.c_void_p(0x1008)) == P.PWQ_EWORKSPACE


def test_binding_refuses_on_the_cpu(P):
    import torch
    x = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        P.quantize_tokens(x)
    with pytest.raises(ValueError):
        P.rms_norm_quantize(x)
    with pytest.raises(ValueError):
        P.quantized_matmul_int8(x.to(torch.int8), torch.ones(4), torch.zeros(8, 32, dtype=torch.int8),
                                torch.ones(8, dtype=torch.float16))
