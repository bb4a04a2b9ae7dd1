"""The norm and the token quantizer at a width of every kernel they choose between, aligned and odd."""
import numpy as np
import pytest
import torch

import oracle as O
import test_gpu_int8 as base
from test_gpu_int8 import DEV, TYPES, check_codes, f64, hidden, norm_case, pwq  # noqa: F401  (the library's fixture)

pytestmark = pytest.mark.gpu

WIDTHS = [(257, 4096), (3, 2560), (2, 4095), (260, 3003), (3, 5120), (2, 5121), (2, 7168), (3, 20480), (2, 20483), (2, 29568),
          (2, 29571), (2, 32768), (1, 32763)]


@pytest.mark.parametrize("T,d", WIDTHS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_tokens(pwq, T, d, dtype):
    base.test_quantize_tokens(pwq, T, d, dtype)


@pytest.mark.parametrize("T,d", WIDTHS)
@pytest.mark.parametrize("dtype,gdt", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", None)])
def test_rms_norm_quantize(pwq, T, d, dtype, gdt):
    rng = np.random.default_rng(T * 70000 + d + 2)
    norm_case(pwq, rng, T, d, dtype, gdt, True, "f16")
    norm_case(pwq, rng, T, d, dtype, gdt, False, None)


@pytest.mark.parametrize("d", [3003, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("place", ["new", "x", "residual", "none"])
def test_rms_norm_rows_past_float32_products(pwq, d, dtype, place):
    base.test_rms_norm_rows_past_float32_products(pwq, d, dtype, place)


@pytest.mark.parametrize("d", [3003, 4096, 32768])
def test_quantize_tokens_ties_and_special_rows(pwq, d):
    base.test_quantize_tokens_ties_and_special_rows(pwq, d)


@pytest.mark.parametrize("d", [1031, 2051, 3003, 4096, 4099, 8191, 16383, 20001, 40001])
@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("dtype,gdt", [("bf16", None), ("f16", "f32"), ("f32", "f32")])
def test_norm_in_place(pwq, d, which, dtype, gdt):
    """h into X or the residual; at odd widths the last piece of a row is read from before its place, over
    elements that other threads write."""
    rng = np.random.default_rng(d)
    T = 70
    X, R = hidden(rng, T, d, dtype), hidden(rng, T, d, dtype)
    G = None if gdt is None else torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).to(TYPES[gdt]).to(DEV)
    h = (X.float() + R.float()).to(X.dtype)
    want = pwq.rms_norm_quantize(X, G, residual=R, want_sums=True)
    dst = X if which == "x" else R
    got = pwq.rms_norm_quantize(X, G, residual=R, want_sums=True, out={"h": dst})
    torch.cuda.synchronize()
    assert torch.equal(dst, h) and all(torch.equal(got[k], want[k]) for k in want)
    g = None if G is None else f64(G)
    check_codes(got, O.rms_norm_quantize(f64(h), g, 1e-5), exact=False, y=O.rms_norm(f64(h), g, 1e-5))


@pytest.mark.parametrize("d", [2048, 40000])
def test_norm_past_127_times_float32(pwq, d):
    """One value and a gain that carry y past what a float32 scale can hold: an infinite scale, codes 0."""
    X = torch.zeros(3, d, device=DEV)
    X[:, 5] = 1.0
    X[1] = 1.0
    G = torch.full((d,), 3e38, device=DEV)
    r = pwq.rms_norm_quantize(X, G, eps=0.0, want_sums=True)
    q, s, n = O.rms_norm_quantize(f64(X), f64(G), 0.0)
    assert (np.isinf(s[[0, 2]]).all() and not q[[0, 2]].any()) == (d == 40000) and np.isfinite(s[1])
    check_codes(r, (q, s, n), exact=True)
