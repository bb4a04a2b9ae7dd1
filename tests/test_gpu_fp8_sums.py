"""Sums of the e4m3 products: every output type's are float32 sums of exact products, unless the caller asks
for the e4m3 instruction's.

Bars, with p = x_scale scale x w, S = the sum of |p| over k of an output.
float32 sums: exact products in float32 sums of at most 128 terms a block, then one scale product, one
multiply-add a block and one addition a split of k, each off by at most a whole step 2^-23 of the sum so far:
(128 + blocks + 16) 2^-23 S, and half a step of the output's type.  At 8192 inputs that is 3e-5 S, about a
third of a percent of a typical output of random signs: a k left out shows.
The e4m3 instruction cuts seven products of each eight at 2^-13 of the largest one's power of two, towards
zero.  What is cut of one is at most that and, evenly spread, a third of its square in the mean; the signs are
those of the products, random here.  So the mean square of an output's error is at most 7 / 3 2^-26 times the
sum over the eights of their largest p^2, which is at most the sum of p^2 over k; twice its root is the bar for
the error's norm over a row or a column of 32 outputs and more, beside half a step of each output and the
float32 sums' bar.  Of one output: 8 times 2^-13 of the largest p of each eight, taken as their sum."""
import numpy as np
import pytest
import torch

from test_gpu_fp8 import DEV, SCALES, TYPES, as_scales, e4m3, f64, pwq, random_codes, random_scales  # noqa: F401
from test_gpu_fp8_plans import LAID, PRODUCTS, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,n,m,E", [(1, 1024, 72, 1), (70, 1024, 130, 1), (2060, 1024, 776, 1), (300, 1024, 520, 3),
                                     (2060, 1024, 776, 3), (40, 1031, 72, 1), (300, 1031, 520, 3), (2400, 1031, 1300, 1)])
def test_small_products_beside_large_ones(pwq, T, n, m, E, out):
    """Of each eight products one is 2^16 or -2^16, in turn, and the others are 4: the large ones cancel and the
    small ones are the result, every step of a float32 sum exact."""
    k = np.arange(n)
    big = (k % 8 == 0) & (k < n // 16 * 16)
    x = np.where(big, np.where(k % 16 == 0, 256.0, -256.0), 2.0).astype(np.float32)
    w = np.where(big, 256.0, 2.0).astype(np.float32)
    want = 4.0 * np.sum(~big)                                # below 2^12: float16 and float32 hold it
    X = torch.from_numpy(x).to(DEV).to(torch.float8_e4m3fn).view(torch.uint8).repeat(T, 1).view(torch.float8_e4m3fn)
    C = torch.from_numpy(w).to(DEV).to(torch.float8_e4m3fn).view(torch.uint8).repeat(E, m, 1).view(torch.float8_e4m3fn)
    G, OB = -(-n // 128), -(-m // 128)
    sx, sw = torch.ones(G, T, device=DEV), torch.ones(E, OB, G, device=DEV)
    if E == 1:
        y = pwq.quantized_matmul_fp8(X, sx, C[0], sw[0], out_dtype=TYPES[out])
    else:
        off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device=DEV)
        y = pwq.quantized_matmul_fp8_grouped(X, sx, C, sw, off, out_dtype=TYPES[out])
    assert (y.double() - want).abs().max() <= want * torch.finfo(TYPES[out]).eps / 2


def products(pwq, T, n, m, E, out, scales, **kw):
    """Random operands' product and, of each expert, (its rows of Y, the exact values, the sums of magnitudes and
    of squares)."""
    rng = np.random.default_rng(T + n + m + E)
    G, OB, dt = -(-n // 128), -(-m // 128), TYPES[out]
    X, C = random_codes(rng, T, n), random_codes(rng, E, m, n)
    e8 = scales == "e8m0"
    sx, sw = random_scales(rng, e8, G, T), random_scales(rng, e8, E, OB, G)
    if e8:
        sx -= 10                                             # float16's range
    else:
        sw *= np.float32(0.25)
    dX, dC, dsx, dsw = e4m3(X), e4m3(C), as_scales(sx), as_scales(sw)
    if E == 1:
        ends, rows = [0, T], np.arange(T)
        Y = pwq.quantized_matmul_fp8(dX, dsx, dC[0], dsw[0], out_dtype=dt, **kw)
    else:
        cut = np.sort(rng.integers(0, T + 1, E - 1))
        ends = [0, *cut.tolist(), T]
        rows = rng.integers(0, T, T).astype(np.int32)
        Y = pwq.quantized_matmul_fp8_grouped(dX, dsx, dC, dsw, torch.tensor(ends, dtype=torch.int32, device=DEV),
                                             rows=torch.from_numpy(rows).to(DEV), out_dtype=dt, **kw)
    bits = (lambda t: t.view(torch.uint8)) if e8 else (lambda t: t)
    at = torch.from_numpy(rows.astype(np.int64)).to(DEV)
    x = values(dX, bits(dsx).t().contiguous().repeat_interleave(128, 1)[:, :n])
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a < b:
            w = values(dC[e], bits(dsw)[e].repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)[:, :n])
            xe = x[at[a:b]]
            yield Y[a:b].double(), xe @ w.t(), xe.abs() @ w.abs().t(), xe.square() @ w.square().t()


@pytest.mark.parametrize("i", range(len(PRODUCTS + LAID)))
def test_sums_in_float32(pwq, i):
    """The sizes that reach every kernel of float32 sums, with outputs of 16 bits."""
    T, n, m, E = (PRODUCTS + LAID)[i]
    out, scales = [("f16", "f32"), ("bf16", "e8m0"), ("f16", "e8m0"), ("bf16", "f32")][i % 4]
    dt = TYPES[out]
    eps = torch.finfo(dt).eps / 2
    for y, want, S, _ in products(pwq, T, n, m, E, out, scales):
        tol = (128 + -(-n // 128) + 16) * 2.0 ** -23 * S
        tol += (want.abs() + tol) * eps + torch.finfo(dt).tiny * eps
        off = (y - want).abs() - tol
        if dt == torch.float16:                              # past 65504 and half a step: infinities
            off[(want.abs() + tol >= 65520) & (y == want.sign() * torch.inf)] = 0.0
        assert (off <= 0).all(), off.max()


@pytest.mark.parametrize("out,scales", [("bf16", "f32"), ("f16", "f32"), ("bf16", "e8m0"), ("f16", "e8m0")])
@pytest.mark.parametrize("T,n,m,E", PRODUCTS + LAID)
def test_sums_of_the_e4m3_instruction(pwq, T, n, m, E, out, scales):
    dt = TYPES[out]
    eps = torch.finfo(dt).eps / 2
    for y, want, S, P in products(pwq, T, n, m, E, out, scales, e4m3_sums=True):
        sure = (128 + -(-n // 128) + 16) * 2.0 ** -23 * S
        tol = sure + 2.0 ** -10 * S
        half = (want.abs() + tol) * eps + torch.finfo(dt).tiny * eps
        off = (y - want).abs()
        if dt == torch.float16:
            off[(want.abs() + tol >= 65520) & (y == want.sign() * torch.inf)] = 0.0
        assert (off <= tol + half).all(), (off - tol - half).max()
        for d in (0, 1):
            if y.shape[d] >= 32:
                bar = 2 * (7 / 3 * 2.0 ** -26 * P.sum(d)).sqrt() + (half + sure).norm(dim=d)
                assert (off.norm(dim=d) <= bar).all(), (off.norm(dim=d) / bar).max()


def test_refusals(pwq):
    q = torch.zeros(8, 256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    c = torch.zeros(1, 64, 256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    sx, sw, off = torch.ones(2, 8, device=DEV), torch.ones(1, 1, 2, device=DEV), torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    for out in (torch.float32, torch.float64, torch.int8):
        with pytest.raises(pwq.PwqError):
            pwq.quantized_matmul_fp8(q, sx, c[0], sw[0], out_dtype=out, e4m3_sums=True)
        with pytest.raises(pwq.PwqError):
            pwq.quantized_matmul_fp8_grouped(q, sx, c, sw, off, out_dtype=out, e4m3_sums=True)
    assert pwq.quantized_matmul_fp8(q, sx, c[0], sw[0], out_dtype=torch.float16, e4m3_sums=True).shape == (8, 64)
