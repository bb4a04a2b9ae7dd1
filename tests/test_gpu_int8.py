"""GPU parity of the 8-bit activation path against the float64 oracle: the token quantizer, the
RMS norm with 8-bit output, the int8 product, and the three together.

Bars.  Token quantizer: codes, scales and sums equal to the last bit (the code is that of the
exact quotient, the scale one float32 division).  Norm: h equal to the last bit (one rounding of
the sum); the scale within one float32 step of the oracle's (2^-23: its float64 value differs by
about 1e-14 at most and may round to either neighbour); a code may differ by 1 only where y / s
lies within 128 * 2^-23 of the border between two codes, what such a step moves it by; y within
half a step of its type plus 2^-24 (it passes float32).  Product: the sum is exact, so three
float32 roundings (the sum's conversion, two scales), 3.001 * 2^-24 relative, and half a step
of the output's type.
"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pwq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_27_amd import pwq as P
    P.lib()
    return P


def half_step(y, dtype):
    a = np.abs(y)
    mant, emin = {torch.float32: (24, -126), torch.float16: (11, -14), torch.bfloat16: (8, -126)}[dtype]
    e = np.maximum(np.floor(np.log2(np.maximum(a, 1e-300))), emin)
    return 2.0 ** (e - mant)


def f64(t):
    return t.double().cpu().numpy()


def hidden(rng, T, d, dtype):
    x = rng.standard_normal((T, d)) * np.where(rng.random(d) < 0.02, 20.0, 1.0)
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype]).to(DEV)


def check_codes(r, want, exact=True, y=None):
    q, s, n = want
    torch.cuda.synchronize()
    gq, gs = r["codes"].cpu().numpy(), r["scales"].cpu().numpy()
    if exact:
        assert np.array_equal(gs, s, equal_nan=True)
        assert np.array_equal(gq, q)
    else:
        assert np.array_equal(np.isnan(gs), np.isnan(s))
        live = ~np.isnan(s)
        assert np.all(np.abs(gs[live].astype(np.float64) - s[live]) <= s[live] * 2.0 ** -23)
        bad = gq != q
        if bad.any():
            assert np.max(np.abs(gq.astype(int) - q)) == 1
            v = (y / s.astype(np.float64)[:, None])[bad]
            assert np.all(np.abs(np.abs(v - np.floor(v)) - 0.5) <= 128 * 2.0 ** -23)
    if "sums" in r:
        assert np.array_equal(r["sums"].cpu().numpy(), gq.sum(axis=1, dtype=np.int32))


# ------------------------------------------------------------------ token quantizer
SIZES = [(1, 1), (3, 7), (2, 8), (5, 500), (9, 512), (257, 768), (6, 1031), (300, 2048), (2, 2048), (261, 4104),
         (4, 4097), (1, 8192), (258, 8192), (2, 8191), (3, 16384), (2, 12345), (2, 28672), (2, 40001), (1, 65528),
         (1, 65535)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_tokens(pwq, T, d, dtype):
    rng = np.random.default_rng(T * 70000 + d)
    X = hidden(rng, T, d, dtype)
    r = pwq.quantize_tokens(X, want_sums=True)
    check_codes(r, O.quantize_tokens(X.float().cpu().numpy()))
    chan = (rng.random(d) * 3 + 0.1).astype(np.float32)
    r = pwq.quantize_tokens(X, channel_scale=torch.from_numpy(chan).to(DEV))
    assert "sums" not in r
    check_codes(r, O.quantize_tokens(X.float().cpu().numpy(), chan))


@pytest.mark.parametrize("d", [513, 2048, 9000])
def test_quantize_tokens_ties_and_special_rows(pwq, d):
    """Whole rows on ties, of zeros, tiny, huge, with NaN and infinities."""
    rng = np.random.default_rng(d)
    T = 12
    X = rng.standard_normal((T, d)).astype(np.float32)
    for t, s in enumerate((1.0, 3.0, 5.0 / 1024, 7.0 * 2.0 ** -100)):            # row t: (k + 1/2) s, exact ties
        X[t] = (rng.integers(-127, 127, d) + 0.5).astype(np.float32) * np.float32(s)
        X[t, d // 2] = np.float32(127 * s)
    X[4] = 0
    X[5, d - 1] = np.nan
    X[6, 0] = np.inf
    X[7, 3] = -np.inf
    X[8] *= np.float32(2.0 ** -122)                                             # near the least scale
    X[9] *= np.float32(2.0 ** -140)
    X[10] *= np.float32(2.0 ** 124)
    X[11, 1:] = 0                                                               # one value alone
    r = pwq.quantize_tokens(torch.from_numpy(X).to(DEV), want_sums=True)
    want = O.quantize_tokens(X)
    assert np.isnan(want[1][5:8]).all() and want[1][4] == 0 and want[1][9] == 0
    check_codes(r, want)


@pytest.mark.parametrize("dtype,d,ldx,off,ldq", [("f16", 264, 300, 1, 270), ("bf16", 96, 104, 8, 96), ("f32", 1024, 1031, 3, 1025),
                                                 ("f16", 2048, 2056, 0, 2051)])
def test_quantize_tokens_strides(pwq, dtype, d, ldx, off, ldq):
    """Rows inside a wider matrix at any offset, codes into a wider matrix: what is around stays."""
    rng = np.random.default_rng(d)
    T = 9
    X = hidden(rng, T, ldx + off, dtype)[:, off:off + d]
    big = torch.full((T, ldq), 55, dtype=torch.int8, device=DEV)
    r = pwq.quantize_tokens(X, out={"codes": big[:, :d]})
    check_codes(r, O.quantize_tokens(X.float().cpu().numpy()))
    assert torch.all(big[:, d:] == 55).item()
    e = pwq.quantize_tokens(X[:0], want_sums=True)
    assert e["codes"].shape == (0, d) and e["scales"].shape == (0,) and e["sums"].shape == (0,)


# ------------------------------------------------------------------ norm
def norm_case(pwq, rng, T, d, dtype, gdt, residual, y_dtype, eps=1e-5, want_codes=True):
    X = hidden(rng, T, d, dtype)
    R = hidden(rng, T, d, dtype) if residual else None
    G = None if gdt is None else torch.from_numpy((1 + 0.3 * rng.standard_normal(d)).astype(np.float32)).to(TYPES[gdt]).to(DEV)
    r = pwq.rms_norm_quantize(X, G, residual=R, eps=eps, want_codes=want_codes, want_sums=want_codes,
                              y_dtype=None if y_dtype is None else TYPES[y_dtype])
    torch.cuda.synchronize()
    h = X
    if residual:
        h = (X.float() + R.float()).to(X.dtype)
        assert torch.equal(r["h"], h)
    else:
        assert "h" not in r
    y = O.rms_norm(f64(h), None if G is None else f64(G), eps)
    if want_codes:
        check_codes(r, O.rms_norm_quantize(f64(h), None if G is None else f64(G), eps), exact=False, y=y)
    else:
        assert "codes" not in r
    if y_dtype is not None:
        assert np.all(np.abs(f64(r["y"]) - y) <= np.abs(y) * 1.001 * 2.0 ** -24 + half_step(y, TYPES[y_dtype]))


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rms_norm_quantize(pwq, T, d, dtype):
    rng = np.random.default_rng(T * 70000 + d + 1)
    norm_case(pwq, rng, T, d, dtype, dtype, True, None)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gdt", [None, "f32", "f16", "bf16"])
@pytest.mark.parametrize("y_dtype", [None, "f32", "f16", "bf16"])
@pytest.mark.parametrize("T,d", [(5, 768), (3, 1001), (2, 10240)])
def test_rms_norm_types(pwq, T, d, dtype, gdt, y_dtype):
    rng = np.random.default_rng(T + d)
    norm_case(pwq, rng, T, d, dtype, gdt, False, y_dtype, eps=1e-6)
    if y_dtype is not None:
        norm_case(pwq, rng, T, d, dtype, gdt, True, y_dtype, want_codes=False)


@pytest.mark.parametrize("d", [96, 1003, 8192])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_rms_norm_in_place(pwq, d, which):
    """h into X or the residual itself."""
    rng = np.random.default_rng(d)
    T = 300
    X, R = hidden(rng, T, d, "bf16"), hidden(rng, T, d, "bf16")
    want = pwq.rms_norm_quantize(X, residual=R)
    dst = X if which == "x" else R
    got = pwq.rms_norm_quantize(X, residual=R, out={"h": dst})
    torch.cuda.synchronize()
    assert torch.equal(dst, want["h"]) and torch.equal(got["codes"], want["codes"]) and torch.equal(got["scales"], want["scales"])


def test_rms_norm_special_rows(pwq):
    T, d = 7, 640
    rng = np.random.default_rng(3)
    X = rng.standard_normal((T, d)).astype(np.float32)
    X[1] = 0
    X[2, 5] = np.nan
    X[3, 6] = np.inf
    X[4] *= 1e30
    X[5] *= 1e-30
    r = pwq.rms_norm_quantize(torch.from_numpy(X).to(DEV), eps=1e-5, want_sums=True)
    want = O.rms_norm_quantize(X, None, 1e-5)
    s = r["scales"].cpu().numpy()
    assert s[1] == 0 and np.isnan(s[2:4]).all() and not r["codes"][1:4].any().item()
    check_codes(r, want, exact=False, y=O.rms_norm(X, None, 1e-5))
    # eps 0: rows of any size, and a row of zeros is not finite
    r = pwq.rms_norm_quantize(torch.from_numpy(X).to(DEV), eps=0.0)
    s = r["scales"].cpu().numpy()
    assert np.isnan(s[1:4]).all() and (s[4:] > 0).all() and not r["codes"][1:4].any().item()
    # a float16 sum past the type's range is infinite, and so is a gain
    big = torch.full((2, 64), 40000.0, dtype=torch.float16, device=DEV)
    r = pwq.rms_norm_quantize(big, residual=big)
    assert torch.isinf(r["h"]).all().item() and torch.isnan(r["scales"]).all().item() and not r["codes"].any().item()
    g = torch.ones(640, device=DEV)
    g[7] = float("nan")
    r = pwq.rms_norm_quantize(torch.from_numpy(X[:1]).to(DEV), g)
    assert torch.isnan(r["scales"]).all().item() and not r["codes"].any().item()


@pytest.mark.parametrize("d", [72, 1003, 2048, 8192, 12000, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("place", ["new", "x", "residual", "none"])
def test_rms_norm_rows_past_float32_products(pwq, d, dtype, place):
    """16-bit rows whose products with the gain leave float32 or its precise range (tiny, huge, mixed,
    zero, not finite), among ordinary ones, with h new, in place or not wanted."""
    rng = np.random.default_rng(d)
    T = 9
    tiny, huge = (1e-30, 1e30) if dtype == "bf16" else (6e-8, 3e4)
    x = rng.standard_normal((T, d)).astype(np.float32)
    x[1] *= tiny
    x[2] = np.clip(x[2] * huge, -3e38 if dtype == "bf16" else -6e4, 3e38 if dtype == "bf16" else 6e4)
    x[3] = 0
    x[4, d // 2] = np.nan
    x[5, d - 1] = np.inf
    x[6, : d // 2] *= tiny
    x[7] = 0
    x[7, 3] = tiny
    X = torch.from_numpy(x).to(TYPES[dtype]).to(DEV)
    R = torch.zeros_like(X)
    R[8] = X[0]
    g = rng.standard_normal(d).astype(np.float32)
    g[:5] *= 1e-20 if dtype == "bf16" else 1e-5
    g[5:8] *= 1e20 if dtype == "bf16" else 1e3
    G = torch.from_numpy(g).to(TYPES[dtype]).to(DEV)
    h = (X.float() + R.float()).to(X.dtype)
    y = O.rms_norm(f64(h), f64(G), 1e-30)
    want = O.rms_norm_quantize(f64(h), f64(G), 1e-30)
    out = {"x": {"h": X}, "residual": {"h": R}}.get(place)
    if place == "none":
        r = pwq.rms_norm_quantize(h, G, eps=1e-30, want_sums=True, y_dtype=torch.float32)
    else:
        r = pwq.rms_norm_quantize(X, G, residual=R, eps=1e-30, want_sums=True, y_dtype=torch.float32, out=out)
        torch.cuda.synchronize()
        assert torch.equal(torch.nan_to_num(r["h"]), torch.nan_to_num(h))
        assert out is None or r["h"] is (X if place == "x" else R)
    assert np.isnan(want[1][4:6]).all() and want[1][3] == 0
    with np.errstate(invalid="ignore"):
        check_codes(r, want, exact=False, y=y)
    got, fin = f64(r["y"]), np.isfinite(y) & (np.abs(y) < 3e38)
    assert np.all(np.abs(got[fin] - y[fin]) <= np.abs(y[fin]) * 1.001 * 2.0 ** -24 + half_step(y[fin], torch.float32))


@pytest.mark.parametrize("T,d", [((1 << 22) + 9, 16), ((1 << 20) + 7, 1040)])
def test_more_rows_than_workgroups(pwq, T, d):
    """Rows that a workgroup takes after its first: equal to calls on those rows alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(d)
    X = torch.randn(T, d, generator=g, device=DEV, dtype=torch.bfloat16)
    G = torch.randn(d, generator=g, device=DEV, dtype=torch.bfloat16)
    few = torch.cat([torch.arange(64), torch.arange((1 << 20) - 5, (1 << 20) + 7), torch.arange(T - 16, T)]).to(DEV)
    few = few[few < T]
    for want_sums in (True, False):
        r, s = pwq.quantize_tokens(X, want_sums=want_sums), pwq.quantize_tokens(X[few], want_sums=want_sums)
        assert torch.equal(r["codes"][few], s["codes"]) and torch.equal(r["scales"][few], s["scales"])
        if want_sums:
            assert torch.equal(r["sums"][few], s["sums"])
            assert torch.equal(r["sums"], r["codes"].sum(1, dtype=torch.int32))
        r, s = pwq.rms_norm_quantize(X, G, want_sums=want_sums), pwq.rms_norm_quantize(X[few], G, want_sums=want_sums)
        # other thread counts sum the squares in another order: the scale may round to its neighbour
        assert torch.all((r["scales"][few] - s["scales"]).abs() <= s["scales"] * 2.0 ** -23).item()
        assert (r["codes"][few].int() - s["codes"].int()).abs().max().item() <= 1
        assert (r["codes"][few] != s["codes"]).float().mean().item() < 1e-3
        if want_sums:
            assert torch.equal(r["sums"], r["codes"].sum(1, dtype=torch.int32))


def test_rms_norm_strides(pwq):
    rng = np.random.default_rng(8)
    T, d = 11, 200
    X = hidden(rng, T, 260, "f16")[:, 3:203]
    R = hidden(rng, T, 208, "f16")[:, :200]
    H = torch.full((T, 216), 9.0, dtype=torch.float16, device=DEV)
    Q = torch.full((T, 201), 7, dtype=torch.int8, device=DEV)
    Y = torch.full((T, 256), 5.0, dtype=torch.float32, device=DEV)
    r = pwq.rms_norm_quantize(X, residual=R, y_dtype=torch.float32, out={"h": H[:, :d], "codes": Q[:, :d], "y": Y[:, :d]})
    torch.cuda.synchronize()
    h = (X.float() + R.float()).half()
    assert torch.equal(r["h"], h)
    check_codes(r, O.rms_norm_quantize(f64(h), None, 1e-5), exact=False, y=O.rms_norm(f64(h), None, 1e-5))
    assert torch.all(H[:, d:] == 9).item() and torch.all(Q[:, d:] == 7).item() and torch.all(Y[:, d:] == 5).item()


# ------------------------------------------------------------------ product
def product_case(pwq, rng, T, n, m, zp, odt, full=False, ldx=None, x_off=0, c_off=0, **kw):
    """Codes drawn over every int8 value (full) or normal; X in rows of ldx from x_off, codes from byte c_off."""
    draw = (lambda *s: rng.integers(-128, 128, s)) if full else (lambda *s: np.clip(np.rint(rng.standard_normal(s) * 32), -127, 127))
    x = draw(T, n).astype(np.int8)
    c = draw(m, n).astype(np.int8)
    z = None
    if zp:
        c = (c.astype(np.int16) + 128).astype(np.uint8)
        z = rng.integers(0, 256, m).astype(np.int16)
    sx = (rng.random(T) * 0.05 + 0.001).astype(np.float32)
    sw = (rng.random((m, 1)) * 0.01 + 0.0005).astype(np.float16)
    ldx = ldx or n
    X = torch.zeros(T * ldx + x_off + 64, dtype=torch.int8, device=DEV)[x_off:x_off + T * ldx].view(T, ldx)[:, :n]
    X.copy_(torch.from_numpy(x))
    C = torch.zeros(m * n + c_off, dtype=torch.uint8 if zp else torch.int8, device=DEV)[c_off:].view(m, n)
    C.copy_(torch.from_numpy(c))
    Y = pwq.quantized_matmul_int8(X, torch.from_numpy(sx).to(DEV), C, torch.from_numpy(sw).to(DEV),
                                  zeros=None if z is None else torch.from_numpy(z).to(DEV),
                                  x_sums=torch.from_numpy(x.sum(axis=1, dtype=np.int32)).to(DEV) if zp else None,
                                  out_dtype=TYPES[odt], **kw)
    torch.cuda.synchronize()
    want = O.quantized_matmul_int8(x, sx, c, sw, zeros=z)
    err = np.abs(f64(Y) - want)
    tol = np.abs(want) * 3.001 * 2.0 ** -24 + half_step(want, TYPES[odt])
    assert np.all(err <= tol), f"T {T} n {n} m {m}: worst {np.max(err / tol):.3f} of the bound, at {np.unravel_index(np.argmax(err / tol), err.shape)}"


@pytest.mark.parametrize("T", [1, 2, 5, 16, 17, 32, 33, 48, 64, 65, 100, 128, 129, 200, 256, 257, 300, 512, 515])
@pytest.mark.parametrize("n,m", [(16, 16), (64, 128), (768, 768), (1024, 260), (1040, 100), (4096, 512), (8208, 384)])
def test_quantized_matmul_int8(pwq, T, n, m):
    """Rows of 16-byte multiples."""
    rng = np.random.default_rng(T * 100000 + n * 10 + m)
    k = T + n // 16 + m
    product_case(pwq, rng, T, n, m, k % 2 == 1, ["f32", "f16", "bf16"][k % 3] if n < 4096 else "f32")


@pytest.mark.parametrize("T,n,m,zp", [(1, 1, 1, False), (1, 1, 1, True), (3, 5, 7, True), (1, 63, 130, False), (40, 65, 129, True),
                                      (130, 1601, 333, True), (16, 127, 1000, False), (129, 255, 257, False),
                                      (2, 9999, 50, True), (70, 770, 130, False), (300, 4100, 300, True)])
def test_quantized_matmul_int8_odd(pwq, T, n, m, zp):
    """Any length and any alignment."""
    rng = np.random.default_rng(T + n + m)
    product_case(pwq, rng, T, n, m, zp, "f32")
    product_case(pwq, rng, T, n, m, zp, "bf16", ldx=n + 3, x_off=1, c_off=5)


@pytest.mark.parametrize("T,n,m,ldx,x_off,c_off", [(5, 256, 64, 272, 16, 16), (5, 256, 64, 260, 0, 0), (33, 1024, 96, 1024, 4, 0),
                                                   (33, 1024, 96, 1024, 0, 8), (200, 512, 256, 528, 32, 48),
                                                   (300, 512, 520, 513, 0, 0)])
def test_quantized_matmul_int8_alignment(pwq, T, n, m, ldx, x_off, c_off):
    rng = np.random.default_rng(T + n + m + ldx)
    for zp in (False, True):
        product_case(pwq, rng, T, n, m, zp, "f32", ldx=ldx, x_off=x_off, c_off=c_off)


@pytest.mark.parametrize("T,n,m", [(1, 4096, 96), (20, 2048, 64), (140, 1008, 200), (270, 1000, 270)])
def test_quantized_matmul_int8_all_values(pwq, T, n, m):
    """Every int8 and uint8 value, -128 among them."""
    rng = np.random.default_rng(n)
    for zp in (False, True):
        product_case(pwq, rng, T, n, m, zp, "f32", full=True)


@pytest.mark.parametrize("n", [65535, 65520])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_quantized_matmul_int8_largest_sums(pwq, T, n):
    """The largest sums int32 has to hold: 65535 * 128 * 255 with a zero-point, 65535 * 128 * 128 without."""
    m = 130
    one = torch.ones(m, dtype=torch.float16, device=DEV)
    X = torch.full((T, n), -128, dtype=torch.int8, device=DEV)
    sx = torch.ones(T, device=DEV)
    sums = torch.full((T,), -128 * n, dtype=torch.int32, device=DEV)
    Y = pwq.quantized_matmul_int8(X, sx, torch.full((m, n), -128, dtype=torch.int8, device=DEV), one, out_dtype=torch.float32)
    assert torch.all(Y == float(np.float32(128 * 128 * n))).item()
    for c, z in ((255, 0), (0, 255)):
        Y = pwq.quantized_matmul_int8(X, sx, torch.full((m, n), c, dtype=torch.uint8, device=DEV), one,
                                      zeros=torch.full((m,), z, dtype=torch.int16, device=DEV), x_sums=sums,
                                      out_dtype=torch.float32)
        assert torch.all(Y == float(np.float32(-128.0 * n * (c - z)))).item()


@pytest.mark.parametrize("T,n,m,zp,odt", [(2000, 2064, 8100, False, "bf16"), (4096, 528, 4100, True, "f16"),
                                          (1000, 8208, 2100, True, "f32"), (70, 28672, 2000, True, "f32"),
                                          (300, 28672, 2000, False, "f16"), (1000, 65520, 300, True, "f32"),
                                          (40, 2064, 8100, False, "f32"), (2, 65520, 1000, True, "bf16"),
                                          (3, 28672, 4096, False, "f32"), (129, 8208, 384, True, "f32"),
                                          (515, 1024, 28672, False, "bf16"), (200, 5000, 3000, True, "f32")])
def test_quantized_matmul_int8_large_sampled(pwq, T, n, m, zp, odt):
    """Sizes that take the larger tiles and splits of k, ragged in every dimension: the oracle on
    sampled tokens by sampled outputs, the edges among them."""
    rng = np.random.default_rng(T + n + m)
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    X = torch.randint(-128, 128, (T, n), generator=g, device=DEV, dtype=torch.int8)
    C = torch.randint(-128, 128, (m, n), generator=g, device=DEV, dtype=torch.int8)
    z = None
    if zp:
        C = C.view(torch.uint8)
        z = torch.randint(0, 256, (m, 1), generator=g, device=DEV, dtype=torch.int16)
    sx = torch.rand(T, generator=g, device=DEV) * 0.01 + 0.001
    sw = (torch.rand(m, 1, generator=g, device=DEV) * 0.003 + 0.0005).half()
    Y = pwq.quantized_matmul_int8(X, sx, C, sw, zeros=z, x_sums=X.sum(1, dtype=torch.int32) if zp else None,
                                  out_dtype=TYPES[odt])
    ts = np.unique(np.concatenate([rng.integers(0, T, 40), [0, T - 1]]))
    os_ = np.unique(np.concatenate([rng.integers(0, m, 90), [0, 1, m - 2, m - 1]]))
    ti, oi = torch.from_numpy(ts).to(DEV), torch.from_numpy(os_).to(DEV)
    want = O.quantized_matmul_int8(X[ti].cpu().numpy(), sx[ti].cpu().numpy(), C[oi].cpu().numpy(), sw[oi].cpu().numpy(),
                                   zeros=None if z is None else z[oi].cpu().numpy())
    err = np.abs(f64(Y[ti][:, oi]) - want)
    tol = np.abs(want) * 3.001 * 2.0 ** -24 + half_step(want, TYPES[odt])
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3f} of the bound"
    # every other output against the same call on other rows: another kernel, the same bits
    half = pwq.quantized_matmul_int8(X[:T // 2], sx[:T // 2], C, sw, zeros=z,
                                     x_sums=X[:T // 2].sum(1, dtype=torch.int32) if zp else None, out_dtype=TYPES[odt])
    assert torch.equal(Y[:T // 2], half)
    one = pwq.quantized_matmul_int8(X[-1:], sx[-1:], C, sw, zeros=z, x_sums=X[-1:].sum(1, dtype=torch.int32) if zp else None,
                                    out_dtype=TYPES[odt])
    assert torch.equal(Y[-1:], one)
    odd = torch.zeros(C.numel() + 1, dtype=C.dtype, device=DEV)[1:].view(m, n)
    odd.copy_(C)
    few = min(T, 130)
    got = pwq.quantized_matmul_int8(X[:few], sx[:few], odd, sw, zeros=z,
                                    x_sums=X[:few].sum(1, dtype=torch.int32) if zp else None, out_dtype=TYPES[odt])
    assert torch.equal(Y[:few], got)


@pytest.mark.parametrize("T,n,m,zp,odt", [(4200, 144, 4100, True, "bf16"), (2100, 400, 9100, False, "f32"),
                                          (4200, 48, 8300, True, "f16"), (2962, 28672, 2756, True, "f16")])
def test_quantized_matmul_int8_several_tiles_per_workgroup(pwq, T, n, m, zp, odt):
    """More tiles than compute units: few steps of k per tile, and a split k on top."""
    test_quantized_matmul_int8_large_sampled(pwq, T, n, m, zp, odt)


@pytest.mark.parametrize("T,n,m,zp,odt", [(333, 1601, 5003, True, "f32"), (16, 8191, 28671, False, "bf16"), (2, 4095, 4099, True, "f16"),
                                          (48, 8190, 4099, False, "f16"), (2000, 5001, 5000, True, "bf16"), (1300, 301, 2002, False, "f32"),
                                          (40, 3001, 9001, True, "f32"), (130, 1023, 28670, True, "bf16"), (65, 65535, 70, True, "f32")])
def test_quantized_matmul_int8_any_alignment(pwq, T, n, m, zp, odt):
    """Rows that start at any byte: sizes that take each tile, with and without splits of k."""
    test_quantized_matmul_int8_large_sampled(pwq, T, n, m, zp, odt)


def test_quantized_matmul_int8_scales(pwq):
    """Scales at the ends of their ranges: a token of scale 0 or NaN, products that a scale alone
    would carry out of float32's range."""
    T, n, m = 6, 64, 48
    rng = np.random.default_rng(1)
    x = rng.integers(-127, 128, (T, n)).astype(np.int8)
    c = rng.integers(-127, 128, (m, n)).astype(np.int8)
    sx = np.array([0.0, np.nan, 1e36, 1e-36, 2.0 ** -120, 1.0], dtype=np.float32)
    sw = np.full(m, 6e-8, dtype=np.float16)
    sw[::2] = 60000.0
    sx[2] = 1e28                                                     # 1e28 * 6e4 * 1e6: finite
    Y = pwq.quantized_matmul_int8(torch.from_numpy(x).to(DEV), torch.from_numpy(sx).to(DEV), torch.from_numpy(c).to(DEV),
                                  torch.from_numpy(sw).to(DEV), out_dtype=torch.float32)
    want = O.quantized_matmul_int8(x, sx, c, sw)
    got = f64(Y)
    assert np.isnan(got[1]).all() and (got[0] == 0).all()
    for t in (2, 3, 4, 5):
        assert np.all(np.abs(got[t] - want[t]) <= np.abs(want[t]) * 3.001 * 2.0 ** -24 + half_step(want[t], torch.float32))


@pytest.mark.parametrize("T,n,m", [(5, 256, 64), (40, 512, 200), (5, 257, 64), (300, 256, 300)])
def test_quantized_matmul_int8_writes_its_columns_alone(pwq, T, n, m):
    rng = np.random.default_rng(T + n)
    out = torch.full((T + 3, m + 9), 3.0, dtype=torch.float32, device=DEV)
    product_case(pwq, rng, T, n, m, False, "f32", out=out[:T, :m])
    assert torch.all(out[T:] == 3).item() and torch.all(out[:, m:] == 3).item()


def test_quantized_matmul_int8_same_bits_every_time(pwq):
    """The sums are exact: two calls, and a call on any rows alone, agree to the last bit."""
    rng = np.random.default_rng(2)
    T, n, m = 300, 4096, 1000
    x = torch.from_numpy(rng.integers(-127, 128, (T, n)).astype(np.int8)).to(DEV)
    c = torch.from_numpy(rng.integers(-127, 128, (m, n)).astype(np.int8)).to(DEV)
    sx = torch.rand(T, device=DEV)
    sw = torch.rand(m, device=DEV).half()
    Y = pwq.quantized_matmul_int8(x, sx, c, sw, out_dtype=torch.float32)
    assert torch.equal(Y, pwq.quantized_matmul_int8(x, sx, c, sw, out_dtype=torch.float32))
    for t0, t1 in ((0, 1), (7, 23), (100, 164), (0, 200)):
        assert torch.equal(Y[t0:t1], pwq.quantized_matmul_int8(x[t0:t1], sx[t0:t1], c, sw, out_dtype=torch.float32))


def test_refusals(pwq):
    X = torch.zeros(4, 64, dtype=torch.int8, device=DEV)
    s = torch.ones(4, device=DEV)
    C = torch.zeros(8, 64, dtype=torch.int8, device=DEV)
    w = torch.ones(8, dtype=torch.float16, device=DEV)
    f = pwq.quantized_matmul_int8
    for args, kw in (((X.float(), s, C, w), {}), ((X, s.double(), C, w), {}), ((X, s[:3], C, w), {}), ((X, s, C[:, :32], w), {}),
                     ((X, s, C.view(torch.uint8), w), {}), ((X, s, C, w.float()), {}), ((X, s, C, w[:4]), {}),
                     ((X, s, C.t().contiguous().t(), w), {}), ((X[:1].expand(4, 64), s, C, w), {}), ((X.t(), s, C, w), {}),
                     ((X, s, C.view(torch.uint8), w), {"zeros": torch.zeros(8, dtype=torch.int16, device=DEV)}),
                     ((X, s, C, w), {"out": torch.empty(4, 9, device=DEV)}), ((X, s.cpu(), C, w), {})):
        with pytest.raises(ValueError):
            f(*args, **kw)
    x = torch.zeros(4, 64, device=DEV)
    for kw in ({"channel_scale": torch.ones(63, device=DEV)}, {"channel_scale": torch.ones(64, device=DEV).half()},
               {"out": {"codes": torch.empty(4, 64, device=DEV)}}, {"out": {"scales": torch.empty(5, device=DEV)}}):
        with pytest.raises(ValueError):
            pwq.quantize_tokens(x, **kw)
    for kw in ({"gain": torch.ones(63, device=DEV)}, {"residual": x.half()}, {"residual": x[:2]},
               {"residual": x, "out": {"h": torch.empty(4, 63, device=DEV)}}):
        with pytest.raises(ValueError):
            pwq.rms_norm_quantize(x, **kw)
    with pytest.raises(pwq.PwqError):
        pwq.rms_norm_quantize(x, want_codes=False)                    # nothing to write
    with pytest.raises(pwq.PwqError):
        pwq.quantize_tokens(torch.zeros(1, 65536, device=DEV))
    with pytest.raises(pwq.PwqError):
        pwq.rms_norm_quantize(x, eps=-1.0)


@pytest.mark.parametrize("n", [256, 250])
def test_offsets_past_32_bits(pwq, n):
    """Rows 2^30 elements apart, so that the last starts behind 2^31 elements."""
    rng = np.random.default_rng(n)
    T, m, ld = 3, 72, (1 << 30) - (0 if n % 16 == 0 else 3)
    rows = lambda dtype, w: torch.empty(T * ld, dtype=dtype, device=DEV).view(T, ld)[:, :w]
    x = torch.from_numpy(rng.standard_normal((T, n))).to(DEV).half()
    X, H, Q = rows(torch.float16, n), rows(torch.float16, n), rows(torch.int8, n)
    X.copy_(x)
    a = pwq.quantize_tokens(X, want_sums=True, out={"codes": Q})
    check_codes(a, O.quantize_tokens(f64(x)), exact=True)
    C = torch.from_numpy(rng.integers(-127, 128, (m, n)).astype(np.int8)).to(DEV)
    sw = torch.from_numpy(rng.random(m) + 0.5).to(DEV).half()
    want = pwq.quantized_matmul_int8(a["codes"].contiguous(), a["scales"], C, sw, out_dtype=torch.float32)
    Y = rows(torch.float32, m)
    got = pwq.quantized_matmul_int8(a["codes"], a["scales"], C, sw, out=Y)
    assert got is Y and torch.equal(Y, want)
    b = pwq.rms_norm_quantize(X, residual=X, want_sums=True, out={"codes": Q, "h": H})
    h = x + x
    assert torch.equal(H, h)
    check_codes(b, O.rms_norm_quantize(f64(h), None, 1e-5), exact=False, y=O.rms_norm(f64(h), None, 1e-5))


def test_tensors_of_out_are_written_or_refused(pwq):
    """A dictionary of an earlier call, used again: nothing in it keeps the earlier call's values."""
    rng = np.random.default_rng(8)
    X = torch.from_numpy(rng.standard_normal((5, 200))).to(DEV).half()
    R = torch.from_numpy(rng.standard_normal((5, 200))).to(DEV).half()
    o = pwq.rms_norm_quantize(X, residual=R, want_sums=True, y_dtype=torch.float32)
    again = pwq.rms_norm_quantize(R, residual=R, out=o)                       # no want_sums, no y_dtype
    want = pwq.rms_norm_quantize(R, residual=R, want_sums=True, y_dtype=torch.float32)
    assert again is o and set(o) == set(want) and all(torch.equal(o[k], want[k]) for k in want)
    with pytest.raises(ValueError):
        pwq.rms_norm_quantize(X, out=o)                                       # its h
    with pytest.raises(ValueError):
        pwq.rms_norm_quantize(X, y_dtype=torch.float16, want_codes=False, out={"sums": o["sums"]})
    with pytest.raises(ValueError):
        pwq.rms_norm_quantize(X, y_dtype=torch.float16, want_codes=False, want_sums=True)
    q = pwq.quantize_tokens(X, want_sums=True)
    pwq.quantize_tokens(R, out=q)
    want = pwq.quantize_tokens(R, want_sums=True)
    assert all(torch.equal(q[k], want[k]) for k in want)


# ------------------------------------------------------------------ together
def layer(pwq, x, res, gain, w1, w2, chan):
    """Norm -> product -> token quantizer (channel scale) -> product, as a decoder's MLP runs them."""
    zp1 = w1.get("zeros")
    a = pwq.rms_norm_quantize(x, gain, residual=res, want_sums=zp1 is not None)
    y = pwq.quantized_matmul_int8(a["codes"], a["scales"], w1["codes"], w1["scales"], zeros=zp1, x_sums=a.get("sums"),
                                  out_dtype=x.dtype)
    b = pwq.quantize_tokens(y, channel_scale=chan)
    return a, y, b, pwq.quantized_matmul_int8(b["codes"], b["scales"], w2["codes"], w2["scales"], out_dtype=x.dtype)


@pytest.mark.parametrize("T,d,f", [(1, 768, 2304), (33, 768, 1000), (300, 1031, 520)])
def test_layer_of_quantized_weights(pwq, T, d, f):
    """The path on weights that the framework quantizes (RTN with zero-points, AWQ's scale and its
    RTN, 8 bits per row): every step equal to the oracle's on that step's own inputs, and the
    output near the float64 product of the weights that were quantized."""
    rng = np.random.default_rng(T + d)
    W1 = torch.from_numpy((rng.standard_normal((f, d)) * 0.03).astype(np.float32)).to(DEV)
    W2 = torch.from_numpy((rng.standard_normal((d, f)) * 0.03).astype(np.float32)).to(DEV)
    w1 = pwq.rtn_quantize_zp(W1, bits=8, group_size=0, want_packed=False)
    cal = torch.from_numpy((rng.standard_normal((256, f)) * (1 + 9 * (rng.random(f) < 0.02))).astype(np.float32)).to(DEV)
    H = torch.zeros((f, f), device=DEV)
    pwq.hessian_accumulate(cal, H)
    w2 = pwq.awq_search(W2, H, 256, pwq.channel_abs_mean(cal), bits=8, group_size=0, n_alpha=5, want_packed=False)
    x, res = hidden(rng, T, d, "f16"), hidden(rng, T, d, "f16")
    gain = torch.from_numpy((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)).to(DEV)
    a, y, b, out = layer(pwq, x, res, gain, w1, w2, w2["s"])
    torch.cuda.synchronize()

    h = (x.float() + res.float()).half()
    assert torch.equal(a["h"], h)
    n = O.rms_norm(f64(h), f64(gain), 1e-5)
    check_codes(a, O.rms_norm_quantize(f64(h), f64(gain), 1e-5), exact=False, y=n)
    want = O.quantized_matmul_int8(a["codes"].cpu().numpy(), a["scales"].cpu().numpy(), w1["codes"].cpu().numpy(),
                                   w1["scales"].cpu().numpy(), zeros=w1["zeros"].cpu().numpy())
    assert np.all(np.abs(f64(y) - want) <= np.abs(want) * 3.001 * 2.0 ** -24 + half_step(want, torch.float16))
    check_codes(b, O.quantize_tokens(y.float().cpu().numpy(), w2["s"].cpu().numpy()))
    want = O.quantized_matmul_int8(b["codes"].cpu().numpy(), b["scales"].cpu().numpy(), w2["codes"].cpu().numpy(),
                                   w2["scales"].cpu().numpy())
    assert np.all(np.abs(f64(out) - want) <= np.abs(want) * 3.001 * 2.0 ** -24 + half_step(want, torch.float16))
    # 8 bits on both sides: steps of 1/127 of a row's largest value leave a few percent at most
    ref = (n @ f64(W1).T) @ f64(W2).T
    assert np.linalg.norm(f64(out) - ref) <= 0.05 * np.linalg.norm(ref)


@pytest.mark.parametrize("sym", [True, False])
@pytest.mark.parametrize("act_order", [False, True])
def test_codes_of_a_gptq_layer(pwq, sym, act_order):
    """A layer quantized by GPTQ to 8 bits, behind the norm: the product of what the calls wrote."""
    rng = np.random.default_rng(5)
    T, n, m = 9, 256, 200
    W = torch.from_numpy((rng.standard_normal((m, n)) * 0.05).astype(np.float32)).to(DEV)
    calib = torch.from_numpy(rng.standard_normal((1024, n)).astype(np.float32)).to(DEV)
    x = torch.from_numpy(rng.standard_normal((T, n))).to(DEV).bfloat16()
    q = pwq.gptq_layer(W, calib, bits=8, group_size=0, act_order=act_order, sym=sym, want_packed=False)
    zeros = None if sym else q["zeros"]
    a = pwq.rms_norm_quantize(x, want_sums=not sym)
    Y = pwq.quantized_matmul_int8(a["codes"], a["scales"], q["codes"], q["scales"], zeros=zeros, x_sums=a.get("sums"),
                                  out_dtype=torch.float32)
    torch.cuda.synchronize()
    want = O.quantized_matmul_int8(a["codes"].cpu().numpy(), a["scales"].cpu().numpy(), q["codes"].cpu().numpy(),
                                   q["scales"].cpu().numpy(), zeros=None if sym else zeros.cpu().numpy())
    assert np.all(np.abs(f64(Y) - want) <= np.abs(want) * 3.001 * 2.0 ** -24)
    # and the layer itself: the codes' steps are the only difference from y W^T with the norm's y
    y = O.rms_norm(f64(x), None, 1e-5)
    sx, sw = a["scales"].cpu().numpy().astype(np.float64), f64(q["scales"]).reshape(-1)
    cw = q["codes"].cpu().numpy().astype(np.float64) - (0 if sym else zeros.cpu().numpy().astype(np.float64).reshape(-1, 1))
    exact = y @ (cw * sw[:, None]).T
    # each activation is off by at most half a step of its token (and the scale's rounding)
    bound = sx[:, None] * 0.5001 * np.sum(np.abs(cw * sw[:, None]), axis=1)[None, :]
    assert np.all(np.abs(f64(Y) - exact) <= bound + np.abs(want) * 2.0 ** -20)


@pytest.mark.parametrize("T,d,f", [(1, 2048, 4096), (40, 770, 512)])
def test_layer_captured_and_replayed(pwq, T, d, f):
    """The path in a HIP graph, replayed on new inputs with eager work between the replays, and on
    another stream than the current one."""
    rng = np.random.default_rng(d)
    w1 = pwq.rtn_quantize(torch.from_numpy((rng.standard_normal((f, d)) * 0.03).astype(np.float32)).to(DEV), 8, 0, want_packed=False)
    w2 = pwq.rtn_quantize(torch.from_numpy((rng.standard_normal((d, f)) * 0.03).astype(np.float32)).to(DEV), 8, 0, want_packed=False)
    gain = torch.ones(d, device=DEV)
    xs = [hidden(rng, T, d, "bf16") for _ in range(4)]
    rs = [hidden(rng, T, d, "bf16") for _ in range(4)]
    want = [layer(pwq, x, r, gain, w1, w2, None)[3].clone() for x, r in zip(xs, rs)]
    x, r = xs[0].clone(), rs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(2):
            assert torch.equal(layer(pwq, xs[i], rs[i], gain, w1, w2, None)[3], want[i])
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(pwq, x, r, gain, w1, w2, None)[3]
    for i in (1, 2, 3, 0, 2):
        x.copy_(xs[i])
        r.copy_(rs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        assert torch.equal(layer(pwq, xs[i], rs[i], gain, w1, w2, None)[3], want[i])


def test_two_streams_at_once(pwq):
    """Calls on two streams with workspaces of their own."""
    rng = np.random.default_rng(4)
    T, n, m = 4, 8192, 512
    c = torch.from_numpy(rng.integers(-127, 128, (m, n)).astype(np.int8)).to(DEV)
    sw = torch.rand(m, device=DEV).half()
    x = [torch.from_numpy(rng.integers(-127, 128, (T, n)).astype(np.int8)).to(DEV) for _ in range(2)]
    sx = torch.rand(T, device=DEV)
    want = [pwq.quantized_matmul_int8(v, sx, c, sw, out_dtype=torch.float32) for v in x]
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                got[i].append(pwq.quantized_matmul_int8(x[i], sx, c, sw, out_dtype=torch.float32))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
