"""The e4m3 products at sizes that reach every kernel the plan chooses between (test_fp8_plan_cpu.py checks
that they do): all outputs against float64 products on the GPU, some of them against the oracle.

Bars as in test_gpu_fp8.py; for all outputs at once the largest product of each eight is taken as their
sum, which is never less."""
import numpy as np
import pytest
import torch

from test_gpu_fp8 import DEV, SCALES, TYPES, as_scales, check_product, e4m3, pwq, random_codes, random_scales, raw  # noqa: F401

pytestmark = pytest.mark.gpu

PRODUCTS = [  # rows, d_in, d_out, experts
    (1, 1040, 40, 1), (130, 1040, 1032, 1), (1300, 48, 6152, 1), (1300, 1040, 6152, 1), (400, 48, 8200, 1), (400, 1040, 8200, 1),
    (1600, 48, 1288, 1), (200, 1040, 8200, 1), (1300, 48, 776, 1), (65, 1040, 8200, 1), (257, 48, 40, 1), (257, 1040, 40, 1),
    (2060, 8208, 72, 1), (17, 6160, 4104, 1), (3, 8208, 40, 1), (17, 8208, 40, 1), (130, 20496, 2696, 1), (130, 16400, 5512, 1),
    (1, 48, 40, 6), (20, 4112, 40, 6), (1030, 400, 136, 6), (1300, 1040, 6152, 6), (65, 1040, 8200, 6), (1600, 48, 2056, 6), (2060, 1040, 776, 6),
    (520, 1040, 3100, 6), (2060, 48, 776, 6), (100, 1040, 3100, 6), (130, 1040, 3100, 6), (1600, 1040, 40, 6), (40, 8208, 40, 6),
    (65, 8208, 40, 6), (100, 6160, 776, 6), (130, 8208, 776, 6), (2060, 8208, 72, 6), (1030, 8208, 200, 6),
    (65, 400, 4104, 1), (65, 8208, 2056, 1), (400, 48, 6152, 6), (24, 1040, 8200, 6), (400, 48, 2696, 1), (1, 12304, 2056, 1), (700, 1040, 2056, 6),
    # rows that start at any byte
    (1, 45, 40, 1), (1, 2065, 40, 1), (100, 1041, 8200, 1), (130, 401, 4104, 1), (257, 1041, 1800, 1), (257, 1041, 5512, 1),
    (700, 149, 5512, 1), (1030, 4113, 72, 1), (1600, 8209, 72, 1), (1600, 8209, 136, 1), (40, 8209, 6152, 1), (1, 1041, 40, 6),
    (700, 1041, 2056, 6), (1030, 1041, 2056, 6), (1600, 1041, 520, 6), (1600, 2065, 520, 6), (1600, 4113, 72, 6), (1600, 401, 5512, 6),
]

# rows of any length that are copied to rows of 16-byte multiples first
LAID = [
    (2208, 131, 4037, 1), (2533, 129, 2294, 1), (2781, 16147, 129, 1), (2358, 583, 1290, 1), (371, 13409, 649, 1), (1295, 2503, 835, 1),
    (1456, 4733, 343, 1), (262, 79215, 202, 1), (4000, 1601, 2003, 1), (3174, 135, 2628, 6), (4000, 129, 2600, 6), (2019, 15035, 403, 6),
    (3167, 9261, 449, 6), (5648, 1807, 516, 6), (3400, 11027, 268, 6), (5000, 4111, 1003, 6), (2422, 30267, 264, 6), (276, 3093, 1, 130),
]


def values(codes, sx):
    s = sx.float().double().cpu().to(DEV) if sx.element_size() == 4 else torch.exp2(sx.view(torch.uint8).double() - 127)
    return codes.double() * s


@pytest.mark.parametrize("out,scales", [("bf16", "f32"), ("f32", "f32"), ("f16", "e8m0"), ("f32", "e8m0")])
@pytest.mark.parametrize("T,n,m,E", PRODUCTS + LAID)
def test_kernels(pwq, T, n, m, E, out, scales):
    rng = np.random.default_rng(T + n + m + E)
    G, OB, dt = -(-n // 128), -(-m // 128), TYPES[out]
    X, C = random_codes(rng, T, n), random_codes(rng, E, m, n)
    e8 = scales == "e8m0"
    sx, sw = random_scales(rng, e8, G, T), random_scales(rng, e8, E, OB, G)
    if e8:
        sx -= 8                                             # float16's range
    dX, dC, dsx, dsw = e4m3(X), e4m3(C), as_scales(sx), as_scales(sw)
    if E == 1:
        ends, rows = [0, T], np.arange(T)
        Y = pwq.quantized_matmul_fp8(dX, dsx, dC[0], dsw[0], out_dtype=dt)
    else:
        cut = np.sort(rng.integers(0, T - T // 20 + 1, E - 1))          # some rows behind the last expert's
        ends = [0, *cut.tolist(), T - T // 20]
        rows = rng.integers(0, T, T).astype(np.int32)
        Y = torch.full((T, m), 7.0, dtype=dt, device=DEV)
        pwq.quantized_matmul_fp8_grouped(dX, dsx, dC, dsw, torch.tensor(ends, dtype=torch.int32, device=DEV),
                                         rows=torch.from_numpy(rows).to(DEV), out=Y)
        assert (Y[ends[-1]:] == 7).all()
    at = torch.from_numpy(rows.astype(np.int64)).to(DEV)
    x = values(dX, dsx.t().contiguous().repeat_interleave(128, 1)[:, :n] if not e8 else
               dsx.view(torch.uint8).t().contiguous().repeat_interleave(128, 1)[:, :n])
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        s = (dsw.view(torch.uint8) if e8 else dsw)[e].repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)[:, :n]
        w = values(dC[e], s)
        xe = x[at[a:b]]
        want, S = xe @ w.t(), xe.abs() @ w.abs().t()
        eps = torch.finfo(dt).eps / 2
        tol = (128 + G + 16) * 2.0 ** -23 * S + want.abs() * eps * 1.0001 + torch.finfo(dt).tiny * eps * 2
        if dt != torch.float32:
            tol += 2.0 ** -10 * S
        y = Y[a:b].double()
        off = (y - want).abs() - tol
        if dt == torch.float16:
            # 65504 + half a step of 32 = 65520 and everything beyond it rounds to infinity, so a value that
            # the bar leaves on either side of 65520 may come out as one of its sign
            off[(want.abs() + tol >= 65520) & (y == want.sign() * torch.inf)] = 0.0
        assert (off <= 0).all(), off.max()
        some = np.unique(np.concatenate([[a, b - 1], rng.integers(a, b, 6)]))
        cols = np.unique(np.concatenate([[0, m - 1], rng.integers(0, m, 30)]))
        for o in np.unique(cols // 128)[:6]:
            c = cols[cols // 128 == o]
            check_product(Y[torch.from_numpy(some).to(DEV)][:, torch.from_numpy(c).to(DEV)], X[rows[some]], sx[:, rows[some]],
                          C[e][c], sw[e][o:o + 1], dt)
