"""The product in 8-bit integers in every kernel that it chooses between, with and without splits of
the inputs: the oracle on sampled tokens by sampled outputs, and equal to the last bit to the same
product through the other kind of kernels (rows at odd addresses, or padded to 16-byte multiples)."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_int8 import DEV, TYPES, f64, half_step, pwq  # noqa: F401  (the library's fixture)

pytestmark = pytest.mark.gpu

# tokens, inputs, outputs; rows of 16-byte multiples, then of any length
PRODUCTS = [
    (1, 1456, 33), (20, 1040, 801), (1, 8192, 1961), (1, 8192, 8192), (4, 8192, 8192), (1, 14336, 4096), (1, 8192, 8190),
    (8, 8192, 2468), (2179, 1584, 3603), (287, 63840, 6207), (1902, 1520, 2182), (973, 8112, 2143), (598, 15104, 805),
    (1370, 1472, 1558), (779, 5600, 1242), (323, 7952, 660), (851, 1440, 1160), (48, 8192, 28672), (2, 17664, 11639),
    (279, 8128, 398), (364, 1456, 367), (397, 4000, 616), (3, 5984, 33),
    (3, 1545, 33), (331, 2705, 420), (2, 4783, 32), (537, 1830, 1852), (257, 37745, 776), (742, 1507, 664),
    (270, 7987, 1413), (342, 5759, 148), (836, 1593, 1160), (801, 5383, 582), (324, 4786, 332), (1604, 1641, 1279),
    (1181, 15508, 1246), (421, 10500, 1173),
]


@pytest.mark.parametrize("T,n,m", PRODUCTS)
@pytest.mark.parametrize("zp", [False, True])
def test_quantized_matmul_int8(pwq, T, n, m, zp):
    rng = np.random.default_rng(T + n + m)
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    X = torch.randint(-128, 128, (T, n), generator=g, device=DEV, dtype=torch.int8)
    C = torch.randint(-128, 128, (m, n), generator=g, device=DEV, dtype=torch.int8)
    z = sums = None
    if zp:
        C = C.view(torch.uint8)
        z = torch.randint(0, 256, (m, 1), generator=g, device=DEV, dtype=torch.int16)
        sums = X.sum(1, dtype=torch.int32)
    sx = torch.rand(T, generator=g, device=DEV) * 0.01 + 0.001
    sw = (torch.rand(m, 1, generator=g, device=DEV) * 0.003 + 0.0005).half()
    # the same operands for the other kind of kernels
    if n % 16 == 0:
        X2, C2 = X, torch.empty(m * n + 1, dtype=C.dtype, device=DEV)[1:].view(m, n)
        C2.copy_(C)
    else:
        X2, C2 = (torch.nn.functional.pad(v, (0, -n % 16)) for v in (X, C))
    ts = np.unique(np.concatenate([rng.integers(0, T, 40), [0, T - 1]]))
    os_ = np.unique(np.concatenate([rng.integers(0, m, 90), [0, 1, m - 2, m - 1]]))
    ti, oi = torch.from_numpy(ts).to(DEV), torch.from_numpy(os_).to(DEV)
    want = O.quantized_matmul_int8(X[ti].cpu().numpy(), sx[ti].cpu().numpy(), C[oi].cpu().numpy(), sw[oi].cpu().numpy(),
                                   zeros=None if z is None else z[oi].cpu().numpy())
    for odt in (torch.float32, torch.bfloat16 if zp else torch.float16):
        Y = pwq.quantized_matmul_int8(X, sx, C, sw, zeros=z, x_sums=sums, out_dtype=odt)
        err = np.abs(f64(Y[ti][:, oi]) - want)
        tol = np.abs(want) * 3.001 * 2.0 ** -24 + half_step(want, odt)
        assert np.all(err <= tol), f"{odt}: worst {np.max(err / tol):.3f} of the bound"
        assert torch.equal(Y, pwq.quantized_matmul_int8(X2, sx, C2, sw, zeros=z, x_sums=sums, out_dtype=odt))
