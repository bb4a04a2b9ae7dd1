"""The grouped e4m3 product with the most experts that a call may have: rows shared out among them, and offsets
that go up and down, whose tiles pass 32 bits when they are counted as they stand."""
import numpy as np
import pytest
import torch

from test_gpu_fp8 import DEV, as_scales, check_product, e4m3, pwq, random_codes, random_scales, raw  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [128, 45])
def test_65536_experts(pwq, n):
    rng = np.random.default_rng(n)
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    E, T, m = 65536, 1 << 20, 24
    X = e4m3(random_codes(rng, T, n))
    C = e4m3(random_codes(rng, 64, m, n)).view(torch.uint8).repeat(E // 64, 1, 1).view(torch.float8_e4m3fn)
    sx, sw = torch.rand(1, T, device=DEV, generator=g) * 1e-3, torch.rand(E, 1, 1, device=DEV, generator=g) * 1e-3
    buf = torch.full((T + 2, m + 2), 7.0, device=DEV)
    cut = torch.randint(5, T - 4, (E - 1,), device=DEV, generator=g).sort().values
    ends = torch.cat([cut.new_tensor([5]), cut, cut.new_tensor([T - 5])]).to(torch.int32)
    pwq.quantized_matmul_fp8_grouped(X, sx, C, sw, ends, out=buf[1:-1, 1:-1])
    torch.cuda.synchronize()
    assert (buf[:6] == 7).all() and (buf[-6:] == 7).all() and (buf[:, 0] == 7).all() and (buf[:, -1] == 7).all()
    of = ends.cpu().numpy()
    for e in [0, 1, 63, 64, 4097, E // 2, E - 2, E - 1, *rng.integers(0, E, 30)]:
        a, b = int(of[e]), int(of[e + 1])
        if a < b:
            check_product(buf[1 + a:1 + b, 1:-1], raw(X[a:b]), raw(sx[:, a:b]), raw(C[e]), raw(sw[e]), torch.float32)
    # 0, T, 0, T, ...: half of the experts have every row
    off = torch.arange(E + 1, device=DEV).remainder(2).mul(T).to(torch.int32)
    for out in (torch.float32, torch.bfloat16):
        buf = torch.full((T + 2, m + 2), 7.0, dtype=out, device=DEV)
        for fast in (False, True)[:1 if out == torch.float32 else 2]:
            pwq.quantized_matmul_fp8_grouped(X, sx, C, sw, off, out=buf[1:-1, 1:-1], e4m3_sums=fast)
            torch.cuda.synchronize()
            assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[:, 0] == 7).all() and (buf[:, -1] == 7).all()
            print("ended", n, out, fast, flush=True)
