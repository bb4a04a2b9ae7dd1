"""Where the 8-bit calls' arguments may lie: columns of one buffer are right, shared memory is refused."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_int8 import DEV, check_codes, f64, hidden, pwq  # noqa: F401  (the library's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d", [(1, 256), (300, 256), (70, 1031), (9, 9000)])
def test_arguments_in_columns_of_one_buffer(pwq, T, d):
    """Each token's record holds x, h, y and the codes; scales and sums lie in one vector's two halves."""
    rng = np.random.default_rng(T + d)
    x, r = hidden(rng, T, d, "f16"), hidden(rng, T, d, "f16")
    want = pwq.rms_norm_quantize(x, residual=r, want_sums=True, y_dtype=torch.float16)
    rec = torch.full((T, 3 * d + (d + 1) // 2 + 5), 7.0, dtype=torch.float16, device=DEV)
    X, H, Y = rec[:, :d], rec[:, d:2 * d], rec[:, 2 * d:3 * d]
    Q = rec.view(torch.int8)[:, 6 * d:7 * d]
    stats = torch.empty(2, T, device=DEV)
    X.copy_(x)
    got = pwq.rms_norm_quantize(X, residual=r, want_sums=True,
                                out={"h": H, "y": Y, "codes": Q, "scales": stats[0], "sums": stats[1].view(torch.int32)})
    torch.cuda.synchronize()
    assert torch.equal(X, x) and all(torch.equal(got[k], want[k]) for k in want)
    assert torch.all(rec[:, 3 * d + (d + 1) // 2:] == 7).item()
    check_codes(got, O.rms_norm_quantize(f64(want["h"]), None, 1e-5), exact=False, y=O.rms_norm(f64(want["h"]), None, 1e-5))

    # the quantizer's codes behind x, then the product behind the codes
    q = pwq.quantize_tokens(X, out={"codes": Q})
    torch.cuda.synchronize()
    check_codes(q, O.quantize_tokens(f64(x)))
    m = 40
    C = torch.from_numpy(rng.integers(-127, 128, (m, d)).astype(np.int8)).to(DEV)
    sw = torch.from_numpy(rng.random(m) + 0.5).half().to(DEV)
    plain = pwq.quantized_matmul_int8(q["codes"].contiguous(), q["scales"], C, sw)
    out = pwq.quantized_matmul_int8(Q, q["scales"], C, sw, out=rec[:, d:d + m])
    assert torch.equal(out, plain) and torch.equal(X, x)


def test_shared_memory_is_refused(pwq):
    T, d, m = 6, 512, 64
    rows = torch.zeros(T, 2 * d, dtype=torch.bfloat16, device=DEV)
    X, R = rows[:, :d], torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    codes = rows.view(torch.int8)
    for out in ({"h": rows[:, 1:d + 1]}, {"h": rows[:, d - 1:2 * d - 1]}, {"codes": codes[:, :d]}, {"codes": codes[:, 2 * d - 1:3 * d - 1]},
                {"y": R}, {"codes": R.view(torch.int8)[:, d:]}, {"scales": R.view(torch.float32).view(-1)[:T]},
                {"h": rows[:, d:], "y": rows[:, d:]}):
        with pytest.raises(pwq.PwqError):
            pwq.rms_norm_quantize(X, residual=R, out=out)
    with pytest.raises(pwq.PwqError):
        pwq.quantize_tokens(X, out={"codes": codes[:, :d]})
    q = torch.zeros(T, d, dtype=torch.int8, device=DEV)
    s = torch.ones(T, device=DEV)
    C = torch.zeros(m, d, dtype=torch.int8, device=DEV)
    w = torch.ones(m, dtype=torch.float16, device=DEV)
    for out in (q.view(torch.float16)[:, :m], C.view(torch.float16).view(-1)[-T * m:].view(T, m)):
        with pytest.raises(pwq.PwqError):
            pwq.quantized_matmul_int8(q, s, C, w, out=out)
    assert not rows.any().item() and not R.any().item() and not q.any().item()
