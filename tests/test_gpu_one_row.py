"""Matrices of one row, whose row stride says nothing: any value of it is taken, and gives what a contiguous row
gives."""
import pytest
import torch

from test_gpu_fp8 import DEV, SCALES, pwq, raw  # noqa: F401

pytestmark = pytest.mark.gpu

STRIDES = [1, 255, 263, 1 << 31]


def one_row(x, stride):
    """x's row with another row stride."""
    return x.as_strided((1, x.shape[1]), (stride, 1))


@pytest.mark.parametrize("stride", STRIDES)
def test_quantizers(pwq, stride):
    x = torch.randn(1, 256, device=DEV).to(torch.bfloat16)
    for call in (pwq.quantize_tokens_fp8, pwq.quantize_blocks_fp8, pwq.quantize_tokens, pwq.rms_norm_quantize):
        want, got = call(x), call(one_row(x, stride))
        assert want.keys() == got.keys()
        assert all(want[k] is got[k] is None or (raw(want[k]) == raw(got[k])).all() for k in want)


@pytest.mark.parametrize("scales", list(SCALES))
def test_experts_of_one_row(pwq, scales):
    """A stack whose matrices are the rows of one."""
    w = torch.randn(5, 256, device=DEV).to(torch.float16)
    want = pwq.quantize_blocks_fp8(w[:, None].contiguous(), scale_dtype=SCALES[scales])
    for v in (w[None].transpose(0, 1), w.as_strided((5, 1, 256), (256, 1 << 31, 1)), w.as_strided((5, 1, 256), (256, 3, 1))):
        got = pwq.quantize_blocks_fp8(v, scale_dtype=SCALES[scales])
        assert all((raw(want[k]) == raw(got[k])).all() for k in want)


@pytest.mark.parametrize("stride", STRIDES)
def test_products(pwq, stride):
    w = pwq.quantize_blocks_fp8(torch.randn(2, 72, 256, device=DEV))
    x = pwq.quantize_tokens_fp8(torch.randn(1, 256, device=DEV))
    q = one_row(x["codes"].view(torch.uint8), stride).view(torch.float8_e4m3fn)
    off = torch.tensor([0, 0, 1], dtype=torch.int32, device=DEV)
    for out in (torch.float32, torch.bfloat16):
        y = torch.empty(1, 72, dtype=out, device=DEV)
        want = pwq.quantized_matmul_fp8(x["codes"], x["scales"], w["codes"][1], w["scales"][1], out_dtype=out)
        pwq.quantized_matmul_fp8(q, x["scales"], w["codes"][1], w["scales"][1], out=one_row(y, stride))
        assert torch.equal(y, want)
        y.zero_()
        pwq.quantized_matmul_fp8_grouped(q, x["scales"], w["codes"], w["scales"], off, out=one_row(y, stride))
        assert torch.equal(y, want)
    c = torch.randint(-127, 128, (72, 256), dtype=torch.int8, device=DEV)
    a, s = pwq.quantize_tokens(torch.randn(1, 256, device=DEV)), torch.rand(72, device=DEV).to(torch.float16)
    want = pwq.quantized_matmul_int8(a["codes"], a["scales"], c, s)
    assert torch.equal(pwq.quantized_matmul_int8(one_row(a["codes"], stride), a["scales"], c, s), want)
