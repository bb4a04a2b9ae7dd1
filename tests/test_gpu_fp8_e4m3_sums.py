"""The e4m3 products with the matrix instruction's own sums: what test_gpu_fp8.py asks of the products with 16-bit
outputs, asked again with e4m3_sums, and how far the sums of either kind are from the exact values on normal data."""
import pytest
import torch

import test_gpu_fp8 as base
from test_gpu_fp8 import DEV, SCALES, TYPES, pwq  # noqa: F401

pytestmark = pytest.mark.gpu


class E4M3Sums:
    """The library with e4m3_sums wherever outputs have 16 bits."""

    def __init__(self, P):
        self.P = P

    def __getattr__(self, name):
        return getattr(self.P, name)

    def _call(self, f, args, kw):
        out = kw["out"].dtype if kw.get("out") is not None else kw.get("out_dtype", torch.float16)
        return f(*args, e4m3_sums=out in (torch.float16, torch.bfloat16), **kw)

    def quantized_matmul_fp8(self, *args, **kw):
        return self._call(self.P.quantized_matmul_fp8, args, kw)

    def quantized_matmul_fp8_grouped(self, *args, **kw):
        return self._call(self.P.quantized_matmul_fp8_grouped, args, kw)


@pytest.fixture(scope="module")
def e4m3_sums(pwq):  # noqa: F811
    return E4M3Sums(pwq)


@pytest.mark.parametrize("scales", list(SCALES))
@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("T,n,m", base.PRODUCTS)
def test_product(e4m3_sums, T, n, m, out, scales):
    base.test_product(e4m3_sums, T, n, m, out, scales)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out,scales", [("bf16", "f32"), ("f16", "e8m0")])
@pytest.mark.parametrize("case", range(len(base.GROUPED)))
def test_grouped(e4m3_sums, case, out, scales, gather):
    base.test_grouped(e4m3_sums, case, out, scales, gather)


@pytest.mark.parametrize("n", [512, 333])
def test_strided(e4m3_sums, n):
    base.test_product_strided(e4m3_sums, n)


@pytest.mark.parametrize("n,out", [(640, "bf16"), (640, "f16"), (643, "f16")])
def test_nan_codes_and_scales(e4m3_sums, n, out):
    base.test_nan_codes_and_scales(e4m3_sums, n, out)


def test_e8m0_extremes(e4m3_sums):
    base.test_e8m0_extremes(e4m3_sums, "bf16")


def test_bad_indexes_and_offsets(e4m3_sums):
    base.test_grouped_bad_indexes_and_offsets(e4m3_sums)


def test_copied_operands(e4m3_sums):
    base.test_copied_operands_of_odd_rows(e4m3_sums)


def test_strides_up_to_32_bit_offsets(e4m3_sums):
    base.test_strides_up_to_32_bit_offsets(e4m3_sums, "bf16")


def test_offsets_past_32_bits(e4m3_sums):
    base.test_offsets_past_32_bits(e4m3_sums)


@pytest.mark.parametrize("scales", list(SCALES))
def test_a_mixture_of_experts_layer(e4m3_sums, scales):
    base.test_a_mixture_of_experts_layer(e4m3_sums, scales)


def test_one_expert_is_the_plain_product(e4m3_sums):
    base.test_one_expert_is_the_plain_product(e4m3_sums)


def test_graphs_and_streams(e4m3_sums):
    base.test_graphs_and_streams(e4m3_sums)


@pytest.mark.parametrize("scales", list(SCALES))
def test_captured_with_splits(pwq, scales):  # noqa: F811
    """Both kinds of sums with k split, and of copied operands, captured together and replayed with eager calls and
    new inputs between."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    sizes = [(17, 8208, 40, 1), (2358, 583, 1290, 1), (130, 8208, 776, 3)]
    calls = []
    for T, n, m, E in sizes:
        w = pwq.quantize_blocks_fp8(torch.randn(E, m, n, device=DEV, generator=g), scale_dtype=SCALES[scales])
        x = torch.randn(T, n, device=DEV, generator=g)
        a = pwq.quantize_tokens_fp8(x, scale_dtype=SCALES[scales])
        off = torch.tensor([0, T // 4, T // 4, T], dtype=torch.int32, device=DEV)
        need = pwq.lib().pwq_quantized_matmul_fp8_grouped_workspace_size(T, n, m, E)
        assert need > 0
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        calls.append((x, a, w, off if E > 1 else None, ws, [torch.empty(T, m, dtype=torch.bfloat16, device=DEV) for _ in range(2)]))

    def run(outs):
        for (x, a, w, off, ws, _), ys in zip(calls, outs):
            pwq.quantize_tokens_fp8(x, out=a)
            for y, e in zip(ys, (False, True)):
                if off is None:
                    pwq.quantized_matmul_fp8(a["codes"], a["scales"], w["codes"][0], w["scales"][0], out=y, ws=ws, e4m3_sums=e)
                else:
                    pwq.quantized_matmul_fp8_grouped(a["codes"], a["scales"], w["codes"], w["scales"], off, out=y, ws=ws, e4m3_sums=e)

    mine = [c[5] for c in calls]
    run(mine)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(mine)
    for _ in range(4):
        for c in calls:
            c[0].normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        eager = [[torch.empty_like(y) for y in ys] for ys in mine]
        run(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(mine, eager) for a, b in zip(p, q))


@pytest.mark.parametrize("scales", list(SCALES))
def test_errors_of_the_norm(pwq, scales):  # noqa: F811
    """Normal data of 8192 inputs.

    float32 sums: an addition is off by at most 2^-24 of the sum so far, evenly spread a third of its square in the
    mean.  With products of unit mean square a sum of j has mean square j: the 128 additions of a block give
    2^-48 128^2 / 6, the 64 blocks 64 times that, and their own 64 additions 2^-48 64 8192 / 6, of 8192.
    e4m3 instruction: 5e-5, as the header says.  Both are seen through the rounding r of 16-bit outputs, where the
    squares add up, but for a product of the two that averages out over the outputs (8 of its deviations)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    T, n, m = 512, 8192, 1024
    a = pwq.quantize_tokens_fp8(torch.randn(T, n, device=DEV, generator=g), scale_dtype=SCALES[scales])
    w = pwq.quantize_blocks_fp8(torch.randn(m, n, device=DEV, generator=g) / 64, scale_dtype=SCALES[scales])

    def f(s):
        return s.float().double() if s.dtype == torch.float32 else torch.exp2(s.view(torch.uint8).double() - 127)
    x = a["codes"].double() * f(a["scales"]).t().contiguous().repeat_interleave(128, 1)
    c = w["codes"].double() * f(w["scales"]).repeat_interleave(128, 0).repeat_interleave(128, 1)
    want = x @ c.t()
    norm = want.norm()

    def off(dtype, **kw):
        y = pwq.quantized_matmul_fp8(a["codes"], a["scales"], w["codes"], w["scales"], out_dtype=dtype, **kw)
        return ((y.double() - want).norm() / norm).item()
    sums = (2.0 ** -48 * (64 * 128 ** 2 + 64 * 8192) / 6 / 8192) ** 0.5
    assert off(torch.float32) <= sums
    for dtype in (torch.float16, torch.bfloat16):
        r = ((want.to(dtype).double() - want).norm() / norm).item()
        cross = 2 * r / (T * m) ** 0.5
        assert abs(off(dtype) ** 2 - r ** 2) <= sums ** 2 + 8 * cross * sums
        assert off(dtype, e4m3_sums=True) ** 2 - r ** 2 <= 5e-5 ** 2 + 8 * cross * 5e-5
