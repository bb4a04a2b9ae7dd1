"""The GPU tests' widths reach every kernel that the norm and the token quantizer choose between."""
import os
import re

from conftest import ROOT


def test_every_range_of_widths_is_tested():
    from test_gpu_int8 import SIZES
    from test_gpu_int8_widths import WIDTHS
    with open(os.path.join(ROOT, "post_weight_quantization_27_amd", "csrc", "tokens.h")) as f:
        text = f.read()
    pick = text[text.index("hipError_t tok_pick("):]
    pick = pick[:pick.index("\n}\n")]
    ends = [int(e) for e in re.findall(r"if \(d <= (\d+)\) return", pick)]
    assert len(ends) >= 5 and ends == sorted(set(ends))
    widths = [d for _, d in SIZES + WIDTHS]
    for lo, hi in zip([0] + ends, ends + [65536]):
        inside = [d for d in widths if lo < -(-d // 8) * 8 <= hi]
        assert any(d % 8 == 0 for d in inside) and any(d % 8 for d in inside), (lo, hi)
