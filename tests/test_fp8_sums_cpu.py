"""The flag of the e4m3 products that asks for the matrix instruction's own sums, without a GPU."""
import os
import re

import pytest

from conftest import ROOT
from test_fp8_cpu import P, _call, far  # noqa: F401


def test_the_binding_has_the_headers_flag(P):
    text = open(os.path.join(ROOT, "include", "pwq.h")).read()
    flag = int(re.search(r"#define PWQ_E4M3_SUMS (0x[0-9a-f]+)", text).group(1), 16)
    assert P.PWQ_E4M3_SUMS == flag and flag & (P.PWQ_F32 | P.PWQ_F16 | P.PWQ_BF16) == 0


@pytest.mark.parametrize("grouped", [False, True])
def test_only_16_bit_outputs_have_e4m3_sums(P, grouped):
    if grouped:
        names = ["X", "nx", "n", "ldx", "sx", "lds", "st", "C", "sw", "m", "E", "off", "rows", "T", "Y", "yt", "ldy", "ws",
                 "wsb", "stream"]
        ok = [far(1), 4, 256, 256, far(2), 4, 1, far(3), far(4), 64, 8, far(7), far(8), 10, far(5), P.PWQ_BF16, 64, far(6),
              1 << 40, None]
        c = _call(P.lib().pwq_quantized_matmul_fp8_grouped, names, ok)
    else:
        names = ["X", "T", "n", "ldx", "sx", "lds", "st", "C", "sw", "m", "Y", "yt", "ldy", "ws", "wsb", "stream"]
        ok = [far(1), 4, 256, 256, far(2), 4, 0, far(3), far(4), 64, far(5), P.PWQ_F16, 64, far(6), 1 << 40, None]
        c = _call(P.lib().pwq_quantized_matmul_fp8, names, ok)
    s = P.PWQ_E4M3_SUMS
    for yt in (P.PWQ_F32 | s, 3 | s, -1, -1 | s, 2 * s | P.PWQ_F16, s >> 1 | P.PWQ_F16):
        assert c(yt=yt) == P.PWQ_EDTYPE, yt
    for yt in (P.PWQ_F16 | s, P.PWQ_BF16 | s):                # the type is right: the other refusals are looked at
        assert c(yt=yt, T=-1) == P.PWQ_EINVAL and c(yt=yt, T=0, X=None) == P.PWQ_OK
        assert c(yt=yt, Y=far(1)) == P.PWQ_EINVAL
