"""The product's choice of a kernel, compiled alone: the GPU tests' shapes reach every kernel, and a
plan covers k and fits its workspace."""
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "post_weight_quantization_27_amd", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "w8a8_plan.h"
int main() {
    long long T, n, m;
    int rows16;
    while (scanf("%lld %lld %lld %d", &T, &n, &m, &rows16) == 4) {
        const pwq::W8Plan p = pwq::w8_plan(T, n, m, rows16 != 0);
        printf("%d %d %lld %lld %d\n", p.kind, p.splits, (long long)p.kper, (long long)pwq::w8_plan_ws_bytes(T, n, m),
               (int)pwq::w8_plan_size_ok(T, m));
    }
    printf("%d %d %d %d %d\n", (int)(sizeof(pwq::w8_tiles) / sizeof(pwq::w8_tiles[0])),
           (int)(sizeof(pwq::w8_any) / sizeof(pwq::w8_any[0])), pwq::W8_ANY, pwq::W8_ROW2, pwq::W8_ROW4);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def run(cases):
        out = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), text=True, check=True,
                             capture_output=True).stdout.strip().split("\n")
        rows = [tuple(int(v) for v in line.split()) for line in out]
        assert len(rows) == len(cases) + 1
        return rows[:-1], rows[-1]
    return run


def test_every_kernel_is_tested(plan):
    from test_gpu_int8_plans import PRODUCTS
    plans, (tiles, anys, any0, row2, row4) = plan([(T, n, m, int(n % 16 == 0)) for T, n, m in PRODUCTS])
    got = {(kind, splits > 1) for kind, splits, *_ in plans}
    kinds = list(range(tiles)) + [any0 + i for i in range(anys)]
    want = {(k, s) for k in kinds for s in (False, True)} | {(row2, False), (row4, False)}
    assert got == want
    # the tiles' loops over k in their steady state (up to five stages in flight), not their ends alone
    assert all(any(p[0] == k and p[1] == 1 and p[2] >= 1024 for p in plans) for k in kinds)


def test_plans_cover_k_and_fit_the_workspace(plan):
    rng = random.Random(3)
    cases = []
    for _ in range(20000):
        T, m = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 16))
        n = min(65535, int(2 ** rng.uniform(0, 16.0)))
        cases.append((T, n, m, 0))
        if n >= 16:
            cases.append((T, n // 16 * 16, m, 1))
    plans, (tiles, anys, any0, row2, row4) = plan(cases)
    for (T, n, m, rows16), (kind, splits, kper, ws, ok) in zip(cases, plans):
        assert ok and (0 <= kind < tiles or kind in (row2, row4) if rows16 else any0 <= kind < any0 + anys)
        assert (splits - 1) * kper < n <= splits * kper
        assert splits == 1 or (kper % 64 == 0 and ws >= splits * T * m * 4 and ws % (T * m * 4) == 0)
        assert kind not in (row2, row4) or (splits == 1 and T <= 1024)
