"""The e4m3 product's choice of a kernel, compiled alone: the GPU tests' shapes reach every kernel, and a
plan covers k and fits its workspace."""
import random
import shutil
import subprocess
import os

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "post_weight_quantization_27_amd", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "fp8_plan.h"
int main() {
    long long T, n, m, E;
    int exact, fast;
    while (scanf("%lld %lld %lld %lld %d %d", &T, &n, &m, &E, &exact, &fast) == 6) {
        const pwq::F8Plan p = pwq::f8_plan(pwq::F8Shape{T, n, m, E, exact != 0, fast != 0});
        printf("%d %d %lld %lld %d %lld %d\n", p.kind, p.splits, (long long)p.kper, (long long)pwq::f8_plan_ws_bytes(T, n, m, E),
               (int)pwq::f8_plan_size_ok(T, m, E), (long long)pwq::f8_tiles_most(T, E, 16), (int)p.lay);
    }
    return 0;
}
"""
ROW1, ROW2, TILES, ANY = -1, -2, 5, (8, 9, 10)
NO_FLOAT16 = (0,)                         # tiles without a form for float32 outputs


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
        assert len(rows) == len(cases)
        return rows
    return run


@pytest.mark.parametrize("exact", [0, 1])
def test_every_kernel_is_tested(plan, exact):
    from test_gpu_fp8_plans import PRODUCTS
    plans = plan([(*p, exact, int(p[1] % 16 == 0)) for p in PRODUCTS])
    got = {(kind, splits > 1) for kind, splits, *_, lay in plans if not lay}
    tiles = [i for i in range(TILES) if not (exact and i in NO_FLOAT16)] + list(ANY)
    assert got == {(k, s) for k in tiles for s in (False, True)} | {(ROW1, False), (ROW2, False)}
    grouped = {kind for (T, n, m, E), (kind, *_, lay) in zip(PRODUCTS, plans) if E > 1 and not lay}
    assert grouped == {*tiles, ROW1, ROW2}
    # the tiles' loops over k in their steady state, not their ends alone
    assert all(any(p[0] == k and p[1] == 1 and p[2] >= 1024 for p in plans) for k in tiles)


def test_copied_operands_are_tested(plan):
    """Rows of any length whose copies take the faster kernels: one matrix and experts, k split and not."""
    from test_gpu_fp8_plans import LAID
    plans = {e: plan([(*p, e, 0) for p in LAID]) for e in (0, 1)}
    assert all(any(plans[e][i][-1] for e in (0, 1)) for i in range(len(LAID)))
    for e in (0, 1):
        got = {(p[3] > 1, q[1] > 1) for p, q in zip(LAID, plans[e]) if q[-1]}
        assert got == {(a, b) for a in (False, True) for b in (False, True)}
    kinds = {q[0] for e in (0, 1) for q in plans[e] if q[-1]}
    assert kinds >= {0, 1, 2, 3, 4} and kinds & {ROW1, ROW2}


def test_plans_cover_k_and_fit_the_workspace(plan):
    rng = random.Random(3)
    cases = []
    for _ in range(20000):
        T, m = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 16))
        n = int(2 ** rng.uniform(0, 16.0))
        E = rng.choice([1, 1, 2, 7, 64, 300])
        exact = rng.randint(0, 1)
        cases.append((T, n, m, E, exact, 0))
        if n >= 16:
            cases.append((T, n // 16 * 16, m, E, exact, 1))
    for (T, n, m, E, exact, fast), (kind, splits, kper, ws, ok, tiles16, lay) in zip(cases, plan(cases)):
        assert ok
        assert kind in (ROW1, ROW2) or 0 <= kind < TILES if fast or lay else kind in ANY
        assert not lay or (not fast and n % 16 and n >= 128)
        assert not (exact and kind in NO_FLOAT16)
        assert (splits - 1) * kper < n <= splits * kper
        assert splits == 1 or kper % 128 == 0
        sums = -(-splits * T * m * 4 // 16) * 16 if splits > 1 else 0
        assert ws >= sums + (lay and (T + E * m) * (-(-n // 16) * 16))
        assert kind not in (ROW1, ROW2) or (splits == 1 and tiles16 <= 65535)


def test_tiles_of_any_shares_fit_the_launch(plan):
    """However the rows are shared out, no more tiles hold rows than are launched."""
    rng = random.Random(4)
    for _ in range(2000):
        E, bt = rng.choice([2, 3, 9, 64]), 16
        counts = [rng.choice([0, 1, 15, 16, 17, rng.randint(0, 200)]) for _ in range(E)]
        T = sum(counts) + rng.choice([0, 0, 5])
        if T == 0:
            continue
        most = T // bt + min(T, E)
        assert sum(-(-c // bt) for c in counts) <= most
