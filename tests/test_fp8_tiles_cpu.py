"""Which tile a workgroup of the e4m3 products takes, compiled alone: every tile once where the offsets do not
decrease, and a place inside the launch whatever they hold."""
import random
import shutil
import subprocess
import os

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "post_weight_quantization_27_amd", "csrc")

# A case: T, m, experts, rows and outputs of a tile, then the offsets, or "alternate" for 0, T, 0, T, ...
# Answers: tiles that were launched, tiles that were counted, the largest sum of 64 experts' tiles, the least and
# largest tile of rows and of outputs, whether every tile was taken once.  Of large launches some workgroups.
PROGRAM = r"""
#include <stdio.h>
#include <string.h>
#include <vector>
#include "fp8_plan.h"
using namespace pwq;
int main() {
    long long T, m, E; int bt, bo; char how[16];
    while (scanf("%lld %lld %lld %d %d %15s", &T, &m, &E, &bt, &bo, how) == 6) {
        std::vector<long long> off(E + 1);
        for (long long i = 0; i <= E; ++i) {
            if (!strcmp(how, "alternate")) off[i] = i & 1 ? T : 0;
            else if (scanf("%lld", &off[i]) != 1) return 1;
        }
        const int most = (int)f8_tiles_most(T, E, bt), tiles_m = (int)f8_cdiv(m, bo);
        uint32_t tiles_t = 0;
        long long sum64 = 0;
        for (long long e0 = 0; e0 < E; e0 += 64) {
            long long n = 0;
            for (long long e = e0; e < e0 + 64 && e < E; ++e) n += f8_own(f8_low(off[e]), f8_high(off[e + 1], T), bt, most);
            sum64 = n > sum64 ? n : sum64;
            tiles_t = f8_upto(tiles_t, (int)n, most);
        }
        const uint32_t grid = (uint32_t)most * (uint32_t)tiles_m, step = grid > 2000000 ? grid / 1000003 + 1 : 1;
        std::vector<unsigned char> taken(step == 1 ? (size_t)tiles_t * tiles_m : 0);
        int t0 = 0, t1 = 0, o0 = 0, o1 = 0;
        bool once = true;
        for (uint32_t bid = 0; bid < grid; bid += step) {
            const F8Place p = f8_place(bid, tiles_t, (uint32_t)tiles_m);
            if (!p.there) continue;
            t0 = p.tt < t0 ? p.tt : t0; t1 = p.tt > t1 ? p.tt : t1; o0 = p.to < o0 ? p.to : o0; o1 = p.to > o1 ? p.to : o1;
            if (step > 1) continue;
            if (p.tt < 0 || p.tt >= (int)tiles_t || p.to < 0 || p.to >= tiles_m || taken[(size_t)p.tt * tiles_m + p.to]++) once = false;
        }
        for (unsigned char c : taken) once = once && c == 1;
        printf("%d %u %lld %d %d %d %d %d\n", most, tiles_t, sum64, t0, t1, o0, o1, (int)once);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("tiles")
    src, exe = d / "tiles.cpp", d / "tiles"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def run(cases):
        text = "\n".join(f"{T} {m} {E} {bt} {bo} " + (off if isinstance(off, str) else "list " + " ".join(map(str, off)))
                         for T, m, E, bt, bo, off in cases)
        out = subprocess.run([str(exe)], input=text, text=True, check=True, capture_output=True).stdout.strip().split("\n")
        rows = [tuple(int(v) for v in line.split()) for line in out]
        assert len(rows) == len(cases)
        return rows
    return run


TILES = [(16, 16), (32, 64), (64, 64), (64, 128), (128, 128), (128, 256), (256, 256)]      # rows, outputs


def test_every_tile_is_taken_once(tiles):
    rng = random.Random(1)
    cases, want = [], []
    for _ in range(400):
        bt, bo = rng.choice(TILES)
        E = rng.choice([1, 1, 2, 9, 63, 64, 65, 130])
        counts = [rng.choice([0, 0, 1, bt - 1, bt, bt + 1, rng.randint(0, 5 * bt)]) for _ in range(E)]
        first, behind = rng.choice([0, 0, 3]), rng.choice([0, 0, 40])
        off = [first]
        for c in counts:
            off.append(off[-1] + c)
        T, m = off[-1] + behind, rng.choice([1, bo, bo + 1, rng.randint(1, 40 * bo)])
        if T:
            cases.append((T, m, E, bt, bo, off))
            want.append(sum(-(-c // bt) for c in counts))
    for (T, m, E, bt, bo, _), w, (most, counted, _, t0, t1, o0, o1, once) in zip(cases, want, tiles(cases)):
        assert counted == w <= most and once
        if w:
            assert (t0, t1, o0, o1) == (0, w - 1, 0, -(-m // bo) - 1)


def test_any_offsets_stay_inside_the_launch(tiles):
    """Offsets that go up and down count rows again and again: 2^20 rows and 65536 experts in tiles of 64 rows
    2^29 times, which eight times over is 0 in 32 bits."""
    rng = random.Random(2)
    cases = [(1 << 20, m, 65536, bt, bo, "alternate") for bt, bo in TILES for m in (1, 64, 5000)]
    cases += [(1 << 28, 64, E, bt, bo, "alternate") for bt, bo in TILES[1:] for E in (2, 3, 300, 65536)]
    for _ in range(200):
        bt, bo = rng.choice(TILES)
        E, T = rng.choice([1, 5, 64, 200]), rng.randint(1, 10 ** 5)
        lo, hi = rng.choice([(-5, T + 5), (-2 ** 31, 2 ** 31 - 1), (0, T)])
        cases.append((T, rng.randint(1, 9000), E, bt, bo, [rng.randint(lo, hi) for _ in range(E + 1)]))
    for (T, m, E, bt, bo, _), (most, counted, sum64, t0, t1, o0, o1, once) in zip(cases, tiles(cases)):
        assert counted <= most and sum64 < 2 ** 31
        assert 0 <= t0 and t1 < max(counted, 1) and 0 <= o0 and o1 < -(-m // bo)
        assert once


def test_a_launch_has_every_share_of_rows(tiles):
    """The launched tiles hold the rows however they are shared out: every expert one row past whole tiles,
    fewer rows than experts, one expert with offsets, all rows at one expert."""
    cases, want = [], []
    for bt, bo in TILES:
        for E in (1, 2, 3, 7, 64, 65, 200):
            for q in (0, 1, 3):
                shares = [[q * bt + 1] * E, [q * bt] * E, [q * bt + bt - 1] * E, [0] * (E - 1) + [q * bt * E + 1],
                          [q * bt * E + E] + [0] * (E - 1), [q * bt + 1] + [1] * (E - 1), [i % 2 for i in range(E)]]
                for counts in shares:
                    if sum(counts):
                        off = [0]
                        for c in counts:
                            off.append(off[-1] + c)
                        cases.append((off[-1], 3 * bo, E, bt, bo, off))
                        want.append(sum(-(-c // bt) for c in counts))
    for w, (most, counted, *_, once) in zip(want, tiles(cases)):
        assert w <= most and counted == w and once
    assert any(w == most for w, (most, *_) in zip(want, tiles(cases)) if w > 1)       # and no fewer would do
