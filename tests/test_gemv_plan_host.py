"""The rule that picks the few-token products' form, compiled on its own: undefined behaviour ends the program, and
what it picks is what a restatement in Python's unbounded numbers picks.  CPU only."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_bit_precision_b200", "csrc")

PROGRAM = r"""
#include "gemv_plan.h"
#include <cstdio>
int main()
{
    long long rows, tiles, fit8, fit16;
    int sms;
    while (std::scanf("%lld %lld %lld %lld %d", &rows, &tiles, &fit8, &fit16, &sms) == 5) {
        const nvfp4::Form f = nvfp4::cheapest_form(rows, tiles, fit8, fit16, sms);
        std::printf("%d %d %d %d %lld\n", f.columns, f.panels, f.plan.seg_rows, f.plan.ctas, (long long)f.plan.cost);
    }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, out = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-I", CSRC,
                    "-o", str(out), str(src)], check=True)
    return str(out)


def pick(program, cases):
    text = "\n".join(" ".join(map(str, c)) for c in cases) + "\n"
    res = subprocess.run([program], input=text, capture_output=True, text=True)
    assert res.returncode == 0
    return [tuple(map(int, line.split())) for line in res.stdout.splitlines()]


def plan(rows, tiles, fit, sms):
    segments = -(-rows // fit)
    seg_rows = -(-rows // segments)
    fewest = -(-segments // sms)
    best = None
    for wave in range(fewest, max(fewest, 4) + 1):
        n = min(tiles, wave * sms // segments)
        cost = wave * (-(-tiles // n) + seg_rows)
        if best is None or cost < best[2]:
            best = (seg_rows, n, cost)
    return best


def expected(rows, tiles, fit8, fit16, sms):
    one, two, panels = plan(rows, tiles, fit8, sms), plan(rows, tiles, fit16, sms), plan(rows, tiles, 8, sms)
    forms = [(20 * one[2], (8, 0) + one), (24 * two[2], (16, 0) + two), (21 * panels[2], (8, 1) + panels)]
    return min(forms, key=lambda f: f[0])[1]


def fits(k):
    """Rows of x that fit whole beside the rings and sums of 8 and of 16 columns: 512 bytes for each 256 columns."""
    room = 216 * 1024
    fixed = [16 * (stages * 2304 + 2 * 4 * 8 * nt * 20) for nt, stages in ((1, 3), (2, 2))]
    steps = -(-k // 256)
    return [min(8 * nt, (room - f) // 512 // steps) for nt, f in zip((1, 2), fixed)]


def test_forms(program):
    cases = []
    for k in (64, 1024, 4096, 5120, 12288, 20480):
        for n in (16, 1536, 4096, 20480):
            for rows in (1, 2, 8, 13, 17, 33, 200, 591 * 8, 592 * 8, 592 * 8 + 1, 4800, 5003, 16384, 100003):
                cases.append((rows, -(-n // 128) * 8, *[max(1, f) for f in fits(k)], 148))
    # as many rows as the call takes (rows x tiles x steps below 2^31), few multiprocessors, one row at a time
    cases += [(2 ** 31 // 8 - 1, 8, 8, 16, 148), (2 ** 28 - 1, 8, 1, 1, 148), (2 ** 20, 2 ** 11, 1, 1, 1), (1, 2 ** 26, 8, 16, 148)]
    for case, got in zip(cases, pick(program, cases)):
        assert got == expected(*case), case


def test_more_segments_than_four_for_each_multiprocessor(program):
    """4800 rows x 4096 x 4096 are 600 segments of 8 rows: 370 of 13 cost less."""
    fit8, fit16 = fits(4096)
    assert (fit8, fit16) == (8, 13)   # (216 KB - 112 KB) / 512 bytes / 16 steps
    (columns, panels, seg_rows, ctas, cost), = pick(program, [(4800, 256, fit8, fit16, 148)])
    assert (columns, panels, seg_rows, ctas, cost) == (16, 0, 13, 1, 3 * (256 + 13))   # 370 segments, three waves
    # 16384 x 4096 x 256: 1024 segments of 16 rows, seven waves of one CTA for each
    (columns, panels, seg_rows, ctas, cost), = pick(program, [(16384, 256, *fits(256), 148)])
    assert (columns, panels, seg_rows, ctas, cost) == (16, 0, 16, 1, 7 * (256 + 16))
