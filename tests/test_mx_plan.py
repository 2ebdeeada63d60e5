"""The rule by which mx_linear divides a product into tiles and chooses CTA pairs: its estimate of
rounds against the schedule itself."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "vocabulary_cross_entropy_gb300", "csrc")
MAIN = r"""
#include "mx_plan.h"
#include <stdio.h>
int main() {
    long long n, v;
    int k, sms;
    while (scanf("%lld %lld %d %d", &n, &v, &k, &sms) == 4) {
        const vce::mx::LinearPlan p = vce::mx::plan_linear(n, v, k, sms);
        printf("%lld %lld %lld %.17g %.17g %d\n", (long long)p.tiles_n, (long long)p.tiles_v, (long long)p.whole_v, p.single,
               p.paired, int(p.pairs));
    }
}
"""


def plans(tmp_path, cases):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(tmp_path / "main.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True, check=True)
    return [[float(x) for x in line.split()] for line in r.stdout.splitlines()]


def test_rounds_are_those_of_the_schedule(tmp_path):
    rng = random.Random(0)
    cases = [(2048, 32000, 32, 152), (1792, 50304, 32, 152), (2048, 128256, 32, 152), (8, 128256, 32, 152), (1, 1, 1, 152)]
    for _ in range(600):
        n, v = int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(0, 18))
        cases.append((n, v, rng.randint(1, 64), rng.choice([152, 148, 20])))
    for (n, v, k, sms), (tiles_n, tiles_v, whole_v, single, paired, pairs) in zip(cases, plans(tmp_path, cases)):
        if not pairs:  # every row and token has a tile, and the CTA with most to do decides
            assert (tiles_n - 1) * 128 < n <= tiles_n * 128
            covered = whole_v * 256 + (tiles_v - whole_v) * 128
            assert v <= covered < v + 256
            load = [0.0] * sms
            for t in range(int(tiles_n * tiles_v)):
                load[t % sms] += 1.0 if t // tiles_n < whole_v else 0.5
            assert single == max(load), (n, v, sms)
        else:
            assert n > 128 and paired < single and tiles_n == -(-n // 256) and tiles_v == whole_v == -(-v // 256)


def test_choices(tmp_path):
    # where one way was measured to take less time (by 4% or more)
    cases = {(256, 128256, 32): 1, (384, 128256, 32): 0, (512, 128256, 32): 1, (640, 128256, 32): 0, (1024, 128256, 32): 1,
             (2048, 128256, 32): 1, (1536, 32000, 32): 1, (1792, 50304, 32): 1, (257, 32001, 17): 0, (1024, 32000, 4): 0,
             (128, 128256, 32): 0}
    got = plans(tmp_path, [c + (152,) for c in cases])
    assert {c: int(g[5]) for c, g in zip(cases, got)} == cases
