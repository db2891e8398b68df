"""Which form the integer product takes, asked of the library's own plan, so that the
GPU tests' sizes reach every form also after its costs change."""
import os
import shutil
import subprocess

import pytest

from test_gpu_int8_forms import SIZES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_gemm_gb300", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "int8_plan.h"
int main() {
  long long M, N, K, sms;
  while (scanf("%lld %lld %lld %lld", &M, &N, &K, &sms) == 4) {
    const q4::Plan p = q4::plan_of(M, N, K, sms);
    printf("%d %d %d %d %d\n", (int)p.pair, p.width, p.splits, p.num_m, p.num_n);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cc").write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", "-O1", "-I", CSRC, "-o", str(at / "plan"), str(at / "plan.cc")], check=True)

    def ask(sizes, sms=152):
        text = "".join(f"{m} {n} {k} {sms}\n" for m, n, k in sizes)
        out = subprocess.run([str(at / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]
    return ask


def test_every_size_takes_the_form_that_it_stands_for(plans):
    for form, sizes in SIZES.items():
        for size, plan in zip(sizes, plans(sizes)):
            assert plan[:3] == form, size


def test_every_form_is_tested(plans):
    """The forms that any size takes, over a grid of all ranges."""
    def steps(least, most):
        v, out = least, []
        while v < most:
            out.append(v)
            v = v * 5 // 4 + 1
        return out + [most]
    grid = [(m, n, 16 * k) for m in steps(1, 9000) for n in steps(1, 40000) for k in steps(1, 8191)]
    assert {p[:3] for p in plans(grid)} == set(SIZES)


def test_kinds_of_pairs(plans):
    sizes = SIZES[(1, 256, 1)]
    several = [p[3] * p[4] > 2 * 76 for p in plans(sizes)]
    runs = [-(-k // 512) for _, _, k in sizes]
    for odd in (0, 1):
        assert any(s and r % 2 == odd and r > 1 and k % 512 for s, r, (_, _, k) in zip(several, runs, sizes))
    assert any(s and r == 1 for s, r in zip(several, runs)) and not all(several)
    assert all(m % 256 for m, _, _ in sizes) and any(n % 256 for _, n, _ in sizes)


def test_parts_and_tiles_stay_in_range(plans):
    """Every K part has a stage, split tiles are all in the grid at once, and tiles
    are counted in 32 bits."""
    sizes = [(m, n, k) for m in (1, 2, 16, 17, 100, 1000, 2 ** 20, 2 ** 30 - 1) for n in (1, 128, 129, 8192, 2 ** 20, 2 ** 30 - 1)
             for k in (16, 128, 144, 272, 400, 8192, 131056) if -(-m // 64) * -(-n // 64) < 2 ** 30]
    for (m, n, k), (pair, width, splits, num_m, num_n) in zip(sizes, plans(sizes)):
        assert num_m == -(-m // width) and num_n == -(-n // (256 if pair else 128)) and num_m * num_n < 2 ** 31
        assert splits == 1 or (not pair and splits <= -(-k // 128) and splits * num_m * num_n <= 152)
