"""Which form the integer product takes, asked of the library's own plan, so that the
GPU tests' sizes reach every form also after its costs change."""
import os
import shutil
import subprocess

import pytest

from test_gpu_int8_forms import SIZES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_gemm_gb300", "csrc")
TILES = r"""
#include <cstdio>
#include <vector>
#include "int8_plan.h"
int main() {
  // every tile once
  for (int width : {16, 32, 64, 128, 256})
    for (int num_m : {1, 2, 15, 16, 17, 63, 64, 65, 300})
      for (int num_n : {1, 3, 40}) {
        std::vector<int> seen(num_m * num_n, 0);
        for (int t = 0; t < num_m * num_n; ++t) {
          const q4::Tile at = q4::tile_at(t, width, num_m, num_n);
          if (at.m < 0 || at.m >= num_m || at.n < 0 || at.n >= num_n || seen[at.m * num_n + at.n]++) return 1;
        }
      }
  // the most weight rows: 2^30 - 1, and the most tokens
  for (int width : {16, 32, 64, 128}) {
    const int num_n = 1 << 23;
    for (int t : {0, 1, num_n / 2, num_n - 1})
      if (q4::tile_at(t, width, 1, num_n).n != t || q4::tile_at(t, width, 1, num_n).m != 0) return 2;
  }
  const int num_m = 1 << 22;
  for (int t : {0, num_m - 1, 2 * num_m, 3 * num_m - 1}) {
    const q4::Tile at = q4::tile_at(t, 256, num_m, 3);
    if (at.m != t / 48 * 16 + t % 48 % 16 || at.n != t % 48 / 16) return 3;
  }
  puts("tiles");
}
"""
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


def _compile(at, text, *flags):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    (at / "program.cc").write_text(text)
    subprocess.run([cc, "-std=c++17", "-O1", *flags, "-I", CSRC, "-o", str(at / "program"), str(at / "program.cc")], check=True)
    return str(at / "program")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    program = _compile(tmp_path_factory.mktemp("plan"), PROGRAM)

    def ask(sizes, sms=152):
        text = "".join(f"{m} {n} {k} {sms}\n" for m, n, k in sizes)
        out = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout
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


def test_tiles(tmp_path):
    """Each tile once, and no step of the way to it beyond 32 bits."""
    program = _compile(tmp_path, TILES, "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error")
    r = subprocess.run([program], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "tiles", (r.returncode, r.stderr)
