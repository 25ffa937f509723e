"""How the gated feed-forward operators' work is cut into launches (csrc/ffn/launch_plan.h), compiled for the host and
asked over a pipe (CPU only)."""

import os
import random
import shutil
import subprocess

import pytest

from tests import ffn_kernel_sizes as sizes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=undefined", "-fno-sanitize-recover=all"]


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "launch_plan")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", *SAN, f"-I{ROOT}/precision_fp8_quant_amd/csrc",
                    os.path.join(ROOT, "tests", "c_client", "ffn_launch_plan.cpp"), "-o", exe], check=True)

    def answers(lines):
        res = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, timeout=120)
        assert res.returncode == 0, res.stderr
        return res.stdout.splitlines()
    return answers


def _cdiv(a, b):
    return -(-a // b)


# (rows, columns, threads) of a workgroup's tile: the streaming kernel's and the LDS-tiled one's, plain and gated
TILES = [(16, 8, 1024), (32, 8, 1024), (16, 16, 512), (16, 16, 1024), (16, 32, 512), (64, 32, 512),
         (64, 64, 512), (64, 32, 1024), (128, 64, 256), (128, 128, 512), (256, 128, 512), (256, 256, 512)]


def test_launches_stay_below_2_to_the_32_threads(ask):
    rng = random.Random(7)
    cases = [(m, n, *t) for t in TILES for m, n in [(1, 1), (4, 1 << 27), (1, (1 << 27) + 40), ((1 << 31) + 3, 8),
                                                    ((1 << 30) + 1, 700), (64, 1 << 29), (1 << 17, 1 << 17)]]
    for _ in range(3000):
        m, n = int(2 ** rng.uniform(0, 34)), int(2 ** rng.uniform(0, 34))
        if _cdiv(m, 16) * _cdiv(n, 16) < 1 << 31:          # the C ABI's limit
            cases.append((m, n, *rng.choice(TILES)))
    cut = 0
    for (m, n, bm, bn, threads), line in zip(cases, ask(["pieces %d %d %d %d %d" % c for c in cases])):
        rows, cols = map(int, line.split())
        assert 0 < rows <= m and 0 < cols <= n
        assert _cdiv(rows, bm) * _cdiv(cols, bn) * threads < 1 << 32
        assert rows == m or rows % bm == 0
        assert cols == n or (cols % bn == 0 and cols % 128 == 0)       # FP8 weights have a scale for 128 columns
        whole = _cdiv(m, bm) * _cdiv(n, bn) * threads < 1 << 32
        assert whole == ((rows, cols) == (m, n))
        cut += not whole
        # no more launches than twice what the threads ask for, and one
        assert _cdiv(m, rows) * _cdiv(n, cols) <= 2 * _cdiv(_cdiv(m, bm) * _cdiv(n, bn) * threads, 1 << 32) + 1
    assert cut > 30


# ---------------------------------------------------------------------------
# Which kernel a size chooses
# ---------------------------------------------------------------------------
def _kernels(ask, gated, sizes):
    return ask([f"kernel {int(gated)} {m} {n} {k}" for m, n, k in sizes])


LISTS = [(False, False, sizes.INT8), (True, False, sizes.INT8_GATED), (True, True, sizes.FP8_GATED)]


@pytest.mark.parametrize("gated, fp8, cases", LISTS, ids=["int8", "int8 gated", "fp8 gated"])
def test_listed_sizes_choose_the_kernels_that_they_are_listed_for(ask, gated, fp8, cases):
    got = _kernels(ask, gated, [c[:3] for c in cases])
    assert got == [c[3] for c in cases]
    for name in {c[3] for c in cases}:
        teams = int(name.split("x")[-1]) if name.startswith("tile") and "+" not in name else 1
        left = {-(-k // 128) % teams for _, _, k, kernel in cases if kernel == name}
        assert left == set(range(teams)), f"{name}: no K with a remainder of {set(range(teams)) - left} groups"


@pytest.mark.parametrize("gated, fp8, cases", LISTS, ids=["int8", "int8 gated", "fp8 gated"])
def test_every_kernel_that_a_size_chooses_is_listed(ask, gated, fp8, cases):
    rng = random.Random(11)
    up = (lambda x: _cdiv(x, 128) * 128) if fp8 else (lambda x: x)
    some = [(int(2 ** rng.uniform(0, 14)), up(int(2 ** rng.uniform(0, 15))), up(int(2 ** rng.uniform(0, 15))))
            for _ in range(60000)]
    few = [(m, up(n), up(1101)) for m in range(1, 70) for n in range(1, 14000, 37)]
    chosen = set(_kernels(ask, gated, some + few))
    # one split behind another takes the same kernels
    chosen = {k for k in chosen if k.count("+") < 2}
    assert chosen == {c[3] for c in cases}


def test_sizes_on_both_sides_of_eight_columns_a_workgroup(ask):
    assert _kernels(ask, True, [(1, 2048, 1101), (16, 2043, 1101), (17, 2041, 1101), (32, 2048, 1101), (32, 2049, 1101),
                                (33, 2048, 1101)]) == \
        ["stream half 1x1x16"] * 2 + ["stream half 2x1x16"] * 2 + ["stream 2x1x16", "tile 64x64x2"]
