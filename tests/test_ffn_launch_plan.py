"""How the gated feed-forward operators' work is cut into launches (csrc/ffn/launch_plan.h), compiled for the host and
asked over a pipe (CPU only)."""

import os
import random
import shutil
import subprocess

import pytest

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
