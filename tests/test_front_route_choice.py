"""When moe_route's merged choice of 4 to 8 experts by shortened FP32 keys (csrc/front/route_choice.h) has to be made again
with all bits: whenever the bits left out matter, and not for what does not matter.  Compiled for the host and asked over a
pipe (CPU only)."""

import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=undefined", "-fno-sanitize-recover=all"]
INF = np.float32(np.inf)


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("choice") / "route_choice")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wno-unknown-pragmas", "-Werror", *SAN,
                    f"-I{ROOT}/precision_fp8_quant_amd/csrc", os.path.join(ROOT, "tests", "c_client", "front_route_choice.cpp"),
                    "-o", exe], check=True)

    def choices(rows, k):
        """(near [T], experts [T][k]) of FP32 logits."""
        room = next(r for r in (64, 128, 256, 512, 1024) if r >= rows.shape[1])
        lines = [f"token {room} {rows.shape[1]} {k} " + " ".join(map(str, r)) for r in rows.view(np.uint32)]
        res = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, timeout=120)
        assert res.returncode == 0, res.stderr
        out = np.array([line.split() for line in res.stdout.splitlines()], int)
        return out[:, 0] != 0, out[:, 1:]
    return choices


def _order(z, k):
    """The k largest, the lower index first; -1 where only minus infinity is left."""
    order = np.argsort(-z.astype(np.float64), axis=1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(z, order, 1) > -INF, order, -1)


def _normal(rng, t, e):
    return (2.0 * rng.standard_normal((t, e))).astype(np.float32)


def _room(e):
    return next(r for r in (64, 128, 256, 512, 1024) if r >= e)


def _kept_bits(z):
    """What a key holds of each logit."""
    return (z + np.float32(0)).view(np.uint32) // _room(z.shape[1])


@pytest.mark.parametrize("k", [4, 5, 6, 7, 8])
@pytest.mark.parametrize("e", [8, 60, 64, 100, 250, 1000])
def test_made_again_wherever_the_keys_may_be_wrong(ask, e, k):
    rng = np.random.default_rng(100 * e + k)
    near = (np.float32(1.5).view(np.int32) + rng.integers(0, 8 * e, (200, e))).astype(np.int32).view(np.float32)
    z = np.concatenate([near, -near, _normal(rng, 200, e)])
    z[::3] = np.where(rng.random((200, e)) < 0.5, -INF, z[::3])
    again, chosen = ask(z, k)
    assert np.array_equal(chosen[~again], _order(z, k)[~again])
    assert again.any()


@pytest.mark.parametrize("e, k", [(4, 4), (5, 4), (6, 4), (7, 7), (6, 5), (8, 8)])
def test_not_made_again_for_few_experts(ask, e, k):
    """Places beyond the row are no choice."""
    z = _normal(np.random.default_rng(e), 400, e)
    bits = np.sort(_kept_bits(z), axis=1)
    apart = (np.diff(bits, axis=1) != 0).all(axis=1)
    again, chosen = ask(z, k)
    assert apart.mean() > 0.9 and not again[apart].any()
    assert np.array_equal(chosen[apart], _order(z, k)[apart])


@pytest.mark.parametrize("e, k, live", [(64, 8, 5), (64, 8, 1), (60, 4, 3), (250, 8, 7), (1000, 6, 6)])
def test_not_made_again_for_experts_taken_out(ask, e, k, live):
    """Rows whose masks leave fewer than k experts, or just as many."""
    rng = np.random.default_rng(e + live)
    z = np.full((300, e), -INF)
    for row in z:
        row[rng.permutation(e)[:live]] = _normal(rng, 1, live)[0]
    bits = np.sort(np.where(z > -INF, _kept_bits(z), 0), axis=1)[:, -live:]
    apart = (np.diff(bits, axis=1) != 0).all(axis=1)
    again, chosen = ask(z, k)
    assert apart.mean() > 0.9 and not again[apart].any()
    assert np.array_equal(chosen[apart], _order(z, k)[apart])


@pytest.mark.parametrize("e", [64, 250])
def test_not_made_again_for_what_comes_behind_the_last_choice(ask, e):
    """Four largest far apart, all the others next to each other."""
    rng = np.random.default_rng(e)
    z = (np.float32(1.5).view(np.int32) + rng.integers(0, 2 * e, (100, e))).astype(np.int32).view(np.float32)
    for row in z:
        row[rng.permutation(e)[:4]] = rng.permutation(np.float32([3, 4, 5, 6]))
    again, chosen = ask(z, 4)
    assert not again.any() and np.array_equal(chosen, _order(z, 4))
    for k in (5, 8):                                       # they matter there
        assert ask(z, k)[0].any()


def test_not_made_again_for_neighbours_in_other_steps(ask):
    """Keys next to each other whose logits differ in the bits that the keys hold."""
    z = np.full((1, 64), -5.0, np.float32)
    z[0, :9] = np.arange(9, 0, -1)
    top = np.float32(20.0).view(np.int32)
    z[0, 63], z[0, 0] = (np.int32(top + 64)).view(np.float32), np.int32(top).view(np.float32)    # keys one apart
    again, chosen = ask(z, 4)
    assert not again.any() and chosen[0, :2].tolist() == [63, 0]
