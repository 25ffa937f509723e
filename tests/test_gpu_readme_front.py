"""The README's example of the operators in front of the projections runs as written and gives what it says."""

import os
import re

import pytest
import torch

from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_front_example_runs():
    require_gpu()
    text = open(os.path.join(ROOT, "README.md")).read()
    block = re.search(r"## In front of the projections\n.*?```python\n(.*?)```", text, re.S).group(1)
    ns = {}
    exec(compile(block, "README.md (In front of the projections)", "exec"), ns)
    torch.cuda.synchronize()
    t, d, e, f, k = (ns[n] for n in "TDEFk")
    assert ns["rows"].shape == (t, k, f) and bool(torch.isfinite(ns["rows"].float()).all())
    # the products of one expert's tokens, from the normed values themselves: FP8's rounding of both operands apart
    rows = ns["token_of_row"][:128].long()
    live = rows >= 0
    want = ns["y"][rows[live]].double() @ ns["w_experts"][:f].double().t()
    got = ns["out"][:128][live].double()
    assert int(ns["group_of_mtile"][0]) == 0 and float((got - want).norm() / want.norm()) < 2 * 2.0 ** -4
    assert float((ns["weights"].sum(1) - 1).abs().max()) < 1e-5 and int(ns["counts"].sum()) == t * k
    # rounding of a sum of rows of dz: each row's is zero
    assert float(ns["d_logits"].float().sum(1).abs().max()) < 64 * 2.0 ** -8 * float(ns["d_logits"].float().abs().max())
    assert ns["dx"].shape == (t, d) and ns["d_gain"].shape == (d,) and ns["qx_t"].shape == (d, t) and ns["q8"].shape == (16, d)
