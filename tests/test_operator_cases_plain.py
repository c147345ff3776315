"""The plain forms and the 64-bit definitions of the operators' cases, on the CPU: every index in range, and whole numbers equal.

(On a GPU an index out of range ends the process; here it is an error that names its line.)"""
import math
import os
import random
import types

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cases():
    path = os.path.join(ROOT, "perf", "more_operators.py")
    with open(path) as f:
        text = f.read().replace('device="cuda"', 'device="cpu"')
    assert '"cuda"' not in text
    m = types.ModuleType("more_operators_on_the_cpu")
    exec(compile(text, path, "exec"), m.__dict__)
    return m


def same(m, case, seed):
    got = m.run(m.prepare(case, seed))
    want = m.exact(case, seed)
    for x, y in zip(got, want, strict=True):
        assert x.shape == y.shape
        if not y.is_floating_point():
            assert torch.equal(x.long(), y.long()), case
        else:
            assert torch.allclose(x.double(), y, rtol=0.02, atol=0.02, equal_nan=True), case


# pools in which no sequence holds a page yet, or all do; one sequence; tables of one page
PLANS = [dict(seqs=2, length=5, new=1999, page=128, spare=1.0), dict(seqs=1, length=1, new=1, page=16, spare=1.0),
         dict(seqs=1, length=1, new=300, page=16, spare=0.5), dict(seqs=3, length=40, new=2, page=64, spare=0.8),
         dict(seqs=7, length=200, new=90, page=16, spare=0.5), dict(seqs=40, length=90, new=33, page=32, spare=0.8)]


@pytest.mark.parametrize("i", range(len(PLANS)))
def test_plans(cases, i):
    case = dict(PLANS[i], op="plan")
    for seed in range(4):
        same(cases, case, seed)


def test_plans_without_kept_tokens(cases, monkeypatch):
    """All pages are free before the step, and again after what it took is given back."""
    case = dict(op="plan", seqs=3, length=10, new=50, page=16, spare=1.0)
    monkeypatch.setattr(cases, "_plan_lengths", lambda case, seed: ([0, 0, 0], [50, 1, 17]))
    same(cases, case, 0)


def test_drawn_cases(cases):
    rng = random.Random(5)
    seen = {}
    for _ in range(4000):
        case = cases.draw(rng)
        size = {"plan": case["seqs"] * case.get("new", 1) if case["op"] == "plan" else 0}.get(case["op"])
        if case["op"] in ("append", "rope"):
            size = case["rows"] * case["heads"] * case["dim"] // 4
        if case["op"] in ("window", "tree"):
            size = case["seqs"] * case["rows"] * case["heads"] * case["length"] * math.isqrt(case["dim"]) // 100
        if size > 20000 or seen.get(case["op"], 0) >= 12:
            continue
        seen[case["op"]] = seen.get(case["op"], 0) + 1
        same(cases, case, seen[case["op"]])
    assert min(seen.get(op, 0) for op in ("plan", "append", "rope", "window", "tree")) >= 6, seen
