"""Which kernels the sizes of the GPU tests take: every case of tests/kernel_cases.py
takes the one it is there for, and together the tests reach every one there is.  A
rule that is tuned again and empties a test fails here."""
import pytest

from tests import kernel_cases as C
from tests import kernel_rules as R
from tests import test_gpu_quantized as Q
from tests import test_gpu_training as T
from tests.segments import spec


def _holds(plan, want):
    got = plan if isinstance(plan, dict) else plan._asdict()
    return {k: got[k] for k in want} == want, got


def _training_plan(p, **kw):
    return {**R.train(p)._asdict(), **R.backward(p, **kw)._asdict()}


@pytest.mark.parametrize("name", C.TRAINING)
def test_training(name):
    case = C.TRAINING[name]
    ok, got = _holds(_training_plan(C.problem(case)), case[4])
    assert ok, got
    if name.startswith("rotated"):
        assert case[2] * 2 % 4096 == 0 and got["input"] != 4
    if name.startswith("units"):   # a run that does not divide the row blocks, or several whole ones
        blocks, runs = -(-case[1] // 256), -(-(-(-case[1] // 256)) // got["div"])
        assert runs > 1 and -(-blocks // runs) == got["div"]


@pytest.mark.parametrize("name", C.QUANTIZED)
def test_quantized(name):
    case = C.QUANTIZED[name]
    for plan, want in zip(R.experts(C.problem(case)), case[4:]):
        ok, got = _holds(plan, want)
        assert ok, got
    if name.startswith("split"):
        assert any(0 < c <= 32 for c in case[0]) and any(c > 32 for c in case[0])
    if name.startswith("blocks"):
        assert max(case[0]) > 96   # all four workgroups of a segment have a block


@pytest.mark.parametrize("name", C.PRODUCTS)
def test_products(name):
    size, want = C.PRODUCTS[name]
    ok, got = _holds(R.product(*size), want)
    assert ok, got


def test_every_training_kernel_has_a_case():
    plans = [_training_plan(spec(c, d, f, dt, **kw)) for c, d, f, dt, kw in T.CASES.values() if dt == "bf16"]
    plans += [_training_plan(C.problem(c)) for c in C.TRAINING.values()]
    for part in ("up", "down", "gate"):
        assert {p[part] for p in plans} == {1, 2, 3, 4}, part
    assert {(p["input"], p["mode"]) for p in plans} == {(h, m) for h in (1, 2, 3, 4)
                                                        for m in (R.WG_LONG, R.WG_SHORT, R.WG_SPLIT)}
    assert {p["div"] for p in plans if p["mode"] == R.WG_SHORT} == {1, 2, 3, 4}
    assert {p["apart"] for p in plans} == {0, 1}


def test_every_8_bit_kernel_has_a_case():
    pairs = [R.experts(spec(c, d, f, "bf16", **kw)) for c, d, f, kw in Q.CASES.values()]
    pairs += [R.experts(C.problem(c)) for c in C.QUANTIZED.values()]
    alone = [R.product(*s) for s in Q.SIZES] + [R.product(*s) for s, _ in C.PRODUCTS.values()]
    gated, down = ([pair[i] for pair in pairs] for i in (0, 1))
    for plans in (gated, down, alone):
        assert {(p.wide, p.low) for p in plans if p.stream} == {(0, 0), (0, 1), (1, 0), (1, 1)}
        assert {p.height for p in plans if p.tiles} == {1, 2, 3, 4}
    for plans in (gated, down):
        assert {(p.wide, p.tiles) for p in plans if p.stream} == {(0, 0), (0, 1), (1, 0), (1, 1)}
        assert {p.wide for p in plans if p.stream and not p.tiles and p.blocks > 1} == {0, 1}


def test_no_workgroups_without_work():
    """Beside tiles a streamed segment has one block of 32 rows: one workgroup for it."""
    for case in C.QUANTIZED.values():
        for plan in R.experts(C.problem(case)):
            if plan.stream and plan.tiles:
                assert plan.blocks == 1
