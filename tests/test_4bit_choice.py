"""Which kernels the sizes of the 4-bit tests take, and that together they take all there
are: a rule that is tuned again and empties a test fails here."""
import pytest

from tests import cases_4bit as C
from tests import rules_4bit as R
from tests.segments import spec


def _holds(plan, want):
    got = plan._asdict()
    return {k: got[k] for k in want} == want, got


@pytest.mark.parametrize("name", C.PRODUCTS)
def test_products(name):
    (M, K, N, _), want = C.PRODUCTS[name]
    ok, got = _holds(R.product(M, K, N), want)
    assert ok, got


@pytest.mark.parametrize("name", C.EXPERTS)
def test_experts(name):
    (counts, d, f, _), *wants = C.EXPERTS[name]
    for plan, want in zip(R.experts(spec(counts, d, f, "bf16")), wants):
        ok, got = _holds(plan, want)
        assert ok, got


def test_every_kernel_has_a_case():
    plans = [(R.product(*s[:3]), s) for s, _ in C.PRODUCTS.values()]
    assert {(p.wide, p.low, p.waves, p.ahead) for p, _ in plans if not p.tiles} == {
        (False, True, 8, False), (False, True, 16, False), (False, False, 8, False), (True, True, 8, False),
        (True, False, 4, False), (True, True, 4, True), (True, False, 4, True)}
    for wide in (False, True):
        assert {s[3] for p, s in plans if not p.tiles and p.wide == wide} == {32, 64, 128}
    tiles = [(p, s) for p, s in plans if p.tiles]
    assert set().union(*(R.heights(s[0], p.bm) for p, s in tiles)) == {4, 6, 8, 10, 12}
    assert {s[3] for p, s in tiles if p.parts == 1} == {s[3] for p, s in tiles if p.parts > 1} == {32, 64, 128}
    assert any(-(-s[1] // 128) == 1 for _, s in tiles) and any(s[1] % 128 == 8 for _, s in tiles)
    gated, down = [], []
    for (counts, d, f, G), *_ in C.EXPERTS.values():
        u, v = R.experts(spec(counts, d, f, "bf16"))
        gated += [(u.tiles, G, h) for c in counts if c for h in R.heights(c, u.bm)]
        down += [(v.tiles, G)]
    assert {(t, G) for t, G, _ in gated} == {(t, G) for t in (False, True) for G in (32, 64, 128)} - {(False, 128)}
    assert {h for t, _, h in gated if t} == {4, 6, 8, 10, 12}
    assert {t for t, _ in down} == {False, True}


def test_parts_cover_all_of_k():
    for M in (1, 40, 65, 130, 300, 700, 2000):
        for K in (8, 136, 1032, 4104, 14344, 100000, 1 << 20):
            for N in (8, 264, 1032, 2040):
                p = R.product(M, K, N)
                kb = -(-K // 128)
                assert (p.parts - 1) * p.per < kb <= p.parts * p.per
                assert p.bm in (64, 128, 192) and p.blocks >= 1
                if p.tiles and p.parts > 1:   # the sums' place: bounded by what the tiles of a round hold
                    assert -(-M // p.bm) * -(-N // 256) * p.parts <= R.CUS
