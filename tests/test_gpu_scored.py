"""Scored routing and the router's gradients against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import combine_router_top_amd as M
from tests.segments import HALF, assert_within, torch_dtype

EPS = 2.0 ** -23   # a fp32 operation that may truncate


def _logits(T, E, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=g) * 1.5
    if kind == "ties":         # few values: most comparisons are equal
        l = torch.randint(-2, 3, (T, E), generator=g).float()
    if kind == "close":        # neighbours in fp32, and sigmoids that fp32 cannot tell apart
        l = torch.where(torch.rand((T, E), generator=g) < 0.5, l.gather(1, torch.zeros((T, E), dtype=torch.int64)), l)
        l = torch.where(torch.rand((T, E), generator=g) < 0.3, torch.nextafter(l, torch.tensor(9.0)), l)
        l[:, E // 2:] = 15 + 2 * torch.rand((T, E - E // 2), generator=g)
    if kind == "masked":
        l[torch.rand((T, E), generator=g) < 0.4] = -math.inf
        l[:, : E // 3] = -math.inf
        l[T // 2] = -math.inf
    return l


def _scores(gate, l):
    l = l.double()
    if gate.score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
    s = e / e.sum(1, keepdim=True)
    return torch.where(top == -math.inf, 0.0, s)


def _choose(gate, k, l, balance):
    """The definition, a token at a time."""
    T, E = l.shape
    s = _scores(gate, l)
    c = s if balance is None else s + balance.double()
    dead = (l == -math.inf) | torch.isnan(c) | (c == -math.inf)
    order = l.double() if gate.score == "softmax" and balance is None else c
    idx = np.empty((T, k), dtype=np.int32)
    per = E // gate.groups
    for t in range(T):
        key = [(1, 0.0) if dead[t, e] else (0, -float(order[t, e])) for e in range(E)]   # ascending: best first
        open_ = range(E)
        if gate.groups > 1:
            value = []
            for q in range(gate.groups):
                best = sorted((-1e300 if dead[t, e] else float(c[t, e]) for e in range(q * per, q * per + per)), reverse=True)
                value.append(-sum(best[: gate.group_top]))
            stay = sorted(range(gate.groups), key=lambda q: (value[q], q))[: gate.topk_groups]
            open_ = sorted(e for q in stay for e in range(q * per, q * per + per))
        idx[t] = sorted(open_, key=lambda e: (key[e], e))[:k]
    top = s.gather(1, torch.from_numpy(idx).long())
    if gate.renorm:
        total = top.sum(1, keepdim=True)
        top = torch.where(total == 0, 0.0, top / total)
    return idx, top * gate.scale


def _spec(T, E, k, d=8, dtype="f32"):
    return M.Spec(T, d, E, k, 8, 0, E, dtype)


def _check_select(gate, k, l, balance, idx, w):
    ri, rw = _choose(gate, k, l, balance)
    assert np.array_equal(idx.cpu().numpy(), ri)
    # score, sum of at most k terms, division and scale in fp32; exp of an argument of some 40
    assert_within(w, rw, (k + 60) * EPS * rw.abs() + 1e-37, "weights")


RULES = [M.Gate(), M.Gate("sigmoid"), M.Gate("softmax", renorm=False, scale=2.5), M.Gate("sigmoid", renorm=False),
         M.Gate("sigmoid", 8, 4, 2, True, 2.5), M.Gate("softmax", 8, 3, 1), M.Gate("softmax", 4, 2, 2, False),
         M.Gate("sigmoid", 3, 2, 1), M.Gate("sigmoid", 64, 9, 2), M.Gate("softmax", 1, 1, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 7, 7), (5, 24, 4), (130, 64, 6), (9, 65, 8), (33, 192, 3), (300, 256, 8), (7, 384, 8),
                                   (5, 1000, 20), (2, 1024, 32)])
@pytest.mark.parametrize("gate", RULES, ids=str)
@pytest.mark.parametrize("bias", [False, True])
def test_select(T, E, k, gate, bias):
    if E % gate.groups or k > gate.topk_groups * (E // gate.groups) or (gate.groups > 1 and gate.group_top > E // gate.groups):
        pytest.skip("no such groups")
    kinds = ("normal", "ties", "close", "masked") if E > 1 else ("normal",)
    for seed, kind in enumerate(kinds):
        l = _logits(T, E, seed + E, kind)
        b = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.2 if bias else None
        if bias and kind == "ties":
            b = (b * 4).round() / 4
        if bias and kind == "masked":
            b[E // 2] = -math.inf
        idx, w = M.select(_spec(T, E, k), gate, l.cuda(), None if b is None else b.cuda())
        _check_select(gate, k, l, b, idx, w)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_values_that_are_not_finite_stay_in_their_row(score, bias):
    T, E, k = 12, 72, 6
    gate = M.Gate(score, 8, 4, 2)
    l = _logits(T, E, 5)
    l[1, 3], l[3, 40], l[5], l[7, 9] = math.nan, -math.nan, math.nan, math.inf
    l[9, 2], l[9, 30], l[11] = math.inf, math.nan, torch.from_numpy(np.full(E, 0xFFFFFFFF, np.uint32).view(np.float32).copy())
    b = torch.linspace(-0.1, 0.1, E) if bias else None
    idx, w = M.select(_spec(T, E, k), gate, l.cuda(), None if b is None else b.cuda())
    idx, w = idx.cpu(), w.cpu()
    assert int(idx.min()) >= 0 and int(idx.max()) < E
    assert all(len(set(r.tolist())) == k for r in idx)
    good = torch.isfinite(l).all(1)
    ri, rw = _choose(gate, k, l[good], b)
    assert np.array_equal(idx[good].numpy(), ri)
    assert_within(w[good], rw, (k + 60) * EPS * rw.abs() + 1e-37, "weights")
    if score == "softmax":
        assert bool(torch.isnan(w[~good]).all())


@pytest.mark.gpu
def test_same_rule_as_route():
    """Softmax scores renormalised over the selected: the library's first router."""
    for T, E, k, d, dtype in ((300, 256, 8, 256, "bf16"), (2000, 128, 8, 512, "bf16"), (40, 16, 2, 64, "bf16"), (17, 12, 3, 64, "f32"), (5, 96, 4, 1024, "bf16")):
        p = _spec(T, E, k, d, dtype)
        g = torch.Generator().manual_seed(T)
        x, wg = ((torch.randn(s, generator=g) / c).to(torch_dtype(dtype)).cuda() for s, c in (((T, d), 1), ((d, E), d ** 0.5)))
        b = torch.randn(E, generator=g).cuda()
        i0, w0, l0 = M.route(p, x, wg, b, want_logits=True)
        i1, w1, l1 = M.route_scored(p, M.Gate(), x, wg, b, want_logits=True)
        # deep splits of K are summed in another order
        assert_within(l1, l0.cpu().double(), 64 * EPS * (l0.abs() + 1).cpu().double(), "logits")
        ri, rw = _choose(M.Gate(), k, l1.cpu(), None)
        assert np.array_equal(i1.cpu().numpy(), ri)
        assert_within(w1, rw, (k + 60) * EPS * rw, "weights")
        same = (l0 == l1).all(1)
        assert torch.equal(i0[same], i1[same])
        i2, w2 = M.select(p, M.Gate(), l1)
        assert torch.equal(i1, i2) and torch.equal(w1, w2)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,d,dtype", [(1, 256, 8, 7168, "bf16"), (70, 256, 8, 512, "bf16"), (1100, 256, 8, 264, "bf16"), (33, 20, 4, 136, "bf16"),
                                           (50, 13, 3, 40, "bf16"), (9, 8, 2, 128, "f32"), (20, 1000, 9, 64, "f32")])
def test_route_scored(T, E, k, d, dtype):
    gate = M.Gate("sigmoid", 4 if E % 4 == 0 else 1, 2 if E % 4 == 0 else 1, 2 if E % 4 == 0 else 1, True, 2.5)
    p, dt = _spec(T, E, k, d, dtype), torch_dtype(dtype)
    g = torch.Generator().manual_seed(T + E)
    x, wg = ((torch.randn(s, generator=g) / c).to(dt) for s, c in (((T, d), 1), ((d, E), d ** 0.5)))
    b, bal = torch.randn(E, generator=g), torch.randn(E, generator=g) * 0.1
    idx, w, l = M.route_scored(p, gate, x.cuda(), wg.cuda(), b.cuda(), bal.cuda(), want_logits=True)
    X, W = x.double(), wg.double()
    assert_within(l, X @ W + b.double(), (d + 8) * EPS * (X.abs() @ W.abs() + b.double().abs()), "logits")
    _check_select(gate, k, l.cpu(), bal, idx, w)


@pytest.mark.gpu
def test_select_on_streams_and_in_graphs():
    p, gate = _spec(500, 256, 8), M.Gate("sigmoid", 8, 4, 2, True, 2.5)
    sets = [_logits(500, 256, s).cuda() for s in (1, 2, 3)]
    bal = (torch.randn(256, generator=torch.Generator().manual_seed(1)) * 0.1).cuda()
    want = [M.select(p, gate, l, bal) for l in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [M.select(p, gate, l, bal, stream=s) for l, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(want, got):
        assert torch.equal(a, c) and torch.equal(b, d)
    held = sets[0].clone()
    out = (torch.empty_like(want[0][0]), torch.empty_like(want[0][1]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        M.select(p, gate, held, bal, out=out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.select(p, gate, held, bal, out=out)
    for i in (1, 2, 0, 1):
        held.copy_(sets[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])


@pytest.mark.gpu
def test_empty_batch():
    p = _spec(0, 16, 2, 8, "bf16")
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    assert M.select(p, M.Gate(), e(0, 16))[0].shape == (0, 2)
    dwg, db = e(8, 16, dt=torch.bfloat16).fill_(3), e(16).fill_(3)
    M.route_backward(p, M.Gate(), e(0, 8, dt=torch.bfloat16), e(8, 16, dt=torch.bfloat16), e(0, 16), e(0, 2, dt=torch.int32),
                     e(0, 2), out=(e(0, 16), e(0, 8, dt=torch.bfloat16), dwg, db))
    assert not bool(dwg.any()) and not bool(db.any())


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
def _grad(gate, l, idx, dw):
    """dlogits by the formulas, in 64 bits, and the size of the terms it is a difference of."""
    l, g, idx = l.double(), dw.double() * gate.scale, idx.long()
    s = _scores(gate, l)
    top = s.gather(1, idx)
    if gate.renorm:
        total = top.sum(1, keepdim=True)
        p = torch.where(total == 0, 0.0, top / total)
        slope = 1 / (1 + torch.exp(l.gather(1, idx))) if gate.score == "sigmoid" else torch.ones_like(top)
        val = p * slope * (g - (g * p).sum(1, keepdim=True))
        size = p * slope * (g.abs() + (g.abs() * p).sum(1, keepdim=True))
    elif gate.score == "sigmoid":
        slope = 1 / (1 + torch.exp(l.gather(1, idx)))
        val = g * top * slope
        size = val.abs()
    else:
        dense = torch.zeros_like(s).scatter_(1, idx, g)
        m, am = (g * top).sum(1, keepdim=True), (g.abs() * top).sum(1, keepdim=True)
        return s * (dense - m), s * (dense.abs() + am)
    return torch.zeros_like(s).scatter_(1, idx, val), torch.zeros_like(s).scatter_(1, idx, size)


@pytest.mark.parametrize("gate", [M.Gate(s, renorm=r, scale=c) for s in ("softmax", "sigmoid") for r in (True, False) for c in (1.0, 2.5)], ids=str)
def test_formulas_against_differences(gate):
    """sum(dtopk_w * topk_w) moved by a step of each logit, the choice held."""
    T, E, k = 6, 11, 4
    l = _logits(T, E, 3).double()
    idx = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(T)])
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(9)).double()

    def loss(v):
        top = _scores(gate, v).gather(1, idx)
        if gate.renorm:
            top = top / top.sum(1, keepdim=True)
        return (top * gate.scale * dw).sum(1)
    dl, _ = _grad(gate, l, idx, dw)
    h = 1e-5
    for e in range(E):
        step = torch.zeros_like(l)
        step[:, e] = h
        # the third derivative of a score is below 1, of a ratio of k of them below 10 k
        assert_within(dl[:, e], (loss(l + step) - loss(l - step)) / (2 * h), torch.full((T,), 1e-7, dtype=torch.float64), f"logit {e}")


def _back_inputs(T, E, k, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + T + E)
    dt = torch_dtype(dtype)
    l = _logits(T, E, seed + 7)
    idx = torch.rand((T, E), generator=g).argsort(1)[:, :k].to(torch.int32).contiguous()
    dw = torch.randn((T, k), generator=g)
    x, wg, add = ((torch.randn(s, generator=g) / c).to(dt) for s, c in (((T, d), 1), ((d, E), d ** 0.5), ((T, d), 1)))
    return l, idx, dw, x, wg, add


def _check_back(gate, dtype, inputs, out, add=None):
    l, idx, dw, x, wg, _ = inputs
    T, E = l.shape
    dl, size = _grad(gate, l, idx, dw)
    # sums over E by a lane and then the wave (at most 16 + 6 additions each), exponentials
    # of arguments up to about 20 (20 half-steps) and some twenty single operations
    slack = 96 * EPS * size + 1e-37
    got, dx, dwg, db = out
    if got is not None:
        assert_within(got, dl, slack, "dlogits")
    half = HALF[dtype]
    X, W = x.double(), wg.double()
    off = slack + (half if dtype == "bf16" else 0) * dl.abs()   # dl as the products take it
    if dx is not None:
        ref = dl @ W.T
        tol = off @ W.abs().T + E * EPS * (dl.abs() @ W.abs().T)
        if add is not None:
            ref = ref + add.double()
            tol = tol + 2 * EPS * (ref.abs() + add.double().abs())
        assert_within(dx, ref, tol * (1 + half) + half * ref.abs() + 1e-37, "dx")
    if dwg is not None:
        ref = X.T @ dl
        tol = X.abs().T @ off + (T + 64) * EPS * (X.abs().T @ dl.abs())
        assert_within(dwg, ref, tol * (1 + half) + half * ref.abs() + 1e-37, "dw_gate")
    if db is not None:
        assert_within(db, dl.sum(0), slack.sum(0) + T * EPS * dl.abs().sum(0) + 1e-37, "dbias")


BACK = [(1, 8, 2, 8, "f32"), (64, 8, 2, 128, "f32"), (33, 13, 3, 40, "f32"), (130, 256, 8, 72, "f32"), (700, 65, 6, 136, "f32"),
        (1, 256, 8, 7168, "bf16"), (5, 1, 1, 8, "bf16"), (70, 13, 3, 40, "bf16"), (300, 256, 8, 512, "bf16"), (1003, 24, 4, 1032, "bf16"),
        (2050, 72, 6, 264, "bf16"), (40, 1000, 9, 128, "bf16"), (257, 384, 32, 520, "bf16"), (5000, 16, 2, 96, "bf16")]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,d,dtype", BACK)
@pytest.mark.parametrize("gate", [M.Gate(), M.Gate("softmax", renorm=False, scale=2.5), M.Gate("sigmoid", scale=2.5), M.Gate("sigmoid", renorm=False)], ids=str)
def test_route_backward(T, E, k, d, dtype, gate):
    inputs = _back_inputs(T, E, k, d, dtype)
    l, idx, dw, x, wg, add = inputs
    dev = [v.cuda() for v in inputs]
    p = _spec(T, E, k, d, dtype)
    out = M.route_backward(p, gate, dev[3], dev[4], dev[0], dev[1], dev[2])
    _check_back(gate, dtype, inputs, out)
    again = M.route_backward(p, gate, dev[3], dev[4], dev[0], dev[1], dev[2])
    assert all(torch.equal(a, b) for a, b in zip(out, again))   # bitwise reproducible
    added = M.route_backward(p, gate, dev[3], dev[4], dev[0], dev[1], dev[2], dx_add=dev[5])
    _check_back(gate, dtype, inputs, added, add)
    place = dev[5].clone()   # the sum in place, nothing else wanted
    M.route_backward(p, gate, None, dev[4], dev[0], dev[1], dev[2], dx_add=place, out=(None, place, None, None))
    assert torch.equal(place, added[1])
    for i in (0, 2, 3):      # each other output alone
        one = [None] * 4
        one[i] = torch.full_like(out[i], 7)
        M.route_backward(p, gate, dev[3] if i == 2 else None, None, dev[0], dev[1], dev[2], out=one)
        assert torch.equal(one[i], out[i]), i


@pytest.mark.gpu
def test_masked_and_saturated_logits_have_finite_gradients():
    T, E, k, d = 40, 64, 6, 64
    for gate in (M.Gate(), M.Gate("softmax", renorm=False), M.Gate("sigmoid"), M.Gate("sigmoid", renorm=False)):
        inputs = list(_back_inputs(T, E, k, d, "bf16"))
        l = inputs[0]
        l[torch.rand((T, E), generator=torch.Generator().manual_seed(3)) < 0.3] = -math.inf
        l[4] = -math.inf
        l[6] = 60.0
        l[7] = -90.0          # every sigmoid below fp32's range, their ratios are not
        l[8, :32] = 300.0
        inputs[0] = l
        dev = [v.cuda() for v in inputs]
        out = M.route_backward(_spec(T, E, k, d, "bf16"), gate, dev[3], dev[4], dev[0], dev[1], dev[2])
        assert all(bool(torch.isfinite(o).all()) for o in out)
        keep = torch.ones(T, dtype=torch.bool)
        keep[7] = gate.score == "softmax" or gate.renorm      # a score that fp32 rounds to a subnormal
        dl, size = _grad(gate, l, inputs[1], inputs[2])
        assert_within(out[0].cpu()[keep], dl[keep], (96 * EPS * size + 1e-37)[keep] * 16, "dlogits")


@pytest.mark.gpu
def test_route_backward_in_graphs_and_on_streams():
    T, E, k, d = 600, 72, 6, 264
    p, gate = _spec(T, E, k, d, "bf16"), M.Gate("sigmoid", 8, 4, 2, True, 2.5)
    sets = [[v.cuda() for v in _back_inputs(T, E, k, d, "bf16", s)] for s in (0, 1)]
    want = [M.route_backward(p, gate, s[3], s[4], s[0], s[1], s[2], dx_add=s[5]) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [M.route_backward(p, gate, s[3], s[4], s[0], s[1], s[2], dx_add=s[5], stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
    held = [v.clone() for v in sets[0]]
    out = tuple(torch.empty_like(v) for v in want[0])
    ws = M.alloc_workspace(p, M.MOE_CALL_ROUTE_BACKWARD)
    call = lambda: M.route_backward(p, gate, held[3], held[4], held[0], held[1], held[2], dx_add=held[5], workspace=ws, out=out)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in (1, 0, 1):
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
