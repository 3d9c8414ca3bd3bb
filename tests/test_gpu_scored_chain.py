"""Scored routing with what it is used with: a layer served with 4-bit experts, and a
training step with the router's gradient, each against 64 bits."""
import pytest
import torch

import combine_router_top_amd as M
from tests.segments import HALF, assert_within
from tests.test_gpu_scored import EPS, _choose, _grad, _scores

pytestmark = pytest.mark.gpu


def _layer(T, d, E, k, f, lo, n, dtype="bf16", seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    r = lambda *s, c=1.0: (torch.randn(s, generator=g) / c).to(dt)  # noqa: E731
    p = M.Spec(T, d, E, k, f, lo, n, dtype)
    return p, r(T, d), r(d, E, c=d ** 0.5), r(n, d, f, c=d ** 0.5), r(n, d, f, c=d ** 0.5), r(n, f, d, c=f ** 0.5), torch.randn(E, generator=g) * 0.1


@pytest.mark.parametrize("T,d,E,k,f,lo,n,G,zero", [(1, 256, 32, 8, 128, 0, 32, 128, False), (40, 264, 16, 4, 136, 4, 8, 64, True),
                                                   (300, 512, 64, 6, 264, 0, 64, 128, False), (900, 128, 8, 2, 256, 2, 5, 32, True)])
def test_served_layer(T, d, E, k, f, lo, n, G, zero):
    p, x, wg, w1, w3, w2, bal = _layer(T, d, E, k, f, lo, n)
    gate = M.Gate("sigmoid", 4, 2, 2, True, 2.5)
    packs = [M.quantize_weights_4bit(w.cuda(), G, zero) for w in (w1, w3, w2)]
    xd = x.cuda()
    idx, w, l = M.route_scored(p, gate, xd, wg.cuda(), None, bal.cuda(), want_logits=True)
    o = M.dispatch(p, idx, xd)
    h, yp = M.expert_gemm_4bit(p, o["x_packed"], o["offsets"], *(t for q in packs for t in q), group=G)
    y = M.combine(p, yp, o["inv"], w)
    ri, rw = _choose(gate, k, l.cpu(), bal)
    assert torch.equal(idx.cpu(), torch.from_numpy(ri))
    # the weights that the packed ones stand for, by a product with ones on the diagonal
    def back(q, e, K):
        eye = torch.eye(K, dtype=torch.bfloat16).cuda()
        return M.gemm_4bit(eye, q[0][e], q[1][e], q[2][e] if zero else None, group=G, dtype=torch.float32).cpu().double()
    full = [[back(q, e, K) for e in range(n)] for q, K in zip(packs, (d, d, f))]
    X, ref, tol = x.double(), torch.zeros(T, d, dtype=torch.float64), torch.zeros(T, d, dtype=torch.float64)
    half = HALF["bf16"]
    for t in range(T):
        for j in range(k):
            e = int(ri[t, j]) - lo
            if not 0 <= e < n:
                continue
            a, b = X[t] @ full[0][e], X[t] @ full[1][e]
            hh = a * torch.sigmoid(a) * b
            dh = half * hh.abs() + 64 * d * EPS * (X[t].abs() @ full[0][e].abs() * 1.1 * b.abs() + X[t].abs() @ full[1][e].abs() * a.abs())
            v = hh @ full[2][e]
            dv = dh @ full[2][e].abs() + half * v.abs() + 64 * f * EPS * (hh.abs() @ full[2][e].abs())
            ref[t] += rw[t, j] * v
            tol[t] += rw[t, j] * dv * (1 + half)
    assert_within(y, ref, tol + half * ref.abs() + (k + 64) * EPS * (tol + ref.abs()) + 1e-6 * tol, "y")


@pytest.mark.parametrize("gate", [M.Gate(), M.Gate("sigmoid", 4, 2, 2, True, 2.5), M.Gate("softmax", renorm=False)], ids=str)
def test_training_step_in_fp32_against_differences(gate):
    """The loss sum(y c) of a whole fp32 layer: gradients of rows and gate matrix by the
    calls, against differences of the layer in 64 bits with the choice held."""
    T, d, E, k, f = 12, 32, 8, 3, 24
    p, x, wg, w1, w3, w2, bal = _layer(T, d, E, k, f, 0, E, "f32", 5)
    dev = [v.cuda() for v in (x, wg, w1, w3, w2)]
    c = torch.randn((T, d), generator=torch.Generator().manual_seed(8))
    idx, w, l = M.route_scored(p, gate, dev[0], dev[1], None, bal.cuda(), want_logits=True)
    o = M.dispatch(p, idx, dev[0])
    g, u, h, yp = M.expert_gemm_train(p, o["x_packed"], o["offsets"], *dev[2:])
    y = M.combine(p, yp, o["inv"], w)
    dyp, dw = M.combine_backward(p, c.cuda(), yp, o["inv"], w)
    dxp = M.expert_gemm_backward(p, o["x_packed"], o["offsets"], *dev[2:], g, u, h, dyp)[0]
    through = M.combine(p, dxp, o["inv"], None)
    _, dx, dwg, db = M.route_backward(p, gate, dev[0], dev[1], l, idx, dw, dx_add=through)

    ix = idx.cpu().long()
    C = c.double()

    def forward(X, W, bias):
        s = _scores(gate, X @ W + bias).gather(1, ix)
        s = (s / s.sum(1, keepdim=True) if gate.renorm else s) * gate.scale
        out = torch.zeros_like(X)
        for e in range(E):
            a, b = X @ w1[e].double(), X @ w3[e].double()
            v = (a * torch.sigmoid(a) * b) @ w2[e].double()
            out += ((ix == e) * s).sum(1, keepdim=True) * v
        return out
    X, W, zero = x.double(), wg.double(), torch.zeros(E, dtype=torch.float64)
    # fp32 throughout: sums of at most 2 f + d + E terms in a chain of five products
    assert_within(y, forward(X, W, zero), torch.full((T, d), 2e-5, dtype=torch.float64), "y")
    eps = 1e-4
    near = lambda a: 3e-5 * (1 + a.abs())  # noqa: E731  differences: eps^2 / 6 of third derivatives below some hundreds
    num = torch.zeros_like(X)
    for i in range(d):
        step = torch.zeros_like(X)
        step[:, i] = eps
        num[:, i] = ((forward(X + step, W, zero) - forward(X - step, W, zero)) * C).sum(1) / (2 * eps)
    assert_within(dx, num, near(num), "dx")
    num = torch.zeros_like(W)
    for i in range(d):
        for e in range(E):
            step = torch.zeros_like(W)
            step[i, e] = eps
            num[i, e] = ((forward(X, W + step, zero) - forward(X, W - step, zero)) * C).sum() / (2 * eps)
    assert_within(dwg, num, near(num), "dw_gate")
    num = torch.zeros(E, dtype=torch.float64)
    for e in range(E):
        step = torch.zeros(E, dtype=torch.float64)
        step[e] = eps
        num[e] = ((forward(X, W, step) - forward(X, W, -step)) * C).sum() / (2 * eps)
    assert_within(db, num, near(num), "dbias")


def test_captured_training_step_of_the_router():
    """Routing, combine's and the router's backward pass in one graph, replayed on new rows."""
    T, d, E, k, f = 200, 264, 32, 4, 136
    gate = M.Gate("sigmoid", 4, 2, 2, True, 2.5)
    p, x, wg, w1, w3, w2, bal = _layer(T, d, E, k, f, 0, E)
    sets = [_layer(T, d, E, k, f, 0, E, seed=s)[1].cuda() for s in (0, 1)]
    wg, w1, w3, w2, bal = (v.cuda() for v in (wg, w1, w3, w2, bal))
    dy = torch.randn((T, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()

    def step(rows):
        idx, w, l = M.route_scored(p, gate, rows, wg, None, bal, want_logits=True)
        o = M.dispatch(p, idx, rows)
        g, u, h, yp = M.expert_gemm_train(p, o["x_packed"], o["offsets"], w1, w3, w2)
        dyp, dw = M.combine_backward(p, dy, yp, o["inv"], w)
        dxp = M.expert_gemm_backward(p, o["x_packed"], o["offsets"], w1, w3, w2, g, u, h, dyp)[0]
        return M.route_backward(p, gate, rows, wg, l, idx, dw, dx_add=M.combine(p, dxp, o["inv"], None)) + (idx, dw, l)
    want = [[v.clone() for v in step(s)] for s in sets]
    dl, size = _grad(gate, want[0][6].cpu(), want[0][4].cpu(), want[0][5].cpu())
    assert_within(want[0][0], dl, 96 * EPS * size + 1e-37, "dlogits")
    held = sets[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(held)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held)
    for i in (1, 0, 1):
        held.copy_(sets[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
