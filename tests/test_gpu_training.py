"""The experts in training: kept forward pass, gradients, combine's gradient,
and the whole layer's gradient through dispatch and combine.

References are the formulas in 64 bits.  Tolerances per element:
  half a step of the output type (2^-8 bf16, 2^-24 fp32) of the value, plus
  half a step for each rounded operand times the sum of absolute products, plus
  K 2^-23 times that sum for the fp32 additions (segments.dot_slack).
The exponential and reciprocal of the activations are good to a few fp32 ulp:
2^-20 relative is allowed for an activation or its derivative.
"""
import numpy as np
import pytest
import torch

import combine_router_top_amd as M
from tests.segments import HALF, SENTINEL, Rows, assert_within, dot_slack, offsets_of, spec

pytestmark = pytest.mark.gpu

ACT = 2.0 ** -20

CASES = {
    # name: (counts, d, f, dtype, spec arguments)
    "one_row": ([1], 64, 64, "bf16", {}),
    "narrow": ([3, 0, 2], 8, 8, "bf16", {}),
    "ragged": ([0, 5, 130, 1, 0, 257], 264, 200, "bf16", {}),        # K tails in every product
    "ragged_whole_k": ([31, 32, 33, 127, 128, 129], 256, 320, "bf16", {}),
    "long": ([700, 0, 300], 136, 72, "bf16", {}),                    # 256-row tiles, K tails
    "long_whole_k": ([513, 255, 256], 288, 544, "bf16", {}),
    "one_long": ([1100], 520, 264, "bf16", {}),
    "mid_k": ([70, 64], 96, 416, "bf16", {}),                        # 3 and 13 stages of K
    # enough tiles for the 256-, 192- and 128-row kernels (fewer take 64-row tiles,
    # as all the others here do), with and without K tails
    "tall_many": ([400 + (37 * e) % 200 - 100 for e in range(64)], 264, 264, "bf16", dict(T=1600, k=16)),
    "tall_many_whole_k": ([400 - (53 * e) % 200 + 100 for e in range(64)], 512, 512, "bf16", dict(T=1600, k=17)),
    "mid_many": ([150 + (29 * e) % 140 - 70 for e in range(128)], 264, 328, "bf16", dict(T=750, k=26)),
    "mid_many_whole_k": ([150 + (31 * e) % 140 - 70 for e in range(128)], 384, 320, "bf16", dict(T=750, k=26)),
    "low_many": ([80 + (23 * e) % 90 - 45 if e % 7 else 0 for e in range(100)], 328, 264, "bf16", dict(T=320, k=25)),
    "low_many_whole_k": ([80 + (19 * e) % 90 - 45 for e in range(100)], 384, 320, "bf16", dict(T=320, k=25)),
    "one_wide": ([2000], 2312, 2568, "bf16", {}),
    # rounds of long tiles: input and weight gradients apart
    "long_many": ([500 + (31 * e) % 41 for e in range(172)], 264, 264, "bf16", dict(T=2800, k=32)),
    "one_deep": ([2000], 4360, 1416, "bf16", {}),
    "many_experts": ([(7 * e) % 5 for e in range(150)], 40, 48, "bf16", dict(T=40, k=8)),
    "no_rows": ([0, 0, 0], 64, 72, "bf16", dict(T=5, k=2)),
    "part_of_experts": ([9, 40, 0, 3], 72, 136, "bf16", dict(T=64, k=2, E=16)),
    "f32_one_row": ([1], 8, 8, "f32", {}),
    "f32_ragged": ([0, 5, 130, 1, 65], 72, 136, "f32", {}),
    "f32_no_rows": ([0, 0], 16, 24, "f32", dict(T=3, k=1)),
}


def _case(name):
    counts, d, f, dtype, kw = CASES[name]
    p = spec(counts, d, f, dtype, **kw)
    r = Rows(p, counts, seed=sum(map(ord, name)))
    n = len(counts)
    v = dict(x=r.draw(r.A, d), w1=r.draw(n, d, f, scale=d ** -0.5), w3=r.draw(n, d, f, scale=d ** -0.5),
             w2=r.draw(n, f, d, scale=f ** -0.5))
    return p, r, v


def _check_forward(p, r, v, got):
    half = HALF[p.dtype]
    for e, s in r.segments():
        x = v["x"][s]
        a, b = x @ v["w1"][e], x @ v["w3"][e]
        ea, eb = dot_slack(x, v["w1"][e]), dot_slack(x, v["w3"][e])
        assert_within(got[0][s], a, half * a.abs() + 2 * ea, "g")
        assert_within(got[1][s], b, half * b.abs() + 2 * eb, "u")
        sig = torch.sigmoid(a)
        act = a * sig
        h = act * b
        # |SiLU'| <= 1.1
        eh = 1.1 * ea * b.abs() + act.abs() * eb + 1.1 * ea * eb + ACT * h.abs()
        assert_within(got[2][s], h, (half + 2 * ACT) * h.abs() + 2 * eh, "h")
        # the down projection from the h that was stored
        hs = got[2][s].cpu().double()
        y = hs @ v["w2"][e]
        assert_within(got[3][s], y, half * y.abs() + 2 * dot_slack(hs, v["w2"][e]), "y")


@pytest.mark.parametrize("name", CASES)
def test_train_forward(name):
    p, r, v = _case(name)
    outs = (r.out(p.f), r.out(p.f), r.out(p.f), r.out(p.d))
    got = M.expert_gemm_train(p, r.packed(v["x"]), offsets_of(r.counts), r.dev(v["w1"]), r.dev(v["w3"]),
                              r.dev(v["w2"]), out=outs)
    torch.cuda.synchronize()
    r.check_tail(*got)
    _check_forward(p, r, v, got)


@pytest.mark.parametrize("name", ["ragged", "long", "one_row", "mid_many", "f32_ragged"])
def test_train_forward_agrees_with_expert_gemm(name):
    """h of both calls: the same formula over fp32 sums that may run in another
    order, so each is within half a step and its sums' error of the exact value."""
    p, r, v = _case(name)
    args = (r.packed(v["x"]), offsets_of(r.counts), r.dev(v["w1"]), r.dev(v["w3"]), r.dev(v["w2"]))
    h, _ = M.expert_gemm(p, *args)
    _, _, h2, _ = M.expert_gemm_train(p, *args)
    for e, s in r.segments():
        x = v["x"][s]
        a, b = x @ v["w1"][e], x @ v["w3"][e]
        ea, eb = dot_slack(x, v["w1"][e]), dot_slack(x, v["w3"][e])
        act = (a * torch.sigmoid(a)).abs()
        eh = 1.1 * ea * b.abs() + act * eb + 1.1 * ea * eb + ACT * (act * b.abs())
        tol = 2 * ((HALF[p.dtype] + 2 * ACT) * (act * b.abs()) + 2 * eh)
        assert_within(h2[s], h[s].cpu().double(), tol, "h")


def _backward_inputs(r, v, p):
    g, u = r.draw(r.A, p.f), r.draw(r.A, p.f)
    h = (g * torch.sigmoid(g) * u).to(r.dt).double()
    return g, u, h, r.draw(r.A, p.d)


def _check_backward(p, r, v, g, u, h, dy, got):
    half = HALF[p.dtype]
    # dg and du are rounded to the storage type; fp32 keeps them as computed
    for e, s in r.segments():
        w1, w3, w2 = v["w1"][e], v["w3"][e], v["w2"][e]
        dh, edh = dy[s] @ w2.T, dot_slack(dy[s], w2.T)
        sig = torch.sigmoid(g[s])
        fg, fu = u[s] * sig * (1 + g[s] * (1 - sig)), g[s] * sig
        dg, du = dh * fg, dh * fu
        # 1 - s loses relative but not absolute precision: its error is 2^-23 g u s dh at most
        eg = half * dg.abs() + 2 * edh * fg.abs() + ACT * (dh * u[s] * sig).abs() * (1 + g[s].abs())
        eu = half * du.abs() + 2 * edh * fu.abs() + ACT * du.abs()
        dx = dg @ w1.T + du @ w3.T
        if got[0] is not None:
            tol = (half * dx.abs() + (1 + half) * (eg @ w1.T.abs() + eu @ w3.T.abs())
                   + 2 * (dot_slack(dg, w1.T) + dot_slack(du, w3.T)) + p.f * 2.0 ** -23 * dx.abs())
            assert_within(got[0][s], dx, tol, "dx")
        x = v["x"][s]
        for k, (left, right, er, what) in enumerate(((x, dg, eg, "dw1"), (x, du, eu, "dw3"), (h[s], dy[s], None, "dw2"))):
            if got[k + 1] is None:
                continue
            ref = left.T @ right
            tol = half * ref.abs() + 2 * dot_slack(left.T, right)
            if er is not None:
                tol = tol + (1 + half) * (left.T.abs() @ er)
            assert_within(got[k + 1][e], ref, tol, what)


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    p, r, v = _case(name)
    g, u, h, dy = _backward_inputs(r, v, p)
    n = len(r.counts)
    outs = (r.out(p.d),) + tuple(torch.full(s, float("nan"), dtype=r.dt, device="cuda")
                                 for s in ((n, p.d, p.f), (n, p.d, p.f), (n, p.f, p.d)))
    got = M.expert_gemm_backward(p, r.packed(v["x"]), offsets_of(r.counts), r.dev(v["w1"]), r.dev(v["w3"]),
                                 r.dev(v["w2"]), r.packed(g), r.packed(u), r.packed(h), r.packed(dy), out=outs)
    torch.cuda.synchronize()
    r.check_tail(got[0])
    _check_backward(p, r, v, g, u, h, dy, got)


@pytest.mark.parametrize("name", ["ragged", "one_long", "f32_ragged"])
@pytest.mark.parametrize("wanted", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (1, 0, 1, 1)])
def test_backward_some_outputs(name, wanted):
    p, r, v = _case(name)
    g, u, h, dy = _backward_inputs(r, v, p)
    n = len(r.counts)
    shapes = (None, (n, p.d, p.f), (n, p.d, p.f), (n, p.f, p.d))
    outs = tuple(None if not w else r.out(p.d) if i == 0 else torch.full(shapes[i], float("nan"), dtype=r.dt, device="cuda")
                 for i, w in enumerate(wanted))
    got = M.expert_gemm_backward(p, r.packed(v["x"]), offsets_of(r.counts), r.dev(v["w1"]), r.dev(v["w3"]),
                                 r.dev(v["w2"]), r.packed(g), r.packed(u), r.packed(h), r.packed(dy), out=outs)
    torch.cuda.synchronize()
    _check_backward(p, r, v, g, u, h, dy, got)


@pytest.mark.parametrize("name", ["ragged", "f32_ragged"])
def test_backward_extreme_gates(name):
    """Gates far out on both sides: s is 0 or 1 there and nothing turns into NaN."""
    p, r, v = _case(name)
    g, u, h, dy = _backward_inputs(r, v, p)
    far = torch.tensor([-3e38, -1e4, -200.0, -90.0, 90.0, 200.0, 1e4, 3e38], dtype=torch.float64).to(r.dt).double()
    g[:, : far.numel()] = far
    u[:, : far.numel()] = u[:, : far.numel()].sign()
    got = M.expert_gemm_backward(p, r.packed(v["x"]), offsets_of(r.counts), r.dev(v["w1"]), r.dev(v["w3"]),
                                 r.dev(v["w2"]), r.packed(g), r.packed(u), r.packed(h), r.packed(dy),
                                 out=(None, torch.empty((len(r.counts), p.d, p.f), dtype=r.dt, device="cuda"), None, None))
    torch.cuda.synchronize()
    s = torch.sigmoid(g)
    for e, seg in r.segments():
        dg = (dy[seg] @ v["w2"][e].T) * u[seg] * s[seg] * (1 + g[seg] * (1 - s[seg]))
        dg[:, : far.numel()] = (dy[seg] @ v["w2"][e].T)[:, : far.numel()] * u[seg][:, : far.numel()] * (far > 0)
        ref = v["x"][seg].T @ dg
        tol = (HALF[p.dtype] * (ref.abs() + 1.1 * (v["x"][seg].T.abs() @ dg.abs()))
               + 3 * dot_slack(v["x"][seg].T, dg)
               + v["x"][seg].T.abs() @ (2 * dot_slack(dy[seg], v["w2"][e].T) * (1 + u[seg].abs()) * 1.1
                                        + ACT * (1 + g[seg].abs().clamp(max=100)) * dg.abs().clamp(min=1e-6)
                                        + ACT * ((dy[seg] @ v["w2"][e].T) * u[seg]).abs()))
        assert_within(got[1][e], ref, tol, "dw1")


def test_backward_empty_batch():
    for dtype in ("bf16", "f32"):
        p = M.Spec(0, 64, 4, 2, 40, 0, 3, dtype)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        z = lambda *s: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        outs = (z(0, 64), *(torch.full(s, float("nan"), dtype=dt, device="cuda")
                            for s in ((3, 64, 40), (3, 64, 40), (3, 40, 64))))
        M.expert_gemm_backward(p, z(0, 64), torch.zeros(4, dtype=torch.int32, device="cuda"), z(3, 64, 40),
                               z(3, 64, 40), z(3, 40, 64), z(0, 40), z(0, 40), z(0, 40), z(0, 64), out=outs)
        torch.cuda.synchronize()
        assert all(bool((o == 0).all()) for o in outs[1:])


def test_backward_empty_batch_rows_alone():
    """Only dx_packed wanted of an empty batch: nothing to do, and no refusal."""
    p = M.Spec(0, 64, 4, 2, 40, 0, 3, "bf16")
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    out = M.expert_gemm_backward(p, z(0, 64), torch.zeros(4, dtype=torch.int32, device="cuda"), z(3, 64, 40), z(3, 64, 40),
                                 z(3, 40, 64), z(0, 40), z(0, 40), z(0, 40), z(0, 64), out=(z(0, 64), None, None, None))
    assert out[0].shape == (0, 64) and out[1:] == (None, None, None)


def _slots(T, k, n, E, seed):
    rng = np.random.default_rng(seed)
    inv = np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        c = rng.choice(E, k, replace=False)
        inv[t][c < n] = 0
    at = np.argwhere(inv.ravel() == 0).ravel()
    flat = inv.ravel()
    flat[at] = rng.permutation(len(at)).astype(np.int32)
    return flat, len(at)


@pytest.mark.parametrize("T,k,n,E,d,dtype", [
    (1, 1, 1, 1, 8, "bf16"), (7, 4, 3, 12, 264, "bf16"), (64, 2, 8, 8, 4096, "bf16"), (33, 32, 64, 64, 72, "bf16"),
    (5, 8, 32, 256, 7168, "bf16"), (9, 3, 2, 5, 8200, "bf16"), (6, 2, 2, 4, 24584, "bf16"),
    (11, 4, 3, 6, 136, "f32"), (3, 2, 2, 2, 4104, "f32"), (40, 1, 1, 16, 64, "bf16")])
def test_combine_backward(T, k, n, E, d, dtype):
    inv, A = _slots(T, k, n, E, seed=T + d)
    p = M.Spec(T, d, E, k, 8, 0, n, dtype)
    r = Rows(p, [A], seed=d)
    r.A = A
    dy, yp = r.draw(T, d), r.draw(A, d)
    w = torch.rand((T, k), generator=r.gen)
    di = torch.from_numpy(inv).cuda()
    dyp, dw = M.combine_backward(p, r.dev(dy), r.packed(yp), di, w.cuda(), out=(r.out(d), torch.full((T, k), 9.0, device="cuda")))
    torch.cuda.synchronize()
    r.check_tail(dyp)
    iv = torch.from_numpy(inv).long().view(T, k)
    for t in range(T):
        for j in range(k):
            row = int(iv[t, j])
            if row < 0:
                assert float(dw[t, j]) == 0.0
                continue
            ref = w[t, j].double() * dy[t]
            # the fp32 product and its rounding
            assert_within(dyp[row], ref, (HALF[dtype] + 2.0 ** -23) * ref.abs(), "dy_packed")
            dot = (dy[t] * yp[row]).sum()
            tol = d * 2.0 ** -23 * (dy[t] * yp[row]).abs().sum()
            assert abs(float(dw[t, j]) - dot) <= tol, (t, j)
    # unit weights, and the rows alone
    one, none = M.combine_backward(p, r.dev(dy), None, di, None, out=(r.out(d), None))
    torch.cuda.synchronize()
    assert none is None
    for t in range(T):
        for j in range(k):
            if iv[t, j] >= 0:
                assert torch.equal(one[int(iv[t, j])].cpu(), dy[t].to(r.dt))


def _layer64(x, w1, w3, w2, idx, w, lo, n):
    """y of the MoE layer with fixed routing, float64, autograd on."""
    y = torch.zeros_like(x)
    for e in range(n):
        t, j = torch.nonzero(idx == lo + e, as_tuple=True)
        if t.numel():
            xe = x[t]
            a = xe @ w1[e]
            out = (a * torch.sigmoid(a) * (xe @ w3[e])) @ w2[e]
            y = y.index_add(0, t, w[t, j][:, None] * out)
    return y


@pytest.mark.parametrize("dtype,T,d,f", [("f32", 50, 72, 56), ("bf16", 300, 136, 200)])
def test_layer_training_step(dtype, T, d, f):
    """dispatch, experts, combine and their gradients together, against autograd
    in 64 bits and against differences of the layer in 64 bits."""
    E, k, lo, n = 8, 3, 2, 5
    p = M.Spec(T, d, E, k, f, lo, n, dtype)
    r = Rows(p, [0], seed=T)
    x = r.draw(T, d)
    w1, w3, w2 = r.draw(n, d, f, scale=d ** -0.5), r.draw(n, d, f, scale=d ** -0.5), r.draw(n, f, d, scale=f ** -0.5)
    wg = r.draw(d, E, scale=d ** -0.5)
    dy = r.draw(T, d)
    idx, wt = M.route(p, r.dev(x), r.dev(wg))
    D = M.dispatch(p, idx, r.dev(x))
    W = (r.dev(w1), r.dev(w3), r.dev(w2))
    g, u, h, yp = M.expert_gemm_train(p, D["x_packed"], D["offsets"], *W)
    y = M.combine(p, yp, D["inv"], wt)
    dyp, dwt = M.combine_backward(p, r.dev(dy), yp, D["inv"], wt)
    dxp, dw1, dw3, dw2 = M.expert_gemm_backward(p, D["x_packed"], D["offsets"], *W, g, u, h, dyp)
    dx = M.combine(p, dxp, D["inv"], None)
    torch.cuda.synchronize()
    leaves = [t.clone().requires_grad_(True) for t in (x, w1, w3, w2, wt.cpu().double())]
    ref = _layer64(*leaves[:4], idx.cpu().long(), leaves[4], lo, n)
    ref.backward(dy)
    # Every value passes at most six roundings to the storage type on its way
    # (x W1, h, y or w dy, dg, dx_packed, the output), each half a step, that
    # add like independent errors of the tensor's norm: 6 half steps bound the
    # relative 2-norm, with the fp32 sums' K 2^-23 on top.
    bound = 6 * HALF[dtype] + (d + f) * 2.0 ** -23
    names = ("y", "dx", "dw1", "dw3", "dw2", "dtopk_w")
    for name, a, b in zip(names, (y, dx, dw1, dw3, dw2, dwt), (ref, *(t.grad for t in leaves))):
        rel = float((a.cpu().double() - b.detach()).norm() / b.detach().norm())
        assert rel <= bound, (name, rel, bound)
    # along a random direction: the loss's central difference in 64 bits
    for i, got in ((0, dx), (1, dw1), (2, dw3), (3, dw2), (4, dwt)):
        with torch.no_grad():
            dirn = torch.randn(leaves[i].shape, generator=r.gen, dtype=torch.float64)
            step = 1e-5
            vals = []
            for sgn in (1, -1):
                moved = [t.detach() + (sgn * step * dirn if j == i else 0) for j, t in enumerate(leaves)]
                vals.append(float((_layer64(*moved[:4], idx.cpu().long(), moved[4], lo, n) * dy).sum()))
            diff = (vals[0] - vals[1]) / (2 * step)
            mine = float((got.cpu().double() * dirn).sum())
            scale = float(leaves[i].grad.norm() * dirn.norm())
            assert abs(mine - diff) <= (bound + 1e-7) * scale, (names[i + 1], mine, diff)


def test_backward_captured():
    """A captured training step replays with new inputs, on a stream of its own."""
    p, r, v = _case("ragged")
    g, u, h, dy = _backward_inputs(r, v, p)
    off = offsets_of(r.counts)
    W = [r.dev(v[k]) for k in ("w1", "w3", "w2")]
    x, dyd = r.packed(v["x"]), r.packed(dy)
    n = len(r.counts)
    ws = M.alloc_workspace(p, M.MOE_CALL_EXPERT_GEMM_BACKWARD)
    fw = tuple(r.out(w) for w in (p.f, p.f, p.f, p.d))
    bw = (r.out(p.d), *(torch.empty(s, dtype=r.dt, device="cuda") for s in ((n, p.d, p.f), (n, p.d, p.f), (n, p.f, p.d))))

    def step():
        M.expert_gemm_train(p, x, off, *W, out=fw)
        M.expert_gemm_backward(p, x, off, *W, *fw[:3], dyd, workspace=ws, out=bw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x[: r.A] = r.dev(r.draw(r.A, p.d))
        dyd[: r.A] = r.dev(r.draw(r.A, p.d))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in (*fw, *bw)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(kept, (*fw, *bw)):
            assert torch.equal(a, b), k


def test_backward_is_reproducible():
    p, r, v = _case("long")
    g, u, h, dy = _backward_inputs(r, v, p)
    args = (r.packed(v["x"]), offsets_of(r.counts), r.dev(v["w1"]), r.dev(v["w3"]), r.dev(v["w2"]), r.packed(g),
            r.packed(u), r.packed(h), r.packed(dy))
    a, b = M.expert_gemm_backward(p, *args), M.expert_gemm_backward(p, *args)
    assert all(torch.equal(s[: r.A] if i == 0 else s, t[: r.A] if i == 0 else t) for i, (s, t) in enumerate(zip(a, b)))


def _busy(stream):
    """Keeps a stream occupied for a few milliseconds."""
    with torch.cuda.stream(stream):
        a = torch.ones((4096, 4096), device="cuda")
        for _ in range(8):
            a = a @ a * 1e-4
    return a


@pytest.mark.parametrize("name", ["ragged", "long", "f32_ragged"])
def test_calls_on_a_given_stream(name):
    """With stream= and nothing else given, what a call allocates (zeroed outputs,
    the workspace) belongs to that stream: the stream is still busy when the call
    returns and other memory is taken and written meanwhile."""
    p, r, v = _case(name)
    g, u, h, dy = _backward_inputs(r, v, p)
    off = offsets_of(r.counts)
    W = [r.dev(v[k]) for k in ("w1", "w3", "w2")]
    x, kept, dyd = r.packed(v["x"]), [r.packed(t) for t in (g, u, h)], r.packed(dy)
    ref = (*M.expert_gemm_train(p, x, off, *W), *M.expert_gemm_backward(p, x, off, *W, *kept, dyd))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy = _busy(s)
    got = (*M.expert_gemm_train(p, x, off, *W, stream=s), *M.expert_gemm_backward(p, x, off, *W, *kept, dyd, stream=s))
    need = M.workspace_bytes(p, M.MOE_CALL_EXPERT_GEMM_BACKWARD)
    spoil = [torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del busy, spoil
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_two_calls_at_once():
    """Two backward passes side by side, each with its own stream and workspace."""
    jobs = []
    for name in ("ragged", "long"):
        p, r, v = _case(name)
        g, u, h, dy = _backward_inputs(r, v, p)
        args = (r.packed(v["x"]), offsets_of(r.counts), *(r.dev(v[k]) for k in ("w1", "w3", "w2")),
                *(r.packed(t) for t in (g, u, h, dy)))
        jobs.append((p, args, M.expert_gemm_backward(p, *args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        got = [M.expert_gemm_backward(p, *args, stream=s) for p, args, _, s in jobs]
        torch.cuda.synchronize()
        for (_, _, ref, _), outs in zip(jobs, got):
            assert all(torch.equal(a, b) for a, b in zip(ref, outs))


@pytest.mark.parametrize("name", ["ragged", "long", "f32_ragged"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_rows_stay_in_their_expert(name, bad):
    """One expert's rows hold a value that is no number: the other experts' rows and
    weight gradients are those of a finite batch."""
    p, r, v = _case(name)
    g, u, h, dy = _backward_inputs(r, v, p)
    off = offsets_of(r.counts)
    W = [r.dev(v[k]) for k in ("w1", "w3", "w2")]
    kept = [r.packed(t) for t in (g, u, h)]

    def run(x, y):
        out = (*M.expert_gemm_train(p, x, off, *W), *M.expert_gemm_backward(p, x, off, *W, *kept, y))
        torch.cuda.synchronize()
        return out

    ref = run(r.packed(v["x"]), r.packed(dy))
    for e, seg in r.segments():
        if seg.start == seg.stop:
            continue
        x, y = r.packed(v["x"]), r.packed(dy)
        x[seg.start], y[seg.stop - 1] = bad, bad
        got = run(x, y)
        assert not bool(torch.isfinite(got[0][seg.start]).all()) and not bool(torch.isfinite(got[7][e]).all())
        rows = torch.ones(r.A, dtype=torch.bool, device="cuda")
        rows[seg] = False
        for a, b in zip(ref[:5], got[:5]):
            assert torch.equal(a[: r.A][rows], b[: r.A][rows])
        others = [k for k in range(len(r.counts)) if k != e]
        for a, b in zip(ref[5:], got[5:]):
            assert torch.equal(a[others], b[others])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combine_backward_padded_rows(dtype):
    """The padded layout: rows of every expert at multiples of the capacity, more
    rows than the compact layout has; rows that no slot names stay as they were."""
    T, k, n, E, d, cap = 13, 3, 4, 6, 72, 13
    p = M.Spec(T, d, E, k, 8, 0, n, dtype)
    r = Rows(p, [n * cap], seed=5)
    gen = np.random.default_rng(5)
    fill, inv = [0] * n, np.full(T * k, -1, dtype=np.int32)
    for t in range(T):
        for j, e in enumerate(gen.choice(E, k, replace=False)):
            if e < n:
                inv[t * k + j] = e * cap + fill[e]
                fill[e] += 1
    dy, yp, w = r.draw(T, d), r.draw(n * cap, d), torch.rand((T, k), generator=r.gen)
    dev = lambda v: v.to(r.dt).cuda()  # noqa: E731
    out = (torch.full((n * cap, d), -77.0, dtype=r.dt, device="cuda"), torch.empty((T, k), device="cuda"))
    dyp, dw = M.combine_backward(p, dev(dy), dev(yp), torch.from_numpy(inv).cuda(), w.cuda(), out=out, rows=n * cap)
    torch.cuda.synchronize()
    named = set(int(i) for i in inv if i >= 0)
    for row in range(n * cap):
        if row not in named:
            assert bool((dyp[row] == -77.0).all())
    for a, row in enumerate(inv):
        if row < 0:
            assert float(dw.view(-1)[a]) == 0.0
            continue
        ref = w.view(-1)[a].double() * dy[a // k]
        assert_within(dyp[int(row)], ref, (HALF[dtype] + 2.0 ** -23) * ref.abs(), "dy_packed")
        each = dy[a // k] * yp[int(row)]
        assert abs(float(dw.view(-1)[a]) - each.sum()) <= d * 2.0 ** -23 * each.abs().sum()


def test_offsets_beyond_32_bits():
    """Rows that lie more than 4 GiB into their buffers, in a segment that is itself
    longer, and in the ones behind it: all training calls, checked on those rows.
    The others hold ones and a zero gradient, which add nothing to the sums."""
    d, f, counts = 8192, 24, [299_950, 0, 10]
    p = spec(counts, d, f, "bf16", k=2)
    assert counts[0] * d * 2 > 2 ** 32
    few = Rows(spec([50, 0, 10], d, f, "bf16"), [50, 0, 10], seed=8)
    v = dict(x=few.draw(60, d), w1=few.draw(3, d, f, scale=d ** -0.5), w3=few.draw(3, d, f, scale=d ** -0.5),
             w2=few.draw(3, f, d, scale=f ** -0.5))
    g, u, h, dy = _backward_inputs(few, v, few.p)
    A = sum(counts)
    at = slice(A - 60, A)

    def buffer(vals, rest):
        t = torch.full((p.rows_max, vals.shape[1]), rest, dtype=torch.bfloat16, device="cuda")
        t[at] = few.dev(vals)
        t[A:] = float("nan")
        return t

    off = offsets_of(counts)
    W = [few.dev(v[k]) for k in ("w1", "w3", "w2")]
    x = buffer(v["x"], 1.0)
    fw = M.expert_gemm_train(p, x, off, *W, out=tuple(torch.full((p.rows_max, n), -77.0, dtype=torch.bfloat16, device="cuda")
                                                      for n in (f, f, f, d)))
    torch.cuda.synchronize()
    assert all(bool((t[A:] == -77.0).all()) for t in fw)
    _check_forward(few.p, few, v, [t[at] for t in fw])
    del fw
    bw = M.expert_gemm_backward(p, x, off, *W, buffer(g, 1.0), buffer(u, 1.0), buffer(h, 1.0), buffer(dy, 0.0))
    torch.cuda.synchronize()
    _check_backward(few.p, few, v, g, u, h, dy, [bw[0][at], *bw[1:]])


def test_combine_backward_beyond_32_bits():
    T, k, d = 40_000, 8, 8192
    p = M.Spec(T, d, 8, k, 8, 0, 8, "bf16")
    assert p.rows_max * d * 2 > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(4)
    dy = torch.randn((T, d), generator=gen, device="cuda").bfloat16()
    yp = torch.randn((8, d), generator=gen, device="cuda").bfloat16().repeat(T, 1)
    w = torch.rand((T, k), generator=gen, device="cuda")
    inv = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0)
    dyp, dw = M.combine_backward(p, dy, yp, inv, w)
    for t in (0, 1, T // 2, T - 1):   # row inv[8 t + j] = 8 (T - t) - 1 - j, whose y_packed is row 7 - j of eight
        rows = torch.arange(8 * (T - t) - 1, 8 * (T - t) - 9, -1)
        ref = w[t].cpu().double()[:, None] * dy[t].cpu().double()
        assert_within(dyp[rows.cuda()], ref, (HALF["bf16"] + 2.0 ** -23) * ref.abs(), "dy_packed")
        each = dy[t].cpu().double() * yp[:8].flip(0).cpu().double()
        assert_within(dw[t], each.sum(1), d * 2.0 ** -23 * each.abs().sum(1), "dtopk_w")


def test_tensors_and_streams_of_another_device_are_refused(monkeypatch):
    """A call runs on the current device; here another number stands for it."""
    p, r, v = _case("one_row")
    x, off, W = r.packed(v["x"]), offsets_of(r.counts), [r.dev(v[k]) for k in ("w1", "w3", "w2")]
    s = torch.cuda.Stream()
    monkeypatch.setattr(M, "_current", lambda: 1)
    with pytest.raises(ValueError, match="x_packed is on device 0, the current device is 1"):
        M.expert_gemm_train(p, x, off, *W)
    with pytest.raises(ValueError, match="x is on device 0"):
        M.quantize_rows(x)
    with pytest.raises(ValueError, match="the stream is on device 0"):
        M._stream_at(1, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [0x7FFFFFFF, 0xFFFFFFFF, 0x7FFF8000, 0x7FC00000])
def test_combine_backward_weights_that_are_no_number(dtype, bits):
    """A NaN weight, of any payload, makes its slot's row NaN and no other."""
    T, k, d = 5, 3, 264
    p = M.Spec(T, d, k, k, 8, 0, k, dtype)
    r = Rows(p, [T * k], seed=2)
    dy, yp = r.dev(r.draw(T, d)), r.dev(r.draw(T * k, d))
    inv = torch.arange(T * k, dtype=torch.int32).flip(0)
    w = torch.rand((T, k), generator=r.gen)
    w[2, 1] = torch.tensor(bits - (bits >> 31 << 32), dtype=torch.int32).view(torch.float32)
    dyp, dw = M.combine_backward(p, dy, yp, inv.cuda(), w.cuda())
    want = torch.zeros((T * k, d), dtype=torch.bool)
    want[int(inv[2 * k + 1])] = True
    assert torch.equal(torch.isnan(dyp).cpu(), want) and bool(torch.isfinite(dw).all())


def test_combine_backward_of_many_tokens():
    """More tokens than workgroups of 256 fit one grid dimension (2^24)."""
    T, d = 2 ** 24 + 3, 8
    p = M.Spec(T, d, 2, 1, 8, 0, 1, "bf16")
    g = torch.Generator(device="cuda").manual_seed(6)
    dy = torch.randn((T, d), generator=g, device="cuda").bfloat16()
    inv = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).contiguous()
    inv[5] = -1   # its row T - 6 is named by no slot
    w = torch.full((T, 1), 0.5, device="cuda")
    out = (torch.full((T, d), SENTINEL, dtype=torch.bfloat16, device="cuda"), torch.full((T, 1), 9.0, device="cuda"))
    dyp, dw = M.combine_backward(p, dy, dy, inv, w, out=out)
    ref = 0.5 * dy.flip(0)   # exact
    ref[T - 6] = SENTINEL
    assert torch.equal(dyp, ref)
    dot = (dy.double() * dy.flip(0).double()).sum(1)
    dot[5] = 0
    each = (dy.double() * dy.flip(0).double()).abs().sum(1)
    assert bool(((dw[:, 0].double() - dot).abs() <= d * 2.0 ** -23 * each).all())
