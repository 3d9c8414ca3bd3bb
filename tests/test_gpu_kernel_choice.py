"""Every kernel of the training and 8-bit calls, at sizes that reach it
(tests/kernel_cases.py says which; tests/test_kernel_choice.py checks that), against
the formulas in 64 bits with the tolerances of test_gpu_training.py and
test_gpu_quantized.py, and captured, on other streams and with rows that are not
finite."""
import pytest
import torch

import combine_router_top_amd as M
from tests import kernel_cases as C
from tests import kernel_rules as R
from tests.segments import HALF, Rows, assert_within, offsets_of
from tests.test_gpu_quantized import _quant
from tests.test_gpu_training import _backward_inputs, _check_backward, _check_forward

pytestmark = pytest.mark.gpu


def test_compute_units():
    """The rules of the cases are those of this device."""
    assert torch.cuda.get_device_properties(0).multi_processor_count == R.CUS


# ---------------------------------------------------------------------------
# training
# ---------------------------------------------------------------------------
class Training:
    def __init__(self, name):
        counts, d, f = C.TRAINING[name][:3]
        self.p = p = C.problem(C.TRAINING[name])
        self.r = r = Rows(p, counts, seed=sum(map(ord, name)))
        n = len(counts)
        self.v = dict(x=r.draw(r.A, d), w1=r.draw(n, d, f, scale=d ** -0.5), w3=r.draw(n, d, f, scale=d ** -0.5),
                      w2=r.draw(n, f, d, scale=f ** -0.5))
        self.off = offsets_of(counts)
        self.W = [r.dev(self.v[k]) for k in ("w1", "w3", "w2")]
        self.x = r.packed(self.v["x"])

    def forward_out(self):
        p, r = self.p, self.r
        return tuple(r.out(w) for w in (p.f, p.f, p.f, p.d))

    def backward_out(self, wanted=(1, 1, 1, 1)):
        p, r, n = self.p, self.r, len(self.r.counts)
        nan = lambda *s: torch.full(s, float("nan"), dtype=r.dt, device="cuda")  # noqa: E731
        make = (lambda: r.out(p.d), lambda: nan(n, p.d, p.f), lambda: nan(n, p.d, p.f), lambda: nan(n, p.f, p.d))
        return tuple(m() if w else None for m, w in zip(make, wanted))


@pytest.mark.parametrize("name", C.TRAINING)
def test_training_forward(name):
    t = Training(name)
    got = M.expert_gemm_train(t.p, t.x, t.off, *t.W, out=t.forward_out())
    torch.cuda.synchronize()
    t.r.check_tail(*got)
    _check_forward(t.p, t.r, t.v, got)


@pytest.mark.parametrize("name", C.TRAINING)
def test_training_backward(name):
    t = Training(name)
    g, u, h, dy = _backward_inputs(t.r, t.v, t.p)
    args = (t.x, t.off, *t.W, *(t.r.packed(a) for a in (g, u, h, dy)))
    got = M.expert_gemm_backward(t.p, *args, out=t.backward_out())
    torch.cuda.synchronize()
    t.r.check_tail(got[0])
    _check_backward(t.p, t.r, t.v, g, u, h, dy, got)
    again = M.expert_gemm_backward(t.p, *args, out=t.backward_out())
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("name", ["units_of_3", "split_192", "long_64", "long_128", "rotated_128"])
@pytest.mark.parametrize("wanted", [(1, 0, 0, 0), (0, 1, 0, 1), (0, 0, 1, 0)])
def test_training_backward_some_outputs(name, wanted):
    """The same values, whatever else is wanted: which kernel a gradient takes depends
    on the others, the order of its sums may too, so both are within the tolerances."""
    t = Training(name)
    g, u, h, dy = _backward_inputs(t.r, t.v, t.p)
    got = M.expert_gemm_backward(t.p, t.x, t.off, *t.W, *(t.r.packed(a) for a in (g, u, h, dy)), out=t.backward_out(wanted))
    torch.cuda.synchronize()
    if got[0] is not None:
        t.r.check_tail(got[0])
    _check_backward(t.p, t.r, t.v, g, u, h, dy, got)


@pytest.mark.parametrize("name", ["rotated_64", "rotated_192", "units_of_2", "units_of_4", "split_256", "long_128"])
def test_training_step_captured(name):
    """Replays of a captured step follow new inputs, with eager steps between them; two
    more steps run at the same time on streams of their own."""
    t = Training(name)
    r, p = t.r, t.p
    dy = r.packed(r.draw(r.A, p.d))
    ws = M.alloc_workspace(p, M.MOE_CALL_EXPERT_GEMM_BACKWARD)
    fw, bw = t.forward_out(), t.backward_out()

    def step():
        M.expert_gemm_train(p, t.x, t.off, *t.W, out=fw)
        M.expert_gemm_backward(p, t.x, t.off, *t.W, *fw[:3], dy, workspace=ws, out=bw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        t.x[: r.A] = r.dev(r.draw(r.A, p.d))
        dy[: r.A] = r.dev(r.draw(r.A, p.d))
        graph.replay()
        torch.cuda.synchronize()
        kept = [a.clone() for a in (*fw, *bw)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, (*fw, *bw)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [M.expert_gemm_backward(p, t.x, t.off, *t.W, *fw[:3], dy, stream=s) for s in streams]
    torch.cuda.synchronize()
    for outs in got:
        assert torch.equal(outs[0][: r.A], bw[0][: r.A]) and all(torch.equal(a, b) for a, b in zip(outs[1:], bw[1:]))


@pytest.mark.parametrize("name", ["rotated_128", "units_of_3", "split_128", "long_128"])
def test_training_rows_that_are_not_finite(name):
    """They reach their own expert's gradients and rows, and no other's."""
    t = Training(name)
    g, u, h, dy = (t.r.packed(a) for a in _backward_inputs(t.r, t.v, t.p))

    def run(x, y):
        out = M.expert_gemm_backward(t.p, x, t.off, *t.W, g, u, h, y)
        torch.cuda.synchronize()
        return out

    ref = run(t.x, dy)
    live = [(e, s) for e, s in t.r.segments() if s.start < s.stop]
    for e, seg in (live[0], live[len(live) // 2], live[-1]):
        x, y = t.x.clone(), dy.clone()
        x[seg.start], y[seg.stop - 1] = float("nan"), float("inf")
        got = run(x, y)
        rows = torch.ones(t.r.A, dtype=torch.bool, device="cuda")
        rows[seg.stop - 1] = False   # every row of dx from its own row of dy
        assert torch.equal(ref[0][: t.r.A][rows], got[0][: t.r.A][rows])
        others = [k for k in range(len(t.r.counts)) if k != e]
        for a, b in zip(ref[1:], got[1:]):
            assert torch.equal(a[others], b[others]) and not bool(torch.isfinite(b[e]).all())


# ---------------------------------------------------------------------------
# 8 bits
# ---------------------------------------------------------------------------
class Quantized:
    def __init__(self, name):
        counts, d, f = C.QUANTIZED[name][:3]
        self.p = C.problem(C.QUANTIZED[name])
        self.r = r = Rows(self.p, counts, seed=sum(map(ord, name)))
        n = len(counts)
        g = torch.Generator().manual_seed(d * f)
        sizes = (("1", d, f), ("3", d, f), ("2", f, d))
        self.w = {k: torch.randint(-127, 128, (n, K, N), generator=g, dtype=torch.int8) for k, K, N in sizes}
        self.s = {k: (torch.rand((n, N), generator=g) + 0.5) / (70.0 * K ** 0.5) for k, K, N in sizes}
        self.xv = r.draw(r.A, d)
        self.x, self.off = r.packed(self.xv), offsets_of(counts)
        self.weights = [t for k in "132" for t in (M.pack_weights(self.w[k].cuda()), self.s[k].cuda())]

    def out(self):
        return self.r.out(self.p.f), self.r.out(self.p.d)

    def check(self, h, y):
        self.r.check_tail(h, y)
        for e, seg in self.r.segments():
            if seg.start == seg.stop:
                continue
            q, sx = _quant(self.xv[seg].numpy())
            q, sx = torch.from_numpy(q).double(), torch.from_numpy(sx).double()[:, None]
            a = q @ self.w["1"][e].double() * sx * self.s["1"][e].double()
            b = q @ self.w["3"][e].double() * sx * self.s["3"][e].double()
            ref = a * torch.sigmoid(a) * b
            # as test_gpu_quantized.test_expert_gemm_quantized
            tol = (HALF["bf16"] + (2.0 ** -20) * (1 + a.abs())) * ref.abs()
            assert_within(h[seg], ref, tol, "h")
            q, sh = _quant(h[seg].float().cpu().numpy())
            ref = torch.from_numpy(q).double() @ self.w["2"][e].double() * torch.from_numpy(sh).double()[:, None] * self.s["2"][e].double()
            assert_within(y[seg], ref, (HALF["bf16"] + 4 * HALF["f32"]) * ref.abs(), "y")


@pytest.mark.parametrize("name", C.QUANTIZED)
def test_quantized_experts(name):
    t = Quantized(name)
    got = M.expert_gemm_quantized(t.p, t.x, t.off, *t.weights, out=t.out())
    torch.cuda.synchronize()
    t.check(*got)


@pytest.mark.parametrize("name", C.QUANTIZED)
def test_quantized_rows_that_are_not_finite(name):
    """They give NaN rows and leave every other row as it was."""
    t = Quantized(name)
    ref = M.expert_gemm_quantized(t.p, t.x, t.off, *t.weights)
    x = t.x.clone()
    hit = sorted({0, t.r.A // 2, t.r.A - 1})
    for row, bad, col in zip(hit, ("nan", "inf", "-inf"), (1, 0, t.p.d - 1)):
        x[row, col] = float(bad)
    got = M.expert_gemm_quantized(t.p, x, t.off, *t.weights)
    torch.cuda.synchronize()
    rest = [i for i in range(t.r.A) if i not in hit]
    for a, b in zip(ref, got):
        assert torch.equal(a[rest], b[rest]) and bool(torch.isnan(b[hit]).all())


@pytest.mark.parametrize("name", ["blocks", "blocks_wide", "split", "split_down", "split_both", "low_wide"])
def test_quantized_captured_and_two_at_once(name):
    t = Quantized(name)
    ws, out = M.alloc_workspace(t.p, M.MOE_CALL_EXPERT_GEMM_QUANTIZED), t.out()

    def step():
        M.expert_gemm_quantized(t.p, t.x, t.off, *t.weights, workspace=ws, out=out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        t.x[: t.r.A] = t.r.dev(t.r.draw(t.r.A, t.p.d))
        graph.replay()
        torch.cuda.synchronize()
        kept = [a.clone() for a in out]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, out))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [M.expert_gemm_quantized(t.p, t.x, t.off, *t.weights, stream=s) for s in streams]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(a[: t.r.A], b[: t.r.A]) for a, b in zip(pair, out))


@pytest.mark.parametrize("name", C.PRODUCTS)
def test_products_are_exact(name):
    (rows, N, K), _ = C.PRODUCTS[name]
    g = torch.Generator().manual_seed(rows + N + K)
    a = torch.randint(-128, 128, (rows, K), generator=g, dtype=torch.int8)
    b = torch.randint(-128, 128, (K, N), generator=g, dtype=torch.int8)
    sa, sb = torch.rand(rows, generator=g) + 0.01, torch.rand(N, generator=g) + 0.01
    packed = M.pack_weights(b.cuda())
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    got = M.gemm_quantized(a.cuda(), one(rows), packed, one(N), dtype=torch.float32)
    ref = a.double() @ b.double()   # exact: below 2^53
    assert torch.equal(got.cpu(), ref.float())
    ref = ref * sa.double()[:, None] * sb.double()
    # three fp32 roundings, and half a step of the output
    for dtype, half in ((torch.float32, 0.0), (torch.bfloat16, HALF["bf16"])):
        got = M.gemm_quantized(a.cuda(), sa.cuda(), packed, sb.cuda(), dtype=dtype)
        assert_within(got, ref, (half + 4 * HALF["f32"]) * ref.abs(), "C")
