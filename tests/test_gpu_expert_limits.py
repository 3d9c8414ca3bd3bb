"""The training and 8-bit calls at the ends of their ranges: the widest rows, as many
experts as there may be, views that start off a cache line, and every call in one
captured step."""
import pytest
import torch

import combine_router_top_amd as M
from tests.segments import HALF, Rows, assert_within, offsets_of, spec
from tests.test_gpu_quantized import _quant
from tests.test_gpu_training import _backward_inputs, _check_backward, _check_forward, _layer64

pytestmark = pytest.mark.gpu

MOST = 1 << 20   # widest d and f of the training calls

WIDE = {
    "d": ([70, 0, 3], MOST, 8, {}),
    "f": ([70, 0, 3], 8, MOST, {}),
    "d_tall": ([193], MOST, 8, dict(T=300, k=1, E=1)),
    "f_tall": ([129], 8, MOST, dict(T=300, k=1, E=1)),
    "experts": ([(5 * e) % 4 if e % 7 else 0 for e in range(1000)], 72, 40, dict(T=64, k=32, E=1024)),
    "experts_long": ([(5 * e) % 61 if e % 7 else 0 for e in range(1000)], 72, 40, dict(T=1000, k=32, E=1024)),
}


@pytest.mark.parametrize("name,dtype", [(n, t) for n in WIDE for t in ("bf16", "f32") if not (n.endswith("tall") and t == "f32")])
def test_training(name, dtype):
    counts, d, f, kw = WIDE[name]
    p = spec(counts, d, f, dtype, **kw)
    r = Rows(p, counts, seed=sum(map(ord, name)))
    n = len(counts)
    v = dict(x=r.draw(r.A, d), w1=r.draw(n, d, f, scale=d ** -0.5), w3=r.draw(n, d, f, scale=d ** -0.5),
             w2=r.draw(n, f, d, scale=f ** -0.5))
    x, off = r.packed(v["x"]), offsets_of(counts)
    W = [r.dev(v[k]) for k in ("w1", "w3", "w2")]
    got = M.expert_gemm_train(p, x, off, *W, out=tuple(r.out(w) for w in (f, f, f, d)))
    torch.cuda.synchronize()
    r.check_tail(*got)
    _check_forward(p, r, v, got)
    g, u, h, dy = _backward_inputs(r, v, p)
    out = (r.out(d), *(torch.full(s, float("nan"), dtype=r.dt, device="cuda") for s in ((n, d, f), (n, d, f), (n, f, d))))
    got = M.expert_gemm_backward(p, x, off, *W, *(r.packed(t) for t in (g, u, h, dy)), out=out)
    torch.cuda.synchronize()
    r.check_tail(got[0])
    _check_backward(p, r, v, g, u, h, dy, got)


@pytest.mark.parametrize("rows,N,K", [(3, 1 << 21, 16), (300, 1 << 21, 16), (300, 16376, 131056)])
def test_widest_products(rows, N, K):
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    a = torch.randint(-128, 128, (rows, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (K, N), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = torch.rand(rows, generator=g, device="cuda") + 0.5, torch.rand(N, generator=g, device="cuda") + 0.5
    packed = M.pack_weights(b)
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    plain = M.gemm_quantized(a, one(rows), packed, one(N), dtype=torch.float32)
    scaled = M.gemm_quantized(a, sa, packed, sb, dtype=torch.float32)
    short = M.gemm_quantized(a, sa, packed, sb)
    for lo in range(0, N, 1 << 19):
        c = slice(lo, min(N, lo + (1 << 19)))
        ref = torch.zeros((rows, c.stop - c.start), dtype=torch.float64, device="cuda")
        for k in range(0, K, 1 << 14):   # exact: below 2^53
            ref += a[:, k : k + (1 << 14)].double() @ b[k : k + (1 << 14), c].double()
        assert torch.equal(plain[:, c], ref.float())
        ref *= sa.double()[:, None] * sb[c].double()
        # three fp32 roundings, and half a step of the output
        assert bool(((scaled[:, c].double() - ref).abs() <= 4 * HALF["f32"] * ref.abs()).all())
        assert bool(((short[:, c].double() - ref).abs() <= (HALF["bf16"] + 4 * HALF["f32"]) * ref.abs()).all())


@pytest.mark.parametrize("name", ["experts", "experts_long"])
def test_quantized_experts(name):
    counts, d, f, kw = WIDE[name]
    p = spec(counts, d, f, "bf16", **kw)
    r = Rows(p, counts, seed=4)
    n = len(counts)
    v = [r.draw(n, *s, scale=s[0] ** -0.5) for s in ((d, f), (d, f), (f, d))]
    packed = [t for w in v for t in M.quantize_weights(r.dev(w))]
    x = r.draw(r.A, d)
    h, y = M.expert_gemm_quantized(p, r.packed(x), offsets_of(counts), *packed, out=(r.out(f), r.out(d)))
    torch.cuda.synchronize()
    r.check_tail(h, y)

    def channels(w):   # [n, K, N] values -> steps and channel scales
        q, s = _quant(w.movedim(1, 2).reshape(-1, w.shape[1]).numpy())
        return (torch.from_numpy(q).view(n, w.shape[2], w.shape[1]).movedim(1, 2).double(),
                torch.from_numpy(s).view(n, w.shape[2]).double())

    (q1, s1), (q3, s3), (q2, s2) = (channels(w) for w in v)
    for e, seg in r.segments():
        if seg.start == seg.stop:
            continue
        q, sx = (torch.from_numpy(t).double() for t in _quant(x[seg].numpy()))
        a, b = (q @ w[e] * sx[:, None] * s[e] for w, s in ((q1, s1), (q3, s3)))
        ref = a * torch.sigmoid(a) * b
        # as test_gpu_quantized.test_expert_gemm_quantized
        assert_within(h[seg], ref, (HALF["bf16"] + 2.0 ** -20 * (1 + a.abs())) * ref.abs(), "h")
        q, sh = (torch.from_numpy(t).double() for t in _quant(h[seg].float().cpu().numpy()))
        ref = q @ q2[e] * sh[:, None] * s2[e]
        assert_within(y[seg], ref, (HALF["bf16"] + 4 * HALF["f32"]) * ref.abs(), "y")


def test_views_off_a_cache_line():
    """Operands that are slices of larger tensors, on 16-byte boundaries but no wider
    ones, give what the same values give elsewhere."""
    counts, d, f = [5, 0, 130, 40], 72, 136
    p = spec(counts, d, f, "bf16")
    r = Rows(p, counts, seed=7)
    n = len(counts)

    def shifted(t, by=16):
        by //= t.element_size()
        big = torch.zeros(t.numel() + by, dtype=t.dtype, device="cuda")
        big[by:] = t.flatten()
        return big[by:].view(t.shape)

    v = [r.draw(r.A, d), r.draw(n, d, f, scale=d ** -0.5), r.draw(n, d, f, scale=d ** -0.5), r.draw(n, f, d, scale=f ** -0.5)]
    x, W, off = r.packed(v[0]), [r.dev(w) for w in v[1:]], offsets_of(counts)
    dy = r.packed(r.draw(r.A, d))
    fw = M.expert_gemm_train(p, x, off, *W)
    bw = M.expert_gemm_backward(p, x, off, *W, *fw[:3], dy)
    fw2 = M.expert_gemm_train(p, shifted(x), shifted(off, 4), *map(shifted, W), out=tuple(shifted(torch.zeros_like(t)) for t in fw))
    bw2 = M.expert_gemm_backward(p, shifted(x), shifted(off, 4), *map(shifted, W), *map(shifted, fw[:3]), shifted(dy),
                                 out=tuple(shifted(torch.zeros_like(t)) for t in bw))
    for a, b in zip((*fw, *bw), (*fw2, *bw2)):
        assert torch.equal(a, b)
    packed = [t for w in W for t in M.quantize_weights(w)]
    again = [t for w in W for t in M.quantize_weights(shifted(w), out=tuple(shifted(torch.zeros_like(t)) for t in packed[:2])
                                                     if w is W[0] else None)]
    assert all(torch.equal(a, b) for a, b in zip(packed, again))
    a = M.expert_gemm_quantized(p, x, off, *packed)
    b = M.expert_gemm_quantized(p, shifted(x), shifted(off, 4), *map(shifted, packed))
    assert all(torch.equal(s[: r.A], t[: r.A]) for s, t in zip(a, b))
    rows = x[: r.A].contiguous()
    q, s = M.quantize_rows(rows)
    q2, s2 = M.quantize_rows(shifted(rows), out=(shifted(torch.zeros_like(q), 8), shifted(torch.zeros_like(s), 4)))
    assert torch.equal(q, q2) and torch.equal(s, s2)
    wide = torch.randint(-128, 128, (r.A, 80), generator=r.gen, dtype=torch.int8).cuda()
    w8 = M.pack_weights(torch.randint(-128, 128, (80, 24), generator=r.gen, dtype=torch.int8).cuda())
    sb = torch.rand(24, generator=r.gen).cuda()
    assert torch.equal(M.gemm_quantized(wide, s, w8, sb), M.gemm_quantized(shifted(wide), shifted(s, 4), shifted(w8), shifted(sb)))


def test_layer_training_step_captured():
    """Route, dispatch, experts, combine and all gradients in one graph, with everything
    that the calls allocate inside it, replayed with new inputs."""
    T, d, f, E, k, lo, n = 200, 136, 72, 8, 3, 2, 5
    p = M.Spec(T, d, E, k, f, lo, n, "bf16")
    r = Rows(p, [0], seed=T)
    x = r.dev(r.draw(T, d))
    W = [r.dev(r.draw(n, *s, scale=s[0] ** -0.5)) for s in ((d, f), (d, f), (f, d))]
    wg = r.dev(r.draw(d, E, scale=d ** -0.5))
    dy = r.dev(r.draw(T, d))

    def step():
        idx, wt = M.route(p, x, wg)
        D = M.dispatch(p, idx, x)
        g, u, h, yp = M.expert_gemm_train(p, D["x_packed"], D["offsets"], *W)
        y = M.combine(p, yp, D["inv"], wt)
        dyp, dwt = M.combine_backward(p, dy, yp, D["inv"], wt)
        dxp, dw1, dw3, dw2 = M.expert_gemm_backward(p, D["x_packed"], D["offsets"], *W, g, u, h, dyp)
        return idx, wt, y, dwt, M.combine(p, dxp, D["inv"], None), dw1, dw3, dw2

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        x.copy_(r.dev(r.draw(T, d)))
        dy.copy_(r.dev(r.draw(T, d)))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))
        # y against the layer in 64 bits: 6 half steps in the 2-norm, as
        # test_gpu_training.test_layer_training_step
        ref = _layer64(x.cpu().double(), *(w.cpu().double() for w in W), kept[0].cpu().long(), kept[1].cpu().double(), lo, n)
        rel = float((kept[2].cpu().double() - ref).norm() / ref.norm())
        assert rel <= 6 * HALF["bf16"] + (d + f) * 2.0 ** -23


def test_quantizers_and_products_captured():
    """Weights and rows quantised and multiplied in one graph."""
    r = Rows(spec([40], 520, 264, "bf16"), [40], seed=1)
    x, w = r.dev(r.draw(40, 520)), r.dev(r.draw(520, 264))
    raw = torch.randint(-128, 128, (528, 264), generator=r.gen, dtype=torch.int8).cuda()

    def step():
        packed, sw = M.quantize_weights(w)
        q, s = M.quantize_rows(x)
        whole = torch.nn.functional.pad(q, (0, 8))   # K a multiple of 16
        return q, s, packed, sw, M.gemm_quantized(whole, s, M.pack_weights(raw), sw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        x.copy_(r.dev(r.draw(40, 520)))
        w.copy_(r.dev(r.draw(520, 264)))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))
        q, sx = _quant(x.cpu().float().numpy())
        assert torch.equal(kept[0].cpu(), torch.from_numpy(q)) and torch.equal(kept[1].cpu(), torch.from_numpy(sx))
