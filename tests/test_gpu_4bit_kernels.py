"""Every kernel of the 4-bit products at sizes that take it, against 64 bits; ranges of rows
and scales; workspaces; views; positions that pass 32 bits."""
import pytest
import torch

import combine_router_top_amd as M
from tests import cases_4bit as C
from tests.segments import HALF, assert_within, offsets_of
from tests.test_gpu_4bit import _check_experts, _dev, _experts, _slack, _weights

pytestmark = pytest.mark.gpu


def _join(K, x, w):
    """K in parts: up to 15 more roundings, each of a sum of at most |x| |W|."""
    return 15 * 2.0 ** -24 * (x.abs() @ w.abs())


@pytest.mark.parametrize("name", C.PRODUCTS)
@pytest.mark.parametrize("zero", [False, True])
def test_products(name, zero):
    (T, K, N, G), _ = C.PRODUCTS[name]
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    q, s, z, w = _weights(K, N, G, zero, T)
    p, X = M.pack_weights_4bit(q.cuda()), x.double()
    ref, slack = X @ w, _slack(X, s, z, G, w) + _join(K, X, w)
    args = (x.cuda(), p, *_dev(s, z))
    for dtype, half in ((torch.bfloat16, HALF["bf16"]), (torch.float32, HALF["f32"])):
        got = M.gemm_4bit(*args, group=G, dtype=dtype)
        assert_within(got, ref, slack * (1 + half) + half * ref.abs(), str(dtype))
        assert torch.equal(got, M.gemm_4bit(*args, group=G, dtype=dtype))


@pytest.mark.parametrize("name", C.EXPERTS)
@pytest.mark.parametrize("zero", [False, True])
def test_experts(name, zero):
    (counts, d, f, G), *_ = C.EXPERTS[name]
    p, r, x, mats, args = _experts(counts, d, f, G, zero)
    h, y = r.out(f), r.out(d)
    size = M.workspace_bytes(p, M.MOE_CALL_EXPERT_GEMM_FOURBIT)
    ws = torch.full((max(size, 1),), 255, dtype=torch.uint8, device="cuda") if size else None   # NaN in every type
    M.expert_gemm_4bit(p, r.packed(x), offsets_of(counts), *args, group=G, workspace=ws, out=(h, y))
    r.check_tail(h, y)
    _check_experts(r, x, mats, G, h, y)


# Rows and scales of very different sizes.  On tiles a row's values are exact in fp16 within
# 2^-31 of its largest and otherwise off by less than 2^-38 of that; scales within 2^-27 of their
# column's largest are exact, others off by less than 2^-34 of it, times up to 15.
@pytest.mark.parametrize("T,K,N,G", [(6, 264, 40, 32), (40, 520, 72, 128), (300, 264, 8200, 64), (130, 14344, 136, 128)])
@pytest.mark.parametrize("zero", [False, True])
def test_ranges(T, K, N, G, zero):
    g = torch.Generator().manual_seed(K)
    exp2 = lambda *s, lo, hi: 2.0 ** torch.randint(lo, hi + 1, s, generator=g)  # noqa: E731
    x = (torch.randn((T, K), generator=g) * exp2(T, 1, lo=-60, hi=60) * exp2(T, K, lo=-40, hi=0)).to(torch.bfloat16)
    x[1] = 0
    q, s, z, _ = _weights(K, N, G, zero, T)
    s = (s.float() * exp2(1, N, lo=-30, hi=30) * exp2(*s.shape, lo=-32, hi=0)).to(torch.bfloat16)
    s[:, 5] = 0
    up = lambda t: t.double().repeat_interleave(G, 0)[:K]  # noqa: E731
    w = (q.double() - (8 if z is None else up(z))) * up(s)
    X = x.double()
    ref = X @ w
    slack = _slack(X, s, z, G, w) + _join(K, X, w)
    slack += 2.0 ** -38 * X.abs().amax(1, keepdim=True) * w.abs().sum(0) + 15 * 2.0 ** -34 * X.abs().sum(1, keepdim=True) * s.double().abs().amax(0)
    slack += K * 2.0 ** -126   # fp32 terms below that may vanish
    got = M.gemm_4bit(x.cuda(), M.pack_weights_4bit(q.cuda()), *_dev(s, z), group=G, dtype=torch.float32)
    assert_within(got, ref, slack * (1 + HALF["f32"]) + HALF["f32"] * ref.abs(), "ranges")
    assert not got[1].any() and not got[:, 5].any()


@pytest.mark.parametrize("T", [3, 300])
def test_largest_and_smallest_rows(T):
    K, N, G = 264, 8200, 64
    x = torch.zeros((T, K), dtype=torch.bfloat16)
    top, low = torch.finfo(torch.bfloat16).max, torch.finfo(torch.bfloat16).tiny
    x[0, 3], x[1, 4], x[2, 263] = top, low, -top
    q, s, z, w = _weights(K, N, G, True, 3, whole=True)   # scales 1/2, 1, 2: products stay finite below 2^127
    s, w = s / 32, w / 32
    got = M.gemm_4bit(x.cuda(), M.pack_weights_4bit(q.cuda()), *_dev(s, z), group=G, dtype=torch.float32).cpu().double()
    ref = x.double() @ w   # one term each: weights and values of few bits, so exact
    normal = (ref == 0) | (ref.abs() >= 2.0 ** -126)
    assert torch.equal(got[normal], ref[normal])
    assert bool(((got - ref).abs()[~normal] <= 2.0 ** -126).all())   # fp32 denormals may be flushed


def test_workspaces():
    """The library's size, filled with NaN, serves calls of the same and of smaller sizes; a
    stream of its own has its own."""
    K, N, G = 264, 8200, 64
    q, s, z, _ = _weights(K, N, G, True, 1)
    p, s, z = M.pack_weights_4bit(q.cuda()), *_dev(s, z)
    x = torch.randn((900, K), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    size = M.gemm_4bit_workspace_bytes(900, N, K)
    assert size > 0
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    want = {T: M.gemm_4bit(x[:T], p, s, z, group=G) for T in (900, 300)}
    for T in (900, 300, 900):
        assert M.gemm_4bit_workspace_bytes(T, N, K) <= size
        assert torch.equal(M.gemm_4bit(x[:T], p, s, z, group=G, workspace=ws), want[T])
    streams = [torch.cuda.Stream() for _ in range(2)]
    held = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    got = [M.gemm_4bit(x, p, s, z, group=G, workspace=w, stream=st) for w, st in zip(held, streams) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[900]) for v in got)
    with pytest.raises(M.MoeError):
        M.gemm_4bit(x, p, s, z, group=G, workspace=ws[: size - 256])


@pytest.mark.parametrize("T", [5, 300])
def test_views(T):
    """Rows from the middle of a buffer, scales and zero points that begin at 8 and 4 bytes;
    what is not dense is refused."""
    K, N, G = 264, 8200, 64
    q, s, z, _ = _weights(K, N, G, True, 1)
    p, s, z = M.pack_weights_4bit(q.cuda()), *_dev(s, z)
    x = torch.randn((T + 7, K), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()

    def shifted(t, by):
        buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
        buf[by:] = t.flatten()
        return buf[by:].view(t.shape)
    want = M.gemm_4bit(x[3: T + 3].clone(), p, s, z, group=G)
    assert torch.equal(M.gemm_4bit(x[3: T + 3], p, shifted(s, 4), shifted(z, 4), group=G), want)
    for bad in (dict(x=x[:T].t().contiguous().t()), dict(s=s.t().contiguous().t()), dict(x=x[:T].float()), dict(z=z[:, :-8])):
        use = {**dict(x=x[:T], s=s, z=z), **bad}
        with pytest.raises(ValueError):
            M.gemm_4bit(use["x"], p, use["s"], use["z"], group=G)
    with pytest.raises(M.MoeError):
        M.gemm_4bit(x[:T], p, shifted(s, 2), z, group=G)


@pytest.mark.parametrize("N", [16, 520])
def test_rows_past_32_bits(N):
    """2.2 * 10^9 values of rows, so that the last ones' bytes start past 2^32: streams (few
    columns) or tiles, compared at some rows of either end."""
    T, K, G = 20000, 110000, 128
    q, s, z, w = _weights(K, N, G, True, 1)
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(1))
    got = M.gemm_4bit(x, M.pack_weights_4bit(q.cuda()), *_dev(s, z), group=G, dtype=torch.float32)
    rows = [0, 63, 9999, 19007, 19990, 19999]
    X = x[rows].cpu().double()
    ref = X @ w
    assert_within(got[rows], ref, (_slack(X, s, z, G, w) + _join(K, X, w)) + HALF["f32"] * ref.abs(), "far rows")


def test_parts_in_graphs_and_on_streams():
    """A product with K in parts, captured beside another of its kind with the same workspace
    in turn, replayed with eager work between."""
    T, K, N, G = 130, 14344, 136, 64
    sets = []
    for seed in (1, 2):
        q, s, z, _ = _weights(K, N, G, True, seed)
        x = torch.randn((2, T, K), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
        sets.append((x, M.pack_weights_4bit(q.cuda()), *_dev(s, z)))
    ws = torch.empty(M.gemm_4bit_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    held = [v[0][0].clone() for v in sets]
    outs = [torch.empty((T, N), dtype=torch.bfloat16, device="cuda") for _ in sets]

    def both():
        for h, (_, p, s, z), o in zip(held, sets, outs):
            M.gemm_4bit(h, p, s, z, group=G, workspace=ws, out=o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in (1, 0, 1):
        for h, v in zip(held, sets):
            h.copy_(v[0][i])
        graph.replay()
        torch.cuda.synchronize()
        for o, (x, p, s, z) in zip(outs, sets):
            assert torch.equal(o, M.gemm_4bit(x[i], p, s, z, group=G))
