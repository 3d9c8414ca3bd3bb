"""4-bit weights: packing, quantiser, products and experts against 64 bits."""
import numpy as np
import pytest
import torch

import combine_router_top_amd as M
from tests.segments import HALF, Rows, assert_within, offsets_of, spec

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -23


def _pack(q):
    """The documented layout, from values [K, N] (numpy)."""
    K, N = q.shape
    kb, nb = -(-K // 128), -(-N // 16)
    out = np.zeros((nb, kb, 64, 4), dtype=np.uint32)
    for k in range(K):
        s, a, v = k % 128 // 32, k % 32 // 8, k % 8
        for c in range(16):
            cols = q[k, c::16].astype(np.uint32)
            out[: cols.size, k // 128, 16 * a + c, s] |= cols << np.uint32(16 * (v % 2) + 4 * (v // 2))
    return (out << np.uint32(3)) | (out >> np.uint32(29))


def _quantise(w, G, zero):
    """The documented steps in single precision: (q, scale fp32 that bf16 holds, zero points)."""
    K, N = w.shape
    w = w.float()
    n = -(-K // G)
    q, s, z = torch.empty((K, N), dtype=torch.uint8), torch.empty((n, N)), torch.full((n, N), 8, dtype=torch.uint8)
    for g in range(n):
        r = w[g * G: g * G + G]
        hi, lo = r.amax(0).clamp(min=0), r.amin(0).clamp(max=0)
        s[g] = ((hi - lo) / 15 if zero else r.abs().amax(0) / 7).to(torch.bfloat16).float()
        live = s[g] > 0
        step = torch.where(live, s[g], 1.0)
        if zero:
            z[g] = torch.where(live, torch.round(-lo / step).clamp(0, 15), 8.0).to(torch.uint8)
        v = torch.round(r / step) + z[g].float()
        q[g * G: g * G + G] = torch.where(live, v.clamp(0 if zero else 1, 15), z[g].float()).to(torch.uint8)
    return q, s, z


def _weights(K, N, G, zero, seed, whole=False):
    """Random values, scales and zero points, and the weights they stand for (float64)."""
    g = torch.Generator().manual_seed(seed + K + N)
    n = -(-K // G)
    q = torch.randint(0, 16, (K, N), generator=g, dtype=torch.uint8)
    s = 2.0 ** torch.randint(-1, 2, (n, N), generator=g) if whole else (torch.rand((n, N), generator=g) + 0.2) / K ** 0.5 / 4
    s = s.to(torch.bfloat16)
    z = torch.randint(0, 16, (n, N), generator=g, dtype=torch.uint8) if zero else None
    up = lambda t: t.double().repeat_interleave(G, 0)[:K]  # noqa: E731
    w = (q.double() - (8 if z is None else up(z))) * up(s)
    return q, s, z, w


def _dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _slack(x, s, z, G, w):
    """Bound of the error of x W before its rounding.  Few rows: part and X are sums of G
    terms of up to 31 |x| each, (16 + z) X is one more rounding; then two per group and the
    waves' join.  Many rows: one sum of x W, K / 32 products of 32 terms (K / 32 + 36 roundings
    cover both), whose weights are exact without zero points and otherwise rounded to 11 bits
    where |q - z| is odd and above 8: (q - z) s is a whole number of at most 15 * 255 < 2^12 times a
    power of two, so from 2^11 on, where not every one has 11 bits, it moves by at most 1, 2^-11 of it."""
    K = x.shape[1]
    per = s.double().abs().repeat_interleave(G, 0)[:K]
    size = x.abs() @ w.abs()
    few = (2 * min(G, K) + 4) * EPS * 31 * (x.abs() @ per) + (2 * s.shape[0] + 20) * EPS * size
    return few + (K / 32 + 36) * EPS * size + (0 if z is None else 2.0 ** -11) * size


@pytest.mark.parametrize("K,N", [(8, 8), (32, 16), (40, 24), (128, 16), (136, 40), (1000, 56)])
def test_pack(K, N):
    q = torch.randint(0, 16, (3, K, N), dtype=torch.uint8, generator=torch.Generator().manual_seed(K))
    got = M.pack_weights_4bit(q.cuda()).cpu().numpy().view(np.uint32)
    for e in range(3):
        assert np.array_equal(got[e], _pack(q[e].numpy()))


@pytest.mark.parametrize("K,N,G", [(8, 8, 32), (128, 16, 128), (136, 40, 64), (264, 24, 32), (1000, 24, 128)])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantise(K, N, G, zero, dtype):
    g = torch.Generator().manual_seed(K + N)
    w = (torch.randn((2, K, N), generator=g) + 0.3).to(dtype)
    w[0, :, 0] = 0             # scale 0
    w[0, :, 1] = 2.5           # one value
    w[1, :, 2] = -w[1, :, 2].abs()
    p, s, z = M.quantize_weights_4bit(w.cuda(), G, zero)
    for e in range(2):
        rq, rs, rz = _quantise(w[e], G, zero)
        assert torch.equal(s[e].cpu().float(), rs)
        assert z is None if not zero else torch.equal(z[e].cpu(), rz)
        assert np.array_equal(p[e].cpu().numpy().view(np.uint32), _pack(rq.numpy()))


@pytest.mark.parametrize("zero", [False, True])
def test_quantised_weights_are_near(zero):
    """Half a step of the scale, and the scale's own rounding at the ends of the range."""
    K, N, G = 256, 64, 64
    w = torch.randn((K, N), generator=torch.Generator().manual_seed(1))
    p, s, z = M.quantize_weights_4bit(w.cuda(), G, zero)
    eye = torch.eye(K, dtype=torch.bfloat16).cuda()
    back = M.gemm_4bit(eye, p, s, z, group=G, dtype=torch.float32)
    step = s.cpu().double().repeat_interleave(G, 0)
    assert_within(back, w.double(), step * (0.5 + 15 * 2.0 ** -8 + 0.5 * zero), "weights")


@pytest.mark.parametrize("M_,K,N,G", [(1, 8, 8, 32), (1, 7168, 2048, 128), (2, 128, 16, 32), (3, 136, 24, 64), (16, 256, 80, 128), (17, 264, 72, 32),
                                      (31, 1000, 56, 128), (33, 512, 128, 64), (64, 384, 264, 128), (65, 640, 136, 32), (100, 4104, 200, 64),
                                      (130, 1024, 520, 128), (257, 328, 264, 128), (300, 2048, 1032, 64), (513, 72, 8, 32), (700, 136, 4104, 32)])
@pytest.mark.parametrize("zero", [False, True])
def test_gemm(M_, K, N, G, zero):
    x = torch.randn((M_, K), generator=torch.Generator().manual_seed(M_)).to(torch.bfloat16)
    q, s, z, w = _weights(K, N, G, zero, M_)
    p = M.pack_weights_4bit(q.cuda())
    X = x.double()
    ref, slack = X @ w, _slack(X, s, z, G, w)
    for dtype, half in ((torch.bfloat16, HALF["bf16"]), (torch.float32, HALF["f32"])):
        got = M.gemm_4bit(x.cuda(), p, *_dev(s, z), group=G, dtype=dtype)
        assert got.dtype == dtype
        assert_within(got, ref, slack * (1 + half) + half * ref.abs(), str(dtype))


@pytest.mark.parametrize("M_,K,N,G", [(1, 1024, 64, 32), (5, 1000, 40, 64), (32, 512, 136, 128), (90, 1152, 264, 64), (200, 392, 520, 32),
                                      (300, 2048, 256, 128), (1000, 136, 72, 128)])
@pytest.mark.parametrize("zero", [False, True])
def test_whole_numbers_are_exact(M_, K, N, G, zero):
    """Small whole rows and scales that are powers of two: every fp32 step is exact."""
    x = torch.randint(-8, 9, (M_, K), generator=torch.Generator().manual_seed(K)).to(torch.bfloat16)
    q, s, z, w = _weights(K, N, G, zero, M_, whole=True)
    assert 31 * 8 * K * 2 * 2 < 2 ** 24
    got = M.gemm_4bit(x.cuda(), M.pack_weights_4bit(q.cuda()), *_dev(s, z), group=G, dtype=torch.float32)
    assert torch.equal(got.cpu().double(), x.double() @ w)


@pytest.mark.parametrize("M_", [4, 40, 400])
def test_values_that_are_not_finite_stay_in_their_row_and_column(M_):
    K, N, G = 264, 136, 64
    x = torch.randn((M_, K), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    q, s, z, w = _weights(K, N, G, True, 3)
    p = M.pack_weights_4bit(q.cuda())
    clean = M.gemm_4bit(x.cuda(), p, *_dev(s, z), group=G)
    x[1, 7], x[3, 260] = float("inf"), float("nan")
    s[2, 40] = float("nan")
    got = M.gemm_4bit(x.cuda(), p, *_dev(s, z), group=G)
    bad = torch.zeros((M_, N), dtype=torch.bool)
    bad[1], bad[3], bad[:, 40] = True, True, True
    assert bool(torch.isnan(got.cpu()[bad]).all())
    assert torch.equal(got.cpu()[~bad], clean.cpu()[~bad])


def _experts(counts, d, f, G, zero, seed=0, **kw):
    p = spec(counts, d, f, "bf16", **kw)
    r = Rows(p, counts, seed)
    x = r.draw(r.A, d)
    mats = [[_weights(K, N, G, zero, 17 * e + m + seed) for e in range(p.n_local)] for m, (K, N) in enumerate(((d, f), (d, f), (f, d)))]
    args = []
    for m in mats:
        args += [M.pack_weights_4bit(torch.stack([v[0] for v in m]).cuda()), torch.stack([v[1] for v in m]).cuda(),
                 torch.stack([v[2] for v in m]).cuda() if zero else None]
    return p, r, x, mats, args


def _check_experts(r, x, mats, G, h, y):
    half = HALF["bf16"]
    hd = h.cpu().double()
    for e, seg in r.segments():
        if seg.start == seg.stop:
            continue
        (_, s1, z1, w1), (_, s3, z3, w3), (_, s2, z2, w2) = (m[e] for m in mats)
        X = x[seg]
        a, b = X @ w1, X @ w3
        ta, tb = _slack(X, s1, z1, G, w1), _slack(X, s3, z3, G, w3)
        sg = torch.sigmoid(a)
        ref = a * sg * b
        # |SiLU'| <= 1.1; the exponential and the reciprocal are each good to a few ulps
        tol = (1.1 * ta * b.abs() + (a * sg).abs() * tb + ta * tb * 1.1) + (16 + 4 * a.abs()) * EPS * ref.abs()
        assert_within(h[seg], ref, tol * (1 + half) + half * ref.abs() + 1e-37, f"h of expert {e}")
        H = hd[seg]   # the product is of the rounded h
        ref = H @ w2
        assert_within(y[seg], ref, _slack(H, s2, z2, G, w2) * (1 + half) + half * ref.abs() + 1e-37, f"y of expert {e}")


@pytest.mark.parametrize("counts,d,f,G,kw", [
    ([1], 8, 8, 32, {}), ([0, 1, 0], 64, 40, 32, {}), ([3, 0, 17, 1], 136, 72, 64, {}), ([40, 5, 0, 33], 264, 136, 128, {}),
    ([0, 0, 0], 64, 64, 64, dict(T=4, k=1)), ([100, 260, 7], 392, 264, 128, {}), ([300], 512, 520, 64, {}),
    ([2, 1, 1, 3, 0, 1, 2, 2], 1024, 384, 128, dict(T=4, k=3)), ([5] * 40, 128, 256, 128, dict(T=8)), ([600, 130], 128, 128, 32, {}),
    ([130, 64, 200, 90], 640, 264, 128, {})])
@pytest.mark.parametrize("zero", [False, True])
def test_experts(counts, d, f, G, kw, zero):
    p, r, x, mats, args = _experts(counts, d, f, G, zero, **kw)
    h, y = r.out(f), r.out(d)
    M.expert_gemm_4bit(p, r.packed(x), offsets_of(counts), *args, group=G, out=(h, y))
    r.check_tail(h, y)
    _check_experts(r, x, mats, G, h, y)
    again = M.expert_gemm_4bit(p, r.packed(x), offsets_of(counts), *args, group=G)
    assert torch.equal(again[0][: r.A], h[: r.A]) and torch.equal(again[1][: r.A], y[: r.A])


def test_zero_points_of_some_matrices_only():
    counts, d, f, G = [9, 30], 136, 72, 64
    p, r, x, mats, args = _experts(counts, d, f, G, True)
    sym = [_weights(d, f, G, False, 5 + e) for e in range(2)]
    mats[1] = sym
    args[3], args[4], args[5] = M.pack_weights_4bit(torch.stack([v[0] for v in sym]).cuda()), torch.stack([v[1] for v in sym]).cuda(), None
    h, y = M.expert_gemm_4bit(p, r.packed(x), offsets_of(counts), *args, group=G)
    _check_experts(r, x, mats, G, h, y)


def test_a_bad_row_changes_no_other():
    counts, d, f, G = [5, 70, 3], 136, 72, 64
    p, r, x, mats, args = _experts(counts, d, f, G, False)
    clean = M.expert_gemm_4bit(p, r.packed(x), offsets_of(counts), *args, group=G)
    x[2, 1], x[40, 3] = float("inf"), float("nan")
    got = M.expert_gemm_4bit(p, r.packed(x), offsets_of(counts), *args, group=G)
    keep = torch.ones(p.rows_max, dtype=torch.bool)
    keep[2] = keep[40] = False
    for a, b in zip(got, clean):
        assert torch.equal(a[: r.A][keep[: r.A]], b[: r.A][keep[: r.A]])
        assert bool(torch.isnan(a[[2, 40]]).all())


def test_streams_and_graphs():
    counts, d, f, G = [20, 3, 0, 50], 264, 136, 64
    sets = [_experts(counts, d, f, G, True, seed) for seed in (0, 1)]
    off = offsets_of(counts)
    xs = [r.packed(x) for _, r, x, _, _ in sets]
    want = [M.expert_gemm_4bit(s[0], v, off, *s[4], group=G) for s, v in zip(sets, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [M.expert_gemm_4bit(s[0], v, off, *s[4], group=G, stream=st) for s, v, st in zip(sets, xs, streams)]
    torch.cuda.synchronize()
    A = sum(counts)
    assert all(torch.equal(a[:A], b[:A]) for w, g in zip(want, got) for a, b in zip(w, g))
    p, _, _, _, args = sets[0]
    held = xs[0].clone()
    out = tuple(torch.zeros_like(v) for v in want[0])
    lin = M.gemm_4bit(held[:A], args[0][0], args[1][0], args[2][0], group=G)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        M.expert_gemm_4bit(p, held, off, *args, group=G, out=out)
        M.gemm_4bit(held[:A], args[0][0], args[1][0], args[2][0], group=G, out=lin)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.expert_gemm_4bit(p, held, off, *args, group=G, out=out)
        M.gemm_4bit(held[:A], args[0][0], args[1][0], args[2][0], group=G, out=lin)
    for i in (1, 0, 1):
        held.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        h, y = M.expert_gemm_4bit(p, held, off, *args, group=G)
        assert torch.equal(out[0][:A], h[:A]) and torch.equal(out[1][:A], y[:A])
        assert torch.equal(lin, M.gemm_4bit(held[:A], args[0][0], args[1][0], args[2][0], group=G))
