"""8-bit rows, weights and products.

The integer sums are exact, so a product is checked through its formula: the
int64 sum rounded to fp32 (one rounding), two fp32 products (two more) and the
store.  fp32 outputs with unit scales must equal the rounded sum itself.
"""
import numpy as np
import pytest
import torch

import combine_router_top_amd as M
from tests.segments import HALF, Rows, assert_within, offsets_of, spec

pytestmark = pytest.mark.gpu


def _quant(x):
    """The quantiser's definition in single precision (numpy)."""
    x = np.asarray(x, dtype=np.float32)
    top = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
    live = top >= np.float32(2.0 ** -119)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(live, np.float32(127) * (np.float32(1) / top), np.float32(0)).astype(np.float32)
    return (np.rint(x * inv[:, None]).astype(np.int8),
            np.where(live, top / np.float32(127), np.float32(0)).astype(np.float32))


@pytest.mark.parametrize("rows,K", [(1, 8), (3, 16), (5, 264), (2, 8192), (3, 8200), (2, 40960), (700, 72), (5000, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_rows(rows, K, dtype):
    g = torch.Generator().manual_seed(rows + K)
    x = (torch.randn((rows, K), generator=g) * torch.rand((rows, 1), generator=g) * 10).to(dtype)
    x[0] = 0                       # scale 0, zeros
    if rows > 1:
        x[1, 1:] = 0               # one value: 127 or -127
    if rows > 3:
        x[3] = x[3].sign() * 2.0 ** -120   # counts as zeros
        x[4] = x[4].sign() * 2.0 ** -119
    if rows > 2:
        x[2, :4] = torch.tensor([2.0, 1.0, -1.0, 0.5]).to(dtype)
    q, s = M.quantize_rows(x.cuda())
    rq, rs = _quant(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("lead,K,N", [((), 8, 8), ((), 64, 16), ((3,), 72, 40), ((2,), 200, 136), ((), 1, 8), ((1,), 130, 24)])
def test_packed_weights(lead, K, N):
    g = torch.Generator().manual_seed(K * N)
    w = torch.randint(-128, 128, lead + (K, N), generator=g, dtype=torch.int8)
    packed = M.pack_weights(w.cuda()).cpu()
    kp, np_ = -(-K // 64) * 64, -(-N // 16) * 16
    full = torch.zeros(lead + (kp, np_), dtype=torch.int8)
    full[..., :K, :N] = w
    ref = full.view(*lead, kp // 64, 4, 16, np_ // 16, 16).movedim((-2, -5, -4, -1, -3), (-5, -4, -3, -2, -1))
    assert torch.equal(packed, ref)
    assert M.packed_weights_bytes(lead[0] if lead else 1, K, N) == packed.numel()
    for dtype in (torch.bfloat16, torch.float32):
        wf = torch.randn(lead + (K, N), generator=g).to(dtype)
        wf[..., 0] = 0             # a channel of zeros
        qp, s = M.quantize_weights(wf.cuda())
        cols = wf.float().movedim(-1, -2).reshape(-1, K).numpy()
        rq, rs = _quant(cols)
        assert np.array_equal(s.cpu().numpy().ravel(), rs)
        rw = torch.from_numpy(rq).view(*lead, N, K).movedim(-1, -2).contiguous()
        assert torch.equal(qp.cpu(), M.pack_weights(rw.cuda()).cpu())


SIZES = [(1, 8, 16), (1, 2048, 7168), (2, 24, 48), (15, 136, 64), (16, 512, 80), (17, 40, 1040), (31, 264, 256),
         (32, 4096, 128), (33, 264, 144), (64, 72, 320), (129, 520, 592), (300, 264, 1040), (257, 1000, 128), (1, 20000, 64),
         (20, 20000, 192), (3, 8, 8192),
         # enough tiles for the 256-, 192- and 128-row kernels
         (4096, 4096, 1040), (2049, 2104, 64), (180, 65528, 80), (70, 33000, 208),
         # deep and narrow: blocks of 32 rows on workgroups of their own, a short one last
         (49, 72, 8208), (100, 136, 2064), (128, 520, 4112), (250, 8, 16400)]


@pytest.mark.parametrize("Mr,N,K", SIZES)
def test_product_is_exact(Mr, N, K):
    g = torch.Generator().manual_seed(Mr + N + K)
    a = torch.randint(-128, 128, (Mr, K), generator=g, dtype=torch.int8)
    b = torch.randint(-128, 128, (K, N), generator=g, dtype=torch.int8)
    a[0] = -128
    b[:, 0] = -128                 # the largest sum
    packed = M.pack_weights(b.cuda())
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    got = M.gemm_quantized(a.cuda(), one(Mr), packed, one(N), dtype=torch.float32)
    ref = (a.double() @ b.double())          # exact: below 2^53
    assert torch.equal(got.cpu(), ref.float())
    # scales, and bf16 output: three fp32 roundings and half a step
    sa, sb = torch.rand(Mr, generator=g) + 0.01, torch.rand(N, generator=g) + 0.01
    got = M.gemm_quantized(a.cuda(), sa.cuda(), packed, sb.cuda())
    ref = ref * sa.double()[:, None] * sb.double()
    assert_within(got, ref, (HALF["bf16"] + 4 * HALF["f32"]) * ref.abs(), "C")


def test_product_extreme_depth():
    """The deepest K: 131056 products of 16384 stay inside int32."""
    K, N = 131056, 8
    for Mr in (2, 40):
        a = torch.full((Mr, K), -128, dtype=torch.int8, device="cuda")
        a[1] = 127
        packed = M.pack_weights(torch.full((K, N), -128, dtype=torch.int8, device="cuda"))
        got = M.gemm_quantized(a, torch.ones(Mr, device="cuda"), packed, torch.ones(N, device="cuda"), dtype=torch.float32)
        assert bool((got[0] == float(np.float32(K * 16384))).all()) and bool((got[1] == float(np.float32(-K * 127 * 128))).all())


CASES = {
    "one_row": ([1], 64, 64, {}),
    "narrow": ([3, 0, 2], 8, 8, {}),
    "streams": ([0, 5, 16, 1, 17, 32], 264, 200, {}),
    "streams_16": ([4, 0, 16, 1], 1032, 328, dict(T=16, k=4)),
    "streams_long": ([0, 5, 128, 33, 1, 64], 264, 200, dict(T=128, k=2, E=48)),   # blocks of 32 rows
    "mixed": ([0, 5, 33, 130, 1, 257], 264, 200, dict(T=257, k=2, E=48)),   # streams and tiles in one call
    "tiles": ([100, 70, 0, 150], 328, 264, {}),
    "tall_tiles": ([700, 0, 300], 136, 72, {}),
    "wide": ([3] * 40, 64, 1032, dict(T=20)),
    "no_rows": ([0, 0, 0], 64, 72, dict(T=5, k=2)),
    # enough tiles for the 256-, 192- and 128-row kernels
    "tall_many": ([400 + (37 * e) % 200 - 100 for e in range(64)], 264, 512, dict(T=1600, k=16)),
    "mid_many": ([150 + (29 * e) % 140 - 70 for e in range(128)], 328, 200, dict(T=750, k=26)),
    "low_many": ([80 + (23 * e) % 90 - 45 if e % 7 else 0 for e in range(100)], 264, 328, dict(T=320, k=25)),
}


@pytest.mark.parametrize("name", CASES)
def test_expert_gemm_quantized(name):
    counts, d, f, kw = CASES[name]
    p = spec(counts, d, f, "bf16", **kw)
    r = Rows(p, counts, seed=d + f)
    n = len(counts)
    g = torch.Generator().manual_seed(d * f)
    x = r.draw(r.A, d)
    w = {k: torch.randint(-127, 128, (n, K, N), generator=g, dtype=torch.int8) for k, K, N in (("1", d, f), ("3", d, f), ("2", f, d))}
    s = {k: (torch.rand((n, N), generator=g) + 0.5) / (70.0 * K ** 0.5) for k, K, N in (("1", d, f), ("3", d, f), ("2", f, d))}
    h, y = M.expert_gemm_quantized(p, r.packed(x), offsets_of(counts), *(t for k in "132" for t in (M.pack_weights(w[k].cuda()), s[k].cuda())),
                                   out=(r.out(f), r.out(d)))
    torch.cuda.synchronize()
    r.check_tail(h, y)
    for e, seg in r.segments():
        if seg.start == seg.stop:
            continue
        q, sx = _quant(x[seg].numpy())
        q, sx = torch.from_numpy(q).double(), torch.from_numpy(sx).double()[:, None]
        a = q @ w["1"][e].double() * sx * s["1"][e].double()
        b = q @ w["3"][e].double() * sx * s["3"][e].double()
        ref = a * torch.sigmoid(a) * b
        # the two products carry three fp32 roundings each, the activation a few
        # ulp that grow with |a| where it decays exponentially (d log SiLU <= 1 + |a|)
        tol = (HALF["bf16"] + (2.0 ** -20) * (1 + a.abs())) * ref.abs()
        assert_within(h[seg], ref, tol, "h")
        # the down projection from the h that was stored
        q, sh = _quant(h[seg].float().cpu().numpy())
        ref = torch.from_numpy(q).double() @ w["2"][e].double() * torch.from_numpy(sh).double()[:, None] * s["2"][e].double()
        assert_within(y[seg], ref, (HALF["bf16"] + 4 * HALF["f32"]) * ref.abs(), "y")


def test_expert_gemm_quantized_near_bf16():
    """Quantised from the same weights: near the bf16 experts (a sanity check of
    scales and layout on real weights; 8-bit steps of a normal row are about 1%)."""
    counts, d, f = [20, 0, 90], 512, 256
    p = spec(counts, d, f, "bf16")
    r = Rows(p, counts, seed=3)
    w = [r.dev(r.draw(3, *s, scale=s[0] ** -0.5)) for s in ((d, f), (d, f), (f, d))]
    x, off = r.packed(r.draw(r.A, d)), offsets_of(counts)
    _, y = M.expert_gemm(p, x, off, *w)
    packed = [t for v in w for t in M.quantize_weights(v)]
    _, yq = M.expert_gemm_quantized(p, x, off, *packed)
    a, b = y[: r.A].double(), yq[: r.A].double()
    # a step is max / 127 and max of ~500 normal values about 3.3 sigma, so each
    # quantised operand is off by 3.3 / 127 / sqrt(12) = 0.75% (h: larger
    # maxima, about 2%); five of them in quadrature stay below 4%
    assert float((a - b).norm() / a.norm()) < 0.04


def test_quantized_captured():
    """Replays follow new inputs, with eager calls between them."""
    counts, d, f = [0, 5, 33, 130], 264, 200
    p = spec(counts, d, f, "bf16", T=130, k=2, E=16)
    r = Rows(p, counts, seed=9)
    w = [t for s in ((d, f), (d, f), (f, d)) for t in M.quantize_weights(r.dev(r.draw(4, *s, scale=s[0] ** -0.5)))]
    x, off = r.packed(r.draw(r.A, d)), offsets_of(counts)
    ws = M.alloc_workspace(p, M.MOE_CALL_EXPERT_GEMM_QUANTIZED)
    out = (r.out(f), r.out(d))

    def step():
        M.expert_gemm_quantized(p, x, off, *w, workspace=ws, out=out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x[: r.A] = r.dev(r.draw(r.A, d))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, out))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [272, 8208])
def test_not_finite_rows_and_channels(dtype, K):
    """A row or channel with an infinity or a NaN: that as its scale and zeros, and
    NaN in every product with it; its neighbours as without it."""
    r = Rows(spec([6], 8, 8, "bf16"), [6], seed=K)
    x = torch.randn((6, K), generator=r.gen).to(dtype)
    rq, rs = _quant(x.float().numpy())
    x[1, 3], x[2, K - 1], x[4, 0], x[4, 7] = float("nan"), float("-inf"), float("inf"), float("nan")
    q, s = M.quantize_rows(x.cuda())
    q, s = q.cpu(), s.cpu()
    assert bool(torch.isnan(s[[1, 4]]).all()) and float(s[2]) == float("inf") and not bool(q[[1, 2, 4]].any())
    for row in (0, 3, 5):
        assert np.array_equal(q[row].numpy(), rq[row]) and float(s[row]) == float(rs[row])
    w = torch.randn((K, 24), generator=r.gen).to(dtype)
    packed, sw = M.quantize_weights(w.cuda())
    bad = w.clone()
    bad[5, 2], bad[K - 1, 17] = float("nan"), float("inf")
    bad_packed, bad_sw = M.quantize_weights(bad.cuda())
    a, sa = M.quantize_rows(x[[0, 3, 5]].contiguous().cuda())
    one, two = M.gemm_quantized(a, sa, packed, sw), M.gemm_quantized(a, sa, bad_packed, bad_sw)
    keep = [c for c in range(24) if c not in (2, 17)]
    assert torch.equal(one[:, keep], two[:, keep]) and bool(torch.isnan(two[:, [2, 17]]).all())
    assert torch.isnan(bad_sw[2]) and torch.isinf(bad_sw[17])


def _experts(counts, d, f, seed, **kw):
    p = spec(counts, d, f, "bf16", **kw)
    r = Rows(p, counts, seed=seed)
    w = [t for s in ((d, f), (d, f), (f, d)) for t in M.quantize_weights(r.dev(r.draw(len(counts), *s, scale=s[0] ** -0.5)))]
    return p, r, w, r.draw(r.A, d), offsets_of(counts)


@pytest.mark.parametrize("name", ["streams", "mixed", "tiles"])
def test_expert_rows_that_are_not_finite(name):
    """They give NaN rows and leave every other row as it was."""
    counts, d, f, kw = CASES[name]
    p, r, w, x, off = _experts(counts, d, f, 11, **kw)
    ref = M.expert_gemm_quantized(p, r.packed(x), off, *w)
    xd = r.packed(x)
    hit = [0, r.A // 2, r.A - 1]
    xd[hit[0], 1], xd[hit[1], 0], xd[hit[2], d - 1] = float("nan"), float("inf"), float("-inf")
    got = M.expert_gemm_quantized(p, xd, off, *w)
    torch.cuda.synchronize()
    rest = [i for i in range(r.A) if i not in hit]
    for a, b in zip(ref, got):
        assert torch.equal(a[rest], b[rest]) and bool(torch.isnan(b[hit]).all())


def test_quantized_on_a_given_stream_and_two_at_once():
    jobs = []
    for seed, (counts, d, f, kw) in enumerate((CASES["mixed"], CASES["tiles"])):
        p, r, w, x, off = _experts(counts, d, f, seed, **kw)
        args = (r.packed(x), off, *w)
        jobs.append((p, args, M.expert_gemm_quantized(p, *args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for p, args, ref, s in jobs:
        with torch.cuda.stream(s):   # still busy when the calls return
            a = torch.ones((4096, 4096), device="cuda")
            for _ in range(8):
                a = a @ a * 1e-4
    got = [M.expert_gemm_quantized(p, *args, stream=s) for p, args, _, s in jobs]
    rows = [M.quantize_rows(args[0], stream=s) for _, args, _, s in jobs]
    spoil = [torch.full((M.workspace_bytes(p, M.MOE_CALL_EXPERT_GEMM_QUANTIZED),), 0x7F, dtype=torch.uint8, device="cuda")
             for p, *_ in jobs for _ in range(3)]
    torch.cuda.synchronize()
    del spoil
    for (p, args, ref, _), out, (q, sc) in zip(jobs, got, rows):
        assert all(torch.equal(a, b) for a, b in zip(ref, out))
        rq, rs = M.quantize_rows(args[0])
        assert torch.equal(q, rq) and torch.equal(sc.view(torch.int32), rs.view(torch.int32))


def test_offsets_beyond_32_bits():
    """Rows more than 4 GiB into their buffers: the sums are exact, so they equal
    the same rows in a small call bit by bit."""
    K, N, rows = 8192, 4104, 530_000
    g = torch.Generator(device="cuda").manual_seed(2)
    some = torch.randn((70, K), generator=g, device="cuda").bfloat16()
    x = some[:1].repeat(rows, 1)
    x[-70:] = some
    q, s = M.quantize_rows(x)
    del x
    q1, s1 = M.quantize_rows(some)
    assert torch.equal(q[-70:], q1) and torch.equal(s[-70:], s1) and q.numel() > 2 ** 32
    packed, sw = M.quantize_weights(torch.randn((K, N), generator=g, device="cuda").bfloat16())
    c = M.gemm_quantized(q, s, packed, sw)
    assert torch.equal(c[-70:], M.gemm_quantized(q1, s1, packed, sw)) and torch.equal(c[0], c[rows // 2])


def test_experts_beyond_32_bits():
    d, f, counts = 8192, 40, [299_950, 0, 10]
    p = spec(counts, d, f, "bf16", k=2)
    few = Rows(spec([50, 0, 10], d, f, "bf16"), [50, 0, 10], seed=8)
    w = [t for s in ((d, f), (d, f), (f, d)) for t in M.quantize_weights(few.dev(few.draw(3, *s, scale=s[0] ** -0.5)))]
    x = few.packed(few.draw(60, d))
    ref = M.expert_gemm_quantized(few.p, x, offsets_of([50, 0, 10]), *w)
    A = sum(counts)
    big = torch.ones((p.rows_max, d), dtype=torch.bfloat16, device="cuda")
    big[A - 60 : A] = x[:60]
    big[A:] = float("nan")
    out = tuple(torch.full((p.rows_max, n), -77.0, dtype=torch.bfloat16, device="cuda") for n in (f, d))
    M.expert_gemm_quantized(p, big, offsets_of(counts), *w, out=out)
    torch.cuda.synchronize()
    for a, b in zip(ref, out):
        assert torch.equal(a[:60], b[A - 60 : A]) and bool((b[A:] == -77.0).all())


@pytest.mark.parametrize("T", [1, 40, 300])
def test_layer_served_in_8_bits(T):
    """Route, dispatch, the 8-bit experts and combine, as a server runs them after
    quantising its weights once, against the layer in 64 bits on the same routing;
    and the experts' call against the same steps through the single products."""
    d, f, E, k, lo, n = 512, 256, 8, 3, 2, 4
    p = M.Spec(T, d, E, k, f, lo, n, "bf16")
    r = Rows(p, [0], seed=T)
    x, wg = r.draw(T, d), r.draw(d, E, scale=d ** -0.5)
    w1, w3, w2 = (r.draw(n, *s, scale=s[0] ** -0.5) for s in ((d, f), (d, f), (f, d)))
    weights = [M.quantize_weights(r.dev(w)) for w in (w1, w3, w2)]
    idx, wt = M.route(p, r.dev(x), r.dev(wg))
    D = M.dispatch(p, idx, r.dev(x))
    h, yp = M.expert_gemm_quantized(p, D["x_packed"], D["offsets"], *(t for pair in weights for t in pair))
    y = M.combine(p, yp, D["inv"], wt)
    torch.cuda.synchronize()
    ref = torch.zeros(T, d, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j]) - lo
            if 0 <= e < n:
                a = x[t] @ w1[e]
                ref[t] += float(wt[t, j]) * ((a * torch.sigmoid(a) * (x[t] @ w3[e])) @ w2[e])
    if float(ref.norm()) == 0:
        assert not bool(y.any())
        return
    # steps of a row or channel whose largest value is c sigma put c / 127 / sqrt(12)
    # on an operand: x (c up to 4.5, in both factors of h) 2%, W1, W3 and W2 (3.3)
    # 0.75% each, h (heavy tails, 9) 2%: 3.2% in quadrature, half as much again
    # for what single rows deviate
    assert float((y.cpu().double() - ref).norm() / ref.norm()) < 0.048
    # the same through the single products: y_packed from the stored h, bit by bit
    off = D["offsets"].cpu().tolist()
    for e in range(n):
        if off[e + 1] > off[e]:
            hq, sh = M.quantize_rows(h[off[e] : off[e + 1]])
            one = M.gemm_quantized(hq, sh, weights[2][0][e], weights[2][1][e])
            assert torch.equal(one, yp[off[e] : off[e + 1]])


def _nan(bits, *shape):
    """fp32 NaN of the given bits; memory filled with 0xFF bytes holds 0xFFFFFFFF."""
    return torch.full(shape, bits - (bits >> 31 << 32), dtype=torch.int32).view(torch.float32)


@pytest.mark.parametrize("bits", [0x7FFFFFFF, 0xFFFFFFFF, 0x7FFF8000, 0x7F800001])
@pytest.mark.parametrize("Mr,N,K", [(6, 24, 8208), (40, 24, 8208), (300, 1040, 1040)])   # the stream, and the tiles
def test_every_nan_gives_nan_products(bits, Mr, N, K):
    """A NaN of any payload, in a row, in a channel or in a given scale, is NaN in
    the bf16 and the fp32 output, and in these rows and columns alone."""
    g = torch.Generator().manual_seed(bits & 0xFFFF)
    x, w = torch.randn((Mr, K), generator=g), torch.randn((K, N), generator=g)
    x[1, 5], w[7, 3] = _nan(bits), _nan(bits)
    q, s = M.quantize_rows(x.cuda())
    packed, sw = M.quantize_weights(w.cuda())
    assert torch.isnan(s[1]) and torch.isnan(sw[3])
    s[4] = _nan(bits).cuda()
    sw[N - 1] = _nan(bits).cuda()
    want = torch.zeros((Mr, N), dtype=torch.bool, device="cuda")
    want[[1, 4]] = True
    want[:, [3, N - 1]] = True
    for dtype in (torch.bfloat16, torch.float32):
        assert torch.equal(torch.isnan(M.gemm_quantized(q, s, packed, sw, dtype=dtype)), want)


@pytest.mark.parametrize("bits", [0x7FFFFFFF, 0xFFFFFFFF])
@pytest.mark.parametrize("name", ["wide", "tiles"])   # the stream, and the tiles
def test_every_nan_scale_gives_nan_rows(bits, name):
    counts, d, f, kw = CASES[name]
    p, r, w, x, off = _experts(counts, d, f, 12, **kw)
    xd = r.packed(x)
    ref = M.expert_gemm_quantized(p, xd, off, *w)
    e, seg = next((e, s) for e, s in r.segments() if s.start < s.stop)
    # channel 5 of the down projection: that column of y alone
    s2 = w[5].clone()
    s2[e, 5] = _nan(bits).cuda()
    h, y = M.expert_gemm_quantized(p, xd, off, *w[:5], s2)
    assert torch.equal(h, ref[0])
    want = torch.zeros((p.rows_max, d), dtype=torch.bool, device="cuda")
    want[seg, 5] = True
    assert torch.equal(torch.isnan(y[: r.A]), want[: r.A])
    # channel 6 of either gated product: that column of h, and then every column of y
    for k in (1, 3):
        scales = list(w)
        scales[k] = w[k].clone()
        scales[k][e, 6] = _nan(bits).cuda()
        h, y = M.expert_gemm_quantized(p, xd, off, *scales)
        want = torch.zeros((p.rows_max, f), dtype=torch.bool, device="cuda")
        want[seg, 6] = True
        assert torch.equal(torch.isnan(h[: r.A]), want[: r.A])
        assert bool(torch.isnan(y[seg]).all()) and torch.equal(y[: r.A][seg.stop :], ref[1][: r.A][seg.stop :])
