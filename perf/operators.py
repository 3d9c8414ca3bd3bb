"""Measured cases of the expert operators for training and for 8-bit serving.

Operators (plain forms below; with ``own`` the library's calls):
  train     forward of the gated expert blocks that keeps what the backward pass reads
  back      backward pass of the gated expert blocks: gradients of the rows and of all weights
  combine   backward pass of the weighted un-permute
  linear    rows quantised to 8 bits, times 8-bit weights with a scale per channel
  experts   gated expert blocks with 8-bit weights and activations

Rows are packed by expert: expert e owns rows offsets[e] .. offsets[e + 1) of buffers that hold
T * min(k, n) rows; the rows behind the last segment stay as they were (zero here).
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    sparse = dict(T=4096, E=256, k=8, n=32, d=7168, f=2048)
    return [
        # a training step's forward through one GPU's 32 of 256 experts, about 128 rows each
        dict(name="train_sparse", op="train", rows=4096, spread="even", dtype="bf16", **sparse),
        # a dense (shared) gated block in training, one segment, sizes off every tile
        dict(name="train_dense", op="train", rows=2000, spread="even", dtype="bf16",
             T=2000, E=1, k=1, n=1, d=4104, f=1416),
        # the backward pass of the sparse layer
        dict(name="back_sparse", op="back", rows=4096, spread="even", dtype="bf16", **sparse),
        # dense routing, long segments: the matrix cores' case and the largest one
        dict(name="back_dense8", op="back", rows=32768, spread="even", dtype="bf16",
             T=16384, E=8, k=2, n=8, d=4096, f=14336),
        # imbalanced routing with experts that got no row, odd widths
        dict(name="back_skew", op="back", rows=1500, spread="skew", dtype="bf16",
             T=1000, E=24, k=4, n=12, d=1032, f=328),
        # the small fp32 layer that numerics are checked with
        dict(name="back_fp32", op="back", rows=128, spread="even", dtype="f32",
             T=64, E=8, k=2, n=8, d=128, f=256),
        # gradient through the weighted un-permute of a 4096-token batch
        dict(name="combine_4096", op="combine", T=4096, E=256, k=8, n=32, d=7168, dtype="bf16"),
        # the same for a few tokens: latency
        dict(name="combine_16", op="combine", T=16, E=8, k=2, n=8, d=4096, dtype="bf16"),
        # one token through an 8-bit projection: a weight stream of a few microseconds
        dict(name="linear_token", op="linear", M=1, K=7168, N=2048),
        # a prefill batch through an 8-bit projection
        dict(name="linear_4096", op="linear", M=4096, K=4096, N=14336),
        # 128 tokens in decode: 4 rows an expert, all weights streamed once
        dict(name="experts_decode", op="experts", rows=128, spread="even",
             T=128, E=256, k=8, n=32, d=7168, f=2048),
        # 4096 tokens in prefill
        dict(name="experts_prefill", op="experts", rows=4096, spread="even", **sparse),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["train", "back", "combine", "linear", "experts"])
    if op == "combine":
        E = _log(rng, 1, 256)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 16)), n=rng.randint(1, E),
                    d=_log(rng, 64, 7168, 8), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 64, 8192, 16), N=_log(rng, 64, 14336, 8))
    n = _log(rng, 1, 48)
    E = n * rng.choice([1, 1, 2, 4, 8])
    k = rng.randint(1, min(E, 8))
    dtype = "bf16" if op == "experts" or rng.random() < 0.85 else "f32"
    small = dtype == "f32"
    T = _log(rng, 1, 256 if small else 8192)
    d = _log(rng, 64, 512 if small else 7168, 8)
    f = _log(rng, 64, 512 if small else 4096, 8)
    rows = max(1, min(T * min(k, n), int(T * k * n / E * rng.uniform(0.5, 1.5))))
    spread = rng.choice(["even", "skew"])
    if T * d * f > 4e10 / 4:   # keep a drawn case below the largest listed one
        T = max(1, int(1e10 / (d * f)))
        rows = max(1, min(rows, T * min(k, n)))
    c = dict(op=op, rows=rows, spread=spread, T=T, E=E, k=k, n=n, d=d, f=f)
    if op != "experts":
        c["dtype"] = dtype
    return c


def _counts(case):
    """Rows of each expert, largest first: mild variation ("even"), or a power law whose last
    experts may get nothing ("skew"); no expert has more rows than there are tokens."""
    n, left, T = case["n"], case["rows"], case["T"]
    w = [(1.0 + 0.3 * math.sin(7.3 * e)) if case["spread"] == "even" else (e + 1.0) ** -1.5 for e in range(n)]
    w.sort(reverse=True)
    out = []
    for e in range(n):
        rest = sum(w[e:])
        c = int(round(left * w[e] / rest)) if e + 1 < n else left
        c = max(min(c, T, left), left - T * (n - e - 1), 0)
        out.append(c)
        left -= c
    return out


def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, shape, scale, dtype):
    """Normal values; drawn in slices of the first axis, so that large weights need no fp32 copy."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    if out.numel() < 1 << 28:
        return out.copy_(torch.randn(shape, generator=g, device="cuda") * scale)
    for i in range(shape[0]):
        out[i].copy_(torch.randn(shape[1:], generator=g, device="cuda") * scale)
    return out


def _weights_i8(g, n, K, N):
    """Weights of n experts quantised per output channel: values [n, K, N], scales [n, N], and the
    values in the order the product reads them: [n, N/16, K/64, 4, 16, 16] with element
    (k, j) at [j / 16, k / 64, (k % 64) / 16, j % 16, k % 16], zero behind K and N."""
    kp, np_ = -(-K // 64) * 64, -(-N // 16) * 16
    q = torch.empty((n, K, N), dtype=torch.int8, device="cuda")
    s = torch.empty((n, N), dtype=torch.float32, device="cuda")
    packed = torch.zeros((n, np_ // 16, kp // 64, 4, 16, 16), dtype=torch.int8, device="cuda")
    for e in range(n):
        w = torch.randn((K, N), generator=g, device="cuda") / math.sqrt(K)
        top = w.abs().amax(0)
        s[e] = top / 127
        q[e] = torch.round(w * (127 / top)).to(torch.int8)
        full = torch.zeros((kp, np_), dtype=torch.int8, device="cuda")
        full[:K, :N] = q[e]
        packed[e] = full.view(kp // 64, 4, 16, np_ // 16, 16).permute(3, 0, 1, 4, 2)
    return q, s, packed


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], _dtype(case)
    st = dict(case=case)
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        st["x"] = _normal(g, (M, K), 1.0, dt)
        q, s, packed = _weights_i8(g, 1, K, N)
        st["w"], st["ws"], st["packed"] = q[0], s[0], packed[0]
        st["out"] = torch.zeros((M, N), dtype=dt, device="cuda")
        return st
    if op == "combine":
        T, k, d, n, E = (case[v] for v in ("T", "k", "d", "n", "E"))
        rows = T * min(k, n)
        # each slot is local with probability n / E, at most min(k, n) of a token's
        score = torch.rand((T, k), generator=g, device="cuda")
        local = score < n / E
        rank = score.argsort(1).argsort(1)
        local &= rank < min(k, n)
        order = torch.rand(T * k, generator=g, device="cuda").masked_fill(~local.view(-1), 2.0).argsort()
        place = torch.empty(T * k, dtype=torch.int64, device="cuda")
        place[order] = torch.arange(T * k, device="cuda")
        st["inv"] = torch.where(local.view(-1), place, torch.full_like(place, -1)).to(torch.int32)
        st["w"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)
        st["dy"] = _normal(g, (T, d), 1.0, dt)
        st["yp"] = _normal(g, (rows, d), 0.5, dt)
        st["out"] = (torch.zeros((rows, d), dtype=dt, device="cuda"), torch.zeros((T, k), device="cuda"))
        return st
    T, k, d, f, n = (case[v] for v in ("T", "k", "d", "f", "n"))
    cap = T * min(k, n)
    counts = _counts(case)
    order = torch.randperm(n, generator=g, device="cuda").tolist()
    counts = [counts[i] for i in order]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    st["longest"] = max(counts)
    st["bounds"] = offsets
    A = offsets[-1]

    def rows_of(width, scale):
        t = torch.zeros((cap, width), dtype=dt, device="cuda")
        t[:A] = _normal(g, (A, width), scale, dt)
        return t

    def zeros(*shape):
        return torch.zeros(shape, dtype=dt, device="cuda")

    st["x"] = rows_of(d, 1.0)
    if op == "experts":
        for name, K, N in (("1", d, f), ("3", d, f), ("2", f, d)):
            st["q" + name], st["s" + name], st["p" + name] = _weights_i8(g, n, K, N)
        st["out"] = (zeros(cap, f), zeros(cap, d))
        return st
    st["w1"] = _normal(g, (n, d, f), 1 / math.sqrt(d), dt)
    st["w3"] = _normal(g, (n, d, f), 1 / math.sqrt(d), dt)
    st["w2"] = _normal(g, (n, f, d), 1 / math.sqrt(f), dt)
    if op == "train":
        st["out"] = (zeros(cap, f), zeros(cap, f), zeros(cap, f), zeros(cap, d))
        return st
    # what the forward pass kept: products with the statistics that the inputs above give
    st["g"], st["u"] = rows_of(f, 1.0), rows_of(f, 1.0)
    st["h"] = (torch.nn.functional.silu(st["g"].float()) * st["u"].float()).to(dt)
    st["dy"] = rows_of(d, 1.0)
    st["out"] = (zeros(cap, d), zeros(n, d, f), zeros(n, d, f), zeros(n, f, d))
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
class _Segments:
    """Rows packed by expert to [n, longest, width] and back."""

    def __init__(self, st):
        off, cap = st["offsets"].long(), st["x"].shape[0]
        n, longest = off.numel() - 1, max(1, st["longest"])
        slot = torch.arange(longest, device="cuda")
        self.valid = (slot < (off[1:] - off[:-1])[:, None])[..., None]
        self.row = (off[:-1, None] + slot).clamp_(max=cap - 1)
        p = torch.arange(cap, device="cuda")
        self.e = torch.searchsorted(off[1:].contiguous(), p, right=True).clamp_(max=n - 1)
        self.slot = (p - off[self.e]).clamp_(0, longest - 1)
        self.live = (p < off[-1])[:, None]

    def spread(self, t):
        return torch.where(self.valid, t[self.row].float(), 0.0)

    def pack(self, t, dtype):
        return torch.where(self.live, t[self.e, self.slot], 0.0).to(dtype)


def _quantise(x):
    top = x.abs().amax(-1, keepdim=True)
    inverse = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    return torch.round(x * inverse), top / 127.0


def _product_i8(a, b):
    """Exact product of 8-bit values held in fp32: slices of 1024 stay below 2^24, their sums in 64 bits."""
    K = a.shape[-1]
    c = -(-K // 1024)
    pad = c * 1024 - K
    a = torch.nn.functional.pad(a, (0, pad)).unflatten(-1, (c, 1024)).movedim(-2, 0).contiguous()
    b = torch.nn.functional.pad(b, (0, 0, 0, pad)).unflatten(-2, (c, 1024)).movedim(-3, 0).contiguous()
    return torch.matmul(a, b).sum(0, dtype=torch.float64)


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    dt = _dtype(case)
    if op == "linear":
        q, s = _quantise(st["x"].float())
        return (_product_i8(q, st["w"].float()).float() * s * st["ws"]).to(dt)
    if op == "combine":
        T, k = st["w"].shape
        inv = st["inv"].long()
        local = inv >= 0
        dy = st["dy"].float()
        token = torch.arange(T * k, device="cuda") // k
        rows = st["yp"].shape[0]
        dyp = torch.zeros((rows + 1, dy.shape[1]), device="cuda")
        dyp[torch.where(local, inv, rows)] = dy[token] * st["w"].view(-1, 1)
        dw = (dy[token] * st["yp"][inv.clamp(min=0)].float()).sum(1)
        return dyp[:rows].to(dt), torch.where(local, dw, 0.0).view(T, k)
    seg = _Segments(st)
    x = seg.spread(st["x"])
    if op == "experts":
        q, s = _quantise(x)
        a = _product_i8(q, st["q1"].float()).float() * s * st["s1"][:, None]
        b = _product_i8(q, st["q3"].float()).float() * s * st["s3"][:, None]
        h = (a / (1 + torch.exp(-a)) * b).to(dt)   # the rows that are quantised next hold dt
        q, s = _quantise(h.float())
        y = _product_i8(q, st["q2"].float()).float() * s * st["s2"][:, None]
        return seg.pack(h.float(), dt), seg.pack(y, dt)
    w1, w3, w2 = st["w1"].float(), st["w3"].float(), st["w2"].float()
    if op == "train":
        a, b = torch.bmm(x, w1), torch.bmm(x, w3)
        h = a / (1 + torch.exp(-a)) * b
        y = torch.bmm(h, w2)
        return seg.pack(a, dt), seg.pack(b, dt), seg.pack(h, dt), seg.pack(y, dt)
    a, b, h, dy = (seg.spread(st[v]) for v in ("g", "u", "h", "dy"))
    dh = torch.bmm(dy, w2.transpose(1, 2))
    s = 1 / (1 + torch.exp(-a))
    da, db = dh * b * s * (1 + a * (1 - s)), dh * a * s
    dx = torch.bmm(da, w1.transpose(1, 2)) + torch.bmm(db, w3.transpose(1, 2))
    xt = x.transpose(1, 2)
    return (seg.pack(dx, dt), torch.bmm(xt, da).to(dt), torch.bmm(xt, db).to(dt),
            torch.bmm(h.transpose(1, 2), dy).to(dt))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    if not own:
        return _plain(st)
    import combine_router_top_amd as moe

    case, op, out = st["case"], st["case"]["op"], st["out"]
    if op == "linear":
        q, s = moe.quantize_rows(st["x"])
        return moe.gemm_quantized(q, s, st["packed"], st["ws"], out=out)
    p = moe.Spec(case["T"], case["d"], case["E"], case["k"], case.get("f", 8), 0, case["n"],
                 case.get("dtype", "bf16"))
    if op == "combine":
        return moe.combine_backward(p, st["dy"], st["yp"], st["inv"], st["w"], out=out)
    if op == "experts":
        return moe.expert_gemm_quantized(p, st["x"], st["offsets"], st["p1"], st["s1"], st["p3"],
                                         st["s3"], st["p2"], st["s2"], out=out)
    if op == "train":
        return moe.expert_gemm_train(p, st["x"], st["offsets"], st["w1"], st["w3"], st["w2"], out=out)
    return moe.expert_gemm_backward(p, st["x"], st["offsets"], st["w1"], st["w3"], st["w2"], st["g"],
                                    st["u"], st["h"], st["dy"], out=out)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    s = 4 if case.get("dtype") == "f32" else 2
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": M * K * 2 + K * N + 4 * N + M * N * 2, "flops": 2 * M * K * N}
    if op == "combine":
        T, k, d = case["T"], case["k"], case["d"]
        rows = T * k * case["n"] / case["E"]
        return {"bytes": T * d * s + 2 * rows * d * s + 12 * T * k, "flops": 3 * rows * d}
    d, f, n, A = case["d"], case["f"], case["n"], case["rows"]
    active = sum(c > 0 for c in _counts(case))
    if op == "experts":
        return {"bytes": A * d * 2 + active * (3 * d * f + 4 * (2 * f + d)) + A * f * 2 + A * d * 2,
                "flops": 6 * A * d * f}
    if op == "train":
        return {"bytes": s * (A * d + active * 3 * d * f + 3 * A * f + A * d), "flops": 6 * A * d * f}
    return {"bytes": s * (2 * A * d + 3 * A * f + active * 3 * d * f + A * d + n * 3 * d * f),
            "flops": 12 * A * d * f}


# ---------------------------------------------------------------------------
# definitions in 64 bits
# ---------------------------------------------------------------------------
def _steps_i8(v):
    """Whole steps and step size of each row, as the quantiser defines them (single precision)."""
    v = v.to(torch.float32)
    big = v.abs().max(dim=1).values
    mul = torch.zeros_like(big)
    mul[big > 0] = 127.0 / big[big > 0]
    return (v * mul[:, None]).round().double(), (big / 127.0).double()


def exact(case, seed):
    st = prepare(case, seed)
    op, dt = case["op"], _dtype(case)
    if op == "linear":
        q, s = _steps_i8(st["x"])
        return q @ st["w"].double() * s[:, None] * st["ws"].double()
    if op == "combine":
        T, k, d = case["T"], case["k"], case["d"]
        inv = st["inv"].view(T, k).long()
        dyp = torch.zeros(st["yp"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        dy = st["dy"].double()
        for j in range(k):
            t = (inv[:, j] >= 0).nonzero()[:, 0]
            r = inv[t, j]
            dyp[r] = st["w"][t, j].double()[:, None] * dy[t]
            dw[t, j] = torch.einsum("td,td->t", dy[t], st["yp"][r].double())
        return dyp, dw
    b, n, d, f, cap = st["bounds"], case["n"], case["d"], case["f"], st["x"].shape[0]

    def full(*shape):
        return torch.zeros(shape, dtype=torch.float64, device="cuda")

    if op == "experts":
        h_all, y_all = full(cap, f), full(cap, d)
        for e in range(n):
            r = slice(b[e], b[e + 1])
            if b[e] == b[e + 1]:
                continue
            q, s = _steps_i8(st["x"][r])
            left = q @ st["q1"][e].double() * s[:, None] * st["s1"][e].double()
            right = q @ st["q3"][e].double() * s[:, None] * st["s3"][e].double()
            h_all[r] = (left * torch.sigmoid(left) * right).to(dt).double()
            q, s = _steps_i8(h_all[r])
            y_all[r] = q @ st["q2"][e].double() * s[:, None] * st["s2"][e].double()
        return h_all, y_all
    if op == "train":
        out = full(cap, f), full(cap, f), full(cap, f), full(cap, d)
        for e in range(n):
            r = slice(b[e], b[e + 1])
            x = st["x"][r].double()
            out[0][r] = x @ st["w1"][e].double()
            out[1][r] = x @ st["w3"][e].double()
            out[2][r] = out[0][r] * torch.sigmoid(out[0][r]) * out[1][r]
            out[3][r] = out[2][r] @ st["w2"][e].double()
        return out
    dx, dw1, dw3, dw2 = full(cap, d), full(n, d, f), full(n, d, f), full(n, f, d)
    for e in range(n):
        r = slice(b[e], b[e + 1])
        x, left, right, h, dy = (st[v][r].double() for v in ("x", "g", "u", "h", "dy"))
        dh = dy @ st["w2"][e].double().T
        gate = torch.sigmoid(left)
        dleft = dh * right * (gate + left * gate * (1 - gate))
        dright = dh * (left * gate)
        dx[r] = dleft @ st["w1"][e].double().T + dright @ st["w3"][e].double().T
        dw1[e], dw3[e], dw2[e] = x.T @ dleft, x.T @ dright, h.T @ dy
    return dx, dw1, dw3, dw2
