"""Measured cases of scored routing with its gradient, and of products with 4-bit weights.

Operators (plain forms below; with ``own`` the library's calls):
  select    experts and weights of every token from its router logits: softmax or sigmoid scores, a
            bias for balance, groups of experts, top-k, weights renormalised or not
  back      backward pass of the router: gradients of logits, rows, gate matrix and gate bias
  linear    rows times 4-bit weights with a scale (and a zero point) for each group of K
  experts   gated expert blocks with such weights

Rows of ``experts`` are packed by expert: expert e owns rows offsets[e] .. offsets[e + 1) of buffers
that hold T * min(k, n) rows; the rows behind the last segment stay as they were (zero here).
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    grouped = dict(E=256, k=8, score="sigmoid", groups=8, topk_groups=4, group_top=2, bias=True, renorm=True, scale=2.5)
    sparse = dict(E=256, k=8, n=32, d=7168, f=2048)
    return [
        # one token in decode: latency of the choice
        dict(name="select_token", op="select", T=1, masked=0, **grouped),
        # a 4096-token batch of the 256-expert layer: sigmoid scores, balance bias, 4 of 8 groups
        dict(name="select_4096", op="select", T=4096, masked=0, **grouped),
        # a long batch over few experts, plain softmax whose weights are not renormalised, one in ten masked out
        dict(name="select_softmax", op="select", T=30011, masked=7, E=72, k=6, score="softmax", groups=1, topk_groups=1,
             group_top=1, bias=False, renorm=False, scale=1.0),
        # the router's gradient in a training step of that layer
        dict(name="back_4096", op="back", T=4096, d=7168, dtype="bf16", **grouped),
        # a dense gradient (softmax over all experts), sizes off every tile
        dict(name="back_softmax", op="back", T=1003, d=1032, dtype="bf16", E=24, k=4, score="softmax", groups=1,
             topk_groups=1, group_top=1, bias=False, renorm=False, scale=1.0),
        # the small fp32 layer that numerics are checked with
        dict(name="back_fp32", op="back", T=64, d=128, dtype="f32", E=8, k=2, score="softmax", groups=1, topk_groups=1,
             group_top=1, bias=False, renorm=True, scale=1.0),
        # one token through a projection: a weight stream of a few microseconds
        dict(name="linear_token", op="linear", M=1, K=7168, N=2048, G=128, zero=False),
        # a few dozen tokens in decode, short groups, a last group that is not full
        dict(name="linear_odd", op="linear", M=37, K=4104, N=1416, G=32, zero=True),
        # a prefill batch
        dict(name="linear_4096", op="linear", M=4096, K=4096, N=14336, G=128, zero=True),
        # one token in decode: the 8 experts it chose, a row each
        dict(name="experts_token", op="experts", T=1, rows=8, spread="one", E=32, k=8, n=32, d=7168, f=2048, G=128, zero=False),
        # 128 tokens in decode: 4 rows an expert, all weights streamed once
        dict(name="experts_decode", op="experts", T=128, rows=128, spread="even", G=128, zero=False, **sparse),
        # 4096 tokens in prefill
        dict(name="experts_prefill", op="experts", T=4096, rows=4096, spread="even", G=128, zero=False, **sparse),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def _gate(rng):
    score = rng.choice(["softmax", "sigmoid"])
    groups = rng.choice([1, 1, 2, 4, 8])
    E = groups * _log(rng, 2, 256 // groups)
    topk_groups = rng.randint(1, groups)
    k = rng.randint(1, min(16, topk_groups * (E // groups)))
    return dict(E=E, k=k, score=score, groups=groups, topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                bias=rng.random() < 0.5, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))


def draw(rng):
    op = rng.choice(["select", "back", "linear", "linear", "experts"])
    if op == "select":
        c = _gate(rng)
        return dict(op=op, T=_log(rng, 1, 32768), masked=rng.choice([0, 0, min(3, c["E"] - 1)]), **c)
    if op == "back":
        f32 = rng.random() < 0.2
        c = _gate(rng)
        return dict(op=op, T=_log(rng, 1, 512 if f32 else 8192), d=_log(rng, 64, 512 if f32 else 7168, 8),
                    dtype="f32" if f32 else "bf16", **c)
    G, zero = rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 64, 8192, 8), N=_log(rng, 64, 14336, 8), G=G, zero=zero)
    n = _log(rng, 1, 48)
    E = n * rng.choice([1, 1, 2, 4, 8])
    k = rng.randint(1, min(E, 8))
    T, d, f = _log(rng, 1, 8192), _log(rng, 64, 7168, 8), _log(rng, 64, 4096, 8)
    rows = max(1, min(T * min(k, n), int(T * k * n / E * rng.uniform(0.5, 1.5))))
    if T * d * f > 1e10:   # keep a drawn case below the largest listed one
        T = max(1, int(1e10 / (d * f)))
        rows = max(1, min(rows, T * min(k, n)))
    return dict(op=op, rows=rows, spread=rng.choice(["even", "skew"]), T=T, E=E, k=k, n=n, d=d, f=f, G=G, zero=zero)


def _counts(case):
    """Rows of each expert, largest first: mild variation ("even"), a power law whose last experts
    may get nothing ("skew"), or one row each until they are gone ("one"); no expert has more rows
    than there are tokens."""
    n, left, T = case["n"], case["rows"], case["T"]
    if case["spread"] == "one":
        return [1 if e < left else 0 for e in range(n)]
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
def _weights(g, n, K, N, G, zero):
    """n matrices of normal weights quantised to 4 bits: values 0 .. 15 as bytes [n, K, N], scales
    bf16 and zero points [n, groups, N] (None: 8 everywhere), and the values as the products read
    them: words [n, N/16, K/128, 64, 4], where lane 16 a + c of a block holds column c, word s its
    k = 32 s + 8 a .. + 7, value 2 p + h of them in bits 16 h + 4 p .. + 3 of the word, which is
    then rotated left by 3 bits; padding holds zeros."""
    ng, kb, nb = -(-K // G), -(-K // 128), -(-N // 16)
    q = torch.empty((n, K, N), dtype=torch.uint8, device="cuda")
    s = torch.empty((n, ng, N), dtype=torch.bfloat16, device="cuda")
    z = torch.empty((n, ng, N), dtype=torch.uint8, device="cuda") if zero else None
    packed = torch.empty((n, nb, kb, 64, 4), dtype=torch.int32, device="cuda")
    shift = torch.tensor([16 * h + 4 * p for p in range(4) for h in range(2)], device="cuda")
    for e in range(n):
        w = torch.randn((K, N), generator=g, device="cuda") / math.sqrt(K)
        if zero:
            w += 0.3 / math.sqrt(K)
        w = torch.nn.functional.pad(w, (0, 0, 0, ng * G - K)).view(ng, G, N)
        if zero:
            lo, hi = w.amin(1).clamp(max=0), w.amax(1).clamp(min=0)
            s[e] = (hi - lo) / 15
            step = s[e].float().clamp(min=1e-30)
            z[e] = torch.round(-lo / step).clamp(0, 15)
            v = torch.round(w / step[:, None]) + z[e][:, None]
        else:
            s[e] = w.abs().amax(1) / 7
            v = torch.round(w / s[e].float().clamp(min=1e-30)[:, None]) + 8
        q[e] = v.clamp_(0, 15).view(ng * G, N)[:K]
        full = torch.zeros((kb * 128, nb * 16), dtype=torch.int64, device="cuda")
        full[:K, :N] = q[e]
        #            k block, word, lane group, value, column block, column
        word = (full.view(kb, 4, 4, 8, nb, 16) << shift[:, None, None]).sum(3)
        word = ((word << 3) | (word >> 29)) & 0xFFFFFFFF
        word = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
        packed[e] = word.permute(3, 0, 2, 4, 1).reshape(nb, kb, 64, 4)
    return q, s, z, packed


def _logits(g, T, E, masked):
    l = torch.randn((T, E), generator=g, device="cuda") * 1.5
    if masked:
        l[:, torch.randperm(E, generator=g, device="cuda")[:masked]] = -math.inf
    return l


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], _dtype(case)
    st = dict(case=case)

    def normal(shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

    if op in ("select", "back"):
        T, E, k = case["T"], case["E"], case["k"]
        st["balance"] = torch.randn(E, generator=g, device="cuda") * 0.1 if case["bias"] else None
        if op == "select":
            st["logits"] = _logits(g, T, E, case["masked"])
            return st
        d = case["d"]
        st["logits"] = _logits(g, T, E, 0)
        # what the forward pass chose: distinct experts of each token, likely ones more often
        noise = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-20)
        st["idx"] = (st["logits"] - torch.log(-torch.log(noise))).argsort(1, descending=True)[:, :k].to(torch.int32).contiguous()
        st["dw"] = torch.randn((T, k), generator=g, device="cuda") * math.sqrt(d) * 0.1
        st["x"], st["wg"] = normal((T, d)), normal((d, E), 1 / math.sqrt(d))
        st["out"] = (torch.zeros((T, E), device="cuda"), torch.zeros((T, d), dtype=dt, device="cuda"),
                     torch.zeros((d, E), dtype=dt, device="cuda"), torch.zeros((E,), device="cuda"))
        return st
    G, zero = case["G"], case["zero"]
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        st["x"] = normal((M, K))
        q, s, z, packed = _weights(g, 1, K, N, G, zero)
        st["q"], st["s"], st["z"], st["w"] = q[0], s[0], None if z is None else z[0], packed[0]
        st["out"] = torch.zeros((M, N), dtype=dt, device="cuda")
        return st
    T, k, d, f, n = (case[v] for v in ("T", "k", "d", "f", "n"))
    cap = T * min(k, n)
    counts = _counts(case)
    order = torch.randperm(n, generator=g, device="cuda").tolist()
    offsets = [0]
    for i in order:
        offsets.append(offsets[-1] + counts[i])
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    st["longest"], st["bounds"] = max(counts), offsets
    st["x"] = torch.zeros((cap, d), dtype=dt, device="cuda")
    st["x"][: offsets[-1]] = normal((offsets[-1], d))
    for name, K, N in (("1", d, f), ("3", d, f), ("2", f, d)):
        st["q" + name], st["s" + name], st["z" + name], st["w" + name] = _weights(g, n, K, N, G, zero)
    st["out"] = (torch.zeros((cap, f), dtype=dt, device="cuda"), torch.zeros((cap, d), dtype=dt, device="cuda"))
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_select(st):
    # scores in 64 bits: in 32 their rounding would decide between neighbours
    case, l = st["case"], st["logits"].double()
    T, E = l.shape
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    c = s if st["balance"] is None else s + st["balance"].double()
    if case["score"] == "softmax" and st["balance"] is None:
        order = l   # the same order, and none of it lost where the exponential underflows
    else:
        order = c
    low = -1e300   # below every value, above the experts of groups that were not chosen
    order, c = (torch.where(l == -math.inf, low, t).clamp(min=low) for t in (order, c))
    if case["groups"] > 1:
        per = E // case["groups"]
        member = c.view(T, case["groups"], per)
        value = member.sort(2, descending=True)[0][..., : case["group_top"]].sum(2)
        best = value.sort(dim=1, descending=True, stable=True)[1][:, : case["topk_groups"]]
        open_ = torch.zeros((T, case["groups"]), dtype=torch.bool, device="cuda").scatter_(1, best, True)
        order = torch.where(open_.repeat_interleave(per, 1), order, -math.inf)
    idx = order.sort(dim=1, descending=True, stable=True)[1][:, : case["k"]]
    w = s.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), (w * case["scale"]).float()


def _plain_back(st):
    case, dt = st["case"], _dtype(st["case"])
    l, idx, dw = st["logits"], st["idx"].long(), st["dw"] * case["scale"]
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    top = s.gather(1, idx)
    if case["renorm"]:
        total = top.sum(1, keepdim=True)
        dw = (dw - (dw * top).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, idx, dw)
    if case["score"] == "sigmoid":
        dl = ds * s * (1 - s)
    else:
        dl = s * (ds - (ds * s).sum(1, keepdim=True))
    dx = dl @ st["wg"].float().t()
    dg = st["x"].float().t() @ dl
    return dl, dx.to(dt), dg.to(dt), dl.sum(0)


def _values(q, s, z, G):
    """The weights that 4-bit values stand for, fp32, [..., K, N]."""
    K = q.shape[-2]
    s, z = (t if t is None else t.float().repeat_interleave(G, -2)[..., :K, :] for t in (s, z))
    return (q.float() - (8.0 if z is None else z)) * s


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


def _plain(st):
    case, op, dt = st["case"], st["case"]["op"], _dtype(st["case"])
    if op == "select":
        return _plain_select(st)
    if op == "back":
        return _plain_back(st)
    if op == "linear":
        return (st["x"].float() @ _values(st["q"], st["s"], st["z"], case["G"])).to(dt)
    seg = _Segments(st)
    x = seg.spread(st["x"])
    a = torch.bmm(x, _values(st["q1"], st["s1"], st["z1"], case["G"]))
    b = torch.bmm(x, _values(st["q3"], st["s3"], st["z3"], case["G"]))
    h = a / (1 + torch.exp(-a)) * b
    y = torch.bmm(h, _values(st["q2"], st["s2"], st["z2"], case["G"]))
    return seg.pack(h, dt), seg.pack(y, dt)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    if not own:
        return _plain(st)
    import combine_router_top_amd as moe

    case, op = st["case"], st["case"]["op"]
    if op == "linear":
        return moe.gemm_4bit(st["x"], st["w"], st["s"], st["z"], group=case["G"], out=st["out"])
    p = moe.Spec(case["T"], case.get("d", 8), case["E"], case["k"], case.get("f", 8), 0, case.get("n", case["E"]),
                 case.get("dtype", "bf16"))
    if op == "experts":
        return moe.expert_gemm_4bit(p, st["x"], st["offsets"], st["w1"], st["s1"], st["z1"], st["w3"], st["s3"],
                                    st["z3"], st["w2"], st["s2"], st["z2"], group=case["G"], out=st["out"])
    gate = moe.Gate(case["score"], groups=case["groups"], topk_groups=case["topk_groups"],
                    group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
    if op == "select":
        return moe.select(p, gate, st["logits"], st["balance"])
    return moe.route_backward(p, gate, st["x"], st["wg"], st["logits"], st["idx"], st["dw"], out=st["out"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "select":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 4 * E + 8 * T * k, "flops": T * E * 4}
    if op == "back":
        T, E, k, d = case["T"], case["E"], case["k"], case["d"]
        s = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * s * (T * d + d * E) + 8 * T * E + 8 * T * k + 4 * E, "flops": 4 * T * d * E}
    G = case["G"]

    def weights(K, N):
        return K * N / 2 + -(-K // G) * N * (3 if case["zero"] else 2)

    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + weights(K, N) + 2 * M * N, "flops": 2 * M * K * N}
    d, f, A = case["d"], case["f"], case["rows"]
    active = sum(c > 0 for c in _counts(case))
    return {"bytes": 4 * A * d + 2 * A * f + active * (2 * weights(d, f) + weights(f, d)), "flops": 6 * A * d * f}


# ---------------------------------------------------------------------------
# definitions in 64 bits
# ---------------------------------------------------------------------------
def _dequantised(q, s, z, G):
    """One matrix [K, N], group by group."""
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for i, lo in enumerate(range(0, q.shape[0], G)):
        base = z[i].double() if z is not None else 8.0
        out[lo: lo + G] = (q[lo: lo + G].double() - base) * s[i].double()
    return out


def _exact_select(st):
    case = st["case"]
    l = st["logits"].double()
    if case["score"] == "sigmoid":
        s = 1 / (1 + (-l).exp())
    else:
        s = (l - torch.logsumexp(l, 1, keepdim=True)).exp()
    sharp = case["score"] == "softmax" and st["balance"] is None
    value = l.clone() if sharp else s + (0 if st["balance"] is None else st["balance"].double())
    value[l == -math.inf] = -1e300
    if case["groups"] > 1:
        of_group = (s if sharp else value).masked_fill(l == -math.inf, -1e300).unflatten(1, (case["groups"], -1))
        total = torch.zeros(of_group.shape[:2], dtype=torch.float64, device="cuda")
        rest = of_group.clone()
        for _ in range(min(case["group_top"], rest.shape[2])):
            top, at = rest.max(2)
            total += top
            rest.scatter_(2, at[..., None], -math.inf)
        # a group's rank: how many groups are better, or as good and before it
        before = torch.arange(case["groups"], device="cuda")
        better = (total[:, None, :] > total[:, :, None]) | ((total[:, None, :] == total[:, :, None]) & (before < before[:, None]))
        shut = better.sum(2) >= case["topk_groups"]
        value = value.unflatten(1, (case["groups"], -1)).masked_fill(shut[..., None], -math.inf).flatten(1)
    chosen = torch.empty((l.shape[0], case["k"]), dtype=torch.int64, device="cuda")
    place = torch.arange(l.shape[1], device="cuda")
    for j in range(case["k"]):
        top = value.amax(1, keepdim=True)
        chosen[:, j] = torch.where(value == top, place, l.shape[1]).amin(1)
        value.scatter_(1, chosen[:, j: j + 1], -math.inf)
    w = s.gather(1, chosen)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return chosen.to(torch.int32), w * case["scale"]


def _exact_back(st):
    case = st["case"]
    l, dw = st["logits"].double(), st["dw"].double()
    picked = torch.nn.functional.one_hot(st["idx"].long(), l.shape[1]).double()     # [T, k, E]
    if case["score"] == "sigmoid":
        s = 1 / (1 + (-l).exp())
    else:
        s = (l - torch.logsumexp(l, 1, keepdim=True)).exp()
    sel = torch.einsum("tke,te->tk", picked, s)
    up = dw * case["scale"]
    if case["renorm"]:
        p = sel / sel.sum(1, keepdim=True)
        up = (up - (up * p).sum(1, keepdim=True)) / sel.sum(1, keepdim=True)
    ds = torch.einsum("tke,tk->te", picked, up)
    dl = ds * s / (1 + l.exp()) if case["score"] == "sigmoid" else ds * s - s * (ds * s).sum(1, keepdim=True)
    return dl, dl @ st["wg"].double().T, st["x"].double().T @ dl, dl.sum(0)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "select":
        return _exact_select(st)
    if op == "back":
        return _exact_back(st)
    if op == "linear":
        return st["x"].double() @ _dequantised(st["q"], st["s"], st["z"], case["G"])
    b, n, d, f, cap = st["bounds"], case["n"], case["d"], case["f"], st["x"].shape[0]
    h_all, y_all = (torch.zeros((cap, v), dtype=torch.float64, device="cuda") for v in (f, d))
    for e in range(n):
        r = slice(b[e], b[e + 1])
        if b[e] == b[e + 1]:
            continue
        m1, m3, m2 = (_dequantised(st["q" + v][e], st["s" + v][e], None if st["z" + v] is None else st["z" + v][e], case["G"])
                      for v in ("1", "3", "2"))
        x = st["x"][r].double()
        left = x @ m1
        h_all[r] = left * torch.sigmoid(left) * (x @ m3)
        y_all[r] = h_all[r] @ m2
    return h_all, y_all
