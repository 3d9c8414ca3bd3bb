"""4-bit products at the ends of what rows, scales and weights can hold."""
import pytest
import torch

import combine_router_top_amd as M
from tests import cases_4bit as C
from tests.segments import HALF, assert_within
from tests.test_gpu_4bit import _dev, _slack, _weights
from tests.test_gpu_4bit_kernels import _join

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", C.PRODUCTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_nan_scale_of_any_payload(name, dtype):
    (T, K, N, G), _ = C.PRODUCTS[name]
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    q, s, z, _ = _weights(K, N, G, True, T)
    p, s, z = M.pack_weights_4bit(q.cuda()), *_dev(s, z)
    clean = M.gemm_4bit(x, p, s, z, group=G, dtype=dtype)
    bits = s.view(torch.int16)
    columns = {1: 0x7FFF, 4: -1, 9: 0x7FC0, 22: 0x7F81}
    for i, (col, payload) in enumerate(columns.items()):
        bits[i % s.shape[0], col] = payload
    got = M.gemm_4bit(x, p, s, z, group=G, dtype=dtype)
    bad = torch.zeros(N, dtype=torch.bool)
    bad[list(columns)] = True
    assert bool(torch.isnan(got[:, bad.cuda()]).all())
    assert torch.equal(got[:, ~bad.cuda()], clean[:, ~bad.cuda()])


# Rows whose values are all of one sign and near the largest (or all tiny).  With scales of 2^-19 to 2^-17
# a group's sum of |x W| is at most 128 * 15 * 2^-17 of the largest, and groups differ in sign.
DENSE = ["narrow, 16 rows", "narrow, long", "narrow, 32 rows", "wide, 16 rows", "wide, 32 rows", "wide, 16 rows, a block ahead",
         "wide, 32 rows, a block ahead", "wide, blocks of rows", "tiles of 64", "K in parts, 64 rows"]


@pytest.mark.parametrize("name", DENSE)
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("exponent", [127, 122, 117, -100, -112, -124, -130])
def test_dense_rows_of_one_sign(name, zero, exponent):
    (T, K, N, G), _ = C.PRODUCTS[name]
    g = torch.Generator().manual_seed(T)
    x = ((1 + 0.99 * torch.rand((T, K), generator=g)) * 2.0 ** exponent).to(torch.bfloat16)
    x[1:2] *= -1
    q, s, z, _ = _weights(K, N, G, zero, T, whole=True)
    s = (s * 2.0 ** (-18 if exponent > 0 else 0)).to(torch.bfloat16)
    up = lambda t: t.double().repeat_interleave(G, 0)[:K]  # noqa: E731
    X, w = x.double(), (q.double() - (8 if z is None else up(z))) * up(s)
    ref, slack = X @ w, _slack(X, s, z, G, w) + _join(K, X, w)
    slack = slack + 3 * s.shape[0] * 2.0 ** -137   # a group's share of the streams' sums in multiples of 2^-137
    args = (x.cuda(), M.pack_weights_4bit(q.cuda()), *_dev(s, z))
    for dtype, half in ((torch.bfloat16, HALF["bf16"]), (torch.float32, HALF["f32"])):
        got = M.gemm_4bit(*args, group=G, dtype=dtype)
        assert_within(got, ref, slack * (1 + half) + half * ref.abs(), str(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantiser_at_the_largest_weights(dtype):
    """With zero points a group's range can pass fp32's largest value; its scale does not."""
    K, N, G = 136, 24, 64
    top = torch.finfo(torch.bfloat16).max
    w = ((torch.rand((K, N), generator=torch.Generator().manual_seed(3)) * 2 - 1) * top).to(dtype)
    w[0], w[1], w[64], w[65], w[128], w[129] = top, -top, top, -top, top, -top
    p, s, z = M.quantize_weights_4bit(w.cuda(), G, True)
    step = torch.tensor(2 * top / 15, dtype=torch.float64).to(torch.bfloat16)
    assert bool((s.cpu() == step).all())
    assert bool((z.cpu() == torch.round(top / step.float())).all())
    values = torch.clamp(torch.round(w.float() / step.float()) + z.cpu().float()[0], 0, 15).to(torch.uint8)
    assert torch.equal(p, M.pack_weights_4bit(values.cuda()))
