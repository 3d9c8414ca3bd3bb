"""The router's gradients at sizes of training, where rows and gate matrix take tiles of 256 x 256
tokens and columns and units of shares of the tokens."""
import pytest
import torch

import combine_router_top_amd as M
from tests.test_gpu_scored import _back_inputs, _check_back, _spec

pytestmark = pytest.mark.gpu

LARGE = [(1030, 300, 8, 7168), (4100, 256, 8, 2056), (8300, 24, 4, 1032), (16500, 13, 3, 264), (600, 1000, 9, 12296), (32700, 8, 2, 64), (10007, 72, 6, 776),
         (4098, 64, 6, 2056)]


@pytest.mark.parametrize("T,E,k,d", LARGE)
@pytest.mark.parametrize("gate", [M.Gate("sigmoid", scale=2.5), M.Gate("softmax", renorm=False)], ids=str)
def test_large(T, E, k, d, gate):
    inputs = _back_inputs(T, E, k, d, "bf16")
    l, idx, dw, x, wg, add = (v.cuda() for v in inputs)
    p = _spec(T, E, k, d, "bf16")
    out = M.route_backward(p, gate, x, wg, l, idx, dw)
    _check_back(gate, "bf16", inputs, out)
    again = M.route_backward(p, gate, x, wg, l, idx, dw)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    added = M.route_backward(p, gate, x, wg, l, idx, dw, dx_add=add)
    _check_back(gate, "bf16", inputs, (None, added[1], None, None), inputs[5])
    assert all(torch.equal(added[i], out[i]) for i in (0, 2, 3))
    place = add.clone()      # in place, nothing else wanted
    M.route_backward(p, gate, None, wg, l, idx, dw, dx_add=place, out=(None, place, None, None))
    assert torch.equal(place, added[1])
    size = M.workspace_bytes(p, M.MOE_CALL_ROUTE_BACKWARD)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")   # NaN in every type
    one = torch.full_like(out[2], 7)
    M.route_backward(p, gate, x, None, l, idx, dw, workspace=ws, out=(None, None, one, None))
    assert torch.equal(one, out[2])
    rows = torch.full_like(x, 7)
    M.route_backward(p, gate, None, wg, l, idx, dw, workspace=ws, out=(None, rows, None, None))
    assert torch.equal(rows, out[1])
