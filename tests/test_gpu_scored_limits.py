"""Choices and weights of scored routing where fp32 alone would go wrong, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import combine_router_top_amd as M
from tests.segments import assert_within
from tests.test_gpu_scored import EPS, _choose, _logits, _scores, _spec


def _choose_all(gate, k, l, balance):
    """What _choose gives for finite values, all tokens at once."""
    T, E = l.shape
    s = _scores(gate, l)
    c = s + balance.double()
    value = c.view(T, gate.groups, -1).sort(2, descending=True)[0][..., : gate.group_top].sum(2)
    stay = value.sort(dim=1, descending=True, stable=True)[1][:, : gate.topk_groups]
    open_ = torch.zeros((T, gate.groups), dtype=torch.bool).scatter_(1, stay, True).repeat_interleave(E // gate.groups, 1)
    idx = torch.where(open_, c, -math.inf).sort(dim=1, descending=True, stable=True)[1][:, :k]
    top = s.gather(1, idx)
    if gate.renorm:
        top = top / top.sum(1, keepdim=True)
    return idx.to(torch.int32).numpy(), top * gate.scale


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,topk_groups,k", [(256, 8, 4, 8), (64, 32, 9, 8), (1024, 64, 20, 9), (160, 8, 3, 6)])
@pytest.mark.parametrize("size", [1.0, 64.0, 1e4, 1e6])
def test_groups_whose_two_best_cancel(score, E, groups, topk_groups, k, size):
    """A group's value is a small difference of large numbers: one expert of each group is lifted
    by ``size``, the others are lowered by as much."""
    T, per = 2048, E // groups
    b = torch.full((E,), -size)
    b[torch.arange(groups) * per + torch.arange(groups) % per] = size
    l = _logits(T, E, int(size) + E)
    gate = M.Gate(score, groups, topk_groups, 2, True, 2.5)
    ri, rw = _choose_all(gate, k, l, b)
    few = _choose(gate, k, l[:8], b)
    assert np.array_equal(few[0], ri[:8]) and torch.equal(few[1], rw[:8])
    idx, w = M.select(_spec(T, E, k), gate, l.cuda(), b.cuda())
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert_within(w, rw, (k + 60) * EPS * rw + 1e-37, "weights")
