"""Choices and weights of scored routing where fp32 alone would go wrong, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import combine_router_top_amd as M
from tests.segments import assert_within
from tests.test_gpu_scored import EPS, _check_select, _choose, _logits, _scores, _spec


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


@pytest.mark.gpu
@pytest.mark.parametrize("score,groups,group_top", [("softmax", 1, 1), ("sigmoid", 1, 1), ("softmax", 8, 1), ("softmax", 8, 2), ("sigmoid", 8, 2)])
@pytest.mark.parametrize("E", [24, 64, 120, 256, 1000])
@pytest.mark.parametrize("where", ["logits", "balance", "both"])
def test_masks_of_the_lowest_value(score, groups, group_top, E, where):
    """Values of the type's lowest come before -inf and after everything else, also where k reaches them."""
    T, k, lowest = 70, 9, torch.finfo(torch.float32).min
    gate = M.Gate(score, groups, max(1, groups // 2), group_top, False)
    g = torch.Generator().manual_seed(E)
    l, b = _logits(T, E, E + 3), None
    if where != "balance":
        pick = torch.rand((T, E), generator=g)
        l[pick < 0.9] = lowest
        l[pick < 0.4] = -math.inf
        l[0], l[1, 1:] = lowest, lowest
    if where != "logits":
        pick = torch.rand(E, generator=g)
        b = torch.randn(E, generator=g) * 0.2
        b[pick < 0.9] = lowest
        b[pick < 0.4] = -math.inf
    idx, w = M.select(_spec(T, E, k), gate, l.cuda(), None if b is None else b.cuda())
    _check_select(gate, k, l, b, idx, w)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,group_top", [(64, 32, 2), (64, 32, 1), (256, 8, 2), (24, 1, 1)])
def test_balances_of_every_size(score, E, groups, group_top):
    T, k = 40, 8
    gate = M.Gate(score, groups, max(1, groups // 3), group_top, False)
    sizes = torch.tensor([3e38, 1e38, 1.0, 0.0, -1.0, -1e38, -3e38, torch.finfo(torch.float32).min, -math.inf])
    for seed in range(12):
        g = torch.Generator().manual_seed(seed)
        b = sizes[torch.randint(0, sizes.numel(), (E,), generator=g)]
        l = _logits(T, E, seed, "masked" if seed % 3 == 0 else "normal")
        idx, w = M.select(_spec(T, E, k), gate, l.cuda(), b.cuda())
        _check_select(gate, k, l, b, idx, w)


@pytest.mark.gpu
@pytest.mark.parametrize("far", [20.0, 80.0, 95.0, 104.0, 200.0])
@pytest.mark.parametrize("groups", [1, 8])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_chosen_far_below_the_best(score, groups, far):
    """The balance chooses experts whose scores fp32 does not hold; under renorm only their ratios count."""
    T, E, k = 300, 64, 6
    l = _logits(T, E, 11) * 0.5
    l[:, : E // 2] += far if score == "softmax" else 0.0
    l[:, E // 2:] -= 0.0 if score == "softmax" else far
    b = torch.zeros(E)
    b[E // 2:] = 4.0
    b += torch.randn(E, generator=torch.Generator().manual_seed(2)) * 0.1
    gate = M.Gate(score, groups, max(1, groups // 2), min(2, groups), True, 2.5)
    idx, w = M.select(_spec(T, E, k), gate, l.cuda(), b.cuda())
    assert int(idx.min()) >= E // 2
    _check_select(gate, k, l, b, idx, w)
