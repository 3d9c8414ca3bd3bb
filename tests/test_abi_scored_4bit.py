"""Host-only checks of the scored-routing and 4-bit calls (no GPU needed): invalid
arguments are rejected with the documented status before anything is launched.
Fake device addresses are never dereferenced.
"""
import copy
import ctypes
import os
import pickle

import pytest
import torch

import combine_router_top_amd as M
from tests.test_abi_training_quantized import BIG, FAKE, INV, ODD, UNS, WS, _p

pytestmark = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="libmoe.so not built")

SELECT = ["logits", "balance", "topk_idx", "topk_w"]
ROUTE = ["x", "w_gate", "bias", "balance", "logits", "topk_idx", "topk_w"]
BACK = ["x", "w_gate", "logits", "topk_idx", "dtopk_w", "dx_add", "dlogits", "dx", "dw_gate", "dbias"]
EXPERTS = ["x_packed", "offsets", "w1", "s1", "z1", "w3", "s3", "z3", "w2", "s2", "z2", "h", "y_packed"]
CALLS = {"moe_select": (SELECT, False), "moe_route_scored": (ROUTE, True), "moe_route_backward": (BACK, True),
         "moe_expert_gemm_fourbit": (EXPERTS, True)}
OPTIONAL = {"balance", "bias", "dx_add", "dlogits", "dx", "dw_gate", "dbias", "z1", "z3", "z2"}
RULE = M.GateRule(M.MOE_SCORE_SIGMOID, 2, 1, 2, 1, 1.0)


def _call(name, p=None, args=None, rule=RULE, group=64, ws=FAKE, wsb=BIG, **named):
    names, has_ws = CALLS[name]
    args = [FAKE] * len(names) if args is None else args
    args = [named.get(n, a) for n, a in zip(names, args)]
    p = _p() if p is None else p
    second = group if name == "moe_expert_gemm_fourbit" else (None if rule is None else ctypes.byref(rule))
    return getattr(M.lib(), name)(ctypes.byref(p), second, *args, *((ws, wsb, None) if has_ws else (None,)))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kw,status", [(dict(T=-1), INV), (dict(k=9), INV), (dict(n_local=0), INV), (dict(flags=0x80), INV),
                                       (dict(d=100), UNS), (dict(f=12), UNS), (dict(dtype=7), UNS)])
def test_problem_validation(name, kw, status):
    assert _call(name, _p(**kw)) == status
    assert M.lib().moe_last_error()


@pytest.mark.parametrize("name", CALLS)
def test_pointers(name):
    aligned = {"x", "w_gate", "dx_add", "dx", "dw_gate", "x_packed", "w1", "w3", "w2", "h", "y_packed", "s1", "s3", "s2"}
    for arg in CALLS[name][0]:
        if arg not in OPTIONAL and not (name == "moe_route_scored" and arg == "logits"):
            assert _call(name, **{arg: None}) == INV, arg
            assert arg.encode() in M.lib().moe_last_error()
        if arg in aligned:
            assert _call(name, **{arg: ODD}) == UNS, arg
            assert arg.encode() in M.lib().moe_last_error()
        if arg in ("z1", "z2", "z3"):
            assert _call(name, **{arg: FAKE + 2}) == UNS, arg


@pytest.mark.parametrize("name", ["moe_select", "moe_route_scored", "moe_route_backward"])
@pytest.mark.parametrize("fields,E,k,status", [
    ((2, 1, 1, 1, 1, 1.0), 8, 2, INV),                 # no such score
    ((0, 0, 1, 1, 1, 1.0), 8, 2, INV), ((0, 3, 1, 1, 1, 1.0), 8, 2, INV), ((0, -2, 1, 1, 1, 1.0), 8, 2, INV),
    ((0, 128, 64, 1, 1, 1.0), 128, 2, UNS),            # more than 64 groups
    ((0, 4, 0, 1, 1, 1.0), 8, 2, INV), ((0, 4, 5, 1, 1, 1.0), 8, 2, INV),
    ((0, 4, 2, 0, 1, 1.0), 8, 2, INV), ((0, 4, 2, 3, 1, 1.0), 8, 2, INV), ((0, 8, 2, 2, 1, 1.0), 8, 2, INV),
    ((0, 4, 1, 1, 1, 1.0), 8, 3, INV),                 # k beyond the groups that stay
    ((0, 1, 1, 1, 2, 1.0), 8, 2, INV), ((0, 1, 1, 1, -1, 1.0), 8, 2, INV),
    ((0, 1, 1, 1, 1, float("nan")), 8, 2, INV), ((1, 1, 1, 1, 0, float("inf")), 8, 2, INV)])
def test_rules(name, fields, E, k, status):
    assert _call(name, _p(E=E, n_local=E, k=k), rule=M.GateRule(*fields)) == status
    assert M.lib().moe_last_error()


@pytest.mark.parametrize("name", ["moe_select", "moe_route_scored", "moe_route_backward"])
def test_no_rule(name):
    assert _call(name, rule=None) == INV and b"gate" in M.lib().moe_last_error()


@pytest.mark.parametrize("name,call", [("moe_route_scored", M.MOE_CALL_ROUTE_SCORED),
                                       ("moe_route_backward", M.MOE_CALL_ROUTE_BACKWARD),
                                       ("moe_expert_gemm_fourbit", M.MOE_CALL_EXPERT_GEMM_FOURBIT)])
def test_workspace(name, call):
    p = _p(T=4096, d=1024, f=1024)   # long segments: also the 4-bit experts have some
    need = M.lib().moe_workspace_bytes(ctypes.byref(p), call)
    assert need > 0
    assert _call(name, p, ws=None) == WS
    assert _call(name, p, wsb=need - 1) == WS
    assert _call(name, p, ws=FAKE + 16) == WS
    assert M.lib().moe_workspace_bytes(ctypes.byref(_p(T=0)), call) == 0


def test_router_gradient_outputs():
    none = dict(dlogits=None, dx=None, dw_gate=None, dbias=None)
    assert _call("moe_route_backward", dx_add=None, **none) == INV
    assert _call("moe_route_backward", **{**none, "dlogits": FAKE}) == INV   # dx_add without dx
    assert b"dx_add" in M.lib().moe_last_error()
    assert _call("moe_route_backward", w_gate=None) == INV and _call("moe_route_backward", x=None) == INV
    assert _call("moe_route_backward", _p(d=(1 << 20) + 8, f=8)) == UNS
    assert _call("moe_route_backward", _p(T=(1 << 27) + 1, d=8, f=8, k=1, dtype=M.MOE_DTYPE_F32)) == UNS


def test_empty_batches_launch_nothing():
    p = _p(T=0)
    nothing = dict(ws=None, wsb=0)
    assert _call("moe_select", p, [None] * 4) == M.MOE_OK
    assert _call("moe_route_scored", p, [None, FAKE] + [None] * 5, **nothing) == M.MOE_OK
    assert _call("moe_route_backward", p, [None] * 10, **nothing) == M.MOE_OK
    assert _call("moe_expert_gemm_fourbit", p, x_packed=None, h=None, y_packed=None, **nothing) == M.MOE_OK
    assert M.lib().moe_gemm_fourbit(0, 64, 64, 32, None, FAKE, FAKE, None, None, M.MOE_DTYPE_BF16, None, 0, None) == M.MOE_OK


def test_experts_take_bf16_rows_and_known_groups():
    assert _call("moe_expert_gemm_fourbit", _p(dtype=M.MOE_DTYPE_F32)) == UNS
    for group in (0, 16, 96, 256, -32):
        assert _call("moe_expert_gemm_fourbit", group=group) == UNS, group
    assert _call("moe_expert_gemm_fourbit", _p(d=(1 << 20) + 8, f=8)) == UNS
    assert _call("moe_expert_gemm_fourbit", _p(f=(1 << 20) + 8, d=8)) == UNS


def test_packed_weights_arguments():
    L = M.lib()
    assert L.moe_packed_weights_fourbit_bytes(1, 128, 16) == 1024
    assert L.moe_packed_weights_fourbit_bytes(3, 136, 24) == 3 * 2 * 2 * 1024
    for n, K, N in ((0, 64, 16), (1, 0, 16), (1, 64, 0), (1025, 64, 16), (1, 12, 16), (1, 64, 12), (1, (1 << 20) + 8, 8),
                    (1, 8, (1 << 21) + 8), (1, 1 << 20, 2048)):
        assert L.moe_packed_weights_fourbit_bytes(n, K, N) == 0 and L.moe_last_error()
        assert L.moe_pack_weights_fourbit(n, K, N, FAKE, FAKE, None) in (INV, UNS)
        assert L.moe_quantize_weights_fourbit(n, K, N, 32, M.MOE_DTYPE_BF16, FAKE, FAKE, FAKE, FAKE, None) in (INV, UNS)
    assert L.moe_pack_weights_fourbit(1, 64, 16, None, FAKE, None) == INV
    assert L.moe_pack_weights_fourbit(1, 64, 16, FAKE, ODD, None) == UNS
    q = lambda g=32, dt=M.MOE_DTYPE_F32, w=FAKE, o=FAKE, s=FAKE, z=FAKE: L.moe_quantize_weights_fourbit(1, 64, 16, g, dt, w, o, s, z, None)  # noqa: E731
    assert q(g=48) == UNS and q(dt=3) == UNS and q(w=ODD) == UNS and q(o=ODD) == UNS and q(s=FAKE + 4) == UNS and q(z=FAKE + 1) == UNS
    assert q(w=None) == INV and q(o=None) == INV and q(s=None) == INV


def test_gemm_4bit_arguments():
    def g(Mr=4, N=16, K=64, G=32, a=FAKE, b=FAKE, s=FAKE, z=FAKE, c=FAKE, dt=M.MOE_DTYPE_BF16, ws=FAKE, wsb=BIG):
        return M.lib().moe_gemm_fourbit(Mr, N, K, G, a, b, s, z, c, dt, ws, wsb, None)
    assert g(Mr=-1) == INV and g(N=0) == INV and g(K=0) == INV
    assert g(Mr=(1 << 30) + 1) == UNS and g(N=(1 << 21) + 8) == UNS and g(K=20) == UNS and g(N=12) == UNS and g(dt=9) == UNS
    assert g(G=0) == UNS and g(G=65) == UNS
    for name in ("a", "b", "s", "c"):
        assert g(**{name: None}) == INV, name
    for name in ("a", "b", "c"):
        assert g(**{name: ODD}) == UNS, name
    assert g(s=FAKE + 4) == UNS and g(z=FAKE + 2) == UNS
    many = dict(Mr=4096, N=1024, K=1024)
    need = M.gemm_4bit_workspace_bytes(4096, 1024, 1024)
    assert need >= 4096 * 1024 * 2
    assert g(ws=None, wsb=0, **many) == WS and g(wsb=need - 1, **many) == WS and g(ws=FAKE + 16, **many) == WS
    assert M.gemm_4bit_workspace_bytes(1, 1024, 1024) == 0 and M.gemm_4bit_workspace_bytes(0, 8, 8) == 0
    for sizes in ((-1, 8, 8), (8, 12, 8), (8, 8, 12)):
        with pytest.raises(M.MoeError):
            M.gemm_4bit_workspace_bytes(*sizes)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    f32, bf, u8, i32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
    z = lambda *s, dt=f32: torch.zeros(s, dtype=dt)  # noqa: E731
    p, gate = M.Spec(4, 16, 8, 2, 8, 0, 8, "bf16"), M.Gate()
    with pytest.raises(ValueError, match="logits must be a contiguous device tensor"):
        M.select(p, gate, z(4, 8))
    with pytest.raises(ValueError, match="logits: expected"):
        M.select(p, gate, z(4, 8, dt=bf))
    with pytest.raises(ValueError, match="x: expected"):
        M.route_scored(p, gate, z(4, 8, dt=bf), z(16, 8, dt=bf))
    with pytest.raises(ValueError, match="logits"):
        M.route_backward(p, gate, None, None, z(4, 4), z(4, 2, dt=i32), z(4, 2))
    with pytest.raises(ValueError, match="score"):
        M.Gate("tanh").c()
    with pytest.raises(ValueError, match="32 bits"):
        M.Gate(groups=1 << 40).c()
    with pytest.raises(ValueError, match="expected \\[n, K, N\\]"):
        M.pack_weights_4bit(z(1, 1, 16, 16, dt=u8))
    with pytest.raises(M.MoeError):
        M.pack_weights_4bit(z(20, 16, dt=u8))
    with pytest.raises(ValueError, match="group: expected"):
        M.quantize_weights_4bit(z(32, 16), group=48)
    with pytest.raises(ValueError, match="w: expected torch.bfloat16 or torch.float32"):
        M.quantize_weights_4bit(z(32, 16, dt=torch.float16))
    with pytest.raises(ValueError, match="group: expected"):
        M.gemm_4bit(z(2, 16, dt=bf), z(1, 1, 64, 4, dt=i32), z(1, 8, dt=bf), group=100)
    with pytest.raises(ValueError, match="a must be"):
        M.gemm_4bit(z(2, 16, dt=bf), z(1, 1, 64, 4, dt=i32), z(1, 8, dt=bf))
    w = (z(8, 1, 1, 64, 4, dt=i32), z(8, 1, 8, dt=bf), None)
    with pytest.raises(ValueError, match="x_packed must be"):
        M.expert_gemm_4bit(p, z(8, 16, dt=bf), z(9, dt=i32), *w, *w, *w)


def test_sizes_beyond_32_bits_are_refused_not_cut_off():
    meta = lambda *s, dt=torch.uint8: torch.empty(s, dtype=dt, device="meta")  # noqa: E731
    wide = 2 ** 32 + 16
    for n, K, N in ((wide, 64, 16), (1, wide, 16), (1, 64, wide)):
        with pytest.raises(ValueError, match="32 bits"):
            M.packed_weights_4bit_bytes(n, K, N)
        with pytest.raises(ValueError, match="32 bits"):
            M.pack_weights_4bit(meta(n, K, N))
    with pytest.raises(ValueError, match="32 bits"):
        M.gemm_4bit(meta(wide, 16, dt=torch.bfloat16), meta(1), meta(1, 16, dt=torch.bfloat16))


def test_a_used_rule_can_be_copied_and_pickled():
    g = M.Gate("sigmoid", 8, 4, 2, True, 2.5)
    g.ref()
    for h in (copy.copy(g), copy.deepcopy(g), pickle.loads(pickle.dumps(g))):
        assert h == g and h.c().scale == 2.5 and h.c().topk_groups == 4
