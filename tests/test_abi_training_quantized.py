"""Host-only checks of the training and 8-bit calls (no GPU needed): invalid
arguments are rejected with the documented status before anything is launched.
Fake device addresses are never dereferenced: validation fails first, or the
call has nothing to do.
"""
import ctypes
import os

import pytest
import torch

import combine_router_top_amd as M

pytestmark = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="libmoe.so not built")

FAKE, ODD = 0x10000, 0x10004   # 16-byte aligned, and not
BIG = 1 << 40
INV, UNS, WS = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED, M.MOE_ERR_WORKSPACE


def _p(**kw):
    base = dict(T=64, d=128, E=8, k=2, f=256, expert_lo=0, n_local=8, dtype=M.MOE_DTYPE_BF16, flags=0)
    base.update(kw)
    return M.Problem(**base)


def _call(name, p, args, ws=FAKE, wsb=BIG, has_ws=True):
    tail = (ws, wsb, None) if has_ws else (None,)
    return getattr(M.lib(), name)(ctypes.byref(p) if p is not None else None, *args, *tail)


TRAIN = ["x_packed", "offsets", "w1", "w3", "w2", "g", "u", "h", "y_packed"]
BACK = ["x_packed", "offsets", "w1", "w3", "w2", "g", "u", "h", "dy_packed", "dx_packed", "dw1", "dw3", "dw2"]
QUANT = ["x_packed", "offsets", "w1", "s1", "w3", "s3", "w2", "s2", "h", "y_packed"]
COMB = ["dy", "y_packed", "inv", "topk_w", "dy_packed", "dtopk_w"]
CALLS = [("moe_expert_gemm_train", TRAIN, False), ("moe_expert_gemm_backward", BACK, True),
         ("moe_expert_gemm_quantized", QUANT, True), ("moe_combine_backward", COMB, False)]


@pytest.mark.parametrize("name,names,has_ws", CALLS)
@pytest.mark.parametrize("kw,status", [(dict(T=-1), INV), (dict(k=9), INV), (dict(n_local=0), INV), (dict(flags=0x80), INV),
                                       (dict(d=100), UNS), (dict(f=12), UNS), (dict(dtype=7), UNS)])
def test_problem_validation(name, names, has_ws, kw, status):
    assert _call(name, _p(**kw), [FAKE] * len(names), has_ws=has_ws) == status
    assert M.lib().moe_last_error()


@pytest.mark.parametrize("name,names,has_ws", CALLS)
def test_null_problem(name, names, has_ws):
    assert _call(name, None, [FAKE] * len(names), has_ws=has_ws) == INV


@pytest.mark.parametrize("name,names,has_ws", CALLS)
def test_pointers(name, names, has_ws):
    # arguments that may be NULL, and those of 4-byte elements read one by one
    may_be_null = {"dx_packed", "dw1", "dw3", "dw2", "topk_w", "dtopk_w"}
    plain = {"offsets", "inv", "topk_w", "dtopk_w"}
    for i, arg in enumerate(names):
        if arg not in may_be_null:
            args = [FAKE] * len(names)
            args[i] = None
            assert _call(name, _p(), args, has_ws=has_ws) == INV, arg
            assert arg.encode() in M.lib().moe_last_error()
        if arg not in plain:
            args = [FAKE] * len(names)
            args[i] = ODD
            assert _call(name, _p(), args, has_ws=has_ws) == UNS, arg
            assert arg.encode() in M.lib().moe_last_error()


@pytest.mark.parametrize("name,names,call", [
    ("moe_expert_gemm_backward", BACK, M.MOE_CALL_EXPERT_GEMM_BACKWARD),
    ("moe_expert_gemm_quantized", QUANT, M.MOE_CALL_EXPERT_GEMM_QUANTIZED)])
def test_workspace(name, names, call):
    p = _p()
    need = M.lib().moe_workspace_bytes(ctypes.byref(p), call)
    assert need > 0
    args = [FAKE] * len(names)
    assert _call(name, p, args, ws=None) == WS
    assert _call(name, p, args, wsb=need - 1) == WS
    assert _call(name, p, args, ws=FAKE + 16) == WS
    assert M.lib().moe_workspace_bytes(ctypes.byref(_p(T=0)), call) == 0


def test_training_widths_are_bounded():
    assert _call("moe_expert_gemm_train", _p(d=(1 << 20) + 8, f=8), [FAKE] * len(TRAIN), has_ws=False) == UNS
    assert _call("moe_expert_gemm_train", _p(f=(1 << 20) + 8, d=8), [FAKE] * len(TRAIN), has_ws=False) == UNS


def test_backward_needs_an_output_and_bounded_widths():
    args = [FAKE] * len(BACK)
    args[9:] = [None] * 4
    assert _call("moe_expert_gemm_backward", _p(), args) == INV
    assert _call("moe_expert_gemm_backward", _p(d=(1 << 20) + 8, f=8), [FAKE] * len(BACK)) == UNS
    assert _call("moe_expert_gemm_backward", _p(f=(1 << 20) + 8, d=8), [FAKE] * len(BACK)) == UNS


def test_quantized_experts_take_bf16_rows_and_exact_depths():
    args = [FAKE] * len(QUANT)
    assert _call("moe_expert_gemm_quantized", _p(dtype=M.MOE_DTYPE_F32), args) == UNS
    assert _call("moe_expert_gemm_quantized", _p(d=131072, f=64), args) == UNS
    assert _call("moe_expert_gemm_quantized", _p(d=64, f=131072), args) == UNS


def test_empty_batches_launch_nothing():
    p = _p(T=0)
    assert _call("moe_expert_gemm_train", p, [None, FAKE, FAKE, FAKE, FAKE] + [None] * 4, ws=None, wsb=0) == M.MOE_OK
    assert _call("moe_expert_gemm_quantized", p, [None] + [FAKE] * 7 + [None] * 2, ws=None, wsb=0) == M.MOE_OK
    assert _call("moe_combine_backward", p, [None] * 6, has_ws=False) == M.MOE_OK
    L = M.lib()
    assert L.moe_quantize_rows(0, 64, M.MOE_DTYPE_BF16, None, None, None, None) == M.MOE_OK
    assert L.moe_gemm_quantized(0, 64, 64, None, None, FAKE, FAKE, None, M.MOE_DTYPE_BF16, None) == M.MOE_OK
    # the backward pass of an empty batch has weight gradients to write: only dx_packed wanted, none
    args = [None, FAKE, FAKE, FAKE, FAKE] + [None] * 4 + [FAKE, None, None, None]
    assert _call("moe_expert_gemm_backward", p, args, ws=None, wsb=0) == M.MOE_OK


def test_quantize_rows_arguments():
    q = lambda rows=4, K=64, dt=M.MOE_DTYPE_BF16, x=FAKE, o=FAKE, s=FAKE: M.lib().moe_quantize_rows(rows, K, dt, x, o, s, None)  # noqa: E731
    assert q(rows=-1) == INV and q(K=0) == INV and q(K=-8) == INV
    assert q(K=12) == UNS and q(dt=5) == UNS and q(x=ODD) == UNS and q(o=ODD) == UNS and q(rows=1 << 40) == UNS
    assert q(x=None) == INV and q(o=None) == INV and q(s=None) == INV


def test_packed_weights_arguments():
    L = M.lib()
    assert L.moe_packed_weights_bytes(1, 64, 16) == 1024
    assert L.moe_packed_weights_bytes(3, 65, 24) == 3 * 2 * 2 * 1024
    for n, K, N in ((0, 64, 16), (1, 0, 16), (1, 64, 0), (1025, 64, 16), (1, 131072, 16), (1, 64, 12), (1, 131064, 16392), (1, 8, (1 << 21) + 8)):
        assert L.moe_packed_weights_bytes(n, K, N) == 0 and L.moe_last_error()
        assert L.moe_pack_weights(n, K, N, FAKE, FAKE, None) in (INV, UNS)
        assert L.moe_quantize_weights(n, K, N, M.MOE_DTYPE_BF16, FAKE, FAKE, FAKE, None) in (INV, UNS)
    assert L.moe_pack_weights(1, 64, 16, None, FAKE, None) == INV
    assert L.moe_pack_weights(1, 64, 16, FAKE, ODD, None) == UNS
    assert L.moe_quantize_weights(1, 64, 16, 3, FAKE, FAKE, FAKE, None) == UNS
    assert L.moe_quantize_weights(1, 64, 16, M.MOE_DTYPE_F32, FAKE, FAKE, None, None) == INV
    assert L.moe_quantize_weights(1, 64, 16, M.MOE_DTYPE_F32, ODD, FAKE, FAKE, None) == UNS


def test_gemm_quantized_arguments():
    def g(Mr=4, N=16, K=64, a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, c=FAKE, dt=M.MOE_DTYPE_BF16):
        return M.lib().moe_gemm_quantized(Mr, N, K, a, sa, b, sb, c, dt, None)
    assert g(Mr=-1) == INV and g(N=0) == INV and g(K=0) == INV
    assert g(Mr=(1 << 30) + 1) == UNS and g(N=(1 << 21) + 8) == UNS and g(K=24) == UNS and g(N=12) == UNS and g(K=131072) == UNS and g(dt=9) == UNS
    for name in ("a", "sa", "b", "sb", "c"):
        assert g(**{name: None}) == INV, name
    for name in ("a", "b", "sb", "c"):
        assert g(**{name: ODD}) == UNS, name


def test_binding_refuses_host_tensors_and_wrong_shapes():
    bf = torch.bfloat16
    p = M.Spec(4, 16, 2, 1, 8, 0, 2, "bf16")
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    off = z(3, dt=torch.int32)
    w = (z(2, 16, 8), z(2, 16, 8), z(2, 8, 16))
    with pytest.raises(ValueError, match="x_packed must be a contiguous device tensor"):
        M.expert_gemm_train(p, z(4, 16), off, *w)
    with pytest.raises(ValueError, match="x_packed: expected"):
        M.expert_gemm_train(p, z(4, 8), off, *w)
    with pytest.raises(ValueError, match="g: expected|x_packed"):
        M.expert_gemm_backward(p, z(4, 16), off, *w, z(4, 16), z(4, 8), z(4, 8), z(4, 16))
    with pytest.raises(ValueError, match="dy"):
        M.combine_backward(p, z(3, 16), z(4, 16), z(4, dt=torch.int32), None)
    with pytest.raises(ValueError, match="x: expected torch.bfloat16 or torch.float32"):
        M.quantize_rows(z(2, 16, dt=torch.float16))
    with pytest.raises(M.MoeError):
        M.pack_weights(z(16, 12, dt=torch.int8))
    with pytest.raises(ValueError, match="expected \\[n, K, N\\]"):
        M.pack_weights(z(1, 1, 16, 16, dt=torch.int8))
    with pytest.raises(ValueError, match="a must be|a: expected"):
        M.gemm_quantized(z(2, 16, dt=torch.int8), z(2, dt=torch.float32), z(1, 1, 4, 16, 16, dt=torch.int8), z(8, dt=torch.float32))


def test_a_used_problem_can_be_copied_and_pickled():
    import copy
    import pickle
    p = M.Spec(4, 16, 2, 1, 8, 0, 2, "bf16", 0)
    need = M.workspace_bytes(p, M.MOE_CALL_EXPERT_GEMM_BACKWARD)
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert q == p and M.workspace_bytes(q, M.MOE_CALL_EXPERT_GEMM_BACKWARD) == need
    # the structure a caller gets is its own
    c = p.c()
    c.T = 400
    assert p.c().T == 4 and M.workspace_bytes(p, M.MOE_CALL_EXPERT_GEMM_BACKWARD) == need


def test_backward_of_an_empty_batch_may_have_no_pointer_for_its_rows():
    """T = 0: an array with a T-sized dimension may be NULL, also the only wanted one."""
    args = [None, FAKE, FAKE, FAKE, FAKE] + [None] * 8
    assert _call("moe_expert_gemm_backward", _p(T=0), args, ws=None, wsb=0) == M.MOE_OK
    assert _call("moe_expert_gemm_backward", _p(), [FAKE] * 9 + [None] * 4) == INV


def test_sizes_beyond_32_bits_are_refused_not_cut_off():
    """Sizes that the C structure and arguments would hold modulo 2^32."""
    meta = lambda *s, dt=torch.int8: torch.empty(s, dtype=dt, device="meta")  # noqa: E731
    wide = 2 ** 32 + 16
    for field in ("T", "d", "f", "E"):
        kw = dict(T=4, d=16, E=2, k=1, f=8, expert_lo=0, n_local=2, dtype="bf16")
        kw[field] = wide
        with pytest.raises(ValueError, match="32 bits"):
            M.workspace_bytes(M.Spec(**kw), M.MOE_CALL_EXPERT_GEMM_BACKWARD)
    with pytest.raises(M.MoeError):   # small negative sizes are the library's to refuse
        M.workspace_bytes(M.Spec(-1, 16, 2, 1, 8, 0, 2, "bf16"), M.MOE_CALL_EXPERT_GEMM_BACKWARD)
    for n, K, N in ((wide, 64, 16), (1, wide, 16), (1, 64, wide)):
        with pytest.raises(ValueError, match="32 bits"):
            M.packed_weights_bytes(n, K, N)
        with pytest.raises(ValueError, match="32 bits"):
            M.pack_weights(meta(n, K, N))
        with pytest.raises(ValueError, match="32 bits"):
            M.quantize_weights(meta(n, K, N, dt=torch.bfloat16))
    with pytest.raises(ValueError, match="32 bits"):
        M.quantize_rows(meta(2, wide, dt=torch.bfloat16))
    f32 = torch.float32
    with pytest.raises(ValueError, match="32 bits"):
        M.gemm_quantized(meta(wide, 16), meta(wide, dt=f32), meta(1, 1, 4, 16, 16), meta(8, dt=f32))
    with pytest.raises(ValueError, match="32 bits"):
        M.gemm_quantized(meta(2, wide), meta(2, dt=f32), meta(1, 1, 4, 16, 16), meta(8, dt=f32))


def test_fp32_rows_of_the_training_calls_are_bounded():
    """Refused as unsupported before anything is launched, not by a failed launch."""
    p = _p(T=(1 << 27) + 1, d=8, f=8, E=1, k=1, n_local=1, dtype=M.MOE_DTYPE_F32)
    assert _call("moe_expert_gemm_train", p, [FAKE] * len(TRAIN), has_ws=False) == UNS
    assert _call("moe_expert_gemm_backward", p, [FAKE] * len(BACK)) == UNS
    assert b"rows" in M.lib().moe_last_error()
