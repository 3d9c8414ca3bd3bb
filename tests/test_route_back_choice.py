"""Which kernels of the router's gradients the sizes of the GPU tests take, and that together
they take all there are."""
import ctypes
import os
import shutil
import subprocess
import tempfile

import pytest

from tests.test_gpu_route_back_kernels import LARGE
from tests.test_gpu_scored import BACK

HERE = os.path.dirname(os.path.abspath(__file__))
CUS = 256


@pytest.fixture(scope="module")
def rules():
    cxx = next((c for c in ("g++", "clang++", "/opt/rocm/llvm/bin/clang++") if shutil.which(c)), None)
    assert cxx, "no host C++ compiler"
    with tempfile.TemporaryDirectory() as tmp:
        out = os.path.join(tmp, "rules.so")
        subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-o", out, os.path.join(HERE, "rules_route_back.cpp")], check=True)
        lib = ctypes.CDLL(out)   # stays mapped after the file is gone
    i64 = ctypes.c_int64
    return (lambda T, d: bool(lib.rules_route_few(i64(CUS), i64(T), d)),
            lambda T, d, E: lib.rules_route_shares(i64(CUS), i64(T), d, E))


def test_every_kernel_has_a_case(rules):
    few, shares = rules
    assert all(few(T, d) for T, E, k, d, dtype in BACK if dtype == "bf16")
    assert not any(few(T, d) for T, E, k, d in LARGE)
    # gate matrices of one and of several blocks of 256 experts, padded rows or not, whole and shared tokens
    assert {(E > 256, E % 8 == 0) for _, E, _, _ in LARGE} == {(a, b) for a in (False, True) for b in (False, True)}
    assert {shares(T, d, E) > 1 for T, E, _, d in LARGE} == {False, True}
    assert any(shares(T, d, E) > 1 for T, E, _, d in LARGE if E > 256 and E % 8)
    # last tiles of few rows and columns, and narrow rows, which are stored another way
    assert any(0 < T % 64 < 4 for T, *_ in LARGE) and any(d % 256 for *_, d in LARGE) and any(d <= 512 for *_, d in LARGE)
    assert {E > 256 for _, E, _, _, dtype in BACK if dtype == "bf16"} == {False, True}


def test_shares_cover_all_tokens(rules):
    _, shares = rules
    for T in (1, 63, 64, 257, 1030, 4097, 32700, 1 << 20):
        for d in (8, 520, 7168):
            for E in (1, 24, 256, 300, 1024):
                n = shares(T, d, E)
                stages = -(-T // 64)
                assert n >= 1 and n * -(-stages // n) >= stages and (n == 1 or stages // n >= 4)
