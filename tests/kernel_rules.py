"""Which kernels a training or 8-bit call takes, from the library's own rules
(csrc/tile_rules.h, compiled for the host), so that a test can say which kernel it
is for and fails when a retuned rule sends its sizes elsewhere."""
import ctypes
import functools
import os
import shutil
import subprocess
import tempfile
from collections import namedtuple

HERE = os.path.dirname(os.path.abspath(__file__))
CUS = 256   # compute units of an MI355X
WG_LONG, WG_SHORT, WG_SPLIT = 0, 1, 2

Train = namedtuple("Train", "up down")
Backward = namedtuple("Backward", "gate input mode div units apart")
I8 = namedtuple("I8", "stream tiles wide low blocks height")


@functools.lru_cache(None)
def _lib():
    cxx = next((c for c in ("g++", "clang++", "/opt/rocm/llvm/bin/clang++") if shutil.which(c)), None)
    assert cxx, "no host C++ compiler"
    with tempfile.TemporaryDirectory() as tmp:
        out = os.path.join(tmp, "kernel_rules.so")
        subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", os.path.join(HERE, "kernel_rules.cpp"),
                        "-o", out], check=True)
        lib = ctypes.CDLL(out)   # stays mapped after the file is gone
    i32, i64 = ctypes.c_int, ctypes.c_int64
    into = ctypes.POINTER(i64)
    lib.rules_train.argtypes = [i64, i64, i32, i32, i32, i32, into]
    lib.rules_backward.argtypes = [i64, i64, i32, i32, i32, i32, i32, i32, into]
    lib.rules_i8.argtypes = [i64, i32, i32, i32, i32, i32, i64, i64, i64, into]
    return lib


def _ask(fn, kind, *args):
    out = (ctypes.c_int64 * len(kind._fields))()
    getattr(_lib(), fn)(CUS, *args, out)
    return kind(*out)


def train(p):
    return _ask("rules_train", Train, p.T * p.k, p.E, p.n_local, p.d, p.f)


def backward(p, input=True, wants=3):
    return _ask("rules_backward", Backward, p.T * p.k, p.E, p.n_local, p.d, p.f, int(input), wants)


def product(M, N, K):
    """gemm_quantized of M rows."""
    return _ask("rules_i8", I8, 0, 0, 1, N, -(-K // 64), M, M, M)


def experts(p):
    """(gated product, down projection) of expert_gemm_quantized."""
    tk = p.T * p.k
    size = (tk // p.E, tk * p.n_local // p.E, p.T)
    return (_ask("rules_i8", I8, 1, 1, p.n_local, p.f, -(-p.d // 64), *size),
            _ask("rules_i8", I8, 0, 1, p.n_local, p.d, -(-p.f // 64), *size))
