"""Which kernels a 4-bit product takes, by the library's own rules."""
import ctypes
import functools
import os
import shutil
import subprocess
import tempfile
from typing import NamedTuple

HERE = os.path.dirname(os.path.abspath(__file__))
CUS = 256


class Plan(NamedTuple):
    tiles: bool
    bm: int
    parts: int
    per: int
    wide: bool
    low: bool
    blocks: int
    waves: int
    ahead: bool


@functools.lru_cache(None)
def _lib():
    cxx = next((c for c in ("g++", "clang++", "/opt/rocm/llvm/bin/clang++") if shutil.which(c)), None)
    assert cxx, "no host C++ compiler"
    with tempfile.TemporaryDirectory() as tmp:
        out = os.path.join(tmp, "rules.so")
        subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-o", out, os.path.join(HERE, "rules_4bit.cpp")], check=True)
        return ctypes.CDLL(out)   # stays mapped after the file is gone


def _plan(gated, segments, n, N, K, mean, rows, most):
    out = (ctypes.c_int64 * 9)()
    i64 = ctypes.c_int64
    _lib().rules_w4(i64(CUS), gated, segments, n, N, -(-K // 128), i64(mean), i64(rows), i64(most), out)
    p = Plan(*out)
    return p._replace(tiles=bool(p.tiles), wide=bool(p.wide), low=bool(p.low), ahead=bool(p.ahead))


def product(M, K, N):
    """Of ``gemm_4bit``."""
    return _plan(0, 0, 1, N, K, M, M, M)


def experts(p):
    """Of the two products of ``expert_gemm_4bit``."""
    tk = p.T * p.k
    mean, rows = tk // p.E, tk * p.n_local // p.E
    return (_plan(1, 1, p.n_local, p.f, p.d, mean, rows, p.T), _plan(0, 1, p.n_local, p.d, p.f, mean, rows, p.T))


def heights(rows, bm):
    """Heights, in row tiles of 16, that the tiles of a segment of ``rows`` rows have."""
    of = lambda r: 4 if r <= 64 else min(2 * -(-r // 32), 12)  # noqa: E731
    return {of(min(bm, rows - r)) for r in range(0, rows, bm)}
