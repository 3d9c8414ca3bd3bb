"""Scalar offsets of the loads of the 4-bit products: none passes the end of its buffer, for
blocks that are loaded ahead of the last, groups that the last block has not, zero points that a
matrix has not and tiles of one row."""
import ctypes
import os
import re
import shutil
import subprocess
import tempfile

import pytest

from combine_router_top_amd import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def offset():
    cxx = next((c for c in ("g++", "clang++", "/opt/rocm/llvm/bin/clang++") if shutil.which(c)), None)
    assert cxx, "no host C++ compiler"
    with tempfile.TemporaryDirectory() as tmp:
        out = os.path.join(tmp, "reach.so")
        subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-o", out, os.path.join(HERE, "reach_4bit.cpp")], check=True)
        lib = ctypes.CDLL(out)   # stays mapped after the file is gone
    lib.reach_offset.restype = ctypes.c_uint32
    return lambda off, size: lib.reach_offset(ctypes.c_uint32(off), ctypes.c_uint32(size)), lib.reach_block


def _stream(K, N, R, group, zero, waves, ahead):
    """(asked for, bytes of the buffer) of every load of every wave."""
    kb, groups, gpb = -(-K // 128), -(-K // group), 128 // group
    per = -(-kb // waves)
    for wave in range(waves):
        s0 = wave * per
        ns = max(0, min(per, kb - s0))
        if ns == 0:
            continue
        ring = 2 if ahead else 1
        blocks = set(range(ring - 1)) | {b + h + ring - 1 for b in range(0, ns, ring) for h in range(ring)}
        for b in blocks:
            yield b * 1024, ns * 1024
            for q in range(4):
                yield ((s0 + b) * 128 + 32 * q) * 2, R * K * 2
            row = (s0 + b) * gpb * N
            yield row * 2, groups * N * 2
            yield row, groups * N if zero else 0


def _tile(K, N, R, group, zero, part, last):
    """(offset, bytes) of weights and rows, and of scales and zero points; ``last``: which block or
    step of a number is copied for one that may lie past it."""
    kb, groups, gpb = -(-K // 128), -(-K // group), 128 // group
    b0, nb = part
    ntn = -(-N // 256)
    for nt in {0, ntn - 1}:
        wsize = (-(-N // 16) - 16 * nt) * kb * 1024 - 1024 * b0
        xsize = R * kb * 256 - 256 * b0
        for b in range(nb + 2):
            yield True, last(b, nb) * 1024, wsize
        for st in {0, 1, 2} | {2 * b + i for b in range(nb) for i in (3, 4)}:
            yield True, last(st, 2 * nb) * 128, xsize
        for bytes_, has in ((2, True), (1, zero)):
            row = N * bytes_
            for u in range(gpb):
                skip = row * (u + b0 * gpb)
                size = groups * row - 256 * nt * bytes_ if has else 0
                for b in range(nb + 2):
                    yield False, last(b, nb) * row * gpb, max(0, size - skip)


SIZES = [(K, N, R, G) for K in (8, 136, 392, 4104) for N in (8, 264) for R in (1, 3, 16) for G in (32, 64, 128)]


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("K,N,R,group", SIZES)
def test_offsets(offset, K, N, R, group, zero):
    offset, block = offset
    kb = -(-K // 128)
    loads = [v for w in (4, 8, 16) for ahead in (False, True) for v in _stream(K, N, R, group, zero, w, ahead)]
    halves = [(0, kb)] + ([(0, (kb + 1) // 2), ((kb + 1) // 2, kb // 2)] if kb > 1 else [])
    tiles = [v for part in halves for v in _tile(K, N, R, group, zero, part, block)]
    assert all(off < size for whole, off, size in tiles if whole)     # by block, as they are
    assert any(off >= size for part in halves for whole, off, size in _tile(K, N, R, group, zero, part, lambda i, n: i) if whole)
    loads += [v[1:] for v in tiles if not v[0]]
    assert any(off > size for off, size in loads)   # what the bound is there for
    for off, size in loads:
        got = offset(off, size)
        assert got <= size and (got == off or off > size)


@pytest.mark.parametrize("src,call", [("expert_4bit.hip", r"__builtin_amdgcn_raw_buffer_load_b\d+"), ("w4_tile.h", r"w4_copy<4>"),
                                      ("w4_tile.h", "xr.issue|w4_issue"), ("route_backward.hip", "bd_copy16")])
def test_every_load_is_bounded(src, call):
    with open(os.path.join(B.CSRC, src)) as f:
        text = f.read()
    found = [text[m.start(): text.index(";", m.start())] for m in re.finditer("(" + call + r")\((?!const)", text)]
    bad = [c for c in found if "st_offset(" not in c and "st_upto(" not in c]
    assert found and not bad, bad
