"""The matrix products that the 4-bit tiles issue by inline asm, in the compiler's listing: the
compiler does not know them for what they are and puts no waits around them, so the order
of the instructions has to leave room.  Compiles both sources as the build does."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from combine_router_top_amd import build as B

SOURCES = ("expert_4bit_up.hip", "expert_4bit_down.hip")


def _listing(src, out):
    path = os.path.join(out, src + ".s")
    subprocess.run([B.hipcc(), "-S", "--cuda-device-only", os.path.join(B.CSRC, src), "-o", path] + B.common_flags() + B.device_flags(),
                   check=True, capture_output=True)
    with open(path) as f:
        return f.read().split("\n")


def _regs(op):
    m = re.match(r"([va])\[(\d+):(\d+)\]$", op)
    if m:
        return {m[1] + str(i) for i in range(int(m[2]), int(m[3]) + 1)}
    return {op} if re.match(r"[va]\d+$", op) else set()


def check(lines):
    """(products, faults): a vector instruction within two wait states before a product that
    takes its result; a sum read within 18 after the product that made it."""
    count, faults, before, at, made = 0, [], [], 0, {}
    for line in lines:
        t = line.split(";")[0].split("//")[0].strip()
        if not line.startswith("\t") or not t or t.startswith("."):
            continue
        name, _, rest = t.partition(" ") if " " in t else t.partition("\t")
        ops = [o.strip().split()[0] for o in rest.split(",") if o.strip()]
        if name == "s_nop":
            at += int(ops[0]) + 1
            continue
        at += 1
        if name in ("s_endpgm", "s_branch"):   # what follows is reached from elsewhere
            before, made = [], {}
            continue
        sets = [_regs(o) for o in ops]
        if name.startswith("v_mfma_f32_16x16x32_f16"):
            count += 1
            use = set().union(*sets[1:])
            faults += [f"{t}: just after {n}" for n, w, when in before if at - when - 1 < 2 and w & use]
            for r in sets[0]:
                made[r] = at
        elif name.startswith(("v_", "ds_write", "buffer_store", "global_store")):
            for r in set().union(*sets) if sets else ():
                if r in made and at - made[r] - 1 < 18:
                    faults.append(f"{t}: soon after the product of {r}")
            if name.startswith("v_"):
                before = before[-4:] + [(name, sets[0] if sets else set(), at)]
                for r in sets[0] if sets else ():
                    made.pop(r, None)
    return count, faults


def test_listing():
    import tempfile
    with tempfile.TemporaryDirectory() as out, cf.ThreadPoolExecutor(2) as pool:
        for src, lines in zip(SOURCES, pool.map(lambda s: _listing(s, out), SOURCES)):
            count, faults = check(lines)
            assert count > 1000, src
            assert not faults, (src, faults[:5])


@pytest.mark.parametrize("text,bad", [
    ("v_pk_add_f16 v1, v2, v3|v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]", 1),
    ("v_pk_add_f16 v1, v2, v3|s_nop 1|v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]", 0),
    ("v_accvgpr_write_b32 a2, 0|s_mov_b32 s0, 0|v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]", 1),
    ("v_pk_add_f16 v1, v2, v3|s_mov_b32 s0, 0|s_mov_b32 s1, 0|v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]", 0),
    ("v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]|s_nop 15|v_accvgpr_read_b32 v9, a3", 1),
    ("v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]|s_nop 15|s_nop 15|v_accvgpr_read_b32 v9, a3", 0),
    ("v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]|v_accvgpr_read_b32 v9, a4", 0)])
def test_check_finds_what_it_is_for(text, bad):
    assert len(check(["\t" + t for t in text.split("|")])[1]) == bad
