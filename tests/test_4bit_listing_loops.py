"""The distances of tests/test_4bit_listing.py along every path: from the end of a loop to its
beginning, and over branches taken or not.  What is open at the end of a block of instructions
(vector results younger than two wait states, sums younger than eighteen) goes on into each block
that may follow it, until nothing new comes in anywhere."""
import concurrent.futures as cf
import re
import tempfile

import pytest

from tests.test_4bit_listing import SOURCES, _listing, _regs

VECTOR, SUM = 2, 18   # wait states


def _blocks(lines):
    """[(instructions, labels that may follow, whether the next block may)] and labels' numbers,
    one list for each function."""
    functions, blocks, labels = [], None, None
    for line in lines:
        t = line.split(";")[0].split("//")[0].rstrip()
        m = re.match(r"([.\w$]+):", t)
        if m and not m[1].startswith("."):          # a function begins
            blocks, labels = [[[], [], True]], {}
            functions.append((blocks, labels))
        elif m and m[1].startswith(".LBB") and blocks is not None:
            blocks.append([[], [], True])
            labels[m[1]] = len(blocks) - 1
        elif t.startswith("\t") and t.strip() and not t.strip().startswith(".") and blocks is not None:
            t = t.strip()
            block = blocks[-1]
            block[0].append(t)
            if t.startswith(("s_branch", "s_cbranch")):
                block[1].append(t.split()[1])
                block[2] = not t.startswith("s_branch")
                blocks.append([[], [], True])
            elif t.startswith("s_endpgm"):
                block[2] = False
                blocks.append([[], [], True])
            elif t.startswith(("s_setpc", "s_swappc", "s_call")):
                raise AssertionError(f"a jump that is not followed: {t}")
    return functions


def _walk(code, vector, sums, faults):
    """Runs a block: ages (wait states since) of vector results and of sums, by register."""
    vector, sums = dict(vector), dict(sums)

    def pass_(n):
        for ages, limit in ((vector, VECTOR), (sums, SUM)):
            for r in [r for r, a in ages.items() if a + n >= limit]:
                del ages[r]
            for r in ages:
                ages[r] += n
    for t in code:
        name, _, rest = t.replace("\t", " ").partition(" ")
        ops = [o.strip().split()[0] for o in rest.split(",") if o.strip()]
        if name == "s_nop":
            pass_(int(ops[0]) + 1)
            continue
        sets = [_regs(o) for o in ops]
        if name.startswith("v_mfma"):
            use = set().union(*sets[1:])
            faults += [f"{t}: {r} just before" for r in use if r in vector]
            pass_(1)
            for r in sets[0]:
                sums[r] = 0
        elif name.startswith(("v_", "ds_write", "buffer_store", "global_store")):
            faults += [f"{t}: soon after the product of {r}" for s in sets for r in s if r in sums]
            pass_(1)
            if name.startswith("v_"):
                for r in sets[0] if sets else ():
                    vector[r] = 0
                    sums.pop(r, None)
        else:
            pass_(1)
    return vector, sums


def check(lines):
    """(products, blocks entered from later ones, faults) of all functions."""
    products = back = 0
    faults = []
    for blocks, labels in _blocks(lines):
        products += sum(t.startswith("v_mfma") for b in blocks for t in b[0])
        state, todo = {0: ({}, {})}, [0]
        while todo:
            i = todo.pop()
            code, jumps, on = blocks[i]
            out = _walk(code, *state[i], [])
            after = [labels[j] for j in jumps] + ([i + 1] if on and i + 1 < len(blocks) else [])
            for j in after:
                if j not in state:
                    state[j] = ({}, {})
                    todo.append(j)
                for mine, new in zip(state[j], out):
                    for r, age in new.items():
                        if age < mine.get(r, 99):
                            mine[r] = age
                            if j not in todo:
                                todo.append(j)
        for i, entry in state.items():
            _walk(blocks[i][0], *entry, faults)
            back += any(labels[j] <= i for j in blocks[i][1])
    return products, back, sorted(set(faults))


def test_listing():
    with tempfile.TemporaryDirectory() as out, cf.ThreadPoolExecutor(2) as pool:
        for src, lines in zip(SOURCES, pool.map(lambda s: _listing(s, out), SOURCES)):
            products, back, faults = check(lines)
            assert products > 1000 and back >= 6 * 5, (src, products, back)   # the K loops of five heights
            assert not faults, (src, len(faults), faults[:5])


MFMA = "v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]"


@pytest.mark.parametrize("text,bad", [
    (f".LBB0_1:|{MFMA}|s_mov_b32 s0, 0|v_pk_add_f16 v1, v2, v3|s_cbranch_scc1 .LBB0_1|s_endpgm", 1),      # around the loop
    (f".LBB0_1:|{MFMA}|v_pk_add_f16 v1, v2, v3|s_nop 0|s_cbranch_scc1 .LBB0_1|s_endpgm", 0),
    (f"v_pk_add_f16 v1, v2, v3|s_cbranch_scc1 .LBB0_2|s_nop 7|.LBB0_2:|{MFMA}|s_endpgm", 1),                # the way that skips
    (f"v_pk_add_f16 v1, v2, v3|s_branch .LBB0_2|.LBB0_1:|{MFMA}|s_endpgm|.LBB0_2:|s_nop 1|s_branch .LBB0_1", 0),
    (f".LBB0_1:|v_accvgpr_read_b32 v9, a3|s_nop 7|{MFMA}|s_nop 15|s_cbranch_scc1 .LBB0_1|s_endpgm", 1),
    (f".LBB0_1:|v_accvgpr_read_b32 v9, a3|s_nop 7|{MFMA}|s_nop 15|s_nop 1|s_cbranch_scc1 .LBB0_1|s_endpgm", 0),
    (f"v_pk_add_f16 v1, v2, v3|s_endpgm|.LBB0_1:|{MFMA}|s_endpgm", 0)])
def test_check_finds_what_it_is_for(text, bad):
    lines = ["f:"] + [t if t.startswith(".L") else "\t" + t for t in text.split("|")]
    assert len(check(lines)[2]) == bad
